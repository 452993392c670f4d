// index_scores.hip - the indexer's scores (dsatopk_scores_paged and
// dsatopk_scores_ragged in include/dsatopk.h):
//
//   score[b, j] = key_scale[j] * sum over heads h of w[b, h] * max(0, q[b, h] . key[j])
//
// for the window positions j of row b. Sums are in fp32 throughout; nothing
// is rounded before the fp32 store.
//
// The product runs on the matrix units with heads as the rows and tokens as
// the columns of 32 x 32 tiles, so one query row of 64 heads fills two tiles
// by itself, for a single token as for a prompt, and a lane holds 16 heads
// of one token: the weighted sum over heads stays inside the lane but for
// one exchange with lane ^ 32 at the end.
//
// A workgroup owns kTile tokens: each wave keeps 64 tokens' keys in
// registers, as they come from memory, and goes over its group of query
// rows, whose heads all four waves read from LDS (swizzled, double
// buffered, copied there without passing through registers). Keys are read
// once per row group, and again only where the table row changes.
//
// 128 rows over 8192 paged keys each (bf16, 64 heads): 62 us, 4.4 TB/s, bound
// by memory, with a table and a score buffer as wide as the rows (wider ones:
// see run_scores). 4 x 1024 rows over 16384 keys each (e4m3, 64 heads): 870 us, 1.23
// PFLOP/s, bound by the matrix units (each 32 x 32 tile's 8 products also need
// 32 vector instructions for the weighting, which other waves' products hide).

#include "serve_common.h"

namespace dsatopk_serve {
namespace {

constexpr int kBlock = 256;
constexpr int kWaveTokens = 64;
constexpr int kTile = kWaveTokens * (kBlock / 64);
constexpr int kMaxHeads = 128;
constexpr int64_t kMaxColumns = int64_t(1) << 30;

struct ScoreParams {
  const char* q;
  int64_t q_row, q_head;  // bytes
  const float* weights;
  int64_t w_row;  // floats
  const char* keys;
  int64_t key_page, key_token;  // bytes
  const float* scales;
  int64_t scale_page;  // floats; a page's scales are contiguous
  int64_t num_pages;   // paged: pages of the cache; ragged: tokens
  const int32_t* seq_lens;
  const int32_t* row_starts;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* table_rows;
  int32_t page_bits, table_width;
  float* out;
  int64_t out_stride;
  int32_t rows, heads, group, columns;
};

// Heads and keys as the matrix units take them: 16-bit elements, 16-byte
// chunks of 8. Bytes become bfloat16 on their way (each e4m3 value is one),
// because the 8-bit products hold their sums to fewer bits than 32: off by up
// to 1.3e-4 of the terms' sizes for 64 products of mixed sizes, against
// 3e-7 by way of bfloat16.
template <int kKind, int kDim>
struct Shape {
  static constexpr int kBytes = kDim * 2;         // of a head in LDS
  static constexpr int kChunks = kBytes / 16;
  static constexpr int kSteps = kDim / 16;        // products over the dimension
  // The chunk that lane half `half` takes in product s. Keys of bytes come 16
  // (two chunks) at a load.
  static __device__ __forceinline__ constexpr int chunk(int s, int half) {
    return kKind == DSATOPK_FP8 ? 4 * (s >> 1) + 2 * half + (s & 1) : 2 * s + half;
  }
};

// 16 bytes as 16 bfloat16 values.
__device__ __forceinline__ void widen(u32x4 v, uint32_t (&out)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    out[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.0f, false));
    out[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.0f, true));
  }
}

template <int kKind>
__device__ __forceinline__ f32x16 product(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (kKind == DSATOPK_FP16)
    return Fp16::mma32(a, b, c);
  else
    return Bf16::mma32(a, b, c);
}

template <int kChunks>
__device__ __forceinline__ constexpr int swizzle_of(int head) {
  return kChunks == 8 ? swizzle8(head) : swizzle16(head);
}

// Row r's heads into LDS, swizzled; heads that the row does not have are
// zeros.
template <int kBytes, int kHeads>
__device__ __forceinline__ void copy_heads(const ScoreParams& p, int32_t r, int wave, int lane,
                                           char* lds) {
  constexpr int kChunks = kBytes / 16;
  constexpr int kCopyRows = 1024 / kBytes;  // heads a wave copies at once
  const char* q = p.q + r * p.q_row;
  const int sub = lane / kChunks, c = lane % kChunks;
#pragma unroll
  for (int i = 0; i < kHeads / kCopyRows / (kBlock / 64); ++i) {
    const int h = (i * (kBlock / 64) + wave) * kCopyRows, hh = h + sub;
    const char* src = hh < p.heads ? q + hh * p.q_head : zero_row();
    copy_to_lds(src + (c ^ swizzle_of<kChunks>(hh)) * 16, lds + h * kBytes);
  }
}

// The same for heads of bytes, by way of registers: a thread loads 16 bytes
// of each of its heads, and later stores them widened.
template <int kDim, int kHeads>
struct ByteHeads {
  static constexpr int kPieces = kDim / 16;                // 16-byte pieces of a head
  static constexpr int kStep = kBlock / kPieces;           // heads of one go
  static constexpr int kGoes = (kHeads + kStep - 1) / kStep;
  u32x4 piece[kGoes];
  __device__ __forceinline__ void load(const ScoreParams& p, int32_t r, int tid) {
    const char* q = p.q + r * p.q_row + (tid % kPieces) * 16;
#pragma unroll
    for (int g = 0; g < kGoes; ++g) {
      const int h = g * kStep + tid / kPieces;
      piece[g] = u32x4{0, 0, 0, 0};
      if (h < p.heads) piece[g] = *reinterpret_cast<const u32x4*>(q + h * p.q_head);
    }
  }
  __device__ __forceinline__ void store(const ScoreParams& p, char* lds, int tid) const {
    constexpr int kBytes = kDim * 2, kChunks = kBytes / 16;
#pragma unroll
    for (int g = 0; g < kGoes; ++g) {
      const int h = g * kStep + tid / kPieces, c = (tid % kPieces) * 2;
      if (kStep * kGoes > kHeads && h >= kHeads) break;
      uint32_t w[8];
      widen(piece[g], w);
#pragma unroll
      for (int x = 0; x < 2; ++x)
        *reinterpret_cast<u32x4*>(lds + h * kBytes + ((c + x) ^ swizzle_of<kChunks>(h)) * 16) =
            u32x4{w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]};
    }
  }
};

// One row's sums over its heads (of this lane's half of each 32) for the
// wave's 2 x 32 tokens, while the next row's heads are copied: the two
// buffers are told apart so that no read of one waits for the other's copy.
// 32 heads at a time: with 64 the weighting of the first could go on beside
// the products of the second, but three waves a SIMD do better at that than
// two with 64 more registers (886 against 922 us for 4 x 1024 rows of 64
// heads over 16384 keys each).
template <int kKind, int kDim, int kHeads, bool kWhole>
__device__ __forceinline__ void row_sums(const ScoreParams& p, const char* __restrict__ heads,
                                         const float* __restrict__ weights,
                                         char* __restrict__ next, int32_t next_row, int wave,
                                         int lane, const u32x4 (&key)[2][Shape<kKind, kDim>::kSteps],
                                         float (&sum)[2]) {
  using S = Shape<kKind, kDim>;
  if (kKind != DSATOPK_FP8 && next_row >= 0)
    copy_heads<S::kBytes, kHeads>(p, next_row, wave, lane, next);
  lane = here(lane);
  const int half = lane >> 5, col = lane & 31;
  // chunk(s, half) ^ swizzle is chunk(s, 0) ^ (chunk(0, half) ^ swizzle)
  const int first = col * S::kBytes + ((S::chunk(0, half) ^ swizzle_of<S::kChunks>(col)) << 4);
#pragma unroll 1
  for (int slab = 0; slab < kHeads / 32; ++slab) {
    f32x16 acc[2] = {};
#pragma unroll
    for (int s = 0; s < S::kSteps; ++s) {
      const u32x4 a = *reinterpret_cast<const u32x4*>(heads + slab * 32 * S::kBytes +
                                                      (first ^ (S::chunk(s, 0) << 4)));
#pragma unroll
      for (int n = 0; n < 2; ++n) acc[n] = product<kKind>(a, key[n][s], acc[n]);
    }
    // Zeros stand in for heads that the row does not have: an infinite key
    // makes no number of them. (Kernels of their own for kHeads heads, which have
    // no such test in the loop: 879 us for the rows above, and 901 with it. A
    // loop over whole slabs with the rest behind it costs the decode rows
    // of 64 heads their third wave a SIMD: 63 and 68 us.)
    if (!kWhole && slab * 32 + 32 > p.heads) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (slab * 32 + 8 * (i / 4) + 4 * half + i % 4 >= p.heads) acc[0][i] = acc[1][i] = 0.0f;
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const f32x4 w = *reinterpret_cast<const f32x4*>(&weights[slab * 32 + 8 * x + 4 * half]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n)
          sum[n] = fmaf(w[i], __builtin_elementwise_maximum(acc[n][4 * x + i], 0.0f), sum[n]);
    }
  }
}

// kWhole: the row has kHeads heads, not fewer.
template <int kKind, int kDim, int kHeads, bool kWhole, bool kPaged>
__global__ __launch_bounds__(kBlock, 2) void scores_kernel(ScoreParams p) {
  using S = Shape<kKind, kDim>;
  constexpr int kBytes = S::kBytes;
  __shared__ __attribute__((aligned(1024))) char heads_lds[2][kHeads * kBytes];
  __shared__ __attribute__((aligned(16))) float w_lds[2][kHeads];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, col = lane & 31;
  const int32_t j0 = (int32_t)blockIdx.x * kTile;
  const int64_t r64 = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * p.group;
  if (r64 >= p.rows) return;
  const int32_t r0 = (int32_t)r64;
  const int32_t r1 = (int32_t)min(r64 + p.group, (int64_t)p.rows);
  const int32_t jw = j0 + wave * kWaveTokens;

  // Lane i has row r0 + i's window in columns, as [lo, hi); the rows whose
  // windows meet this workgroup's tokens are a bit each.
  int32_t lo = 0, hi = 0, from = 0;
  if (r0 + lane < r1) {
    const int32_t r = r0 + lane;
    if constexpr (kPaged)
      from = p.table_rows ? p.table_rows[r] : r;
    else
      lo = p.row_starts[r];
    hi = (int32_t)min((int64_t)lo + max(p.seq_lens[r], 0), (int64_t)p.columns);
    lo = max(lo, 0);
  }
  uint64_t todo = __ballot(lo < j0 + kTile && hi > j0 && hi > lo);
  if (todo == 0) return;

  // This thread's weight of a row, 0 for heads that it does not have.
  auto weight_of = [&](int32_t r) { return tid < p.heads ? p.weights[r * p.w_row + tid] : 0.0f; };

  u32x4 key[2][S::kSteps];
  float scale[2] = {1.0f, 1.0f};
  bool there[2] = {true, true};  // the lane's tokens have a key
  auto load_keys = [&](int64_t table_row) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int32_t j = jw + n * 32 + col;
      const char* src = zero_row();
      if constexpr (kPaged) {
        const int32_t e = j >> p.page_bits, in = j & ((1 << p.page_bits) - 1);
        const int32_t page = e < p.table_width ? p.table[table_row * p.table_stride + e] : -1;
        there[n] = page >= 0 && page < p.num_pages;
        if (there[n]) {
          src = p.keys + page * p.key_page + in * p.key_token;
          scale[n] = p.scales ? p.scales[page * p.scale_page + in] : 1.0f;
        }
      } else if (j < p.num_pages) {
        src = p.keys + j * p.key_token;
        scale[n] = p.scales ? p.scales[j] : 1.0f;
      }
      if constexpr (kKind == DSATOPK_FP8) {
#pragma unroll
        for (int s = 0; s < kDim / 32; ++s) {
          uint32_t w[8];
          widen(load16(src + (2 * s + half) * 16), w);
          key[n][2 * s] = u32x4{w[0], w[1], w[2], w[3]};
          key[n][2 * s + 1] = u32x4{w[4], w[5], w[6], w[7]};
        }
      } else {
#pragma unroll
        for (int s = 0; s < S::kSteps; ++s) key[n][s] = load16(src + S::chunk(s, half) * 16);
      }
    }
  };

  int at = __builtin_ctzll(todo);
  todo &= todo - 1;
  int buf = 0;
  int32_t have = -1;
  ByteHeads<kDim, kHeads> bytes;
  if constexpr (kKind == DSATOPK_FP8) {
    bytes.load(p, r0 + at, tid);
    bytes.store(p, heads_lds[0], tid);
  } else {
    copy_heads<kBytes, kHeads>(p, r0 + at, wave, lane, heads_lds[0]);
  }
  if (tid < kHeads) w_lds[0][tid] = weight_of(r0 + at);
  if constexpr (!kPaged) load_keys(0);
  for (;;) {
    if constexpr (kPaged) {
      const int32_t want = __builtin_amdgcn_readlane(from, at);
      if (want != have) load_keys(have = want);
    }
    const int next = todo ? __builtin_ctzll(todo) : -1;
    todo &= todo - 1;
    copies_barrier();  // the row's heads are there, the other buffer is free
    float weight = 0.0f;
    if (next >= 0) {
      weight = weight_of(r0 + next);
      if constexpr (kKind == DSATOPK_FP8) bytes.load(p, r0 + next, tid);
    }
    float sum[2] = {0.0f, 0.0f};
    row_sums<kKind, kDim, kHeads, kWhole>(p, heads_lds[buf], w_lds[buf], heads_lds[buf ^ 1],
                                          next >= 0 ? r0 + next : -1, wave, lane, key, sum);
    if (next >= 0) {
      if constexpr (kKind == DSATOPK_FP8) bytes.store(p, heads_lds[buf ^ 1], tid);
      if (tid < kHeads) w_lds[buf ^ 1][tid] = weight;
    }
    // both halves' heads; then lane l keeps token l of the wave's 64
    float t0 = (sum[0] + other_half(sum[0])) * scale[0];
    float t1 = (sum[1] + other_half(sum[1])) * scale[1];
    if constexpr (kPaged) {  // 0 without a key, whatever the row holds
      t0 = there[0] ? t0 : 0.0f;
      t1 = there[1] ? t1 : 0.0f;
    }
    const int32_t j = jw + lane;
    if (j >= __builtin_amdgcn_readlane(lo, at) && j < __builtin_amdgcn_readlane(hi, at))
      p.out[(r0 + at) * p.out_stride + j] = half ? t1 : t0;
    if (next < 0) break;
    at = next;
    buf ^= 1;
  }
}

template <int kKind, int kDim, int kHeads>
int launch_heads(const ScoreParams& p, bool paged, dim3 grid, void* stream) {
  const auto kernel = p.heads == kHeads ? paged ? scores_kernel<kKind, kDim, kHeads, true, true>
                                                : scores_kernel<kKind, kDim, kHeads, true, false>
                      : paged           ? scores_kernel<kKind, kDim, kHeads, false, true>
                                        : scores_kernel<kKind, kDim, kHeads, false, false>;
  return launch(kernel, grid, dim3(kBlock), p, stream);
}

template <int kKind, int kDim>
int launch_scores(const ScoreParams& p, bool paged, dim3 grid, void* stream) {
  return p.heads <= 32   ? launch_heads<kKind, kDim, 32>(p, paged, grid, stream)
         : p.heads <= 64 ? launch_heads<kKind, kDim, 64>(p, paged, grid, stream)
                         : launch_heads<kKind, kDim, kMaxHeads>(p, paged, grid, stream);
}

int run_scores(ScoreParams p, int32_t type, int32_t dim, bool paged, void* stream) {
  const int64_t tiles = ((int64_t)p.columns + kTile - 1) / kTile;
  if (tiles == 0) return DSATOPK_OK;
  // Rows a workgroup: enough workgroups to fill the card come first, then
  // keys read for as many rows as possible, up to a lane for each. With 1024 /
  // 2048 / 4096 as enough (us): 128 rows of 8192 paged keys 69 / 64 / 64, of two
  // and four rows a request 82 / 76 / 76 and 106 / 100 / 99; 256 rows over
  // 16384 keys 74 / 75 / 80, 1024 over 4096 69 / 70 / 75, 4096 over 16384 868 to 870.
  // The rows' lengths are on the device: what counts here is the buffer's and the
  // table's width, and in ones much wider than the rows few of the groups have work.
  // The 128 rows of 8192 in a table of 131072 take 228 us instead of 64.
  constexpr int64_t kEnough = 2048, kMostY = 65535;
  int64_t group = p.rows * tiles / kEnough;
  group = group < 1 ? 1 : group > 64 ? 64 : group;
  const int64_t groups = (p.rows + group - 1) / group;
  p.group = (int32_t)group;
  const dim3 grid((unsigned)tiles, (unsigned)(groups < kMostY ? groups : kMostY),
                  (unsigned)((groups + kMostY - 1) / kMostY));
  switch (type * 2 + (dim == 128)) {
    case 0: return launch_scores<0, 64>(p, paged, grid, stream);
    case 1: return launch_scores<0, 128>(p, paged, grid, stream);
    case 2: return launch_scores<1, 64>(p, paged, grid, stream);
    case 3: return launch_scores<1, 128>(p, paged, grid, stream);
    case 4: return launch_scores<2, 64>(p, paged, grid, stream);
    default: return launch_scores<2, 128>(p, paged, grid, stream);
  }
}

// What both forms check. Strides come in elements. What has no entries (no
// pages or tokens, no columns) may be null.
int check_scores(const void* q, int64_t q_row, int64_t q_head, const float* weights,
                 int64_t w_row, const void* keys, int64_t num_keys, int64_t key_token,
                 const int32_t* seq_lens,
                 int32_t type, int32_t heads, int32_t dim, int32_t rows, const float* out,
                 int64_t out_stride, int64_t columns) {
  if (rows < 0 || heads < 1 || heads > kMaxHeads || (dim != 64 && dim != 128) ||
      type < DSATOPK_BF16 || type > DSATOPK_FP8 || columns < 0 || columns > kMaxColumns ||
      out_stride < columns || q_row < 0 || q_head < 0 || key_token < 0 || w_row < 0)
    return DSATOPK_ERR_INVALID_ARG;
  if (rows == 0) return DSATOPK_OK;
  if (!q || !weights || (num_keys && !keys) || !seq_lens || (columns && !out))
    return DSATOPK_ERR_INVALID_ARG;
  const int64_t size = type == DSATOPK_FP8 ? 1 : 2;
  if (!aligned16(q) || !aligned16(keys) || (q_row * size) % 16 || (q_head * size) % 16 ||
      (key_token * size) % 16 || !aligned4(out) || !aligned4(weights))
    return DSATOPK_ERR_ALIGNMENT;
  return DSATOPK_OK;
}

}  // namespace
}  // namespace dsatopk_serve

using namespace dsatopk_serve;

extern "C" {

int dsatopk_scores_paged(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                         const float* weights, int64_t weight_stride, const void* keys,
                         int64_t num_pages, int64_t key_page_stride, int64_t key_token_stride,
                         const float* key_scales, int64_t scale_page_stride, int32_t type,
                         int32_t num_heads, int32_t head_dim, const int32_t* seq_lens,
                         const int32_t* page_table, int64_t page_table_stride,
                         int32_t page_table_width, int32_t page_size, const int32_t* table_rows,
                         int32_t num_rows, float* out, int64_t out_stride, int64_t columns,
                         void* stream) {
  const int st = check_scores(q, q_row_stride, q_head_stride, weights, weight_stride, keys,
                              num_pages, key_token_stride, seq_lens, type, num_heads, head_dim, num_rows,
                              out, out_stride, columns);
  if (st != DSATOPK_OK || num_rows == 0) return st;
  if (!page_table || page_table_width < 1 || page_table_stride < page_table_width ||
      !pow2(page_size) || page_size > (1 << 20) || num_pages < 0 || key_page_stride < 0 ||
      scale_page_stride < 0)
    return DSATOPK_ERR_INVALID_ARG;
  const int64_t size = type == DSATOPK_FP8 ? 1 : 2;
  if ((key_page_stride * size) % 16) return DSATOPK_ERR_ALIGNMENT;
  ScoreParams p{};
  p.q = static_cast<const char*>(q);
  p.q_row = q_row_stride * size;
  p.q_head = q_head_stride * size;
  p.weights = weights;
  p.w_row = weight_stride;
  p.keys = static_cast<const char*>(keys);
  p.key_page = key_page_stride * size;
  p.key_token = key_token_stride * size;
  p.scales = key_scales;
  p.scale_page = scale_page_stride;
  p.num_pages = num_pages;
  p.seq_lens = seq_lens;
  p.table = page_table;
  p.table_stride = page_table_stride;
  p.table_rows = table_rows;
  p.page_bits = log2_of(page_size);
  p.table_width = page_table_width;
  p.out = out;
  p.out_stride = out_stride;
  p.rows = num_rows;
  p.heads = num_heads;
  const int64_t most = (int64_t)page_table_width * page_size;
  p.columns = (int32_t)(columns < most ? columns : most);
  return run_scores(p, type, head_dim, true, stream);
}

int dsatopk_scores_ragged(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                          const float* weights, int64_t weight_stride, const void* keys,
                          int64_t num_keys, int64_t key_stride, const float* key_scales,
                          int32_t type, int32_t num_heads, int32_t head_dim,
                          const int32_t* seq_lens, const int32_t* row_starts, int32_t num_rows,
                          float* out, int64_t out_stride, int64_t columns, void* stream) {
  const int st = check_scores(q, q_row_stride, q_head_stride, weights, weight_stride, keys,
                              num_keys, key_stride, seq_lens, type, num_heads, head_dim, num_rows, out,
                              out_stride, columns);
  if (st != DSATOPK_OK || num_rows == 0) return st;
  if (!row_starts || num_keys < 0) return DSATOPK_ERR_INVALID_ARG;
  const int64_t size = type == DSATOPK_FP8 ? 1 : 2;
  ScoreParams p{};
  p.q = static_cast<const char*>(q);
  p.q_row = q_row_stride * size;
  p.q_head = q_head_stride * size;
  p.weights = weights;
  p.w_row = weight_stride;
  p.keys = static_cast<const char*>(keys);
  p.key_token = key_stride * size;
  p.scales = key_scales;
  p.num_pages = num_keys;
  p.seq_lens = seq_lens;
  p.row_starts = row_starts;
  p.out = out;
  p.out_stride = out_stride;
  p.rows = num_rows;
  p.heads = num_heads;
  p.columns = (int32_t)(columns < num_keys ? columns : num_keys);
  return run_scores(p, type, head_dim, false, stream);
}

}  // extern "C"
