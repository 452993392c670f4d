// expanded_attend.hip - latent attention in its expanded form
// (dsatopk_attend_expanded in include/dsatopk.h), for prompts:
//
//   s[i, j] = scale * (q[i, h][:128] . k[j, h] + q[i, h][128:] . k_rope[j])
//   out[i, h] = sum_j softmax(s[i, :])[j] * v[j, h]
//
// over a ragged batch: request r's queries are rows q_starts[r] ..
// q_starts[r + 1] - 1, its keys rows k_starts[r] .. k_starts[r + 1] - 1, and
// query i (of n) sees the keys up to its own place counted from the end (the
// last query sees all). The rotary key is one for all heads: it is
// read from its own tensor instead of being copied into every head's key.
//
// A workgroup takes kRows queries of one head and goes over the keys, kTile
// at a time, copied to LDS one tile ahead. Both products are transposed: S' = K
// Q' has a query in each lane and keys in its registers, which are, rounded,
// the B operand of O' = V' P'; V's columns come from LDS column reads. See
// latent_attend.hip, whose tile is the same but for its sharing one tensor.
// Queries stay in registers throughout.
//
// Weights are rounded to the inputs' type for the second product; scores,
// maxima, sums and accumulators are fp32.

#include "serve_common.h"

namespace dsatopk_serve {
namespace {

constexpr int kBlock = 256;
constexpr int kWaves = kBlock / 64;
constexpr int kRows = 32 * kWaves;
constexpr int kTile = 64;
constexpr int kNope = 128, kRope = 64, kValue = 128;
constexpr int kKeyBytes = kNope * 2, kRopeBytes = kRope * 2, kValueBytes = kValue * 2;
constexpr int kRopeAt = kTile * kKeyBytes, kValueAt = kRopeAt + kTile * kRopeBytes;
constexpr int kBuffer = kValueAt + kTile * kValueBytes;
constexpr int kSteps = (kNope + kRope) / 16;
constexpr int kBlocks = kValue / 32;
constexpr float kGrow = 8.0f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct ExpandParams {
  const char* q;
  int64_t q_row, q_head;  // bytes, all of them
  const char* k;
  int64_t k_row, k_head;
  const char* v;
  int64_t v_row, v_head;
  const char* rope;
  int64_t rope_row;
  const int32_t* q_starts;
  const int32_t* k_starts;
  int32_t requests, heads, tiles, num_q, num_k, causal;
  float scale2;
  char* out;
  float* lse;
};

// Copies keys j0 .. j0 + 63 (of the request's `keys`; rows past them repeat
// the last) of all three tensors, swizzled: a wave takes 16.
__device__ __forceinline__ void copy_tile(const ExpandParams& p, char* tile, const char* k,
                                          const char* v, const char* rope, int32_t j0,
                                          int32_t keys, int wave, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = wave * 16 + i * 4 + (lane >> 4);
    const int64_t j = min(j0 + t, keys - 1);
    const int at = ((lane & 15) ^ swizzle32(t)) * 16;
    copy_to_lds(k + j * p.k_row + at, tile + (wave * 16 + i * 4) * kKeyBytes);
    copy_to_lds(v + j * p.v_row + at, tile + kValueAt + (wave * 16 + i * 4) * kValueBytes);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = wave * 16 + i * 8 + (lane >> 3);
    const int64_t j = min(j0 + t, keys - 1);
    copy_to_lds(rope + j * p.rope_row + ((lane & 7) ^ swizzle8(t)) * 16,
                tile + kRopeAt + (wave * 16 + i * 8) * kRopeBytes);
  }
}

struct State {
  f32x16 o[kBlocks];
  float top, sum;
};

// One tile of 64 keys for the wave's 32 queries, and first the next tile's
// copies. `seen`: how many of the tile's keys this lane's query sees (may be
// negative or above 64); `whole`: all of them, for every lane of the wave.
template <class T>
__device__ __forceinline__ void tile_step(const ExpandParams& p, State& st,
                                          const u32x4 (&q)[kSteps], const char* __restrict__ cur,
                                          char* __restrict__ next, const char* k, const char* v,
                                          const char* rope, int32_t next_j, int32_t keys,
                                          int32_t seen, bool whole, int wave, int lane) {
  if (next_j < keys) copy_tile(p, next, k, v, rope, next_j, keys, wave, lane);
  const int col = lane & 31, half = lane >> 5;
  f32x16 s[2] = {};
  {
    const int swz = swizzle32(col);
    const char* row = cur + col * kKeyBytes;
    const char* tail = cur + kRopeAt + col * kRopeBytes;
#pragma unroll
    for (int i = 0; i < kNope / 16; ++i)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        s[x] = T::mma32(*reinterpret_cast<const u32x4*>(row + (((2 * i + half) ^ swz) << 4) + x * 32 * kKeyBytes),
                        q[i], s[x]);
#pragma unroll
    for (int i = 0; i < kRope / 16; ++i)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        s[x] = T::mma32(*reinterpret_cast<const u32x4*>(tail + (((2 * i + half) ^ swizzle8(col)) << 4) + x * 32 * kRopeBytes),
                        q[kNope / 16 + i], s[x]);
  }
  if (!whole) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (x * 32 + 8 * (i / 4) + 4 * half + i % 4 >= seen) s[x][i] = -INFINITY;
  }
  float top = s[0][0];
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, s[x][i]);
  top = fmaxf(top, other_half(top)) * p.scale2;
  if (__any(top > st.top + kGrow)) {
    const float to = fmaxf(st.top, top);
    const float by = st.top == -INFINITY ? 0.0f : exp2_fast(st.top - to);
    st.top = to;
    st.sum *= by;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) st.o[b] *= by;
  }
  const float ref = st.top == -INFINITY ? 0.0f : st.top;
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[x][i] = exp2_fast(fmaf(s[x][i], p.scale2, -ref));
      st.sum += s[x][i];
    }
  // lane i of 16 points at row i / 4, 8 bytes i % 4 of a 4 x 32 byte block
  const int in = lane & 15, side = (lane >> 4) & 1;
  const int tok = 4 * half + (in >> 2);
  const int swz = swizzle32(tok);
  int at[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    at[j] = tok * kValueBytes + (((4 * j + 2 * side + ((in & 3) >> 1)) ^ swz) << 4) + 8 * (in & 1);
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const u32x4 w = {T::pack(s[x][8 * g], s[x][8 * g + 1]), T::pack(s[x][8 * g + 2], s[x][8 * g + 3]),
                       T::pack(s[x][8 * g + 4], s[x][8 * g + 5]), T::pack(s[x][8 * g + 6], s[x][8 * g + 7])};
      const char* rows = cur + kValueAt + (x * 32 + g * 16) * kValueBytes;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        const u32x2 lo = read_columns(rows + at[b]);
        const u32x2 hi = read_columns(rows + (at[b] ^ 32) + 8 * kValueBytes);  // swizzle32(t + 8) = swizzle32(t) ^ 2
        st.o[b] = T::mma32(u32x4{lo[0], lo[1], hi[0], hi[1]}, w, st.o[b]);
      }
    }
}

template <class T>
__global__ __launch_bounds__(kBlock, 2) void expand_kernel(ExpandParams p) {
  __shared__ __attribute__((aligned(1024))) char tiles[2 * kBuffer];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, half = lane >> 5;

  // Workgroup -> (request and head, rows). Neighbouring numbers run on
  // different XCDs: the row tiles of one head, which read the same keys, are
  // 8 apart so that they share an L2. Late rows see most keys: they go first.
  const uint32_t pairs = (uint32_t)(p.requests * p.heads);
  const uint32_t id = blockIdx.x;
  const uint32_t pair = id / (8 * p.tiles) * 8 + id % 8;
  if (pair >= pairs) return;
  const int tile = p.tiles - 1 - (int)(id / 8 % p.tiles);
  const int r = pair / p.heads, head = pair % p.heads;

  const int32_t q0 = max(p.q_starts[r], 0), q1 = min(p.q_starts[r + 1], p.num_q);
  const int32_t k0 = max(p.k_starts[r], 0), k1 = min(p.k_starts[r + 1], p.num_k);
  const int32_t rows = q1 - q0, keys = max(k1 - k0, 0);
  const int32_t first = tile * kRows;
  if (first >= rows) return;

  const int32_t row = first + wave * 32 + col;  // of the request
  const int64_t at = q0 + min(row, rows - 1);
  // Keys that the row sees, and the most and the fewest that any of the workgroup's (wave's) sees.
  auto sees = [&](int32_t i) {
    return p.causal ? min(max(i + 1 + keys - rows, 0), keys) : keys;
  };
  const int32_t mine = sees(row < rows ? row : rows - 1);
  const int32_t most = sees(min(first + kRows, rows) - 1);
  const int32_t least = sees(min(first + wave * 32, rows - 1));

  u32x4 q[kSteps];
  const char* qh = p.q + at * p.q_row + head * p.q_head;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) q[i] = *reinterpret_cast<const u32x4*>(qh + (2 * i + half) * 16);

  State st;
  st.top = -INFINITY;
  st.sum = 0.0f;
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) st.o[b] = f32x16{};

  const char* k = p.k + k0 * p.k_row + head * p.k_head;
  const char* v = p.v + k0 * p.v_row + head * p.v_head;
  const char* rope = p.rope + k0 * p.rope_row;
  if (most > 0) copy_tile(p, tiles, k, v, rope, 0, keys, wave, lane);
  int buf = 0;
  for (int32_t j = 0; j < most; j += kTile) {
    copies_barrier();
    tile_step<T>(p, st, q, tiles + buf * kBuffer, tiles + (buf ^ 1) * kBuffer, k, v, rope,
                 j + kTile < most ? j + kTile : keys, keys, mine - j, least >= j + kTile, wave, lane);
    buf ^= 1;
  }
  if (row >= rows) return;
  const float sum = st.sum + other_half(st.sum);
  const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
  char* to = p.out + ((at * p.heads + head) * kValue + 4 * half) * 2;
#pragma unroll
  for (int b = 0; b < kBlocks; ++b)
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *reinterpret_cast<u32x2*>(to + (b * 32 + 2 * i) * 2) =
          u32x2{T::pack(st.o[b][i] * by, st.o[b][i + 1] * by),
                T::pack(st.o[b][i + 2] * by, st.o[b][i + 3] * by)};
  if (p.lse && half == 0) p.lse[at * p.heads + head] = (st.top + log2f(sum)) * kLn2;
}

}  // namespace
}  // namespace dsatopk_serve

using namespace dsatopk_serve;

extern "C" int dsatopk_attend_expanded(
    const void* q, int64_t q_row_stride, int64_t q_head_stride, const void* k,
    int64_t k_row_stride, int64_t k_head_stride, const void* v, int64_t v_row_stride,
    int64_t v_head_stride, const void* k_rope, int64_t rope_row_stride, int32_t type,
    int32_t num_heads, int32_t nope_dim, int32_t rope_dim, int32_t value_dim, float scale,
    int32_t causal, const int32_t* q_starts, const int32_t* k_starts, int32_t num_requests,
    int32_t num_queries, int32_t num_keys, int32_t max_queries, void* out, float* lse,
    void* stream) {
  if (num_requests < 0 || num_queries < 0 || num_keys < 0 || max_queries < 0 || num_heads < 1 ||
      num_heads > 1024 || nope_dim != kNope || rope_dim != kRope || value_dim != kValue ||
      (type != DSATOPK_BF16 && type != DSATOPK_FP16) || !(scale > 0.0f) || !(scale < INFINITY) ||
      q_row_stride < 0 || q_head_stride < 0 || k_row_stride < 0 || k_head_stride < 0 ||
      v_row_stride < 0 || v_head_stride < 0 || rope_row_stride < 0)
    return DSATOPK_ERR_INVALID_ARG;
  if (num_requests == 0 || num_queries == 0 || max_queries == 0) return DSATOPK_OK;
  if (!q || !out || !q_starts || !k_starts || (num_keys && (!k || !v || !k_rope)))
    return DSATOPK_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(k_rope) ||
      (reinterpret_cast<uintptr_t>(out) & 7u) || !aligned4(lse) || q_row_stride % 8 ||
      q_head_stride % 8 || k_row_stride % 8 || k_head_stride % 8 || v_row_stride % 8 ||
      v_head_stride % 8 || rope_row_stride % 8)
    return DSATOPK_ERR_ALIGNMENT;
  ExpandParams p{};
  p.q = static_cast<const char*>(q);
  p.q_row = q_row_stride * 2;
  p.q_head = q_head_stride * 2;
  p.k = static_cast<const char*>(k);
  p.k_row = k_row_stride * 2;
  p.k_head = k_head_stride * 2;
  p.v = static_cast<const char*>(v);
  p.v_row = v_row_stride * 2;
  p.v_head = v_head_stride * 2;
  p.rope = static_cast<const char*>(k_rope);
  p.rope_row = rope_row_stride * 2;
  p.q_starts = q_starts;
  p.k_starts = k_starts;
  p.requests = num_requests;
  p.heads = num_heads;
  p.num_q = num_queries;
  p.num_k = num_keys;
  p.causal = causal != 0;
  p.scale2 = scale * kLog2e;
  p.out = static_cast<char*>(out);
  p.lse = lse;
  const int32_t longest = max_queries < num_queries ? max_queries : num_queries;
  p.tiles = (longest + kRows - 1) / kRows;
  const int64_t groups = ((int64_t)num_requests * num_heads + 7) / 8 * 8 * p.tiles;
  if (groups > INT32_MAX) return DSATOPK_ERR_INVALID_ARG;
  const dim3 grid((unsigned)groups);
  return type == DSATOPK_BF16 ? launch(expand_kernel<Bf16>, grid, dim3(kBlock), p, stream)
                              : launch(expand_kernel<Fp16>, grid, dim3(kBlock), p, stream);
}
