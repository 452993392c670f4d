// latent_attend.hip - latent attention in its absorbed form
// (dsatopk_attend_selected and dsatopk_attend_paged in include/dsatopk.h).
//
// Every head of query row b attends to the same cached vectors c[j] =
// (latent, rotary part):
//
//   s[h, j] = scale * q[b, h] . c[j],   out[b, h] = sum_j softmax(s[h, :])[j] * latent(c[j])
//
// over the tokens j that the row reads: its selected slots, or the first
// seq_len positions of its page table's row. A cached vector is read once
// for both products and for all heads of the workgroup.
//
// Both products are computed transposed: S' = C Q' has a head in each lane
// (column) and tokens in its registers (rows), so the softmax's maximum and
// sum are reductions inside a lane but for one or two lane exchanges, and
// the rounded weights are, register for register, the B operand of O' =
// latent' P' (the order of tokens along that contraction is free, and is
// taken as S' leaves it). O' has a head in each lane too: rescaling it is a
// multiplication by the lane's own factor, done only where weights outgrow
// the reference in use (by 2^8; kMost of the type). The A operand of O' needs the
// tile by columns; the LDS column reads give it from the same tile that the
// rows were read from.
//
// A workgroup takes one row, up to 128 heads and a range of tokens (split
// over workgroups when there are few rows; a second kernel joins the parts),
// a tile of 32 or 64 tokens at a time, copied to LDS one tile ahead without
// passing through registers. Its waves are WH groups of 16 heads by WT groups
// of a tile's tokens; token groups keep sums of their own and join them at
// the end. A wave's sums take 128 registers and its queries 72, so eight waves
// fill a CU: for up to 64 heads two workgroups of four, which do not wait for
// each other (1024 rows of 64 heads: 342 us, and 370 as one workgroup of eight
// with tiles of 64 tokens), for more heads one of eight.
//
// 1024 prompt rows of 2048 slots and 64 heads (out of 4 x 16384 tokens) take
// 347 us, 0.84 PFLOP/s: copies and products each take about 300 by themselves
// and overlap in part. 128 decode rows of 128 heads take 117 us (2.9 TB/s), 8 rows
// of 131072 tokens and 16 heads 238 us: 5.1 TB/s, where sums along the rows of a
// 4 GB matrix read 6.2.
//
// Weights are rounded to the inputs' 16-bit type for the second product (off
// by at most 2^-8 of each in bfloat16; in half precision by 2^-11 of each or
// 2^-35 of the row's largest, see kLift); scores, maxima, sums and both
// products' accumulators are fp32.

#include "latent_tiles.h"

namespace dsatopk_serve {
namespace {

struct AttendParams {
  const char* q;
  int64_t q_row, q_head;  // bytes
  Cache cache;
  const int32_t* slots;  // selected form: [rows, slot_stride], the first `selected` of a row
  int64_t slot_stride;
  const int32_t* seq_lens;  // paged form
  const int32_t* table;
  int64_t table_stride;
  const int32_t* table_rows;
  int32_t table_width, selected, blocks;
  float scale2;  // scale * log2 e
  Joined to;
};

template <class T, class P, bool kPaged>
__global__ __launch_bounds__(P::kBlock, P::kOwn ? 1 : 2) void attend_kernel(AttendParams p) {
  __shared__ __attribute__((aligned(1024))) char tiles[2 * P::kBuffer];
  __shared__ uint32_t masks[2][P::kWaves];
  __shared__ float joined[2][P::kWaves][16];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t id = blockIdx.x;
  const int split = id % p.to.splits;
  const int block = (id / p.to.splits) % p.blocks;
  const int64_t row = id / p.to.splits / p.blocks;

  // the tokens of this workgroup
  int32_t len = p.selected;
  const int32_t* list;
  if constexpr (kPaged) {
    const int64_t most = min((int64_t)p.table_width << p.cache.page_bits, (int64_t)(INT32_MAX - P::kTile));
    len = (int32_t)min((int64_t)max(p.seq_lens[row], 0), most);
    list = p.table + (p.table_rows ? p.table_rows[row] : row) * p.table_stride;
  } else {
    list = p.slots + row * p.slot_stride;
  }
  const int32_t tiles_all = (len + P::kTile - 1) / P::kTile;
  const int32_t per = (tiles_all + p.to.splits - 1) / p.to.splits;
  const int32_t first = split * per;
  const int32_t last = min(first + per, tiles_all);

  const Places<P> places(wave, lane);
  State<P> st;
  st.top = -INFINITY;
  st.sum = 0.0f;
#pragma unroll
  for (int b = 0; b < P::kBlocks; ++b) st.o[b] = f32x4{};

  const int head = (block * P::kWH + wave % P::kWH) * 16 + (lane & 15);
  const char* qh = head < p.to.heads ? p.q + row * p.q_row + head * p.q_head : zero_row();
  attend_range<T, P, kPaged, false>(st, tiles, masks, p.cache, list, 0, len, first, last, qh, 0, places,
                                    wave, lane, p.scale2);

  float sum = head_sum(st.sum);
  float top = st.top;
  if constexpr (P::kWT > 1) {
    join_groups<P>(st, top, sum, tiles, joined, wave, lane);
    if (wave / P::kWH > 0) return;
  }
  if (head >= p.to.heads) return;
  put<T, P>(st, top, sum, p.to, row, head, split, lane);
}

// Heads a workgroup: 16, 32, 64 or 128.
int head_block(int32_t heads) { return heads <= 16 ? 16 : heads <= 32 ? 32 : heads <= 64 ? 64 : 128; }

constexpr int kUnit = 64;

// Parts of the token axis. Costs in 64 tokens of one CU's time, which runs one
// workgroup: a part costs its tiles and about kPart more (first loads, last
// sums, the join). Rows as long as they may be go in rounds of 256
// workgroups; rows of mixed lengths end with the longest row's parts, after
// all rows' work has been shared out. The lengths are on the device, so the
// rule weighs both, even rows twice.
int32_t splits_for(int32_t rows, int32_t heads, int64_t tokens) {
  constexpr double kCus = 256, kPart = 3;
  constexpr int kTry[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 24, 32, 48, 64, 96, 128, 192, 256};
  const int hb = head_block(heads);
  const double groups = (double)rows * ((heads + hb - 1) / hb);
  const int64_t tiles = (tokens + kUnit - 1) / kUnit;
  int32_t best = 1;
  double least = 0;
  for (const int s : kTry) {
    if (s > 1 && s > tiles) break;
    const double part = (double)((tiles + s - 1) / s) + kPart;
    const double rounds = (double)(int64_t)((groups * s + kCus - 1) / kCus);
    const double cost = 2 * rounds * part + part + groups * ((double)tiles + s * kPart) / kCus;
    if (s == 1 || cost < least) {
      best = s;
      least = cost;
    }
  }
  return best;
}

template <class T, class P, bool kPaged>
int launch_plan(const AttendParams& p, void* stream) {
  const dim3 grid((unsigned)((int64_t)p.to.rows * p.blocks * p.to.splits));
  return launch(attend_kernel<T, P, kPaged>, grid, dim3(P::kBlock), p, stream);
}

template <class T, int kLatent, bool kPaged>
int launch_attend(AttendParams p, void* stream) {
  const int hb = head_block(p.to.heads);
  p.blocks = (p.to.heads + hb - 1) / hb;
  const int st = hb == 16   ? launch_plan<T, Plan<1, 4, 64, kLatent>, kPaged>(p, stream)
                 : hb == 32 ? launch_plan<T, Plan<2, 2, 32, kLatent>, kPaged>(p, stream)
                 : hb == 64 ? launch_plan<T, Plan<4, 1, 32, kLatent>, kPaged>(p, stream)
                            : launch_plan<T, Plan<8, 1, 64, kLatent>, kPaged>(p, stream);
  if (st != DSATOPK_OK || p.to.splits == 1) return st;
  return launch_join<T, kLatent>(p.to, stream);
}

// Checks and fills what both forms share; `tokens` bounds a row's tokens.
int check_attend(AttendParams& p, const void* q, int64_t q_row, int64_t q_head, const void* cache,
                 int64_t num_pages, int64_t page_stride, int64_t token_stride, int32_t page_size,
                 int32_t type, int32_t heads, int32_t latent, int32_t rope, float scale,
                 int32_t rows, int64_t tokens, void* out, float* lse, void* workspace,
                 size_t workspace_bytes) {
  if (rows < 0 || heads < 1 || heads > 1024 || (latent != 256 && latent != 512) || rope != kRope ||
      (type != DSATOPK_BF16 && type != DSATOPK_FP16) || !(scale > 0.0f) || !(scale < INFINITY) ||
      num_pages < 0 || page_stride < 0 || token_stride < 0 || !pow2(page_size) ||
      page_size > (1 << 20) || q_row < 0 || q_head < 0 || tokens < 0 || tokens > INT32_MAX - kUnit)
    return DSATOPK_ERR_INVALID_ARG;
  if (rows == 0) return DSATOPK_OK;
  if (!q || !out || (num_pages && !cache)) return DSATOPK_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(cache) || (reinterpret_cast<uintptr_t>(out) & 7u) ||
      !aligned4(lse) || q_row % 8 || q_head % 8 || page_stride % 8 || token_stride % 8)
    return DSATOPK_ERR_ALIGNMENT;
  p.to.splits = splits_for(rows, heads, tokens);
  if (p.to.splits > 1) {
    if (!workspace || workspace_bytes < part_floats(rows, heads, latent, p.to.splits) * sizeof(float))
      return DSATOPK_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned16(workspace)) return DSATOPK_ERR_ALIGNMENT;
    p.to.part = static_cast<float*>(workspace);
    p.to.state = p.to.part + (size_t)rows * p.to.splits * heads * latent;
  }
  p.q = static_cast<const char*>(q);
  p.q_row = q_row * 2;
  p.q_head = q_head * 2;
  p.cache.at = static_cast<const char*>(cache);
  p.cache.page = page_stride * 2;
  p.cache.token = token_stride * 2;
  p.cache.pages = num_pages;
  p.cache.page_bits = log2_of(page_size);
  p.to.rows = rows;
  p.to.heads = heads;
  p.scale2 = scale * kLog2e;
  p.to.out = static_cast<char*>(out);
  p.to.lse = lse;
  return DSATOPK_OK;
}

template <bool kPaged>
int run_attend(const AttendParams& p, int32_t type, int32_t latent, void* stream) {
  if (type == DSATOPK_BF16)
    return latent == 256 ? launch_attend<Bf16, 256, kPaged>(p, stream)
                         : launch_attend<Bf16, 512, kPaged>(p, stream);
  return latent == 256 ? launch_attend<Fp16, 256, kPaged>(p, stream)
                       : launch_attend<Fp16, 512, kPaged>(p, stream);
}

}  // namespace
}  // namespace dsatopk_serve

using namespace dsatopk_serve;

extern "C" {

size_t dsatopk_attend_bytes(int32_t num_rows, int32_t num_heads, int32_t latent_dim,
                            int64_t max_tokens) {
  if (num_rows < 1 || num_heads < 1 || latent_dim < 1 || max_tokens < 0) return 0;
  return part_floats(num_rows, num_heads, latent_dim,
                     splits_for(num_rows, num_heads, max_tokens)) * sizeof(float);
}

int dsatopk_attend_selected(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                            const void* cache, int64_t num_pages, int64_t page_stride,
                            int64_t token_stride, int32_t page_size, int32_t type,
                            int32_t num_heads, int32_t latent_dim, int32_t rope_dim, float scale,
                            const int32_t* slots, int64_t slot_stride, int32_t k,
                            int32_t num_rows, void* out, float* lse, void* workspace,
                            size_t workspace_bytes, void* stream) {
  AttendParams p{};
  if (k < 0 || slot_stride < k || (num_rows > 0 && k && !slots)) return DSATOPK_ERR_INVALID_ARG;
  const int st = check_attend(p, q, q_row_stride, q_head_stride, cache, num_pages, page_stride,
                              token_stride, page_size, type, num_heads, latent_dim, rope_dim,
                              scale, num_rows, k, out, lse, workspace, workspace_bytes);
  if (st != DSATOPK_OK || num_rows == 0) return st;
  p.slots = slots;
  p.slot_stride = slot_stride;
  p.selected = k;
  return run_attend<false>(p, type, latent_dim, stream);
}

int dsatopk_attend_paged(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                         const void* cache, int64_t num_pages, int64_t page_stride,
                         int64_t token_stride, int32_t page_size, int32_t type, int32_t num_heads,
                         int32_t latent_dim, int32_t rope_dim, float scale,
                         const int32_t* seq_lens, const int32_t* page_table,
                         int64_t page_table_stride, int32_t page_table_width,
                         const int32_t* table_rows, int64_t max_seq_len, int32_t num_rows,
                         void* out, float* lse, void* workspace, size_t workspace_bytes,
                         void* stream) {
  AttendParams p{};
  if (page_table_width < 1 || page_table_stride < page_table_width ||
      (num_rows > 0 && (!seq_lens || !page_table)))
    return DSATOPK_ERR_INVALID_ARG;
  const int st = check_attend(p, q, q_row_stride, q_head_stride, cache, num_pages, page_stride,
                              token_stride, page_size, type, num_heads, latent_dim, rope_dim,
                              scale, num_rows, max_seq_len, out, lse, workspace, workspace_bytes);
  if (st != DSATOPK_OK || num_rows == 0) return st;
  p.seq_lens = seq_lens;
  p.table = page_table;
  p.table_stride = page_table_stride;
  p.table_rows = table_rows;
  p.table_width = page_table_width;
  return run_attend<true>(p, type, latent_dim, stream);
}

}  // extern "C"
