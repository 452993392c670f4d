// shared_attend.hip - latent attention in its absorbed form for rows that share
// their first tokens (dsatopk_attend_shared in include/dsatopk.h).
//
// Row b of group g attends to len_b tokens. The first shared_g of them are the
// same cached vectors for every row of the group, so they are read once for
// all rows' heads; the others are the row's own. With the partial sums over a
// set J of tokens, by a reference m,
//
//   n_J = sum_j exp(s_j - m),   o_J = sum_j exp(s_j - m) * latent(c_j)
//
// the row's result is the quotient of the sums over its sets, each brought to
// the largest reference. One launch computes the parts (the shared tokens of
// each group's heads, the own tokens of each row), a second one joins them.
//
// The shared parts are products of all heads of several rows, packed 16 a wave
// and up to 128 a workgroup, with a head of its own row in each lane; a lane
// counts how many of the tokens its row sees (drafted tokens, whose rows see
// one token more each). Tiles, products and softmax are those of one row's heads
// (latent_tiles.h).

#include "latent_tiles.h"

namespace dsatopk_serve {
namespace {

struct SharedParams {
  const char* q;
  int64_t q_row, q_head;  // bytes
  Cache cache;
  const int32_t* seq_lens;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* table_rows;
  const int32_t* group_starts;
  const int32_t* shared_lens;
  int32_t groups, table_width;
  int32_t shared_splits, own_splits, own_blocks;
  uint32_t slots, shared_jobs;  // blocks of lanes that the groups may have, workgroups for them
  float scale2;
  Joined to;
};

// First row of group g; the first group starts at row 0 and the last one ends
// behind the last row, whatever the list says.
__device__ __forceinline__ int32_t start_of(const SharedParams& p, int32_t g) {
  return g <= 0 ? 0 : g >= p.groups ? p.to.rows : min(max(p.group_starts[g], 0), p.to.rows);
}

__device__ __forceinline__ int32_t positions(const SharedParams& p) {
  return (int32_t)min((int64_t)p.table_width << p.cache.page_bits, (int64_t)(INT32_MAX - 64));
}

__device__ __forceinline__ int32_t shared_of(const SharedParams& p, int32_t g) {
  return p.shared_splits ? min(max(p.shared_lens[g], 0), positions(p)) : 0;
}

__device__ __forceinline__ int32_t length_of(const SharedParams& p, int64_t row) {
  return min(max(p.seq_lens[row], 0), positions(p));
}

__device__ __forceinline__ const int32_t* pages_of(const SharedParams& p, int64_t row) {
  return p.table + (p.table_rows ? p.table_rows[row] : row) * p.table_stride;
}

template <class P>
__device__ __forceinline__ void clear(State<P>& st) {
  st.top = -INFINITY;
  st.sum = 0.0f;
#pragma unroll
  for (int b = 0; b < P::kBlocks; ++b) st.o[b] = f32x4{};
}

// This workgroup's share of `tiles` tiles, part `split` of `splits`.
__device__ __forceinline__ void share(int32_t tiles, int32_t splits, int32_t split, int32_t& first,
                                      int32_t& last) {
  const int32_t per = (tiles + splits - 1) / splits;
  first = min(split * per, tiles);
  last = min(first + per, tiles);
}

// Part `split` of a group's shared tokens, for block `slot` of lanes. Group g's
// blocks begin at number start_g * heads / lanes + g, which leaves room
// for all of them.
template <class T, class P>
__device__ __forceinline__ void shared_part(const SharedParams& p, char* tiles,
                                            uint32_t (*masks)[P::kWaves], float (*joined)[P::kWaves][16],
                                            uint32_t slot, int32_t split, int wave, int lane) {
  constexpr int kLanes = P::kWH * 16;
  const int32_t heads = p.to.heads;
  auto first_slot = [&](int32_t g) { return (int64_t)start_of(p, g) * heads / kLanes + g; };
  const int32_t g = last_below(p.groups, slot, lane, first_slot);
  const int32_t row0 = start_of(p, g), rows = start_of(p, g + 1) - row0;
  const int64_t begin = ((int64_t)slot - first_slot(g)) * kLanes, lanes = (int64_t)rows * heads;
  if (begin < 0 || begin >= lanes) return;  // starts that do not rise may say anything
  const int32_t shared = shared_of(p, g);

  // Lane i of the block: its row, its head, the tokens that it sees.
  const int32_t row1 = row0 + (int32_t)(begin / heads), head1 = (int32_t)(begin % heads);
  const int32_t count = (int32_t)min(lanes - begin, (int64_t)kLanes);
  auto row_of = [&](int32_t i) { return row1 + (head1 + i) / heads; };
  auto sees = [&](int32_t i) { return min(length_of(p, row_of(i)), shared); };
  int32_t most = 0;
#pragma unroll
  for (int i = 0; i < kLanes; i += 64)
    if (i + lane < count) most = max(most, sees(i + lane));
#pragma unroll
  for (int d = 32; d; d >>= 1) most = max(most, __shfl_xor(most, d));
  most = __builtin_amdgcn_readfirstlane(most);

  int32_t first, last;
  share((most + P::kTile - 1) / P::kTile, p.shared_splits, split, first, last);
  State<P> st;
  clear<P>(st);
  {
    const int32_t i = wave % P::kWH * 16 + (lane & 15);
    const bool real = i < count;
    const int32_t mine = real ? sees(i) : INT32_MAX;
    const char* qh = real ? p.q + row_of(i) * p.q_row + (head1 + i) % heads * p.q_head : zero_row();
    // a lane that sees nothing of these tokens must not ask for a reference at every tile
    if (mine <= first * P::kTile) st.top = 0.0f;
    const Places<P> places(wave, lane);
    attend_range<T, P, true, true>(st, tiles, masks, p.cache, pages_of(p, row0), 0, most, first, last,
                                   qh, mine, places, wave, lane, p.scale2);
  }
  // which lane this is, anew: until here the registers are the tokens'
  const int32_t i = wave % P::kWH * 16 + (here(lane) & 15);
  const bool real = i < count;
  const int64_t row = row_of(i);
  const int head = (head1 + i) % heads;
  float sum = head_sum(st.sum);
  float top = real && sees(i) <= first * P::kTile ? -INFINITY : st.top;
  if constexpr (P::kWT > 1) {
    join_groups<P>(st, top, sum, tiles, joined, wave, lane);
    if (wave / P::kWH > 0) return;
  }
  if (real) put<T, P>(st, top, sum, p.to, row, head, split, lane);
}

// Part `split` of a row's own tokens, for block `block` of its heads.
template <class T, class P>
__device__ __forceinline__ void own_part(const SharedParams& p, char* tiles, uint32_t (*masks)[P::kWaves],
                                         float (*joined)[P::kWaves][16], int64_t row, int32_t block,
                                         int32_t split, int wave, int lane) {
  const int32_t g = last_below(p.groups, row, lane, [&](int32_t i) { return (int64_t)start_of(p, i); });
  const int32_t len = length_of(p, row), base = min(shared_of(p, g), len);
  int32_t first, last;
  share((len - base + P::kTile - 1) / P::kTile, p.own_splits, split, first, last);
  State<P> st;
  clear<P>(st);
  {
    const int head = (block * P::kWH + wave % P::kWH) * 16 + (lane & 15);
    const char* qh = head < p.to.heads ? p.q + row * p.q_row + head * p.q_head : zero_row();
    const Places<P> places(wave, lane);
    attend_range<T, P, true, false>(st, tiles, masks, p.cache, pages_of(p, row), base, len - base, first,
                                    last, qh, 0, places, wave, lane, p.scale2);
  }
  const int head = (block * P::kWH + wave % P::kWH) * 16 + (here(lane) & 15);
  float sum = head_sum(st.sum);
  float top = st.top;
  if constexpr (P::kWT > 1) {
    join_groups<P>(st, top, sum, tiles, joined, wave, lane);
    if (wave / P::kWH > 0) return;
  }
  if (head < p.to.heads) put<T, P>(st, top, sum, p.to, row, head, p.shared_splits + split, lane);
}

// PS for the shared parts, PO for the own ones: workgroups of the same size.
template <class T, class PS, class PO>
__global__ __launch_bounds__(PS::kBlock, 2) void shared_kernel(SharedParams p) {
  static_assert(PS::kBlock == PO::kBlock && PS::kBuffer == PO::kBuffer, "one launch for both");
  __shared__ __attribute__((aligned(1024))) char tiles[2 * PS::kBuffer];
  __shared__ uint32_t masks[2][PS::kWaves];
  __shared__ float joined[2][PS::kWaves][16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  uint32_t id = blockIdx.x;
  if (id < p.shared_jobs) {
    // Blocks that read the same tokens are 8 apart, on one XCD, where there
    // are that many parts.
    const uint32_t each = p.shared_splits % 8 ? p.shared_splits : 8;
    const uint32_t slot = id / each % p.slots;
    const int32_t split = id / each / p.slots * each + id % each;
    shared_part<T, PS>(p, tiles, masks, joined, slot, split, wave, lane);
  } else {
    id -= p.shared_jobs;
    const int32_t split = id % p.own_splits, block = id / p.own_splits % p.own_blocks;
    own_part<T, PO>(p, tiles, masks, joined, id / p.own_splits / p.own_blocks, block, split, wave, lane);
  }
}

// How a call is cut: heads packed into a workgroup for the shared tokens, and
// parts of the token axes.
struct Cut {
  int32_t lanes, shared_splits, own_splits;
};

int head_block(int32_t heads) { return heads <= 32 ? 32 : heads <= 64 ? 64 : 128; }

Cut cut_of(int32_t rows, int32_t heads, int32_t groups, int64_t max_shared, int64_t max_own) {
  constexpr int kUnit = 64;
  constexpr double kPart = 4;
  constexpr int kTry[] = {1, 2, 4, 8, 16, 24, 32, 40, 48, 64, 96, 128};
  const int64_t each = ((int64_t)rows + groups - 1) / groups * heads;  // lanes of a mean group
  Cut c;
  c.lanes = each <= 32 ? 32 : each <= 64 ? 64 : 128;
  const int hb = head_block(heads) < c.lanes ? head_block(heads) : c.lanes;
  const double places = c.lanes == 128 ? 256 : 512;
  const double blocks = (double)groups * ((each + c.lanes - 1) / c.lanes);
  const double own = (double)rows * ((heads + hb - 1) / hb);
  const int64_t shared_tiles = (max_shared + kUnit - 1) / kUnit, own_tiles = (max_own + kUnit - 1) / kUnit;
  double least = -1;
  c.shared_splits = 0;
  c.own_splits = 1;
  for (const int s : kTry) {
    if (s > 1 && s > shared_tiles) break;
    for (const int o : kTry) {
      if (o > 1 && o > own_tiles) break;
      const double a = max_shared ? (double)((shared_tiles + s - 1) / s) + kPart : 0;
      const double b = max_own ? (double)((own_tiles + o - 1) / o) + kPart : 0;
      const double work = blocks * s * a + own * o * b;
      const double cost = work / places + (a > b ? a : b);
      if (least < 0 || cost < least) {
        least = cost;
        c.shared_splits = max_shared ? s : 0;
        c.own_splits = max_own || !max_shared ? o : 0;
      }
    }
  }
  return c;
}

template <class T, class PS, class PO>
int launch_parts(SharedParams p, void* stream) {
  const int64_t slots = (int64_t)p.to.rows * p.to.heads / (PS::kWH * 16) + p.groups;
  p.own_blocks = (p.to.heads + PO::kWH * 16 - 1) / (PO::kWH * 16);
  const int64_t shared = slots * p.shared_splits;
  const int64_t own = (int64_t)p.to.rows * p.own_blocks * p.own_splits;
  if (shared + own > INT32_MAX) return DSATOPK_ERR_INVALID_ARG;
  p.slots = (uint32_t)slots;
  p.shared_jobs = (uint32_t)shared;
  return launch(shared_kernel<T, PS, PO>, dim3((unsigned)(shared + own)), dim3(PS::kBlock), p, stream);
}

template <class T, int kLatent>
int launch_shared(const SharedParams& p, int32_t lanes, void* stream) {
  const int hb = head_block(p.to.heads);
  const int st =
      lanes == 32 ? launch_parts<T, Plan<2, 2, 32, kLatent>, Plan<2, 2, 32, kLatent>>(p, stream)
      : lanes == 64 ? hb == 32 ? launch_parts<T, Plan<4, 1, 32, kLatent>, Plan<2, 2, 32, kLatent>>(p, stream)
                               : launch_parts<T, Plan<4, 1, 32, kLatent>, Plan<4, 1, 32, kLatent>>(p, stream)
      : hb == 32 ? launch_parts<T, Plan<8, 1, 64, kLatent>, Plan<2, 4, 64, kLatent>>(p, stream)
      : hb == 64 ? launch_parts<T, Plan<8, 1, 64, kLatent>, Plan<4, 2, 64, kLatent>>(p, stream)
                 : launch_parts<T, Plan<8, 1, 64, kLatent>, Plan<8, 1, 64, kLatent>>(p, stream);
  if (st != DSATOPK_OK || p.to.splits == 1) return st;
  return launch_join<T, kLatent>(p.to, stream);
}

}  // namespace
}  // namespace dsatopk_serve

using namespace dsatopk_serve;

extern "C" {

size_t dsatopk_shared_bytes(int32_t num_rows, int32_t num_heads, int32_t latent_dim,
                            int32_t num_groups, int64_t max_shared_len, int64_t max_own_len) {
  if (num_rows < 1 || num_heads < 1 || latent_dim < 1 || num_groups < 1 || max_shared_len < 0 ||
      max_own_len < 0)
    return 0;
  const Cut c = cut_of(num_rows, num_heads, num_groups, max_shared_len, max_own_len);
  return part_floats(num_rows, num_heads, latent_dim, c.shared_splits + c.own_splits) * sizeof(float);
}

int dsatopk_attend_shared(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                          const void* cache, int64_t num_pages, int64_t page_stride,
                          int64_t token_stride, int32_t page_size, int32_t type, int32_t num_heads,
                          int32_t latent_dim, int32_t rope_dim, float scale, const int32_t* seq_lens,
                          const int32_t* page_table, int64_t page_table_stride,
                          int32_t page_table_width, const int32_t* table_rows,
                          const int32_t* group_starts, const int32_t* shared_lens,
                          int32_t num_groups, int64_t max_shared_len, int64_t max_own_len,
                          int32_t num_rows, void* out, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream) {
  SharedParams p{};
  if (num_rows < 0 || num_heads < 1 || num_heads > 1024 || (latent_dim != 256 && latent_dim != 512) ||
      rope_dim != kRope || (type != DSATOPK_BF16 && type != DSATOPK_FP16) || !(scale > 0.0f) ||
      !(scale < INFINITY) || num_pages < 0 || page_stride < 0 || token_stride < 0 ||
      !pow2(page_size) || page_size > (1 << 20) || q_row_stride < 0 || q_head_stride < 0 ||
      page_table_width < 1 || page_table_stride < page_table_width || num_groups < 0 ||
      max_shared_len < 0 || max_own_len < 0 || max_shared_len > INT32_MAX - 64 ||
      max_own_len > INT32_MAX - 64)
    return DSATOPK_ERR_INVALID_ARG;
  if (num_rows == 0) return DSATOPK_OK;
  if (!q || !out || (num_pages && !cache) || !seq_lens || !page_table || num_groups < 1 ||
      !group_starts || !shared_lens)
    return DSATOPK_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(cache) || (reinterpret_cast<uintptr_t>(out) & 7u) ||
      !aligned4(lse) || q_row_stride % 8 || q_head_stride % 8 || page_stride % 8 || token_stride % 8)
    return DSATOPK_ERR_ALIGNMENT;
  const Cut c = cut_of(num_rows, num_heads, num_groups, max_shared_len, max_own_len);
  p.shared_splits = c.shared_splits;
  p.own_splits = c.own_splits;
  p.to.splits = c.shared_splits + c.own_splits;
  if (p.to.splits > 1) {
    if (!workspace ||
        workspace_bytes < part_floats(num_rows, num_heads, latent_dim, p.to.splits) * sizeof(float))
      return DSATOPK_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned16(workspace)) return DSATOPK_ERR_ALIGNMENT;
    p.to.part = static_cast<float*>(workspace);
    p.to.state = p.to.part + (size_t)num_rows * p.to.splits * num_heads * latent_dim;
  }
  p.q = static_cast<const char*>(q);
  p.q_row = q_row_stride * 2;
  p.q_head = q_head_stride * 2;
  p.cache.at = static_cast<const char*>(cache);
  p.cache.page = page_stride * 2;
  p.cache.token = token_stride * 2;
  p.cache.pages = num_pages;
  p.cache.page_bits = log2_of(page_size);
  p.seq_lens = seq_lens;
  p.table = page_table;
  p.table_stride = page_table_stride;
  p.table_rows = table_rows;
  p.table_width = page_table_width;
  p.group_starts = group_starts;
  p.shared_lens = shared_lens;
  p.groups = num_groups;
  p.scale2 = scale * kLog2e;
  p.to.rows = num_rows;
  p.to.heads = num_heads;
  p.to.out = static_cast<char*>(out);
  p.to.lse = lse;
  if (type == DSATOPK_BF16)
    return latent_dim == 256 ? launch_shared<Bf16, 256>(p, c.lanes, stream)
                             : launch_shared<Bf16, 512>(p, c.lanes, stream);
  return latent_dim == 256 ? launch_shared<Fp16, 256>(p, c.lanes, stream)
                           : launch_shared<Fp16, 512>(p, c.lanes, stream);
}

}  // extern "C"
