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

#include "serve_common.h"

namespace dsatopk_serve {
namespace {

constexpr int kRope = 64;
constexpr int kRopeBytes = kRope * 2;
constexpr int kFewSplits = 4;  // joined in one go
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttendParams {
  const char* q;
  int64_t q_row, q_head;  // bytes
  const char* cache;
  int64_t page, token;  // bytes
  int64_t num_pages;
  const int32_t* slots;  // selected form: [rows, slot_stride], the first `selected` of a row
  int64_t slot_stride;
  const int32_t* seq_lens;  // paged form
  const int32_t* table;
  int64_t table_stride;
  const int32_t* table_rows;
  int32_t table_width, page_bits;
  int32_t rows, heads, selected, blocks, splits;
  float scale2;  // scale * log2 e
  char* out;
  float* lse;
  float* part;   // [rows, splits, heads, latent], then [rows, splits, heads, 2]
  float* state;
};

// Waves of a workgroup: WH groups of 16 heads by WT groups of tokens.
template <int kWH_, int kWT_, int kTile_, int kLatent_>
struct Plan {
  static constexpr int kWH = kWH_, kWT = kWT_, kWaves = kWH * kWT;
  static constexpr int kTile = kTile_;          // tokens
  static constexpr int kBlock = kWaves * 64;
  static constexpr int kLatent = kLatent_;
  static constexpr int kRow = kLatent * 2;      // bytes of a latent vector
  static constexpr int kBuffer = kTile * (kRow + kRopeBytes);
  static constexpr int kTokens = kTile / kWT;   // a wave's of a tile
  static constexpr int kGo = kTokens == 16 ? 1 : 2;  // 16 tokens each, taken at once
  static constexpr int kCopy = kTile / kWaves;  // tokens that a wave copies
  static constexpr int kSteps = kLatent / 32;   // contraction steps over the latent part
  static constexpr int kRopeSteps = kRope / 32;
  static constexpr int kBlocks = kLatent / 16;  // output blocks
  static constexpr bool kOwn = kWH == 1;        // a wave copies what it reads
};

// Largest (sum) over the lanes that hold the same head.
__device__ __forceinline__ float head_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float head_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// The chunk that a lane group takes in step i of the contraction over the
// latent part (its order is free, as long as queries and keys share it).
// 16-byte reads go through 16 lanes at a time, 8 of them from the next lane
// group: rows 0-3 and 12-15 of one, rows 4-11 of the other. With chunks 2
// apart in neighbouring groups swizzle16 keeps these on different banks too;
// chunks 1 apart cost a second cycle for each.
__device__ __forceinline__ constexpr int chunk_of(int i, int group) {
  return 8 * (i >> 1) + 2 * group + (i & 1);
}

// A lane's places in a tile, in bytes, from which the others follow by
// exclusive or: of the swizzled chunks that differ in bits of their number
// only, within the row's first 256 bytes.
template <class P>
struct Places {
  int copy;  // chunk of a copied vector, for the wave's token 0
  int row;   // chunk of token lane % 16, for step 0 of the contraction
  int rope;  // the same of its rotary part
  int column;  // of the column reads of output block 0

  __device__ __forceinline__ Places(int wave, int lane) {
    const int col = lane & 15, group = lane >> 4;
    const int first = wave * P::kCopy;
    copy = P::kRow == 1024 ? (lane ^ swizzle16(first)) * 16
                           : ((lane & 31) ^ swizzle16(first + (lane >> 5))) * 16;
    row = col * P::kRow + ((chunk_of(0, group) ^ swizzle16(col)) << 4);
    rope = P::kTile * P::kRow + col * kRopeBytes + ((group ^ swizzle8(col)) << 4);
    // lane i of 16 points at row i / 4, 8 bytes i % 4 of a 4 x 32 byte block
    const int tok = 4 * group + (col >> 2);
    column = tok * P::kRow + ((((col & 3) >> 1) ^ swizzle16(tok)) << 4) + 8 * (col & 1);
  }
};

// Copies the wave's P::kCopy tokens of a tile; `at` is the address of token
// lane % P::kCopy of them.
template <class P>
__device__ __forceinline__ void copy_tokens(char* tile, uint64_t at, int place, int wave, int lane) {
  constexpr int kPer = 1024 / P::kRow;  // tokens a copy
  const uint32_t lo = (uint32_t)at, hi = (uint32_t)(at >> 32);
  const int first = wave * P::kCopy;
#pragma unroll
  for (int t = 0; t < P::kCopy; t += kPer) {
    // tokens t of 8 (16) on: swizzle16(first + t) is swizzle16(first) ^ swizzle16(t)
    const uint32_t chunk = place ^ (swizzle16(t) * 16);
    const uint64_t base = ((uint64_t)__builtin_amdgcn_readlane(hi, t) << 32) |
                          (uint32_t)__builtin_amdgcn_readlane(lo, t);
    char* to = tile + (first + t) * P::kRow;
    if constexpr (kPer == 2) {
      const uint64_t second = ((uint64_t)__builtin_amdgcn_readlane(hi, t + 1) << 32) |
                              (uint32_t)__builtin_amdgcn_readlane(lo, t + 1);
      copy_to_lds(reinterpret_cast<const char*>(lane < 32 ? base : second) + chunk, to);
    } else {
      copy_to_lds(reinterpret_cast<const char*>(base) + chunk, to);
    }
  }
#pragma unroll
  for (int t = 0; t < P::kCopy; t += 8) {
    const int mine = t + (lane >> 3);
    const uint64_t base = ((uint64_t)(uint32_t)__shfl((int)hi, mine) << 32) |
                          (uint32_t)__shfl((int)lo, mine);
    const uint32_t chunk = ((lane & 7) ^ swizzle8(first + mine)) * 16;
    copy_to_lds(reinterpret_cast<const char*>(base) + P::kRow + chunk,
                tile + P::kTile * P::kRow + (first + t) * kRopeBytes);
  }
}

// A wave's running state.
template <class P>
struct State {
  f32x4 o[P::kBlocks];
  float top, sum;  // the reference (log2), this lane's part of the sum
};

// Scores, weights and sums of the wave's next P::kGo * 16 tokens, from tile row
// `from` on, and first the next tile's copies if `more`: the two buffers are
// told apart so that no read of one waits for the other's copies. `valid`: a
// bit for each token.
template <class T, class P>
__device__ __forceinline__ void attend_tokens(State<P>& st, const u32x4 (&q)[P::kSteps + P::kRopeSteps],
                                              const char* __restrict__ cur, char* __restrict__ next,
                                              bool more, uint64_t next_at, const Places<P>& places,
                                              int wave, int from, uint64_t valid, int lane,
                                              float scale2) {
  constexpr int kGo = P::kGo;
  if (more) copy_tokens<P>(next, next_at, here(places.copy), wave, here(lane));
  const int group = lane >> 4;
  f32x4 s[kGo];
  {
    const int row = here(places.row), rope = here(places.rope);
    const char* rows = cur + from * P::kRow;  // `from` is a multiple of 16: the swizzle starts over
    const char* ropes = cur + from * kRopeBytes;
#pragma unroll
    for (int x = 0; x < kGo; ++x) s[x] = f32x4{};
    // Reads go kAhead steps before the products that take them, and no
    // further: registers are what a wave has least of.
    constexpr int kAhead = 3, kAll = P::kSteps + P::kRopeSteps;
    auto read = [&](int i, int x) {
      if (i < P::kSteps)
        return *reinterpret_cast<const u32x4*>(
            rows + (row ^ ((chunk_of(i, 0) & 15) << 4)) + (i >> 2) * 256 + x * 16 * P::kRow);
      return *reinterpret_cast<const u32x4*>(
          ropes + (rope ^ ((i - P::kSteps) << 6)) + x * 16 * kRopeBytes);
    };
    u32x4 a[kAhead][kGo];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int x = 0; x < kGo; ++x) a[i][x] = read(i, x);
#pragma unroll
    for (int i = 0; i < kAll; ++i) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int x = 0; x < kGo; ++x) {
        s[x] = T::mma16(a[i % kAhead][x], q[i], s[x]);
        if (i + kAhead < kAll) a[i % kAhead][x] = read(i + kAhead, x);
      }
    }
  }
  // register i of product x holds its token 4 * group + i
  constexpr uint32_t kEvery = kGo == 2 ? ~0u : 0xffffu;
  if ((uint32_t)valid != kEvery) {
    const uint32_t mine = (uint32_t)valid >> (4 * group);
#pragma unroll
    for (int x = 0; x < kGo; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!((mine >> (x * 16 + i)) & 1)) s[x][i] = -INFINITY;
  }
  const int column = here(places.column);
  const char* columns = cur + from * P::kRow;
  auto column_of = [&](int b) {
    u32x4 v = {};
#pragma unroll
    for (int x = 0; x < kGo; ++x) {
      const u32x2 w = read_columns(columns + (column ^ ((b & 7) << 5)) + (b >> 3) * 256 + x * 16 * P::kRow);
      v[2 * x] = w[0];
      v[2 * x + 1] = w[1];
    }
    return v;
  };

  // The weights, by the reference in use. It only has to be near
  // enough: a lane's sum over kMost (or not a number) tells that it is not,
  // as no row's maximum is looked for otherwise.
  float w[kGo][4], sum;
  auto weigh = [&]() {
    const float ref = st.top == -INFINITY ? 0.0f : st.top;
    sum = 0.0f;
#pragma unroll
    for (int x = 0; x < kGo; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[x][i] = exp2_fast(fmaf(s[x][i], scale2, -ref));
        sum += w[x][i];
      }
  };
  weigh();
  if (__any(!(sum <= T::kMost) || st.top == -INFINITY)) {
    float top = s[0][0];
#pragma unroll
    for (int x = 0; x < kGo; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, s[x][i]);
    const float to = fmaxf(st.top, head_max(top) * scale2 - T::kLift);
    const float by = st.top == -INFINITY ? 0.0f : exp2_fast(st.top - to);
    st.top = to;
    st.sum *= by;
#pragma unroll
    for (int b = 0; b < P::kBlocks; ++b) st.o[b] *= by;
    weigh();
  }
  st.sum += sum;

  // The sums. kAhead is what the registers leave: one more block ahead spills,
  // and a reload waits for every copy in flight (375 -> 480 us for 1024 rows
  // of 2048 slots and 64 heads, when they were one workgroup a CU).
  constexpr int kAhead = kGo == 1 ? 8 : 4;
  u32x4 a[kAhead];
#pragma unroll
  for (int b = 0; b < kAhead; ++b) a[b] = column_of(b);
  if constexpr (kGo == 1) {
    const u32x2 v = {T::pack(w[0][0], w[0][1]), T::pack(w[0][2], w[0][3])};
#pragma unroll
    for (int b = 0; b < P::kBlocks; ++b) {
      __builtin_amdgcn_sched_barrier(0);
      st.o[b] = T::mma16_half(u32x2{a[b % kAhead][0], a[b % kAhead][1]}, v, st.o[b]);
      if (b + kAhead < P::kBlocks) a[b % kAhead] = column_of(b + kAhead);
    }
  } else {
    const u32x4 v = {T::pack(w[0][0], w[0][1]), T::pack(w[0][2], w[0][3]),
                     T::pack(w[1][0], w[1][1]), T::pack(w[1][2], w[1][3])};
#pragma unroll
    for (int b = 0; b < P::kBlocks; ++b) {
      __builtin_amdgcn_sched_barrier(0);
      st.o[b] = T::mma16(a[b % kAhead], v, st.o[b]);
      if (b + kAhead < P::kBlocks) a[b % kAhead] = column_of(b + kAhead);
    }
  }
}

template <class T, class P, bool kPaged>
__global__ __launch_bounds__(P::kBlock, P::kOwn ? 1 : 2) void attend_kernel(AttendParams p) {
  constexpr int kWH = P::kWH, kWT = P::kWT;
  __shared__ __attribute__((aligned(1024))) char tiles[2 * P::kBuffer];
  __shared__ uint32_t masks[2][P::kWaves];
  __shared__ float joined[2][P::kWaves][16];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wh = wave % kWH, wt = wave / kWH;
  const uint32_t id = blockIdx.x;
  const int split = id % p.splits;
  const int block = (id / p.splits) % p.blocks;
  const int64_t row = id / p.splits / p.blocks;

  // the tokens of this workgroup
  int32_t len = p.selected;
  const int32_t* list;
  if constexpr (kPaged) {
    const int64_t most = min((int64_t)p.table_width << p.page_bits, (int64_t)(INT32_MAX - P::kTile));
    len = (int32_t)min((int64_t)max(p.seq_lens[row], 0), most);
    list = p.table + (p.table_rows ? p.table_rows[row] : row) * p.table_stride;
  } else {
    list = p.slots + row * p.slot_stride;
  }
  const int32_t tiles_all = (len + P::kTile - 1) / P::kTile;
  const int32_t per = (tiles_all + p.splits - 1) / p.splits;
  const int32_t first = split * per;
  const int32_t last = min(first + per, tiles_all);

  // The entry (slot or page) of token lane % P::kCopy of this wave's share of a tile, -1: none.
  auto entry_of = [&](int32_t tile) {
    const int32_t j = tile * P::kTile + wave * P::kCopy + lane % P::kCopy;
    if (tile >= last || j >= len) return -1;
    return list[kPaged ? j >> p.page_bits : j];
  };
  // Its address, or that of zeros.
  auto address_of = [&](int32_t tile, int32_t entry, bool& there) {
    int64_t page = entry;
    int32_t in = tile * P::kTile + wave * P::kCopy + lane % P::kCopy;
    if constexpr (!kPaged) {
      page = entry >> p.page_bits;
      in = entry;
    }
    in &= (1 << p.page_bits) - 1;
    there = entry >= 0 && page < p.num_pages;
    const char* at = there ? p.cache + page * p.page + in * p.token : zero_row();
    return (uint64_t)(uintptr_t)at;
  };
  auto bits_of = [&](bool there) { return (uint32_t)(__ballot(there) & ((1ull << P::kCopy) - 1)); };

  const Places<P> places(wave, lane);
  State<P> st;
  st.top = -INFINITY;
  st.sum = 0.0f;
#pragma unroll
  for (int b = 0; b < P::kBlocks; ++b) st.o[b] = f32x4{};

  const int col = lane & 15, group = lane >> 4;
  const int head = (block * kWH + wh) * 16 + col;
  if (first < last) {
    int32_t entry = entry_of(first);
    bool there;
    uint64_t at = address_of(first, entry, there);
    uint32_t mask = bits_of(there);
    if (!P::kOwn && lane == 0) masks[0][wave] = mask;
    copy_tokens<P>(tiles, at, places.copy, wave, lane);
    entry = entry_of(first + 1);

    u32x4 q[P::kSteps + P::kRopeSteps];
    const char* qh = head < p.heads ? p.q + row * p.q_row + head * p.q_head : zero_row();
#pragma unroll
    for (int i = 0; i < P::kSteps + P::kRopeSteps; ++i)
      q[i] = load16(qh + (i < P::kSteps ? chunk_of(i, group) : 4 * i + group) * 16);

    for (int32_t t = first; t < last; ++t) {
      const int buf = (t - first) & 1;
      uint64_t valid;
      if constexpr (P::kOwn) {
        wait_copies();
        valid = mask;
      } else {
        copies_barrier();
        uint64_t all = 0;
        constexpr int kParts = P::kTokens / P::kCopy;  // waves whose copies this one reads
#pragma unroll
        for (int w = 0; w < kParts; ++w)
          all |= (uint64_t)masks[buf][wt * kParts + w] << (w * P::kCopy);
        valid = (uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(all >> 32)) << 32 |
                (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)all);
      }
      const bool more = t + 1 < last;
      if (more) {
        at = address_of(t + 1, entry, there);
        mask = bits_of(there);
        if (!P::kOwn && lane == 0) masks[buf ^ 1][wave] = mask;
        entry = entry_of(t + 2);
      }
#pragma unroll 1
      for (int from = 0; from < P::kTokens; from += P::kGo * 16)
        attend_tokens<T, P>(st, q, tiles + buf * P::kBuffer, tiles + (buf ^ 1) * P::kBuffer,
                            more && from == 0, at, places, wave, wt * P::kTokens + from, valid >> from,
                            lane, p.scale2);
    }
  }

  float sum = head_sum(st.sum);
  float top = st.top;
  if constexpr (kWT > 1) {
    // join the token groups: each wave's sums to the common maximum, then into group 0
    if (lane < 16) {
      joined[0][wave][lane] = top;
      joined[1][wave][lane] = sum;
    }
    __syncthreads();
    float all = -INFINITY, total = 0.0f;
#pragma unroll
    for (int w = 0; w < kWT; ++w) all = fmaxf(all, joined[0][w * kWH + wh][col]);
#pragma unroll
    for (int w = 0; w < kWT; ++w) {
      const float x = joined[0][w * kWH + wh][col];
      total += joined[1][w * kWH + wh][col] * (x == -INFINITY ? 0.0f : exp2_fast(x - all));
    }
    const float by = top == -INFINITY ? 0.0f : exp2_fast(top - all);
#pragma unroll
    for (int b = 0; b < P::kBlocks; ++b) st.o[b] *= by;
    // the upper half of the groups gives to the lower, until one is left
    constexpr int kShare = P::kBlocks * 256;  // floats of a wave
    static_assert(kWH * (kWT / 2) * kShare * 4 <= 2 * P::kBuffer, "the tiles' space holds what is given");
    float* give = reinterpret_cast<float*>(tiles) + lane * 4;
#pragma unroll
    for (int step = kWT / 2; step; step /= 2) {
      __syncthreads();
      if (wt >= step && wt < 2 * step) {
        float* to = give + ((wt - step) * kWH + wh) * kShare;
#pragma unroll
        for (int b = 0; b < P::kBlocks; ++b) *reinterpret_cast<f32x4*>(to + b * 256) = st.o[b];
      }
      __syncthreads();
      if (wt < step) {
        const float* from = give + (wt * kWH + wh) * kShare;
#pragma unroll
        for (int b = 0; b < P::kBlocks; ++b) st.o[b] += *reinterpret_cast<const f32x4*>(from + b * 256);
      }
    }
    if (wt > 0) return;
    top = all;
    sum = total;
  }
  if (head >= p.heads) return;

  // register i of block b: element b * 16 + 4 * group + i of the head's vector
  if (p.splits == 1) {
    const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
    char* to = p.out + ((row * p.heads + head) * P::kLatent + 4 * group) * 2;
#pragma unroll
    for (int b = 0; b < P::kBlocks; ++b)
      *reinterpret_cast<u32x2*>(to + b * 32) = u32x2{T::pack(st.o[b][0] * by, st.o[b][1] * by),
                                                     T::pack(st.o[b][2] * by, st.o[b][3] * by)};
    if (p.lse && group == 0) p.lse[row * p.heads + head] = (top + log2f(sum)) * kLn2;
  } else {
    const int64_t at = (row * p.splits + split) * p.heads + head;
    if (group == 0) {
      p.state[at * 2] = top;
      p.state[at * 2 + 1] = sum;
    }
    // parts of many that saw nothing are skipped by the join
    if (p.splits > kFewSplits && top == -INFINITY && sum == 0.0f) return;
    float* to = p.part + at * P::kLatent + 4 * group;
#pragma unroll
    for (int b = 0; b < P::kBlocks; ++b) *reinterpret_cast<f32x4*>(to + b * 16) = st.o[b];
  }
}

// Joins few splits: kLatent / 4 threads for each row's head, 4 elements a
// thread, every thread by itself and all loads at once (parts that saw
// nothing are zeros). For two parts of 128 rows of 128 heads this takes 6 us
// less than the kernel below; for eight parts that one is faster by 1 us.
template <class T, int kLatent>
__global__ __launch_bounds__(256) void join_few_kernel(AttendParams p) {
  constexpr int kEach = kLatent / 4;
  const int64_t at = (int64_t)blockIdx.x * (256 / kEach) + threadIdx.x / kEach;
  if (at >= (int64_t)p.rows * p.heads) return;
  const int64_t row = at / p.heads;
  const int64_t base = row * p.splits * p.heads + at % p.heads;
  const int e = threadIdx.x % kEach * 4;
  float x[kFewSplits], n[kFewSplits], top = -INFINITY, sum = 0.0f;
  f32x4 v[kFewSplits], o = {};
#pragma unroll
  for (int s = 0; s < kFewSplits; ++s) {
    x[s] = -INFINITY;
    n[s] = 0.0f;
    v[s] = f32x4{};
    if (s < p.splits) {
      const int64_t part = base + (int64_t)s * p.heads;
      x[s] = p.state[part * 2];
      n[s] = p.state[part * 2 + 1];
      v[s] = *reinterpret_cast<const f32x4*>(p.part + part * kLatent + e);
    }
    top = fmaxf(top, x[s]);
  }
#pragma unroll
  for (int s = 0; s < kFewSplits; ++s) {
    const float by = exp2_fast(x[s] - (top == -INFINITY ? 0.0f : top));
    sum += n[s] * by;
    o += v[s] * by;
  }
  const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
  *reinterpret_cast<u32x2*>(p.out + (at * kLatent + e) * 2) =
      u32x2{T::pack(o[0] * by, o[1] * by), T::pack(o[2] * by, o[3] * by)};
  if (p.lse && e == 0) p.lse[at] = (top + log2f(sum)) * kLn2;
}

// Joins the splits of 4 * kEach elements of one row's head. First a thread
// for each split: the common maximum and the factors; then kEach threads for
// each of kJoinBlock / kEach sets of splits, 4 elements each. Many splits
// mean few rows: a workgroup takes 128 elements then (64 parts of 8 rows of 16
// heads: 8 us, and 20 by whole heads); up to kMidSplits, a head (8 parts of
// 66 rows of 40 heads: 10 us, and 14 by quarters).
constexpr int kMaxSplits = 256, kMidSplits = 16;
constexpr int kJoinBlock = 256;

template <class T, int kLatent, int kEach>
__global__ __launch_bounds__(kJoinBlock) void join_kernel(AttendParams p) {
  constexpr int kSides = kJoinBlock / kEach, kSlices = kLatent / (4 * kEach);
  __shared__ float tops[kJoinBlock / 64], sums[kJoinBlock / 64];
  __shared__ float factor[kMaxSplits];
  __shared__ __attribute__((aligned(16))) float half[kJoinBlock * 4];
  const int tid = threadIdx.x, wave = tid >> 6;
  const uint32_t which = blockIdx.x / kSlices, slice = blockIdx.x % kSlices;
  const int64_t row = which / p.heads;
  const int head = which % p.heads;
  const int64_t base = row * p.splits * p.heads + head;

  float x = -INFINITY, n = 0.0f;
  if (tid < p.splits) {
    const float* s = p.state + (base + (int64_t)tid * p.heads) * 2;
    x = s[0];
    n = s[1];
  }
  float top = x;
#pragma unroll
  for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  if ((tid & 63) == 0) tops[wave] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinBlock / 64; ++w) top = fmaxf(top, tops[w]);
  const bool empty = x == -INFINITY && n == 0.0f;  // such a split has written no vector
  const float by = empty ? 0.0f : exp2_fast(x - (top == -INFINITY ? 0.0f : top));
  factor[tid] = empty ? -1.0f : by;
  float sum = n * by;
#pragma unroll
  for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
  if ((tid & 63) == 0) sums[wave] = sum;
  __syncthreads();
  sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinBlock / 64; ++w) sum += sums[w];

  const int side = tid / kEach;
  const int e = (slice * kEach + tid % kEach) * 4;
  f32x4 o = {};
#pragma unroll 4
  for (int s = side; s < p.splits; s += kSides) {
    const float f = factor[s];
    if (f < 0.0f) continue;
    o += *reinterpret_cast<const f32x4*>(p.part + (base + (int64_t)s * p.heads) * kLatent + e) * f;
  }
  *reinterpret_cast<f32x4*>(half + tid * 4) = o;
  __syncthreads();
  if (side) return;
#pragma unroll
  for (int s = 1; s < kSides; ++s)
    o += *reinterpret_cast<const f32x4*>(half + (s * kEach + tid) * 4);
  const float scale = sum == 0.0f ? 0.0f : 1.0f / sum;
  *reinterpret_cast<u32x2*>(p.out + ((row * p.heads + head) * kLatent + e) * 2) =
      u32x2{T::pack(o[0] * scale, o[1] * scale), T::pack(o[2] * scale, o[3] * scale)};
  if (p.lse && e == 0) p.lse[row * p.heads + head] = (top + log2f(sum)) * kLn2;
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
  const dim3 grid((unsigned)((int64_t)p.rows * p.blocks * p.splits));
  return launch(attend_kernel<T, P, kPaged>, grid, dim3(P::kBlock), p, stream);
}

template <class T, int kLatent, bool kPaged>
int launch_attend(AttendParams p, void* stream) {
  const int hb = head_block(p.heads);
  p.blocks = (p.heads + hb - 1) / hb;
  const int st = hb == 16   ? launch_plan<T, Plan<1, 4, 64, kLatent>, kPaged>(p, stream)
                 : hb == 32 ? launch_plan<T, Plan<2, 2, 32, kLatent>, kPaged>(p, stream)
                 : hb == 64 ? launch_plan<T, Plan<4, 1, 32, kLatent>, kPaged>(p, stream)
                            : launch_plan<T, Plan<8, 1, 64, kLatent>, kPaged>(p, stream);
  if (st != DSATOPK_OK || p.splits == 1) return st;
  if (p.splits <= kFewSplits) {
    constexpr int kPer = 256 / (kLatent / 4);
    return launch(join_few_kernel<T, kLatent>,
                  dim3((unsigned)(((int64_t)p.rows * p.heads + kPer - 1) / kPer)), dim3(256), p, stream);
  }
  const int64_t heads = (int64_t)p.rows * p.heads;
  return p.splits <= kMidSplits
             ? launch(join_kernel<T, kLatent, kLatent / 4>, dim3((unsigned)heads), dim3(kJoinBlock), p, stream)
             : launch(join_kernel<T, kLatent, 32>, dim3((unsigned)(heads * (kLatent / 128))), dim3(kJoinBlock),
                      p, stream);
}

size_t part_floats(int32_t rows, int32_t heads, int32_t latent, int32_t splits) {
  return splits <= 1 ? 0 : (size_t)rows * splits * heads * (latent + 2);
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
  p.splits = splits_for(rows, heads, tokens);
  if (p.splits > 1) {
    if (!workspace || workspace_bytes < part_floats(rows, heads, latent, p.splits) * sizeof(float))
      return DSATOPK_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned16(workspace)) return DSATOPK_ERR_ALIGNMENT;
    p.part = static_cast<float*>(workspace);
    p.state = p.part + (size_t)rows * p.splits * heads * latent;
  }
  p.q = static_cast<const char*>(q);
  p.q_row = q_row * 2;
  p.q_head = q_head * 2;
  p.cache = static_cast<const char*>(cache);
  p.page = page_stride * 2;
  p.token = token_stride * 2;
  p.num_pages = num_pages;
  p.page_bits = log2_of(page_size);
  p.rows = rows;
  p.heads = heads;
  p.scale2 = scale * kLog2e;
  p.out = static_cast<char*>(out);
  p.lse = lse;
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
