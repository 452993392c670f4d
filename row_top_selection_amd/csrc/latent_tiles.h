// latent_tiles.h - what the kernels of absorbed latent attention share: tiles
// of cached vectors in LDS, the scores, weights and sums of a tile, a range of
// tokens, and the join of the parts that a row's tokens were split into.
#ifndef DSATOPK_LATENT_TILES_H_
#define DSATOPK_LATENT_TILES_H_

#include "serve_common.h"

namespace dsatopk_serve {
namespace {

constexpr int kRope = 64;
constexpr int kRopeBytes = kRope * 2;
constexpr int kFewSplits = 4;  // joined in one go
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The paged cache.
struct Cache {
  const char* at;
  int64_t page, token;  // bytes
  int64_t pages;
  int32_t page_bits;
};

// Results, and the parts that they are joined from.
struct Joined {
  int32_t rows, heads, splits;
  char* out;
  float* lse;
  float* part;   // [rows, splits, heads, latent], then [rows, splits, heads, 2]
  float* state;
};

// Waves of a workgroup: WH groups of 16 heads by WT groups of tokens.
template <int kWH_, int kWT_, int kTile_, int kLatent_>
struct Plan {
  static constexpr int kWH = kWH_, kWT = kWT_, kWaves = kWH * kWT, kCols = 16, kLanes = kWH * kCols;
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
// bit for each token; with kLane a lane's head sees `seen` of them at most (may be
// negative).
template <class T, class P, bool kLane>
__device__ __forceinline__ void attend_tokens(State<P>& st, const u32x4 (&q)[P::kSteps + P::kRopeSteps],
                                              const char* __restrict__ cur, char* __restrict__ next,
                                              bool more, uint64_t next_at, const Places<P>& places,
                                              int wave, int from, uint64_t valid, int32_t seen,
                                              int lane, float scale2) {
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
    // Reads are issued kAhead steps before the products that take them, and no
    // further: registers are what a wave has least of. (While the next tile's copies
    // are under way they are waited for together, every few products: copy_to_lds.)
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
  if ((uint32_t)valid != kEvery || (kLane && __any(seen < 16 * kGo))) {
    uint32_t bits = (uint32_t)valid;
    if (kLane && seen < 32) bits = seen <= 0 ? 0 : bits & ((1u << seen) - 1);
    const uint32_t mine = bits >> (4 * group);
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

// Tiles `first` to `last` of `len` tokens, the entries of which are in `list`:
// slots, or (paged) pages, from position `base` on. The lane's head has the queries `qh`,
// and sees, with kLane, the first `mine` tokens. The wave's tokens of a tile
// go into its own sums.
template <class T, class P, bool kPaged, bool kLane>
__device__ __forceinline__ void attend_range(State<P>& st, char* tiles, uint32_t (*masks)[P::kWaves],
                                             const Cache& c, const int32_t* list, int32_t base,
                                             int32_t len, int32_t first, int32_t last, const char* qh,
                                             int32_t mine, const Places<P>& places, int wave,
                                             int lane, float scale2) {
  const int wt = wave / P::kWH, group = lane >> 4;
  // The entry (slot or page) of token lane % P::kCopy of this wave's share of a tile, -1: none.
  auto entry_of = [&](int32_t tile) {
    const int32_t j = tile * P::kTile + wave * P::kCopy + lane % P::kCopy;
    if (tile >= last || j >= len) return -1;
    return list[kPaged ? (base + j) >> c.page_bits : j];
  };
  // Its address, or that of zeros.
  auto address_of = [&](int32_t tile, int32_t entry, bool& there) {
    int64_t page = entry;
    int32_t in = base + tile * P::kTile + wave * P::kCopy + lane % P::kCopy;
    if constexpr (!kPaged) {
      page = entry >> c.page_bits;
      in = entry;
    }
    in &= (1 << c.page_bits) - 1;
    there = entry >= 0 && page < c.pages;
    const char* at = there ? c.at + page * c.page + in * c.token : zero_row();
    return (uint64_t)(uintptr_t)at;
  };
  auto bits_of = [&](bool there) { return (uint32_t)(__ballot(there) & ((1ull << P::kCopy) - 1)); };

  if (first >= last) return;
  int32_t entry = entry_of(first);
  bool there;
  uint64_t at = address_of(first, entry, there);
  uint32_t mask = bits_of(there);
  if (!P::kOwn && lane == 0) masks[0][wave] = mask;
  copy_tokens<P>(tiles, at, places.copy, wave, lane);
  entry = entry_of(first + 1);

  u32x4 q[P::kSteps + P::kRopeSteps];
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
      attend_tokens<T, P, kLane>(st, q, tiles + buf * P::kBuffer, tiles + (buf ^ 1) * P::kBuffer,
                          more && from == 0, at, places, wave, wt * P::kTokens + from, valid >> from,
                                 kLane ? mine - t * P::kTile - wt * P::kTokens - from : 0, lane, scale2);
  }
}

// Joins the sums of the workgroup's token groups, each wave's by the common
// maximum, into those of group 0. `joined`, and the tiles' space: to pass them on.
template <class P>
__device__ __forceinline__ void join_groups(State<P>& st, float& top, float& sum, char* tiles,
                                            float (*joined)[P::kWaves][16], int wave, int lane) {
  constexpr int kWH = P::kWH, kWT = P::kWT;
  const int wh = wave % kWH, wt = wave / kWH, col = lane & 15;
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
  top = all;
  sum = total;
}

// What the wave's sums come to: the result, if its tokens are not split, or part `split`.
template <class T, class P>
__device__ __forceinline__ void put(const State<P>& st, float top, float sum, const Joined& to, int64_t row,
                                    int head, int split, int lane) {
  const int group = lane >> 4;
  // register i of block b: element b * 16 + 4 * group + i of the head's vector
  if (to.splits == 1) {
    const float by = 1.0f / sum;
    char* out = to.out + ((row * to.heads + head) * P::kLatent + 4 * group) * 2;
#pragma unroll
    for (int b = 0; b < P::kBlocks; ++b) {
      const u32x2 v = {T::pack(st.o[b][0] * by, st.o[b][1] * by), T::pack(st.o[b][2] * by, st.o[b][3] * by)};
      // (zeros where nothing was seen: the sums may not be, by infinite numbers that others saw)
      *reinterpret_cast<u32x2*>(out + b * 32) = sum == 0.0f ? u32x2{} : v;
    }
    if (to.lse && group == 0) to.lse[row * to.heads + head] = (top + log2f(sum)) * kLn2;
  } else {
    const int64_t at = (row * to.splits + split) * to.heads + head;
    if (group == 0) {
      to.state[at * 2] = top;
      to.state[at * 2 + 1] = sum;
    }
    // parts of many that saw nothing are skipped by the join
    if (to.splits > kFewSplits && top == -INFINITY && sum == 0.0f) return;
    float* part = to.part + at * P::kLatent + 4 * group;
#pragma unroll
    for (int b = 0; b < P::kBlocks; ++b) *reinterpret_cast<f32x4*>(part + b * 16) = st.o[b];
  }
}

// Joins few splits: kLatent / 4 threads for each row's head, 4 elements a
// thread, every thread by itself and all loads at once (parts that saw
// nothing are zeros). For two parts of 128 rows of 128 heads this takes 6 us
// less than the kernel below; for eight parts that one is faster by 1 us.
template <class T, int kLatent>
__global__ __launch_bounds__(256) void join_few_kernel(Joined p) {
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
__global__ __launch_bounds__(kJoinBlock) void join_kernel(Joined p) {
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

template <class T, int kLatent>
int launch_join(const Joined& p, void* stream) {
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

inline size_t part_floats(int32_t rows, int32_t heads, int32_t latent, int32_t splits) {
  return splits <= 1 ? 0 : (size_t)rows * splits * heads * (latent + 2);
}

}  // namespace
}  // namespace dsatopk_serve

#endif  // DSATOPK_LATENT_TILES_H_
