// expanded_attend.hip - latent attention in its expanded form
// (dsatopk_attend_expanded and dsatopk_attend_expanded_shared in
// include/dsatopk.h), for prompts:
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
// A workgroup of 4 or 8 waves takes 32 queries a wave of one head and goes
// over the keys, 8 a wave at a time, through a ring of tiles in LDS. Both
// products are transposed: S' = K Q' has a query in each lane and keys in its
// registers, which are, rounded, the B operand of O' = V' P'; V's columns
// come from LDS column reads. Queries stay in registers throughout.
//
// A wave takes the softmax of 32 keys between the reads for the scores of the
// next 32 and their products. Two waves a SIMD fill each other's pauses, one's
// products beside the other's exponentials.
//
// Few rows of many keys are split over workgroups by keys; a second kernel
// joins the parts.
//
// With shared keys a workgroup takes the next 32 queries a wave of those that
// stand together, whichever requests they are of, and goes over segments of
// keys: those that the requests share, once for all of them that stand
// together, then each request's own. A lane counts the keys of a segment that its query sees; waves
// none of whose queries are in a segment only copy. Prompts of 16 tokens fill
// tiles that way, which would be nearly empty if every request had its own.
//
// 4 x 1024 queries behind 15360 earlier tokens, 16 heads: 620 us, 1.07 PFLOP/s
// (a large library product of random numbers reaches 1.37 here). The clock
// falls with what the matrix units switch: the same call on zeros takes 530
// us.
//
// 16 x 512 queries that share 16384 keys, 16 heads: 1250 ... 1320 us by card, 1.1 PFLOP/s.
//
// Weights are rounded to the inputs' type for the second product (off by at
// most 2^-8 of each in bfloat16; in half precision by 2^-11 of each or 2^-35
// of the row's largest, see kLift); scores, maxima, sums and accumulators are
// fp32.

#include "serve_common.h"

namespace dsatopk_serve {
namespace {

constexpr int kKeys = 32;  // taken at once
constexpr int kNope = 128, kRope = 64, kValue = 128;
constexpr int kKeyBytes = kNope * 2, kRopeBytes = kRope * 2, kValueBytes = kValue * 2;
constexpr int kSteps = (kNope + kRope) / 16;
constexpr int kBlocks = kValue / 32;
constexpr int64_t kMostStride = int64_t(1) << 27;  // of a key, in elements: 8 of them are 2^31 bytes
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Eight waves share what four would each copy for themselves (a workgroup a
// CU, tiles of 64 keys); four leave room for a second workgroup, and suit
// short and few prompts.
template <int kWaves_>
struct Shape {
  static constexpr int kWaves = kWaves_, kBlock = kWaves * 64, kRows = kWaves * 32;
  static constexpr int kTile = kWaves * 8;
  static constexpr int kRing = kWaves == 4 ? 4 : 3;  // tiles in LDS: kRing - 1 ahead
  static constexpr int kRopeAt = kTile * kKeyBytes;
  static constexpr int kValueAt = kRopeAt + kTile * kRopeBytes;
  static constexpr int kBuffer = kValueAt + kTile * kValueBytes;
};

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
  const int32_t* shared_starts;  // shared form
  const int32_t* shared_lens;
  int32_t requests, heads, tiles, num_q, num_k, causal, splits;
  float scale2;
  char* out;
  float* lse;
  float* part;   // [splits, num_q, heads, kValue], then [splits, num_q, heads, 2]
  float* state;
};

// A lane's places in a tile and in its copies, in bytes; the others follow
// by exclusive or of the chunk numbers' bits.
template <class S>
struct Places {
  uint32_t k, v, rope;  // offset of the lane's row of 4 (8) in a copy
  int chunk, tail;      // its chunk there, of k and v and of the rotary part
  int row, rope_row;    // of key lane % 32, step 0 of the contraction
  int column;           // of the column reads of output block 0

  __device__ __forceinline__ Places(const ExpandParams& p, int lane) {
    const int col = lane & 31, half = lane >> 5;
    k = (lane >> 4) * (uint32_t)p.k_row;
    v = (lane >> 4) * (uint32_t)p.v_row;
    rope = (lane >> 3) * (uint32_t)p.rope_row;
    chunk = ((lane & 15) ^ swizzle32(lane >> 4)) * 16;
    tail = ((lane & 7) ^ swizzle8(lane >> 3)) * 16;
    row = col * kKeyBytes + ((half ^ swizzle32(col)) << 4);
    rope_row = S::kRopeAt + col * kRopeBytes + ((half ^ swizzle8(col)) << 4);
    // lane i of 16 points at row i / 4, 8 bytes i % 4 of a 4 x 32 byte block
    const int in = lane & 15, side = (lane >> 4) & 1, tok = 4 * half + (in >> 2);
    column = S::kValueAt + tok * kValueBytes + (((2 * side + ((in & 3) >> 1)) ^ swizzle32(tok)) << 4) +
             8 * (in & 1);
  }
};

constexpr int kCopies = 5;  // a wave's of a tile

// Copies keys j0 .. j0 + kTile - 1 (of the request's `keys`; rows past them repeat
// the last) of all three tensors, swizzled: a wave takes 8.
template <class S>
__device__ __forceinline__ void copy_tile(const ExpandParams& p, char* tile, const char* k,
                                          const char* v, const char* rope, int32_t j0,
                                          int32_t keys, const Places<S>& at, int wave, int lane) {
  const int t0 = wave * 8;
  char* rope_to = tile + S::kRopeAt + t0 * kRopeBytes;
  if (j0 + S::kTile <= keys) {
    // whole: a uniform address and the lane's offset
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t j = j0 + t0 + i * 4;
      const uint32_t c = at.chunk ^ (swizzle32(t0 + i * 4) * 16);
      copy_to_lds(k + j * p.k_row + (at.k + c), tile + (t0 + i * 4) * kKeyBytes);
      copy_to_lds(v + j * p.v_row + (at.v + c), tile + S::kValueAt + (t0 + i * 4) * kValueBytes);
    }
    copy_to_lds(rope + (int64_t)(j0 + t0) * p.rope_row +
                    (at.rope + (uint32_t)(at.tail ^ (swizzle8(t0) * 16))),
                rope_to);
  } else {
    lane = here(lane);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = t0 + i * 4 + (lane >> 4);
      const int64_t j = min(j0 + t, keys - 1);
      const int c = ((lane & 15) ^ swizzle32(t)) * 16;
      copy_to_lds(k + j * p.k_row + c, tile + (t0 + i * 4) * kKeyBytes);
      copy_to_lds(v + j * p.v_row + c, tile + S::kValueAt + (t0 + i * 4) * kValueBytes);
    }
    const int t = t0 + (lane >> 3);
    const int64_t j = min(j0 + t, keys - 1);
    copy_to_lds(rope + j * p.rope_row + ((lane & 7) ^ swizzle8(t)) * 16, rope_to);
  }
}

struct State {
  f32x16 o[kBlocks];
  float top, sum;
};

// Weight i of scores s by the reference `ref` (log2).
__device__ __forceinline__ float weight_of(const f32x16& s, int i, float scale2, float ref) {
  return exp2_fast(fmaf(s[i], scale2, -ref));
}

// The scores of the 32 keys `part` of a tile for the wave's 32 queries, and with them
// the weights of `s` (if there is one). Reads are issued at least kAhead steps before
// their products: left alone, the compiler puts each read right before its product,
// waits for it there, and takes the weights after all products. Written as here, a few
// weights behind each product, it issues all reads and takes the weights first, and
// the products run through behind them.
template <class T, class S>
__device__ __forceinline__ f32x16 scores_of(const char* tile, int part, const u32x4 (&q)[kSteps],
                                            const Places<S>& places, const f32x16* s, float scale2,
                                            float ref, f32x16* w, float* sum) {
  constexpr int kAhead = 4;
  const int row = here(places.row), rope_row = here(places.rope_row);
  auto read = [&](int i) {
    return *reinterpret_cast<const u32x4*>(
        i < kNope / 16 ? tile + part * kKeys * kKeyBytes + (row ^ (i << 5))
                       : tile + part * kKeys * kRopeBytes + (rope_row ^ ((i - kNope / 16) << 5)));
  };
  u32x4 a[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) a[i] = read(i);
  f32x16 next = {};
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    __builtin_amdgcn_sched_barrier(0);
    next = T::mma32(a[i % kAhead], q[i], next);
    if (i + kAhead < kSteps) a[i % kAhead] = read(i + kAhead);
    if (s) {
#pragma unroll
      for (int e = 16 * i / kSteps; e < 16 * (i + 1) / kSteps; ++e) {
        (*w)[e] = weight_of(*s, e, scale2, ref);
        *sum += (*w)[e];
      }
    }
  }
  __builtin_amdgcn_sched_barrier(0);
  return next;
}

// 32 keys: the weights of their scores `s` and their part of the sums, and
// the scores of the 32 after them (`after`) in their place. First, if `copy`,
// the copies of the tile at key copy_j. The tiles are told apart so that no
// read of one waits for the copies of another. `seen`: how many of the 32 keys
// this lane's query sees (may be negative or above 32); `whole`: all of them, for
// every lane of the wave. With kApart nothing of keys that a query sees none of goes into
// its sums, whatever their values are (a weight of 0 times an infinite one is NaN).
template <class T, class S, bool kApart = false>
__device__ __forceinline__ void keys_step(const ExpandParams& p, State& st, f32x16& s,
                                          const u32x4 (&q)[kSteps], const char* __restrict__ cur,
                                          int part, const char* __restrict__ after, int after_part,
                                          char* __restrict__ copy_to, const char* k,
                                          const char* v, const char* rope, bool copy, int32_t copy_j,
                                          int32_t keys, int32_t seen, bool whole,
                                          const Places<S>& places, int wave, int lane) {
  if (copy) copy_tile<S>(p, copy_to, k, v, rope, copy_j, keys, places, wave, lane);
  const int half = lane >> 5;
  if (!whole) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (8 * (i / 4) + 4 * half + i % 4 >= seen) s[i] = -INFINITY;
  }
  // The weights are taken by the reference in use, which only has to
  // be near enough: a lane's sum over kMost (or not a number) tells that it
  // is not, and the scores' maximum is looked for. A query that sees none of
  // these keys needs no reference for them.
  const bool wants = st.top == -INFINITY && seen > 0;
  f32x16 w;
  float sum = 0.0f;
  const f32x16 next = scores_of<T, S>(after, after_part, q, places, &s, p.scale2,
                                      st.top == -INFINITY ? 0.0f : st.top, &w, &sum);
  const int column = here(places.column);
  // Step n: block n % kBlocks of 16 keys' share, n / kBlocks of 2. Reads go
  // kAhead steps before their products.
  constexpr int kAll = 2 * kBlocks, kAhead = 5;
  auto read = [&](int n) {
    const int b = n % kBlocks;
    const char* rows = cur + part * kKeys * kValueBytes + (n / kBlocks) * 16 * kValueBytes;
    const u32x2 lo = read_columns(rows + (column ^ (b << 6)));
    // swizzle32(t + 8) = swizzle32(t) ^ 2
    const u32x2 hi = read_columns(rows + (column ^ (b << 6) ^ 32) + 8 * kValueBytes);
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  };
  u32x4 a[kAhead];
  if constexpr (!kApart) {
#pragma unroll
    for (int n = 0; n < kAhead; ++n) a[n] = read(n);
  }
  if (__any(!(sum <= T::kMost) || wants)) {
    float top = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
    const float to = fmaxf(st.top, fmaxf(top, other_half(top)) * p.scale2 - T::kLift);
    const float by = st.top == -INFINITY ? 0.0f : exp2_fast(st.top - to);
    st.top = to;
    st.sum *= by;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) st.o[b] *= by;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      w[i] = weight_of(s, i, p.scale2, to == -INFINITY ? 0.0f : to);
      sum += w[i];
    }
  }
  st.sum += sum;
  s = next;

  auto weights = [&](int g) {
    return u32x4{T::pack(w[8 * g], w[8 * g + 1]), T::pack(w[8 * g + 2], w[8 * g + 3]),
                 T::pack(w[8 * g + 4], w[8 * g + 5]), T::pack(w[8 * g + 6], w[8 * g + 7])};
  };
  if constexpr (kApart) {
    const u32x4 y[2] = {weights(0), weights(1)};
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      const f32x16 o = T::mma32(read(kBlocks + b), y[1], T::mma32(read(b), y[0], f32x16{}));
#pragma unroll
      for (int i = 0; i < 16; ++i) st.o[b][i] += seen > 0 ? o[i] : 0.0f;
    }
    return;
  }
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const u32x4 y = weights(g);
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      const int n = g * kBlocks + b;
      __builtin_amdgcn_sched_barrier(0);
      st.o[b] = T::mma32(a[n % kAhead], y, st.o[b]);
      if (n + kAhead < kAll) a[n % kAhead] = read(n + kAhead);
    }
  }
}

// What the wave's sums come to, for the lane's query `at`: the result, or part `split`.
template <class T>
__device__ __forceinline__ void put(const ExpandParams& p, const State& st, int64_t at, int head, int split,
                                    int half) {
  const float sum = st.sum + other_half(st.sum);
  if (p.splits > 1) {
    const int64_t to = ((int64_t)split * p.num_q + at) * p.heads + head;
    if (half == 0) {
      p.state[to * 2] = st.top;
      p.state[to * 2 + 1] = sum;
    }
    if (st.top == -INFINITY && sum == 0.0f) return;  // nothing seen: the join skips it
    float* part = p.part + to * kValue + 4 * half;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<f32x4*>(part + b * 32 + 2 * i) =
            f32x4{st.o[b][i], st.o[b][i + 1], st.o[b][i + 2], st.o[b][i + 3]};
    return;
  }
  const float by = 1.0f / sum;
  char* to = p.out + ((at * p.heads + head) * kValue + 4 * half) * 2;
#pragma unroll
  for (int b = 0; b < kBlocks; ++b)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const u32x2 v = {T::pack(st.o[b][i] * by, st.o[b][i + 1] * by),
                       T::pack(st.o[b][i + 2] * by, st.o[b][i + 3] * by)};
      // (zeros where nothing was seen: the sums may not be, by infinite values that others saw)
      *reinterpret_cast<u32x2*>(to + (b * 32 + 2 * i) * 2) = sum == 0.0f ? u32x2{} : v;
    }
  if (p.lse && half == 0) p.lse[at * p.heads + head] = (st.top + log2f(sum)) * kLn2;
}

template <class T, class S>
__global__ __launch_bounds__(S::kBlock, 2) void expand_kernel(ExpandParams p) {
  constexpr int kRows = S::kRows, kTile = S::kTile, kRing = S::kRing, kBuffer = S::kBuffer;
  __shared__ __attribute__((aligned(1024))) char tiles[kRing * kBuffer];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, half = lane >> 5;

  // Workgroup -> (request and head, rows). Neighbouring numbers run on
  // different XCDs: the row tiles of one head, which read the same keys, are
  // 8 apart so that they share an L2. Late rows see most keys: they go first.
  const uint32_t pairs = (uint32_t)(p.requests * p.heads);
  const uint32_t id = blockIdx.x;
  const int split = blockIdx.y;
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
  const int32_t all = sees(min(first + kRows, rows) - 1);
  const int32_t least = sees(min(first + wave * 32, rows - 1));
  // this part's keys: [start, most)
  const int32_t share = ((all + kTile - 1) / kTile + p.splits - 1) / p.splits * kTile;
  const int32_t start = min(split * share, all);
  const int32_t most = min(start + share, all);

  u32x4 q[kSteps];
  const char* qh = p.q + at * p.q_row + head * p.q_head;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) q[i] = load16(qh + (2 * i + half) * 16);

  State st;
  st.top = -INFINITY;
  st.sum = 0.0f;
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) st.o[b] = f32x16{};

  const char* k = p.k + k0 * p.k_row + head * p.k_head;
  const char* v = p.v + k0 * p.v_row + head * p.v_head;
  const char* rope = p.rope + k0 * p.rope_row;
  const Places<S> places(p, lane);
  if (start < most) {
    constexpr int kAheadTiles = kRing - 1, kParts = kTile / kKeys;
#pragma unroll
    for (int n = 0; n < kAheadTiles; ++n)
      if (start + n * kTile < most)
        copy_tile<S>(p, tiles + n * kBuffer, k, v, rope, start + n * kTile, keys, places, wave, lane);
    copies_barrier();
    f32x16 s = scores_of<T, S>(tiles, 0, q, places, nullptr, 0.0f, 0.0f, nullptr, nullptr);
    int n = 0;
    for (int32_t j0 = start; j0 < most; j0 += kTile, ++n) {
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
        const bool last = part + 1 == kParts;
        if (last) {
          // Tile n + 1 has arrived (later ones may be under way, unless they
          // are the last), and all waves are done with tile n - 1, whose
          // place is the next copy's.
          if (kAheadTiles > 2 && j0 + kAheadTiles * kTile < most + kTile)
            wait_copies_but<(kAheadTiles - 2) * kCopies>();
          else
            wait_copies();
          __syncthreads();
        }
        const int32_t j = j0 + part * kKeys, copy_j = j0 + kAheadTiles * kTile;
        if (part > 0 && j >= most) break;
        keys_step<T, S>(p, st, s, q, tiles + n % kRing * kBuffer, part,
                        tiles + (n + last) % kRing * kBuffer, last ? 0 : part + 1,
                        tiles + (n + kAheadTiles) % kRing * kBuffer, k, v, rope,
                        last && copy_j < most, copy_j, keys, mine - j, least >= j + kKeys, places,
                        wave, lane);
      }
    }
  }
  if (row < rows) put<T>(p, st, at, head, split, half);
}

// Keys that some queries see: rows base .. base + len - 1 of the keys, for the
// queries from .. to - 1, of which query i sees the first i + diag (not fewer than
// 0, nor more than len).
struct Segment {
  int32_t base, len, from, to, diag;

  __device__ __forceinline__ int32_t seen(int32_t i) const {
    return i >= from && i < to ? min(max(i + diag, 0), len) : 0;
  }
};

// A workgroup's queries: tile `index` of the batch's stretches, each cut into tiles from its own
// first query on. A stretch is a run of requests with the same shared keys. (In tiles of the
// whole batch, one that two runs meet in goes over both runs' keys, twice what the others take:
// 2 x 4 prompts of up to 777 tokens behind 2000, 16 heads, took 200 us and take 105.) Where
// there are many requests for the queries (kPacked), all runs of less than half a tile that
// stand together are one stretch, or single tokens might each need a workgroup. Threads take chunks
// of the requests, and what is before or behind a chunk from the others.
struct Tile {
  int32_t q0, q1, first;  // queries; the stretch's first request
};
template <class S, bool kPacked>
__device__ __forceinline__ Tile tile_of(const ExpandParams& p, int32_t index, char* space, int tid, int wave,
                                        int lane) {
  struct Room {
    int32_t last[S::kWaves], next[S::kWaves], cuts[S::kWaves], tiles[S::kWaves];
    Tile tile;
  };
  Room& room = *reinterpret_cast<Room*>(space);
  const int32_t chunk = p.requests / S::kBlock + 1;
  const int32_t r0 = min(tid * chunk, p.requests), r1 = min(r0 + chunk, p.requests);
  auto start = [&](int32_t r) { return min(max(p.q_starts[r], 0), p.num_q); };
  auto queries = [&](int32_t from, int32_t to) { return max(start(to) - start(from), 0); };
  auto begins = [&](int32_t r) {
    return r == 0 || p.shared_starts[r] != p.shared_starts[r - 1] || p.shared_lens[r] != p.shared_lens[r - 1];
  };
  // the largest of the threads before this one, 0 if there is none; `all` of a wave each
  auto before = [&](int32_t x, int32_t* all) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int32_t o = __shfl_up(x, d);
      if (lane >= d) x = max(x, o);
    }
    if (lane == 63) all[wave] = x;
    __syncthreads();
    x = __shfl_up(x, 1);
    if (lane == 0) x = 0;
#pragma unroll
    for (int w = 0; w < S::kWaves; ++w)
      if (w < wave) x = max(x, all[w]);
    return x;
  };
  // runs: where the one before the chunk begins, and the first one behind it
  int32_t last = 0, next = p.requests;
  for (int32_t r = r1 - 1; r >= r0; --r)
    if (begins(r)) {
      last = max(last, r);
      next = r;
    }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t o = __shfl_down(next, d);
    if (lane + d < 64) next = min(next, o);
  }
  if (lane == 0) room.next[wave] = next;
  if (tid == 0) room.tile = Tile{0, 0, 0};
  last = before(last, room.last);
  next = __shfl_down(next, 1);
  if (lane == 63) next = p.requests;
#pragma unroll
  for (int w = 0; w < S::kWaves; ++w)
    if (w > wave) next = min(next, room.next[w]);
  // Stretches begin where a run does; packed, if that or the one before it is long.
  auto stretches = [&](auto&& what) {
    int32_t run = last;
    for (int32_t r = r0; r < r1; ++r) {
      if (!begins(r)) continue;
      if (!kPacked) {
        what(r);
        continue;
      }
      int32_t end = r + 1;
      while (end < r1 && !begins(end)) ++end;
      if (end == r1) end = next;
      if (r == 0 || 2 * queries(run, r) >= S::kRows || 2 * queries(r, end) >= S::kRows) what(r);
      run = r;
    }
  };
  int32_t cut = 0;
  stretches([&](int32_t r) { cut = r; });
  cut = before(cut, room.cuts);
  // tiles of the stretches that end in the chunk
  auto each = [&](auto&& what) {
    int32_t from = cut;
    stretches([&](int32_t r) {
      if (r > 0) what(from, r);
      from = r;
    });
    if (r0 < r1 && r1 == p.requests) what(from, r1);
  };
  auto count = [&](int32_t from, int32_t to) { return (queries(from, to) + S::kRows - 1) / S::kRows; };
  int32_t tiles = 0;
  each([&](int32_t from, int32_t to) { tiles += count(from, to); });
  int32_t below = tiles;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t o = __shfl_up(below, d);
    if (lane >= d) below += o;
  }
  if (lane == 63) room.tiles[wave] = below;
  __syncthreads();
  below -= tiles;
#pragma unroll
  for (int w = 0; w < S::kWaves; ++w)
    if (w < wave) below += room.tiles[w];
  if (index >= below && index < below + tiles)
    each([&](int32_t from, int32_t to) {
      const int32_t n = count(from, to);
      if (index >= below && index < below + n) {
        const int32_t q0 = start(from) + (index - below) * S::kRows;
        room.tile = Tile{q0, min(q0 + S::kRows, start(to)), from};
      }
      below += n;
    });
  __syncthreads();
  const Tile tile{__builtin_amdgcn_readfirstlane(room.tile.q0), __builtin_amdgcn_readfirstlane(room.tile.q1),
                  __builtin_amdgcn_readfirstlane(room.tile.first)};
  __syncthreads();  // before the space is taken for tiles of keys
  return tile;
}

// The segments of the queries q0 .. q1 - 1, a tile of keys at a time. The same in
// all lanes.
template <class S, bool kPacked>
struct Walk {
  const ExpandParams& p;
  int32_t q0, q1;
  int32_t request;  // whose own keys come next, or with whom a new run begins
  int32_t run;      // the first request behind those that share with it
  Segment at;
  int32_t j;  // first key of the tile, in the segment
  bool done;

  __device__ __forceinline__ Walk(const ExpandParams& params, int32_t first, int32_t last, int32_t r)
      : p(params), q0(first), q1(last), request(r), run(r), at{}, j(0), done(false) {
    if (kPacked) {
      next();
    } else {  // one run: its shared keys, and then requests only
      share(r, q0, q1);
      if (at.len == 0) next();
    }
  }
  __device__ __forceinline__ int32_t starts(int32_t r) const { return max(p.q_starts[r], 0); }
  __device__ __forceinline__ int32_t ends(int32_t r) const { return min(p.q_starts[r + 1], p.num_q); }
  // The keys that request r shares, for the queries from .. to - 1.
  __device__ __forceinline__ void share(int32_t r, int32_t from, int32_t to) {
    at.base = min(max(p.shared_starts[r], 0), p.num_k);
    at.len = min(max(p.shared_lens[r], 0), p.num_k - at.base);
    at.from = from;
    at.to = to;
    at.diag = at.len;
  }

  __device__ __forceinline__ void next() {
    j = 0;
    while (true) {
      if (kPacked && request >= run) {
        while (request < p.requests && starts(request) >= ends(request)) ++request;
        if (request < p.requests && starts(request) < q1) {
          const int32_t first = p.shared_starts[request], len = p.shared_lens[request];
          run = request + 1;
          while (run < p.requests && starts(run) < q1 &&
                 (starts(run) >= ends(run) || (p.shared_starts[run] == first && p.shared_lens[run] == len)))
            ++run;
          share(request, max(starts(request), q0), min(ends(run - 1), q1));
          if (at.len > 0 && at.from < at.to) return;
        }
      }
      if (request >= p.requests || starts(request) >= q1) {
        done = true;
        return;
      }
      const int32_t r = request++;
      const int32_t first = starts(r), rows = ends(r) - first;
      at.base = min(max(p.k_starts[r], 0), p.num_k);
      const int32_t keys = max(min(p.k_starts[r + 1], p.num_k) - at.base, 0);
      at.from = max(first, q0);
      at.to = min(first + rows, q1);
      if (at.from >= at.to) continue;
      at.diag = p.causal ? keys - rows + 1 - first : keys;
      at.len = min(max(at.to - 1 + at.diag, 0), keys);
      if (at.len > 0) return;
    }
  }
  __device__ __forceinline__ void advance() {
    j += S::kTile;
    if (j >= at.len) next();
  }
  // n tiles on.
  __device__ __forceinline__ void skip(int32_t n) {
    while (n > 0 && !done) {
      const int32_t here = (at.len - j + S::kTile - 1) / S::kTile;
      if (here > n) {
        j += n * S::kTile;
        return;
      }
      n -= here;
      next();
    }
  }
  __device__ __forceinline__ int32_t tiles() {
    int32_t n = 0;
    for (; !done; next()) n += (at.len + S::kTile - 1) / S::kTile;
    return n;
  }
};

// Dies that one head's workgroups are on, of 8: all on one leave the others idle where heads are few (2 x 6 prompts
// of up to 243 behind 9373, one head: 47 us, on one die 139; 8 of up to 600 behind 4000, four heads, 100 and 139).
__host__ __device__ constexpr int dies_of(int heads) { return heads < 8 ? 8 / heads : 1; }

// The sums of the queries q0 .. q1 - 1, the first of which are of request r, over part `split` of their keys.
template <class T, class S, bool kPacked, bool kApart>
__device__ __forceinline__ void attend_segments(const ExpandParams& p, State& st, char* tiles, int32_t q0, int32_t q1,
                                                int32_t r, int head, int split, int wave, int lane) {
  constexpr int kTile = S::kTile, kRing = S::kRing, kBuffer = S::kBuffer;
  constexpr int kAheadTiles = kRing - 1, kParts = kTile / kKeys;
  const int col = lane & 31, half = lane >> 5;
  const int32_t w0 = q0 + wave * 32;
  const int32_t at = min(w0 + col, q1 - 1);

  u32x4 q[kSteps];
  const char* qh = p.q + (int64_t)at * p.q_row + head * p.q_head;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) q[i] = load16(qh + (2 * i + half) * 16);

  st.top = -INFINITY;
  st.sum = 0.0f;
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) st.o[b] = f32x16{};

  using Keys = Walk<S, kPacked>;
  Keys use(p, q0, q1, r);
  int32_t most = INT32_MAX;
  if (p.splits > 1) {
    const int32_t all = Keys(use).tiles();
    const int32_t per = (all + p.splits - 1) / p.splits;
    most = per;
    use.skip(split * per);
  }
  Keys copy(use);
  const Places<S> places(p, lane);
  int32_t copied = 0;
  auto keys_at = [&](const char* base, int64_t head_bytes, int64_t row_bytes) {
    return base + copy.at.base * row_bytes + head * head_bytes;
  };
  while (copied < kAheadTiles && copied < most && !copy.done) {
    copy_tile<S>(p, tiles + copied * kBuffer, keys_at(p.k, p.k_head, p.k_row), keys_at(p.v, p.v_head, p.v_row),
                 keys_at(p.rope, 0, p.rope_row), copy.j, copy.at.len, places, wave, lane);
    copy.advance();
    ++copied;
  }
  if (copied) {
    copies_barrier();
    f32x16 s = {};
    bool have = false;  // s holds the scores of the next 32 keys
    for (int32_t n = 0; n < copied; ++n) {
      const Segment seg = use.at;
      const int32_t j0 = use.j;
      use.advance();
      // what the wave's queries see of the segment, at most and at least
      const int32_t top = w0 < seg.to ? seg.seen(min(w0 + 31, seg.to - 1)) : 0;
      const int32_t low = w0 + 31 < seg.to ? seg.seen(w0) : 0;
      const int32_t sees = seg.seen(at);  // lanes past the last query do as that does
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
        const bool last = part + 1 == kParts;
        if (last) {
          // tile n + 1 has arrived, and all waves are done with tile n - 1
          if (kAheadTiles > 2 && copied - n >= kAheadTiles)
            wait_copies_but<(kAheadTiles - 2) * kCopies>();
          else
            wait_copies();
          __syncthreads();
        }
        const bool more = last && copied < most && !copy.done;
        const int32_t j = j0 + part * kKeys;
        const char* cur = tiles + n % kRing * kBuffer;
        char* to = tiles + (n + kAheadTiles) % kRing * kBuffer;
        const char* k = keys_at(p.k, p.k_head, p.k_row);
        const char* v = keys_at(p.v, p.v_head, p.v_row);
        const char* rope = keys_at(p.rope, 0, p.rope_row);
        if (j < top) {
          if (!have)
            s = scores_of<T, S>(cur, part, q, places, nullptr, 0.0f, 0.0f, nullptr, nullptr);
          keys_step<T, S, kApart>(p, st, s, q, cur, part, tiles + (n + last) % kRing * kBuffer, last ? 0 : part + 1, to,
                          k, v, rope, more, copy.j, copy.at.len, sees - j, low >= j + kKeys, places, wave, lane);
        } else if (more) {
          copy_tile<S>(p, to, k, v, rope, copy.j, copy.at.len, places, wave, lane);
        }
        have = j < top;
        if (more) {
          copy.advance();
          ++copied;
        }
      }
    }
  }
}

// Uniform values, and the arguments as they are in memory, from which what follows is computed anew: nothing of it is kept
// from before, in registers that a loop in between is short of.
__device__ __forceinline__ int32_t anew(int32_t x) {
  asm volatile("" : "+s"(x));
  return x;
}
__device__ __forceinline__ const ExpandParams& params_anew() {
  auto* p = (const __attribute__((address_space(4))) ExpandParams*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const ExpandParams*)p;
}

template <class T, class S, bool kPacked>
__global__ __launch_bounds__(S::kBlock, 2) void expand_shared_kernel(ExpandParams p) {
  __shared__ __attribute__((aligned(1024))) char tiles[S::kRing * S::kBuffer];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // Workgroup -> (head, queries), as above: those of one head are 8 apart. Less than 8 heads have several dies each.
  const uint32_t id = blockIdx.x, slot = id % 8;
  const int split = blockIdx.y, dies = dies_of(p.heads);
  const int head = dies > 1 ? slot / dies : id / (8 * p.tiles) * 8 + slot;
  const int index = dies > 1 ? id / 8 * dies + slot % dies : id / 8 % p.tiles;
  if (head >= p.heads || index >= p.tiles) return;
  const Tile tile = tile_of<S, kPacked>(p, p.tiles - 1 - index, tiles, tid, wave, lane);
  const int32_t q0 = tile.q0, q1 = tile.q1;
  if (q0 >= q1) return;
  const int32_t r = max(tile.first, last_below(p.requests, q0, lane, [&](int32_t i) { return (int64_t)p.q_starts[i]; }));
  State st;
  attend_segments<T, S, kPacked, false>(p, st, tiles, q0, q1, r, head, split, wave, lane);
  if (min(p.q_starts[r + 1], p.num_q) < q1) {
    // Queries of several requests: infinite values or NaN of one request's keys have made NaN of them all, by
    // weights of 0. If any result is not finite, all are computed once more, each of what it sees only. (The
    // lane's number is asked for anew: the sums leave no register to keep it in.)
    float odd = 0.0f;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) odd = fmaf(st.o[b][i], 0.0f, odd);
    int32_t* odds = reinterpret_cast<int32_t*>(tiles);
    const bool mine = __any(odd != 0.0f);
    __syncthreads();  // nobody reads the tiles any more
    if (__lane_id() == 0) odds[wave] = mine;
    __syncthreads();
    int32_t any = 0;
#pragma unroll
    for (int w = 0; w < S::kWaves; ++w) any |= odds[w];
    any = __builtin_amdgcn_readfirstlane(any);
    __syncthreads();  // before the space is taken for tiles
    if (any)
      attend_segments<T, S, kPacked, true>(params_anew(), st, tiles, anew(q0), anew(q1), anew(r), anew(head), anew(split),
                                           wave, __lane_id());
  }
  const int32_t w0 = q0 + wave * 32;
  const int now = here(__lane_id());
  if (w0 + (now & 31) < q1) put<T>(p, st, w0 + (now & 31), head, split, now >> 5);
}

// Joins the parts of the rows' heads: 32 threads for each, 4 elements a
// thread. Rows of no request, or past their request's max_queries, have not
// been computed and are left alone.
constexpr int kJoinBlock = 256, kJoinEach = kValue / 4;

template <class T>
__global__ __launch_bounds__(kJoinBlock) void expand_join_kernel(ExpandParams p) {
  const int64_t at = (int64_t)blockIdx.x * (kJoinBlock / kJoinEach) + threadIdx.x / kJoinEach;
  const int64_t each = (int64_t)p.num_q * p.heads;
  if (at >= each) return;
  const int32_t row = (int32_t)(at / p.heads);
  int lo = 0, hi = p.requests;  // q_starts[lo] <= row < q_starts[hi], if it is in a request
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.q_starts[mid] <= row)
      lo = mid;
    else
      hi = mid;
  }
  if (row < p.q_starts[lo] || row >= p.q_starts[lo + 1] ||
      row - p.q_starts[lo] >= p.tiles * Shape<4>::kRows)
    return;
  float top = -INFINITY;
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) top = fmaxf(top, p.state[(s * each + at) * 2]);
  const float ref = top == -INFINITY ? 0.0f : top;
  f32x4 o = {};
  float sum = 0.0f;
  const int e = threadIdx.x % kJoinEach * 4;
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) {
    const float x = p.state[(s * each + at) * 2], n = p.state[(s * each + at) * 2 + 1];
    if (x == -INFINITY && n == 0.0f) continue;
    const float by = exp2_fast(x - ref);
    sum += n * by;
    o += *reinterpret_cast<const f32x4*>(p.part + (s * each + at) * kValue + e) * by;
  }
  const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
  *reinterpret_cast<u32x2*>(p.out + (at * kValue + e) * 2) =
      u32x2{T::pack(o[0] * by, o[1] * by), T::pack(o[2] * by, o[3] * by)};
  if (p.lse && e == 0) p.lse[at] = (top + log2f(sum)) * kLn2;
}

// Workgroups of a batch, and the parts that its keys are cut into: where four
// waves a workgroup leave half the card's places (two a CU) empty, as many
// as fill them, of 512 keys at least by the requests' mean. Measured with
// 256 / 512 / 1024 keys at least (us): 2 x 164 queries over 4906 keys each, one
// head, 33 / 28 / 41; 8 over 8200, four heads, 29 / 27 / 36; one over 20000, 42 /
// 40 / 39; 1500 over 13500, one head, 163 / 135 / 118; but 4 x 64 over 2064, two
// heads, 18 / 23 / 34 and 8 x 32 over 1532, one head, 17 / 27 / 41.
struct Cut {
  int64_t pairs;
  int32_t longest, splits;
  bool wide;
};
Cut cut_of(int32_t requests, int32_t heads, int32_t queries, int32_t keys, int32_t max_queries) {
  Cut c;
  c.pairs = ((int64_t)requests * heads + 7) / 8 * 8;
  c.longest = max_queries < queries ? max_queries : queries;
  // Eight waves where they fill the card's 256 CUs, if all prompts are of the
  // longest's length. Measured with eight waves and with four (us): 4 x 1024
  // queries behind 15360 earlier tokens, 16 heads (256 workgroups of eight) 619
  // and 668; 2 x 1024 (128) 490 and 346; uneven prompts of up to 777 (240) 42
  // and 33, of up to 1500 (480) 115 and 114. Of the two, the rule takes the slower
  // for 3 x 1024 (192: 517 and 566) and where a last workgroup is mostly empty:
  // 4 x 300 behind 4096, 64 heads, 350 and 308.
  c.wide = c.pairs * (c.longest / 256) >= 256;
  const int64_t groups = (int64_t)requests * heads * ((c.longest + 127) / 128);
  int64_t s = groups > 0 ? 512 / groups : 1;
  const int64_t most = requests > 0 ? keys / requests / 512 : 1;
  if (s > most) s = most;
  c.splits = c.wide || s < 2 ? 1 : s > 64 ? 64 : (int32_t)s;
  return c;
}

template <class T, class S>
int launch_expand(ExpandParams p, const Cut& c, void* stream) {
  p.tiles = (c.longest + S::kRows - 1) / S::kRows;
  p.splits = c.splits;
  const int st = launch(expand_kernel<T, S>, dim3((unsigned)(c.pairs * p.tiles), (unsigned)c.splits),
                        dim3(S::kBlock), p, stream);
  if (st != DSATOPK_OK || c.splits == 1) return st;
  const int64_t each = (int64_t)p.num_q * p.heads;
  constexpr int kPer = kJoinBlock / kJoinEach;
  return launch(expand_join_kernel<T>, dim3((unsigned)((each + kPer - 1) / kPer)), dim3(kJoinBlock), p,
                stream);
}

// The same for the shared form, whose queries stand together: as for one request, but eight
// waves from 160 workgroups of them on (8 x 341 queries behind 2001 keys, 16 heads, 160 whole
// ones: 104 us, by four waves 119; 128 and 192 above).
Cut shared_cut_of(int32_t heads, int32_t queries, int32_t max_keys) {
  Cut c = cut_of(1, heads, queries, max_keys, queries);
  c.wide = (int64_t)heads * (queries / 256) >= 160;
  if (c.wide) c.splits = 1;
  return c;
}
// Tiles that its stretches may have (every one may end in a part of one): there are no more than requests,
// nor, packed, than long runs and what lies between them. Packed where that leaves fewer, and they would be
// several times what the card holds at once. With and without (us), behind 2000 shared keys, 16 heads: 64
// requests of 1 query 127 and 135, 256 of 1 237 and 290, 1000 of 3 319 and 538, 256 of 16 157 and 188; but 18
// of 1 or 2, one head, behind three sets of up to 2244 keys, 87 and 33; and where every run is a tile or more,
// packing has nothing to leave out and its longer walk over the keys costs up to 5%: 2 x 4 prompts of up to 777
// 113 and 107.
struct Tiles {
  int32_t most;
  bool packed;
};
Tiles shared_tiles(int32_t queries, int32_t requests, int64_t each, int rows) {
  const int64_t whole = queries / rows, runs = 2 * ((int64_t)queries / (rows / 2)) + 1;
  const bool packed = requests > runs && each * (whole + requests) > 2048;
  const int64_t n = whole + (packed ? runs : requests);
  return {(int32_t)(n < queries ? n : queries), packed};
}

template <class T, class S>
int launch_shared(ExpandParams p, const Cut& c, void* stream) {
  const Tiles tiles = shared_tiles(p.num_q, p.requests, (int64_t)p.heads * c.splits, S::kRows);
  const int dies = dies_of(p.heads);
  const int64_t groups = dies > 1 ? ((int64_t)tiles.most + dies - 1) / dies * 8 : c.pairs * tiles.most;
  p.tiles = tiles.most;
  p.splits = c.splits;
  const int st = launch(tiles.packed ? expand_shared_kernel<T, S, true> : expand_shared_kernel<T, S, false>,
                        dim3((unsigned)groups, (unsigned)c.splits), dim3(S::kBlock), p, stream);
  if (st != DSATOPK_OK || c.splits == 1) return st;
  p.tiles = INT32_MAX / Shape<4>::kRows;  // every row of a request has been computed
  const int64_t each = (int64_t)p.num_q * p.heads;
  constexpr int kPer = kJoinBlock / kJoinEach;
  return launch(expand_join_kernel<T>, dim3((unsigned)((each + kPer - 1) / kPer)), dim3(kJoinBlock), p,
                stream);
}

size_t part_floats(const Cut& c, int32_t queries, int32_t heads) {
  return c.splits == 1 ? 0 : (size_t)c.splits * queries * heads * (kValue + 2);
}

}  // namespace
}  // namespace dsatopk_serve

using namespace dsatopk_serve;

extern "C" size_t dsatopk_expanded_bytes(int32_t num_requests, int32_t num_heads, int32_t num_queries,
                                         int32_t num_keys, int32_t max_queries) {
  if (num_requests < 1 || num_heads < 1 || num_queries < 1 || num_keys < 0 || max_queries < 1) return 0;
  return part_floats(cut_of(num_requests, num_heads, num_queries, num_keys, max_queries), num_queries,
                     num_heads) * sizeof(float);
}

namespace dsatopk_serve {
namespace {

// Checks and fills what both forms share.
int check_expanded(ExpandParams& p, const void* q, int64_t q_row, int64_t q_head, const void* k,
                   int64_t k_row, int64_t k_head, const void* v, int64_t v_row, int64_t v_head,
                   const void* k_rope, int64_t rope_row, int32_t type, int32_t heads, int32_t nope,
                   int32_t rope, int32_t value, float scale, int32_t causal, const int32_t* q_starts,
                   const int32_t* k_starts, int32_t requests, int32_t queries, int32_t keys,
                   int32_t max_queries, void* out, float* lse) {
  if (requests < 0 || queries < 0 || keys < 0 || max_queries < 0 || heads < 1 || heads > 1024 ||
      nope != kNope || rope != kRope || value != kValue ||
      (type != DSATOPK_BF16 && type != DSATOPK_FP16) || !(scale > 0.0f) || !(scale < INFINITY) ||
      q_row < 0 || q_head < 0 || k_row < 0 || k_head < 0 || v_row < 0 || v_head < 0 || rope_row < 0 ||
      k_row > kMostStride || v_row > kMostStride || rope_row > kMostStride)
    return DSATOPK_ERR_INVALID_ARG;
  if (requests == 0 || queries == 0 || max_queries == 0) return DSATOPK_OK;
  if (!q || !out || !q_starts || !k_starts || (keys && (!k || !v || !k_rope)))
    return DSATOPK_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(k_rope) ||
      (reinterpret_cast<uintptr_t>(out) & 7u) || !aligned4(lse) || q_row % 8 || q_head % 8 || k_row % 8 ||
      k_head % 8 || v_row % 8 || v_head % 8 || rope_row % 8)
    return DSATOPK_ERR_ALIGNMENT;
  p.q = static_cast<const char*>(q);
  p.q_row = q_row * 2;
  p.q_head = q_head * 2;
  p.k = static_cast<const char*>(k);
  p.k_row = k_row * 2;
  p.k_head = k_head * 2;
  p.v = static_cast<const char*>(v);
  p.v_row = v_row * 2;
  p.v_head = v_head * 2;
  p.rope = static_cast<const char*>(k_rope);
  p.rope_row = rope_row * 2;
  p.q_starts = q_starts;
  p.k_starts = k_starts;
  p.requests = requests;
  p.heads = heads;
  p.num_q = queries;
  p.num_k = keys;
  p.causal = causal != 0;
  p.scale2 = scale * kLog2e;
  p.out = static_cast<char*>(out);
  p.lse = lse;
  return DSATOPK_OK;
}

// The workspace of a call that is cut as `c`.
int check_room(ExpandParams& p, const Cut& c, void* workspace, size_t workspace_bytes) {
  if (c.pairs * ((c.longest + 127) / 128) > INT32_MAX) return DSATOPK_ERR_INVALID_ARG;
  if (c.splits == 1) return DSATOPK_OK;
  if (!workspace || workspace_bytes < part_floats(c, p.num_q, p.heads) * sizeof(float))
    return DSATOPK_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned16(workspace)) return DSATOPK_ERR_ALIGNMENT;
  p.part = static_cast<float*>(workspace);
  p.state = p.part + (size_t)c.splits * p.num_q * p.heads * kValue;
  return DSATOPK_OK;
}

}  // namespace
}  // namespace dsatopk_serve

extern "C" int dsatopk_attend_expanded(
    const void* q, int64_t q_row_stride, int64_t q_head_stride, const void* k,
    int64_t k_row_stride, int64_t k_head_stride, const void* v, int64_t v_row_stride,
    int64_t v_head_stride, const void* k_rope, int64_t rope_row_stride, int32_t type,
    int32_t num_heads, int32_t nope_dim, int32_t rope_dim, int32_t value_dim, float scale,
    int32_t causal, const int32_t* q_starts, const int32_t* k_starts, int32_t num_requests,
    int32_t num_queries, int32_t num_keys, int32_t max_queries, void* out, float* lse,
    void* workspace, size_t workspace_bytes, void* stream) {
  ExpandParams p{};
  int st = check_expanded(p, q, q_row_stride, q_head_stride, k, k_row_stride, k_head_stride, v,
                          v_row_stride, v_head_stride, k_rope, rope_row_stride, type, num_heads,
                          nope_dim, rope_dim, value_dim, scale, causal, q_starts, k_starts,
                          num_requests, num_queries, num_keys, max_queries, out, lse);
  if (st != DSATOPK_OK || !p.q) return st;
  const Cut c = cut_of(num_requests, num_heads, num_queries, num_keys, max_queries);
  st = check_room(p, c, workspace, workspace_bytes);
  if (st != DSATOPK_OK) return st;
  const bool bf16 = type == DSATOPK_BF16;
  return c.wide ? bf16 ? launch_expand<Bf16, Shape<8>>(p, c, stream)
                       : launch_expand<Fp16, Shape<8>>(p, c, stream)
         : bf16 ? launch_expand<Bf16, Shape<4>>(p, c, stream)
                : launch_expand<Fp16, Shape<4>>(p, c, stream);
}

extern "C" size_t dsatopk_expanded_shared_bytes(int32_t num_heads, int32_t num_queries,
                                                int32_t max_keys) {
  if (num_heads < 1 || num_queries < 1 || max_keys < 0) return 0;
  return part_floats(shared_cut_of(num_heads, num_queries, max_keys), num_queries, num_heads) *
         sizeof(float);
}

extern "C" int dsatopk_attend_expanded_shared(
    const void* q, int64_t q_row_stride, int64_t q_head_stride, const void* k,
    int64_t k_row_stride, int64_t k_head_stride, const void* v, int64_t v_row_stride,
    int64_t v_head_stride, const void* k_rope, int64_t rope_row_stride, int32_t type,
    int32_t num_heads, int32_t nope_dim, int32_t rope_dim, int32_t value_dim, float scale,
    int32_t causal, const int32_t* q_starts, const int32_t* k_starts, const int32_t* shared_starts,
    const int32_t* shared_lens, int32_t num_requests, int32_t num_queries, int32_t num_keys,
    int32_t max_keys, void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  ExpandParams p{};
  // a query's number and a count of keys are added in 32 bits
  if (num_queries > (1 << 30) || num_keys > (1 << 30) || max_keys < 0) return DSATOPK_ERR_INVALID_ARG;
  int st = check_expanded(p, q, q_row_stride, q_head_stride, k, k_row_stride, k_head_stride, v,
                          v_row_stride, v_head_stride, k_rope, rope_row_stride, type, num_heads,
                          nope_dim, rope_dim, value_dim, scale, causal, q_starts, k_starts,
                          num_requests, num_queries, num_keys, num_queries, out, lse);
  if (st != DSATOPK_OK || !p.q) return st;
  if (!shared_starts || !shared_lens) return DSATOPK_ERR_INVALID_ARG;
  p.shared_starts = shared_starts;
  p.shared_lens = shared_lens;
  const Cut c = shared_cut_of(num_heads, num_queries, max_keys);
  if (c.pairs * shared_tiles(num_queries, num_requests, (int64_t)num_heads * c.splits, 128).most > INT32_MAX) return DSATOPK_ERR_INVALID_ARG;
  st = check_room(p, c, workspace, workspace_bytes);
  if (st != DSATOPK_OK) return st;
  const bool bf16 = type == DSATOPK_BF16;
  return c.wide ? bf16 ? launch_shared<Bf16, Shape<8>>(p, c, stream)
                       : launch_shared<Fp16, Shape<8>>(p, c, stream)
         : bf16 ? launch_shared<Bf16, Shape<4>>(p, c, stream)
                : launch_shared<Fp16, Shape<4>>(p, c, stream);
}
