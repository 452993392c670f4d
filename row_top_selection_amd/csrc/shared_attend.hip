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
// A block is the heads of several rows, up to 32, 64 or 128, with a head of its own
// row in each lane; a lane counts how many of the tokens its row sees
// (drafted tokens, whose rows see one token more each). Tiles, products and
// softmax are those of one row's heads (latent_tiles.h), but 128 heads of vectors of 512
// have a loop of their own (wide_tiles.h): in four waves, where those of 256 take eight.
//
// How many tokens there are of which kind only the device knows. Each workgroup
// adds up the tiles of all blocks and
// takes its equal share of them, in their order: the end of one block,
// blocks as a whole, the beginning of the last one. So the card is full from
// the first to the last tile whatever the lengths are, and a block has as
// many parts as workgroups worked on it. What one workgroup did alone it
// writes as the result.
//
// 64 rows of 16 heads behind 262144 tokens take 620 ... 645 us, 920 TFLOP/s (a large
// library product reaches 1370): the matrix units are busy two fifths of the
// time, and the reads of LDS, which would fit beside them, are waited for
// (wide_tiles.h). What
// comes on top for shorter work is the parts: 256 workgroups of 128 heads write
// and read 64 MB, 25 us; and 12 us until the first tile is there (share, pages,
// tokens: a chain of loads). 33 groups of 4 drafts behind 2500 ... 5000 tokens: 70 us,
// where reading the tokens takes 23. Every workgroup looks at all groups and rows:
// 20 us for each thousand groups (1000 of one empty row 25 us, 10000 222), 9 for each
// thousand rows of one group (10000: 90 us).
//
// Where little is shared dsatopk_attend_paged, which reads the shared tokens for every row, is
// faster, by 4 to 10 us: up to about 300000 rows times shared tokens of 16 heads (4 rows
// behind 65536 48 and 47 us, 64 behind 4096 48 and 42, 32 behind 16384 58 and 83).

#include <cstddef>
#include <type_traits>

#include "wide_tiles.h"

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
  int32_t groups, table_width, rows, heads;
  int32_t lanes, own_lanes, own_blocks;  // heads of a shared block, of an own one; own blocks of a row
  bool shares, owns;
  float scale2;
  char* out;
  float* lse;
  // Parts: vectors [number, lanes / cols, latent / 4, cols, 4], as the lanes of a product hold them; references
  // and sums [number, lanes, 2]; first and last part of each block [blocks, 2].
  int32_t cols;
  int32_t shared_most, own_most;  // numbers that there are
  float* shared_part;
  float* shared_state;
  int32_t* shared_numbers;
  float* own_part;
  float* own_state;
  int32_t* own_numbers;
};

// The arguments as they are in memory, to be loaded anew: by itself the compiler keeps
// them all in registers, and spills, across the loops over tokens.
using Args = const __attribute__((address_space(4))) SharedParams;
__device__ __forceinline__ Args& args() {
  Args* p = (Args*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *p;
}

constexpr int kTile = 64;   // tokens of a unit of work
// A block costs its tiles and this many: first loads, last sums, the join. With 2 / 4 / 6 / 8, 22 rows of
// 128 heads behind 32768 tokens, 257 own ones, take 337 / 242 / 227 / 226 us, and 64 rows of 16 behind
// 16384, 1000 own, 93 / 81 / 80 / 83.
constexpr int kBegin = 6;
constexpr int kLeast = 2;   // units that a workgroup is started for (4: 31 us for 4 rows behind 512 tokens, 2: 25)
constexpr int kStarts = 1024;  // groups whose starts are kept in LDS

__device__ __forceinline__ int32_t positions(Args& p) {
  return (int32_t)min((int64_t)p.table_width << p.cache.page_bits, (int64_t)(INT32_MAX - kTile));
}
__device__ __forceinline__ int32_t shared_of(Args& p, int32_t g) {
  return p.shares ? min(max(p.shared_lens[g], 0), positions(p)) : 0;
}
__device__ __forceinline__ int32_t length_of(Args& p, int64_t row) {
  return min(max(p.seq_lens[row], 0), positions(p));
}
__device__ __forceinline__ const int32_t* pages_of(Args& p, int64_t row) {
  return p.table + (p.table_rows ? p.table_rows[row] : row) * p.table_stride;
}

// First rows of the groups: of the first one 0, and the last one ends behind the last
// row, whatever the list says.
__device__ __forceinline__ int32_t start_of(Args& p, int32_t g) {
  return g <= 0 ? 0 : g >= p.groups ? p.rows : min(max(p.group_starts[g], 0), p.rows);
}
struct Starts {
  Args& p;
  const int32_t* kept;  // in LDS, if they fit
  __device__ __forceinline__ int32_t operator()(int32_t g) const {
    return p.groups <= kStarts && g < p.groups ? kept[max(g, 0)] : start_of(p, g);
  }
  // The group of a row, a lane by itself.
  __device__ __forceinline__ int32_t of(int32_t row) const {
    int32_t lo = 0, hi = p.groups;
    while (hi - lo > 1) {
      const int32_t mid = (lo + hi) >> 1;
      if ((*this)(mid) <= row)
        lo = mid;
      else
        hi = mid;
    }
    return lo;
  }
};

// Group g's blocks of lanes are numbered from here on, which leaves room for all
// of those of the groups before it.
__device__ __forceinline__ int64_t first_block(Args& p, int32_t start, int32_t g) {
  return (int64_t)start * p.heads / p.lanes + g;
}

// The work in its order: the shared tokens of each group, then the own ones of
// each row; `blocks` times `tiles`.
struct Entry {
  int32_t tiles, blocks;
  __device__ __forceinline__ int64_t units() const { return tiles > 0 ? (int64_t)blocks * (tiles + kBegin) : 0; }
};
__device__ __forceinline__ Entry entry_of(Args& p, const Starts& starts, int32_t e, int32_t& g) {
  if (e < p.groups) {
    const int64_t lanes = (int64_t)max(starts(e + 1) - starts(e), 0) * p.heads;
    return {lanes ? (shared_of(p, e) + kTile - 1) / kTile : 0, (int32_t)((lanes + p.lanes - 1) / p.lanes)};
  }
  const int32_t row = e - p.groups;
  if (g < 0 || starts(g) > row) g = starts.of(row);
  while (g + 1 < p.groups && starts(g + 1) <= row) ++g;
  const int32_t own = length_of(p, row) - shared_of(p, g);
  return {p.owns && own > 0 ? (own + kTile - 1) / kTile : 0, p.own_blocks};
}

// Where a lane's part goes: its vector (4 elements of each `step` floats), and its reference and sum.
struct Slot {
  float *part, *state;
  int32_t step;
};

// This lane's head of a part: into the result if the part is all that there is, else to its place.
template <class T, class P>
__device__ __forceinline__ void put_part(Args& p, const State<P>& st, float top, float sum,
                                         bool whole, int64_t row, int32_t head, const Slot& to, int lane) {
  const int group = lane >> 4;
  if (whole) {
    Joined out{};
    out.heads = p.heads;
    out.splits = 1;
    out.out = p.out;
    out.lse = p.lse;
    put<T, P>(st, top, sum, out, row, head, 0, lane);
    return;
  }
  if (group == 0) {
    to.state[0] = top;
    to.state[1] = sum;
  }
  if (top == -INFINITY && sum == 0.0f) return;  // nothing seen: the join skips it
  float* part = to.part + group * to.step;
#pragma unroll
  for (int b = 0; b < P::kBlocks; ++b) *reinterpret_cast<f32x4*>(part + b * 4 * to.step) = st.o[b];
}

// The same for 32 heads a wave, where register i of block b holds element 32 * b + 8 * (i / 4) + 4 *
// (lane / 32) + i % 4.
template <class T>
__device__ __forceinline__ void put_wide(Args& p, const WideState& st, bool whole, int64_t row, int32_t head,
                                         const Slot& to, int lane) {
  const int half = lane >> 5;
  const float by = whole ? 1.0f / st.sum : 1.0f;
  char* out = p.out + ((row * p.heads + head) * Wide::kLatent + 4 * half) * 2;
  float* part = to.part + half * to.step;
  if (whole) {
    if (p.lse && half == 0) p.lse[row * p.heads + head] = (st.top + log2f(st.sum)) * kLn2;
  } else {
    if (half == 0) {
      to.state[0] = st.top;
      to.state[1] = st.sum;
    }
    if (st.top == -INFINITY && st.sum == 0.0f) return;  // nothing seen: the join skips it
  }
#pragma unroll
  for (int b = 0; b < Wide::kBlocks; ++b)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const f32x4 v = f32x4{st.o[b][i], st.o[b][i + 1], st.o[b][i + 2], st.o[b][i + 3]} * by;
      const u32x2 y = {T::pack(v[0], v[1]), T::pack(v[2], v[3])};
      if (whole)  // (zeros where nothing was seen, whatever others saw)
        *reinterpret_cast<u32x2*>(out + (b * 32 + 2 * i) * 2) = st.sum == 0.0f ? u32x2{} : y;
      else
        *reinterpret_cast<f32x4*>(part + (8 * b + i / 2) * to.step) = v;
    }
}

template <class P>
__device__ __forceinline__ void clear(State<P>& st) {
  st.top = -INFINITY;
  st.sum = 0.0f;
#pragma unroll
  for (int b = 0; b < P::kBlocks; ++b) st.o[b] = f32x4{};
}
// What a workgroup is at, in LDS, for the same reason.
struct Job {
  int64_t at, end;     // units, of all
  int64_t in;          // units into the entry
  int64_t number;      // of the part
  int32_t entry;
  int32_t row0, rows;  // of the group; the row, of own tokens
  int32_t shared, block, first, last;
  int32_t whole;       // the block's only part
};

__device__ __forceinline__ Cache cache_of(Args& p) {
  return Cache{p.cache.at, p.cache.page, p.cache.token, p.cache.pages, p.cache.page_bits};
}
__device__ __forceinline__ int32_t uniform(int32_t x) { return __builtin_amdgcn_readfirstlane(x); }

// The block of lanes of a job: lane i's row, its head, the tokens that it sees; and where its part goes.
struct Block {
  Args& p;
  bool own;
  int32_t row, head, heads, count, shared;
  __device__ __forceinline__ Block(Args& args, const Job& job, int32_t lanes)
      : p(args), own(uniform(job.entry) >= args.groups), heads(args.heads), shared(uniform(job.shared)) {
    const int64_t begin = (int64_t)uniform(job.block) * (own ? p.own_lanes : lanes);
    row = uniform(job.row0) + (int32_t)(begin / heads);
    head = (int32_t)(begin % heads);
    count = (int32_t)min((int64_t)uniform(job.rows) * heads - begin, (int64_t)(own ? p.own_lanes : lanes));
  }
  __device__ __forceinline__ int32_t row_of(int32_t i) const { return row + (head + i) / heads; }
  __device__ __forceinline__ int32_t head_of(int32_t i) const { return (head + i) % heads; }
  // Of a group's shared tokens; of a row's own ones, all.
  __device__ __forceinline__ int32_t sees(int32_t i) const {
    const int32_t len = length_of(p, row_of(i));
    return own ? len - shared : min(len, shared);
  }
  __device__ __forceinline__ const char* queries(int32_t i) const {
    return i < count ? p.q + row_of(i) * p.q_row + head_of(i) * p.q_head : zero_row();
  }
  // Whether the job's part, if it is the block's only one, is all that there is of the row.
  __device__ __forceinline__ bool alone(int32_t i) const {
    return own ? shared == 0 : !p.owns || length_of(p, row_of(i)) <= shared;
  }
  template <class P>
  __device__ __forceinline__ Slot slot(const Job& job, int32_t i) const {
    const int64_t at = job.number * (own ? p.own_lanes : P::kLanes);
    return {(own ? p.own_part : p.shared_part) + at * P::kLatent +
                ((int64_t)(i / P::kCols) * (P::kLatent / 4) * P::kCols + i % P::kCols) * 4,
            (own ? p.own_state : p.shared_state) + (at + i) * 2, P::kCols * 4};
  }
};

// A job's tiles: of a group's shared tokens, or of a row's own.
template <class T, class P, bool kOwn>
__device__ __forceinline__ void attend_job(const Job& job, char* tiles, uint32_t (*masks)[P::kWaves],
                                           float (*joined)[P::kWaves][16], int wave, int lane) {
  constexpr int kLanes = P::kLanes, kPer = kTile / P::kTile;
  int32_t len = 0, base, first, last;  // tokens that any lane sees, and where they begin
  {
    const Block block(args(), job, kLanes);
#pragma unroll
    for (int i = 0; i < kLanes; i += 64)
      if (i + lane < block.count) len = max(len, block.sees(i + lane));
#pragma unroll
    for (int d = 32; d; d >>= 1) len = max(len, __shfl_xor(len, d));
    len = uniform(len);
    base = block.own ? block.shared : 0;
    first = uniform(job.first) * kPer;
    last = min(uniform(job.last) * kPer, (len + P::kTile - 1) / P::kTile);
  }
  // What the lane's head is, and sees, from its place in the workgroup: when it is needed.
  auto queries = [&](int32_t i) { return Block(args(), job, kLanes).queries(i); };
  auto mine = [&](int32_t i) {
    const Block block(args(), job, kLanes);
    return i < block.count ? block.sees(i) : INT32_MAX;
  };
  if constexpr (std::is_same_v<P, Wide>) {
    auto done = [&](const WideState& st) {
      const Block block(args(), job, kLanes);
      const int32_t now = here(lane), i = wave * 32 + now % 32;
      if (i < block.count)
        put_wide<T>(block.p, st, job.whole && block.alone(i), block.row_of(i), block.head_of(i),
                    block.slot<P>(job, i), now);
    };
    Args& p = args();
    const bool idle = wave * 32 >= Block(p, job, kLanes).count;
    attend_wide<T>(tiles, masks, cache_of(p), pages_of(p, uniform(job.row0)), base, len, first, last, idle,
                   [&](int now) { return queries(wave * 32 + now % 32); },
                   [&](int now) { return mine(wave * 32 + now % 32); }, done, wave, lane, p.scale2);
  } else {
    State<P> st;
    clear<P>(st);
    {
      const int32_t i = wave % P::kWH * 16 + (lane & 15);
      // a lane that sees none of the wave's tokens must not ask for a reference at every tile
      if (!kOwn && mine(i) <= first * P::kTile + wave / P::kWH * P::kTokens) st.top = 0.0f;
      Args& p = args();
      const Places<P> places(wave, lane);
      attend_range<T, P, true, !kOwn>(st, tiles, masks, cache_of(p), pages_of(p, uniform(job.row0)), base, len,
                                      first, last, queries(i), kOwn ? 0 : mine(i), places, wave, lane, p.scale2);
    }
    const int32_t now = here(lane), i = wave % P::kWH * 16 + (now & 15);
    float sum = head_sum(st.sum);
    float top = !kOwn && mine(i) <= job.first * kTile + wave / P::kWH * P::kTokens ? -INFINITY : st.top;
    if constexpr (P::kWT > 1) join_groups<P>(st, top, sum, tiles, joined, wave, now);
    const Block block(args(), job, kLanes);
    if (wave / P::kWH == 0 && i < block.count)
      put_part<T, P>(block.p, st, top, sum, job.whole && block.alone(i), block.row_of(i), block.head_of(i),
                     block.slot<P>(job, i), now);
  }
}

__device__ __forceinline__ int64_t uniform(int64_t x) {
  return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int32_t)(x >> 32)) << 32 |
                   (uint32_t)__builtin_amdgcn_readfirstlane((int32_t)x));
}
__device__ __forceinline__ int64_t from_below(int64_t x, int d) {
  return (int64_t)((uint64_t)(uint32_t)__shfl_up((int32_t)(x >> 32), d) << 32 | (uint32_t)__shfl_up((int32_t)x, d));
}

// The next job of a workgroup, from its units: false if there is none. The same in all lanes.
__device__ __forceinline__ bool next_job(Job& job, const Starts& starts, int tid, int lane) {
  Args& p = args();
  const int32_t entries = p.groups + (p.owns ? p.rows : 0);
  int32_t e = uniform(job.entry);
  int64_t in = uniform(job.in), at = uniform(job.at);
  const int64_t end = uniform(job.end);
  __syncthreads();  // before the next one is written
  while (at < end) {
    int32_t g = -1;
    const Entry x = entry_of(p, starts, e, g);
    if (in >= x.units()) {
      // the next entry that has any work, 64 at a time
      in = 0;
      uint64_t some = 0;
      for (++e; e < entries; e += 64) {
        int32_t mine = -1;
        some = __ballot(e + lane < entries && entry_of(p, starts, min(e + lane, entries - 1), mine).units() > 0);
        if (some) break;
      }
      if (!some) return false;
      e += __builtin_ctzll(some);
      continue;
    }
    const int32_t each = x.tiles + kBegin;
    const int32_t block = (int32_t)(in / each), unit = (int32_t)(in - (int64_t)block * each);
    const int32_t n = (int32_t)min((int64_t)(each - unit), end - at);
    const int32_t first = max(unit - kBegin, 0), last = unit + n - kBegin;
    in += n;
    at += n;
    if (last <= first) continue;
    // The parts of a block are numbered as its workgroups are: by the workgroup's
    // number and the block's, of which one at least grows from part to part.
    const bool own = e >= p.groups;
    const int32_t row0 = own ? e - p.groups : starts(e);
    const int64_t which = own ? (int64_t)row0 * p.own_blocks + block : first_block(p, row0, e) + block;
    const int64_t number = which + blockIdx.x;
    if (tid == 0) {
      int32_t* numbers = (own ? p.own_numbers : p.shared_numbers) + which * 2;
      if (first == 0) numbers[0] = (int32_t)number;
      if (last == x.tiles) numbers[1] = (int32_t)number;
      job = Job{at, end, in, number, e, row0, own ? 1 : starts(e + 1) - row0, shared_of(p, own ? g : e), block,
                first, last, first == 0 && last == x.tiles};
    }
    return true;
  }
  return false;
}

// PS for the shared parts, PO for the own ones: workgroups of the same size.
template <class T, class PS, class PO>
__global__ __launch_bounds__(PS::kBlock, (std::is_same_v<PS, Wide> ? 1 : 2)) void shared_kernel(SharedParams) {
  constexpr int kWaves = PS::kWaves;
  constexpr int kSpace = std::is_same_v<PS, Wide> ? Wide::kRing * Wide::kBuffer : 2 * PS::kBuffer;
  static_assert(PS::kBlock == PO::kBlock && 2 * PO::kBuffer <= kSpace, "one launch for both");
  struct Rest {
    Job job;
    int64_t sums[kWaves];
    float joined[2][kWaves][16];
    int32_t kept[kStarts];
    alignas(16) uint32_t masks[Wide::kRing][kWaves];  // (read 16 bytes at a time)
  };
  static_assert(kSpace % 16 == 0 && offsetof(Rest, masks) % 16 == 0, "masks are aligned as they are read");
  __shared__ __attribute__((aligned(1024))) char tiles[kSpace + sizeof(Rest)];
  Rest& rest = *reinterpret_cast<Rest*>(tiles + kSpace);
  auto& job = rest.job;
  auto& sums = rest.sums;
  auto& joined = rest.joined;
  auto& kept = rest.kept;
  auto& masks = rest.masks;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  {
    Args& p = args();
    if (p.groups <= kStarts)
      for (int g = tid; g < p.groups; g += PS::kBlock) kept[g] = start_of(p, g);
    __syncthreads();
    const Starts starts{p, kept};

    // all units, and those before this thread's entries
    const int32_t entries = p.groups + (p.owns ? p.rows : 0);
    const int32_t chunk = (entries + PS::kBlock - 1) / PS::kBlock;
    const int32_t e0 = min(tid * chunk, entries), e1 = min(e0 + chunk, entries);
    int64_t units = 0;
    int32_t g = -1;
    for (int32_t e = e0; e < e1; ++e) units += entry_of(p, starts, e, g).units();
    int64_t below = units;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t o = from_below(below, d);
      if (lane >= d) below += o;
    }
    if (lane == 63) sums[wave] = below;
    __syncthreads();
    int64_t all = 0;
    below -= units;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) below += sums[w];
      all += sums[w];
    }
    const int64_t per = max((all + gridDim.x - 1) / gridDim.x, (int64_t)kLeast);
    const int64_t at = blockIdx.x * per, end = min(at + per, all);
    if (uniform(at) >= uniform(end)) return;
    if (at >= below && at < below + units) {
      g = -1;
      for (int32_t e = e0; e < e1; ++e) {
        const int64_t n = entry_of(p, starts, e, g).units();
        if (at < below + n) {
          job.at = at;
          job.end = end;
          job.in = at - below;
          job.entry = e;
          break;
        }
        below += n;
      }
    }
  }
  while (true) {
    __syncthreads();  // the job is there, the tiles' space is free
    const int now = here(tid);  // what is made of it is made in every round, not kept across them
    if (!next_job(job, Starts{args(), kept}, now, now & 63)) return;
    __syncthreads();
    if (!std::is_same_v<PS, PO> && uniform(job.entry) >= args().groups)
      attend_job<T, PO, true>(job, tiles, masks, joined, wave, now & 63);
    else
      attend_job<T, PS, false>(job, tiles, masks, joined, wave, now & 63);
  }
}

// Joins the parts of 32 heads, 8 elements of each: a lane's are 4 elements of its head, and wave w of kSides takes
// every kSides-th part from w on, four at a time, by the largest reference so far; then wave 0 joins
// the waves' sums. Parts are as the products' lanes left them, so that a load of a wave is of
// whole lines. What is a single part has been written as the result.
constexpr int kPlaces = 512;  // workgroups at most, and so parts of a block but one
constexpr int kXcds = 8;
constexpr int kFew = 16;  // waves that join few heads' parts

// Parts of a block, by its first and last number. Starts that do not rise may leave blocks that nobody
// has numbered: they have none.
__device__ __forceinline__ int32_t parts_of(const int32_t* numbers, int32_t most) {
  const int32_t a = numbers[0], b = numbers[1];
  return a >= 0 && a <= b && b < most && b - a <= kPlaces ? b - a + 1 : 0;
}

template <class T, int kLatent, int kSides>
__global__ __launch_bounds__(kSides * 64) void shared_join_kernel(SharedParams) {
  Args& p = args();
  constexpr int kPairs = kLatent / 8, kAtOnce = 4;
  __shared__ __attribute__((aligned(16))) char space[kSides * 64 * 24];
  f32x4* vectors = reinterpret_cast<f32x4*>(space);
  float* tops = reinterpret_cast<float*>(space + kSides * 64 * 16);
  float* sums = tops + kSides * 64;
  const int tid = threadIdx.x, lane = tid & 63, side = tid >> 6;
  // Workgroups of the same heads on the same die, whose cache puts their results together; those of few heads on
  // all of them (32 heads of 512 parts: 13.5 us, on one die 22.9).
  constexpr uint32_t kDies = kSides == kFew ? 1 : kXcds;
  const uint32_t set = blockIdx.x / kDies;
  const int64_t heads = (int64_t)p.rows * p.heads, x0 = ((int64_t)(set / kPairs) * kDies + blockIdx.x % kDies) * 32;
  const int32_t e4 = (set % kPairs) * 2 + (lane >> 5);
  if (x0 >= heads) return;
  const int64_t x = min(x0 + (lane & 31), heads - 1);
  const int32_t row = (int32_t)(x / p.heads), head = (int32_t)(x - (int64_t)row * p.heads);
  int32_t g = last_below(p.groups, (int32_t)(x0 / p.heads), lane, [&](int32_t i) { return (int64_t)start_of(p, i); });
  while (g + 1 < p.groups && start_of(p, g + 1) <= row) ++g;
  const int32_t shared = shared_of(p, g);
  int32_t n = 0, m = 0;  // shared parts, own parts
  int64_t first = 0, own = 0;
  const int32_t start = start_of(p, g);
  // (where starts do not rise a row may be before its group: no part is its own then)
  if (shared > 0 && start <= row) {
    const int64_t i = x - (int64_t)start * p.heads;
    const int32_t* numbers = p.shared_numbers + (first_block(p, start, g) + i / p.lanes) * 2;
    n = parts_of(numbers, p.shared_most);
    first = (int64_t)(n ? numbers[0] : 0) * p.lanes + i % p.lanes;
  }
  if (p.owns && length_of(p, row) > shared) {
    const int32_t* numbers = p.own_numbers + ((int64_t)row * p.own_blocks + head / p.own_lanes) * 2;
    m = parts_of(numbers, p.own_most);
    own = (int64_t)(m ? numbers[0] : 0) * p.own_lanes + head % p.own_lanes;
  }
  const int32_t parts = n + m, cols = p.cols;
  // (lanes of a block are a multiple of cols)
  auto vector = [&](const float* part, int64_t at) {
    return part + (at / cols * cols * (kLatent / 4) + (int64_t)e4 * cols + at % cols) * 4;
  };
  const float* shared_part = vector(p.shared_part, first);
  const float* own_part = vector(p.own_part, own);
  const float *shared_state = p.shared_state + first * 2, *own_state = p.own_state + own * 2;

  float top = -INFINITY, sum = 0.0f;
  f32x4 o = {};
  auto join = [&](const float (&tops)[kAtOnce], const float (&ns)[kAtOnce], const f32x4 (&v)[kAtOnce]) {
    float most = top;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) most = fmaxf(most, tops[k]);
    const float ref = most == -INFINITY ? 0.0f : most;
    const float by = exp2_fast(top - ref);
    o *= by;
    sum *= by;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (tops[k] == -INFINITY && ns[k] == 0.0f) continue;  // such a part has no vector
      const float f = exp2_fast(tops[k] - ref);
      o += v[k] * f;
      sum += ns[k] * f;
    }
    top = most;
  };
  for (int32_t s = side; s < parts; s += kAtOnce * kSides) {
    float xs[kAtOnce], ns[kAtOnce];
    f32x4 v[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int32_t i = s + k * kSides;
      xs[k] = -INFINITY;
      ns[k] = 0.0f;
      v[k] = f32x4{};
      if (i >= parts) continue;
      const int64_t skip = i < n ? (int64_t)i * p.lanes : (int64_t)(i - n) * p.own_lanes;
      const float* state = (i < n ? shared_state : own_state) + skip * 2;
      xs[k] = state[0];
      ns[k] = state[1];
      v[k] = *reinterpret_cast<const f32x4*>((i < n ? shared_part : own_part) + skip * kLatent);
    }
    join(xs, ns, v);
  }
  if (side) {
    vectors[tid] = o;
    tops[tid] = top;
    sums[tid] = sum;
  }
  __syncthreads();
  if (side || parts == 1 || x0 + (lane & 31) >= heads) return;
  for (int s = 1; s < kSides; s += kAtOnce) {
    float xs[kAtOnce], ns[kAtOnce];
    f32x4 v[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const bool is = s + k < kSides;
      xs[k] = is ? tops[(s + k) * 64 + lane] : -INFINITY;
      ns[k] = is ? sums[(s + k) * 64 + lane] : 0.0f;
      v[k] = is ? vectors[(s + k) * 64 + lane] : f32x4{};
    }
    join(xs, ns, v);
  }
  const float scale = sum == 0.0f ? 0.0f : 1.0f / sum;
  *reinterpret_cast<u32x2*>(p.out + (x * kLatent + e4 * 4) * 2) =
      u32x2{T::pack(o[0] * scale, o[1] * scale), T::pack(o[2] * scale, o[3] * scale)};
  if (p.lse && e4 == 0) p.lse[x] = (top + log2f(sum)) * kLn2;
}

// How a call is cut: heads packed into a workgroup for the shared tokens and for a
// row's own, workgroups, and numbers that blocks and parts may have.
struct Cut {
  int32_t lanes, cols, own_lanes, own_blocks, places;
  int64_t shared_blocks, own;
  size_t shared_parts, own_parts;  // lanes of all parts
  int32_t latent;

  Cut(int32_t rows, int32_t heads, int32_t latent, int32_t groups, int64_t max_shared, int64_t max_own)
      : latent(latent) {
    const bool shares = max_shared > 0, owns = max_own > 0 || !shares;
    const int64_t each = ((int64_t)rows + groups - 1) / groups * heads;  // lanes of a mean group
    lanes = each <= 32 ? 32 : each <= 64 ? 64 : 128;
    // 64 lanes, two workgroups a CU, also for larger groups, where their tiles are few for each workgroup or
    // most are single rows' of few heads, which leave waves of 32 heads idle. Measured with 64 and with
    // 128 (us), 16 heads: 8 rows behind 2048 tokens and 200 own ones 26 and 33, 32 behind 4096 38 and 39, behind
    // 16384 and 1000 own ones 59 and 59, 64 behind 16384 83 and 74, behind 65536 220 and 173; 128 rows of 2000 own
    // tokens 73 and 97. With vectors of 256, in the same order: 22 and 24, 30 and 31, 40 and 41, 51 and 49, 122 and
    // 109; 22 rows of 128 heads behind 32768 159 and 141; but 64 of 16 behind 16384 and 1000 own ones 54 and 58.
    const double shared_tiles = (double)((max_shared + kTile - 1) / kTile) * (double)((int64_t)rows * heads / 64 + groups);
    const double own_tiles = owns ? (double)((max_own + kTile - 1) / kTile) * rows * ((heads + 63) / 64) : 0.0;
    if (lanes == 128 && (shared_tiles + own_tiles <= 8.0 * kPlaces || (heads <= 64 && own_tiles >= 4.0 * shared_tiles)))
      lanes = 64;
    const int32_t most = heads <= 32 ? 32 : heads <= 64 || lanes == 64 ? 64 : 128;
    cols = lanes == 128 && latent == Wide::kLatent ? Wide::kCols : 16;
    own_lanes = heads < most ? (heads + cols - 1) / cols * cols : most;
    own_blocks = (heads + most - 1) / most;
    shared_blocks = shares ? (int64_t)rows * heads / lanes + groups : 0;
    own = owns ? (int64_t)rows * own_blocks : 0;
    // as many as run at once, or as the bounds have work for
    const double units = (double)shared_blocks * (double)((max_shared + kTile - 1) / kTile + kBegin) +
                         (double)own * (double)((max_own + kTile - 1) / kTile + kBegin);
    const int32_t most_places = lanes == 128 ? 256 : kPlaces;
    places = units / kLeast >= most_places ? most_places : 1 + (int32_t)(units / kLeast);
    shared_parts = shares ? (size_t)(shared_blocks + places) * lanes : 0;
    own_parts = owns ? (size_t)(own + places) * own_lanes : 0;
  }
  size_t bytes() const {
    return (shared_parts + own_parts) * (latent + 2) * sizeof(float) +
           ((size_t)(shared_blocks + own) * 2 * sizeof(int32_t) + 15) / 16 * 16;
  }
};

template <class T, class PS, class PO>
int launch_parts(const SharedParams& p, const Cut& c, void* stream) {
  return launch(shared_kernel<T, PS, PO>, dim3((unsigned)c.places), dim3(PS::kBlock), p, stream);
}

template <class T, int kLatent>
int launch_cut(const SharedParams& p, const Cut& c, void* stream) {
  using Two = Plan<2, 2, 32, kLatent>;
  using Four = Plan<4, 1, 32, kLatent>;
  if (c.lanes == 32) return launch_parts<T, Two, Two>(p, c, stream);
  if (c.lanes == 64)
    return p.heads <= 32 ? launch_parts<T, Four, Two>(p, c, stream) : launch_parts<T, Four, Four>(p, c, stream);
  if constexpr (kLatent == Wide::kLatent)
    return launch_parts<T, Wide, Wide>(p, c, stream);
  else
    return p.heads <= 32   ? launch_parts<T, Plan<8, 1, 64, kLatent>, Plan<2, 4, 64, kLatent>>(p, c, stream)
           : p.heads <= 64 ? launch_parts<T, Plan<8, 1, 64, kLatent>, Plan<4, 2, 64, kLatent>>(p, c, stream)
                           : launch_parts<T, Plan<8, 1, 64, kLatent>, Plan<8, 1, 64, kLatent>>(p, c, stream);
}

template <class T, int kLatent>
int launch_shared(SharedParams p, const Cut& c, void* workspace, void* stream) {
  p.lanes = c.lanes;
  p.own_lanes = c.own_lanes;
  p.own_blocks = c.own_blocks;
  p.cols = c.cols;
  p.shared_most = (int32_t)(c.shared_blocks + c.places);
  p.own_most = (int32_t)(c.own + c.places);
  p.shared_part = static_cast<float*>(workspace);
  p.own_part = p.shared_part + c.shared_parts * kLatent;
  p.shared_state = p.own_part + c.own_parts * kLatent;
  p.own_state = p.shared_state + c.shared_parts * 2;
  p.shared_numbers = reinterpret_cast<int32_t*>(p.own_state + c.own_parts * 2);
  p.own_numbers = p.shared_numbers + c.shared_blocks * 2;
  const int st = launch_cut<T, kLatent>(p, c, stream);
  if (st != DSATOPK_OK) return st;
  const int64_t tiles = ((int64_t)p.rows * p.heads + 31) / 32;
  const auto grid = [&](int64_t dies) {
    return dim3((unsigned)((tiles + dies - 1) / dies * dies * (kLatent / 8)));
  };
  // A wave by itself for many heads (2112 heads of 16 parts: 12.6 us, 20.4 by four); few are too few waves to have
  // the memory busy (1024 heads of 33 parts: 11.7 us by four, 14.5 by eight), and may have a part of every workgroup.
  return tiles >= 64   ? launch(shared_join_kernel<T, kLatent, 1>, grid(kXcds), dim3(64), p, stream)
         : tiles >= 16 ? launch(shared_join_kernel<T, kLatent, 4>, grid(kXcds), dim3(256), p, stream)
                       : launch(shared_join_kernel<T, kLatent, kFew>, grid(1), dim3(kFew * 64), p, stream);
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
  return Cut(num_rows, num_heads, latent_dim, num_groups, max_shared_len, max_own_len).bytes();
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
  p.shares = max_shared_len > 0;
  p.owns = max_own_len > 0 || !p.shares;
  const Cut c(num_rows, num_heads, latent_dim, num_groups, max_shared_len, max_own_len);
  // parts are numbered, and the join's threads counted, in 32 bits
  if ((int64_t)num_rows * num_heads * (latent_dim / 4) > INT32_MAX || c.shared_blocks + kPlaces > INT32_MAX ||
      c.own + kPlaces > INT32_MAX || (int64_t)num_groups + num_rows > INT32_MAX)
    return DSATOPK_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < c.bytes()) return DSATOPK_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned16(workspace)) return DSATOPK_ERR_ALIGNMENT;
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
  p.rows = num_rows;
  p.heads = num_heads;
  p.out = static_cast<char*>(out);
  p.lse = lse;
  if (type == DSATOPK_BF16)
    return latent_dim == 256 ? launch_shared<Bf16, 256>(p, c, workspace, stream)
                             : launch_shared<Bf16, 512>(p, c, workspace, stream);
  return latent_dim == 256 ? launch_shared<Fp16, 256>(p, c, workspace, stream)
                           : launch_shared<Fp16, 512>(p, c, workspace, stream);
}

}  // extern "C"
