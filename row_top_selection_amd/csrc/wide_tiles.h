// wide_tiles.h - absorbed latent attention for many heads that read the same
// tokens: 32 heads a wave, 128 a workgroup of four waves, one on a CU.
//
// The products and the softmax are transposed as in latent_tiles.h, by matrix
// instructions of 32 x 32: a vector that is read from LDS feeds twice as many
// products as with 16 heads a wave. The sums of 32 heads (256 registers) and
// their queries (144) leave room for one wave a SIMD, which has to be kept busy by
// itself: the scores of the next 32 tokens are computed before the sums of the
// current ones, and reads are issued up to eight products ahead.
//
// A tile of 32 tokens takes a wave 68 products of 32 cycles, 2176, and the four
// waves' reads of it (278528 bytes) as many cycles of LDS; it is done in 2.35 us,
// about 5600. Between these lie the waits: with copies under way (copy_to_lds) all
// reads are waited for at every eighth product, the last of which has only been
// issued, nine times a tile; and the compiler takes all weights behind the last
// product, not between them. With 16
// heads a wave and eight waves (twice the reads) 64 rows of 16 heads behind 262144
// tokens take 748 us, with these 620 ... 645; behind 16384, up to 1000 own ones, 87 and 79.
#ifndef DSATOPK_WIDE_TILES_H_
#define DSATOPK_WIDE_TILES_H_

#include "latent_tiles.h"

namespace dsatopk_serve {
namespace {

struct Wide {
  static constexpr int kLatent = 512, kRow = kLatent * 2;
  static constexpr int kWaves = 4, kBlock = kWaves * 64, kCols = 32, kLanes = kWaves * kCols;
  static constexpr int kTile = 32, kRing = 4;  // tokens of a tile, tiles in LDS
  static constexpr int kRopeAt = kTile * kRow;
  static constexpr int kBuffer = kRopeAt + kTile * kRopeBytes;
  static constexpr int kCopy = kTile / kWaves;           // tokens that a wave copies
  static constexpr int kCopies = kCopy + kCopy / 8;      // in as many instructions
  static constexpr int kSteps = kLatent / 16, kAll = kSteps + kRope / 16;
  static constexpr int kBlocks = kLatent / 32;
  // What a lane's weights of a tile may add up to before they need another reference, which costs 2.7 us here, a
  // tile 2.35. bfloat16's weights are as exact far from theirs as near it: up to 2^24 (sums stay finite for values up
  // to 2^80). 64 rows of 16 heads behind 16384 tokens and 1000 own ones with scores that spread by 0.9 / 1.7 /
  // 3.5 / 6.9: 85 / 86 / 86 / 96 us, in half precision 86 / 96 / 131 / 147 (64 heads a workgroup 101 ... 106).
  template <class T>
  static constexpr float most() {
    return T::kLift == 0.0f ? 0x1p24f : T::kMost;
  }
};

struct WideState {
  f32x16 o[Wide::kBlocks];
  float top, sum;
};

// A lane's places in a tile, in bytes; the others follow by exclusive or.
struct WidePlaces {
  int row, rope;  // of token lane % 32, step 0 of the contraction
  int column;     // of the column reads of output block 0

  __device__ __forceinline__ explicit WidePlaces(int lane) {
    const int col = lane & 31, half = lane >> 5, in = lane & 15, side = (lane >> 4) & 1;
    row = col * Wide::kRow + ((half ^ swizzle32(col)) << 4);
    rope = Wide::kRopeAt + col * kRopeBytes + ((half ^ swizzle8(col)) << 4);
    const int tok = 4 * half + (in >> 2);
    column = tok * Wide::kRow + (((2 * side + ((in & 3) >> 1)) ^ swizzle32(tok)) << 4) + 8 * (in & 1);
  }
};

// Where a job's tokens are: `len` of them from position `base` of the pages in `list` on.
struct WideTokens {
  Cache c;
  const int32_t* list;
  int32_t base, len, last;  // last: behind the job's last tile

  // The page of token lane % 8 of the wave's share of a tile, -1: none.
  __device__ __forceinline__ int32_t page_of(int32_t tile, int wave, int lane) const {
    const int32_t j = tile * Wide::kTile + wave * Wide::kCopy + lane % Wide::kCopy;
    return tile < last && j < len ? list[(base + j) >> c.page_bits] : -1;
  }
};

// A copy of the wave's share of a tile, in kCopies instructions. Tokens that are not there are
// copied from zeros.
struct WideCopy {
  uint64_t at, rope;  // of token lane % 8; the lane's own of the rotary parts
  uint32_t there;     // a bit for each token

  __device__ __forceinline__ WideCopy(const WideTokens& x, int32_t page, int32_t tile, int wave, int lane) {
    const int32_t j = tile * Wide::kTile + wave * Wide::kCopy + lane % Wide::kCopy;
    const bool is = page >= 0 && page < x.c.pages;
    const char* from = x.c.at + page * x.c.page + ((x.base + j) & ((1 << x.c.page_bits) - 1)) * x.c.token;
    at = (uint64_t)(uintptr_t)(is ? from : zero_row());
    there = (uint32_t)__ballot(is) & ((1u << Wide::kCopy) - 1);
    const int mine = lane >> 3;
    rope = ((uint64_t)(uint32_t)__shfl((int)(at >> 32), mine) << 32 | (uint32_t)__shfl((int)at, mine)) + Wide::kRow +
           ((lane & 7) ^ swizzle8(wave * Wide::kCopy + mine)) * 16;
  }
  __device__ __forceinline__ void piece(char* to, int k, int wave, int lane) const {
    const int first = wave * Wide::kCopy;
    if (k == Wide::kCopy) {
      copy_to_lds(reinterpret_cast<const char*>(rope), to + Wide::kRopeAt + first * kRopeBytes);
    } else {
      const uint64_t base = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(at >> 32), k) << 32 |
                            (uint32_t)__builtin_amdgcn_readlane((int)at, k);
      // (first is a multiple of 8: the bit of the swizzle that it may have is added)
      copy_to_lds(reinterpret_cast<const char*>(base) +
                      (uint32_t)((lane * 16) ^ ((swizzle32(k) | (first >> 3 & 1) << 1) * 16)),
                  to + (first + k) * Wide::kRow);
    }
  }
};

// A product of scores, its sums in vector registers: the accumulation registers
// are all taken by the output's, and the compiler's own choice for every
// product of a kernel that has them. Products that add to the sums of the one before need
// no wait between them; what else reads them goes through settled().
template <class T>
__device__ __forceinline__ void score_first(f32x16& c, u32x4 a, u32x4 b);
template <>
__device__ __forceinline__ void score_first<Bf16>(f32x16& c, u32x4 a, u32x4 b) {
  asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, 0" : "=&v"(c) : "v"(a), "v"(b));
}
template <>
__device__ __forceinline__ void score_first<Fp16>(f32x16& c, u32x4 a, u32x4 b) {
  asm volatile("v_mfma_f32_32x32x16_f16 %0, %1, %2, 0" : "=&v"(c) : "v"(a), "v"(b));
}
template <class T>
__device__ __forceinline__ void score_next(f32x16& c, u32x4 a, u32x4 b);
template <>
__device__ __forceinline__ void score_next<Bf16>(f32x16& c, u32x4 a, u32x4 b) {
  asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
}
template <>
__device__ __forceinline__ void score_next<Fp16>(f32x16& c, u32x4 a, u32x4 b) {
  asm volatile("v_mfma_f32_32x32x16_f16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
}
__device__ __forceinline__ void settled(f32x16& c) {
  asm volatile("s_nop 15\n\ts_nop 7" : "+v"(c));  // 24 cycles; a product of eight passes is read after 11
}

// Reads of a tile's rows, for step i of the scores.
__device__ __forceinline__ u32x4 read_scores(const char* tile, int row, int rope, int i) {
  return *reinterpret_cast<const u32x4*>(i < Wide::kSteps ? tile + (row ^ ((i & 7) << 5)) + (i >> 3) * 256
                                                          : tile + (rope ^ ((i - Wide::kSteps) << 5)));
}

// Reads of a tile's columns, for step n of the sums: output block n % kBlocks, tokens 16 * (n / kBlocks) on.
__device__ __forceinline__ u32x4 read_sums(const char* tile, int column, int n) {
  const int b = n % Wide::kBlocks;
  const char* rows = tile + (n / Wide::kBlocks) * 16 * Wide::kRow + (b >> 2) * 256;
  const u32x2 lo = read_columns(rows + (column ^ ((b & 3) << 6)));
  const u32x2 hi = read_columns(rows + (column ^ ((b & 3) << 6) ^ 32) + 8 * Wide::kRow);
  return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

// The scores of a tile's tokens for the wave's 32 heads.
template <class T>
__device__ __forceinline__ f32x16 wide_scores(const char* tile, const u32x4 (&q)[Wide::kAll], const WidePlaces& places) {
  constexpr int kAhead = 8;
  u32x4 a[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) a[i] = read_scores(tile, places.row, places.rope, i);
  f32x16 s;
#pragma unroll
  for (int i = 0; i < Wide::kAll; ++i) {
    __builtin_amdgcn_sched_barrier(0);
    if (i == 0)
      score_first<T>(s, a[0], q[0]);
    else
      score_next<T>(s, a[i % kAhead], q[i]);
    if (i + kAhead < Wide::kAll) a[i % kAhead] = read_scores(tile, places.row, places.rope, i + kAhead);
  }
  settled(s);
  return s;
}

// Scores of tokens that a lane's head does not see, or that are not there, count nothing.
__device__ __forceinline__ void wide_mask(f32x16& s, uint32_t valid, int32_t seen, int lane) {
  if (valid != ~0u || __any(seen < Wide::kTile)) {
    uint32_t bits = valid;
    if (seen < 32) bits = seen <= 0 ? 0 : bits & ((1u << seen) - 1);
    bits >>= 4 * (lane >> 5);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!((bits >> (8 * (i / 4) + i % 4)) & 1)) s[i] = -INFINITY;
  }
}

// Weights of a tile's tokens, rounded, two in a word, and their sum.
struct Weights {
  uint32_t y[8];
  float sum;

  // Two of them, those of registers 2 * i and 2 * i + 1 of the scores.
  template <class T>
  __device__ __forceinline__ void take(const f32x16& s, int i, float scale2, float ref) {
    const float a = exp2_fast(fmaf(s[2 * i], scale2, -ref)), b = exp2_fast(fmaf(s[2 * i + 1], scale2, -ref));
    sum += a + b;
    y[i] = T::pack(a, b);
  }
};

// One tile, `cur`, the weights of which are there: a copy of a later one, the scores of the one after it, and the
// sums, and those scores become weights. The tiles are told apart so that no read of one
// waits for the copies of another. `valid`, `seen`: as for wide_mask, of the tile after it.
// One wave a SIMD has nobody to fill its pauses: reads are issued kAhead products ahead, also from the scores into
// the sums, and the copy's addresses and instructions stand between the scores' products. That order holds, but the
// reads are waited for all at once, every kAhead products (copy_to_lds); and the weights, written between the sums'
// products, end up behind them.
template <class T>
__device__ __forceinline__ void wide_step(f32x16 (&o)[Wide::kBlocks], Weights& w, const u32x4 (&q)[Wide::kAll],
                                          const char* __restrict__ cur, const char* __restrict__ after,
                                          char* __restrict__ to, const WideTokens& tokens, int32_t& page,
                                          int32_t tile, uint32_t& there, uint32_t valid, int32_t seen,
                                          const WidePlaces& places, float ref, float scale2, int wave, int lane0) {
  const int lane = here(lane0);
  constexpr int kScores = Wide::kAll, kAll = kScores + 2 * Wide::kBlocks, kAhead = 8;
  const int row = here(places.row), rope = here(places.rope), column = here(places.column);
  auto read = [&](int i) {
    return i < kScores ? read_scores(after, row, rope, i) : read_sums(cur, column, i - kScores);
  };
  u32x4 a[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) a[i] = read(i);
  __builtin_amdgcn_sched_barrier(0);
  const WideCopy copy(tokens, page, tile, wave, lane);
  there = copy.there;
  page = tokens.page_of(tile + 1, wave, lane);
  f32x16 s;
#pragma unroll
  for (int i = 0; i < kScores; ++i) {
    __builtin_amdgcn_sched_barrier(0);
    if (i == 0)
      score_first<T>(s, a[0], q[0]);
    else
      score_next<T>(s, a[i % kAhead], q[i]);
    a[i % kAhead] = read(i + kAhead);
    if (i % 4 == 1) copy.piece(to, i / 4, wave, lane);
  }
  settled(s);
  __builtin_amdgcn_sched_barrier(0);
  wide_mask(s, valid, seen, lane);
  Weights next;
  next.sum = 0.0f;
#pragma unroll
  for (int i = kScores; i < kAll; ++i) {
    __builtin_amdgcn_sched_barrier(0);
    const int n = i - kScores, b = n % Wide::kBlocks, g = 4 * (n / Wide::kBlocks);
    o[b] = T::mma32(a[i % kAhead], u32x4{w.y[g], w.y[g + 1], w.y[g + 2], w.y[g + 3]}, o[b]);
    if (i + kAhead < kAll) a[i % kAhead] = read(i + kAhead);
    if (n % 4 == 1) next.take<T>(s, n / 4, scale2, ref);
  }
  w = next;
}

// Tiles `first` to `last` of `len` tokens from position `base` of the pages in
// `list` on. queries() gives the lane's head's, mine() how many of the tokens it sees.
// done(st) gets the sums. Weights are taken by a reference that holds until they
// outgrow it; the loop over tiles is left then, and the sums are brought to another one. An
// `idle` wave, which has no heads, only copies.
template <class T, class Queries, class Mine, class Done>
__device__ __forceinline__ void attend_wide(char* tiles, uint32_t (*masks)[Wide::kWaves], const Cache& c,
                                            const int32_t* list, int32_t base, int32_t len, int32_t first,
                                            int32_t last, bool idle, Queries queries, Mine mine_of, Done done,
                                            int wave, int lane, float scale2) {
  constexpr int kTile = Wide::kTile, kRing = Wide::kRing, kAheadTiles = kRing - 1, kBuffer = Wide::kBuffer;
  const WideTokens tokens{c, list, base, len, last};
  int32_t pages[kAheadTiles + 1];
#pragma unroll
  for (int n = 0; n <= kAheadTiles; ++n) pages[n] = tokens.page_of(first + n, wave, lane);
#pragma unroll
  for (int n = 0; n < kAheadTiles; ++n) {
    const WideCopy copy(tokens, pages[n], first + n, wave, lane);
#pragma unroll
    for (int k = 0; k < Wide::kCopies; ++k) copy.piece(tiles + n * kBuffer, k, wave, lane);
    if (lane == 0) masks[n][wave] = copy.there;
  }
  int32_t page = pages[kAheadTiles];
  // Bits of a tile's tokens, in every lane.
  auto valid_of = [&](int n) { return *reinterpret_cast<const u32x4*>(masks[n % kRing]); };
  auto joined = [&](u32x4 v) {
    static_assert(Wide::kWaves == 4 && Wide::kCopy == 8, "a byte of each wave");
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)(v[0] | v[1] << 8 | v[2] << 16 | v[3] << 24));
  };
  // (for all of them: the compiler lets reads in the loop go ahead of copies only if none are under way when it begins)
  copies_barrier();

  if (idle) {
#pragma unroll 1
    for (int32_t t = first; t < last; ++t) {
      const int n = t - first + kAheadTiles, now = here(lane);
      wait_copies_but<Wide::kCopies>();
      __syncthreads();
      const WideCopy copy(tokens, page, first + n, wave, now);
#pragma unroll
      for (int k = 0; k < Wide::kCopies; ++k) copy.piece(tiles + n % kRing * kBuffer, k, wave, now);
      if (now == 0) masks[n % kRing][wave] = copy.there;
      page = tokens.page_of(first + n + 1, wave, now);
    }
    wait_copies();
    return;
  }
  WideState st;
  st.top = -INFINITY;
  st.sum = 0.0f;
#pragma unroll
  for (int b = 0; b < Wide::kBlocks; ++b) st.o[b] = f32x16{};
  if (first < last) {
    u32x4 q[Wide::kAll];
    const char* qh = queries(lane) + (lane >> 5) * 16;
#pragma unroll
    for (int i = 0; i < Wide::kAll; ++i) q[i] = load16(qh + 32 * i);
    const int32_t mine = mine_of(lane);
    int32_t t = first;
#pragma unroll 1
    while (true) {
      const int now = here(lane);
      const WidePlaces places(now);
      Weights w;
      w.sum = 0.0f;
      {
        f32x16 s = wide_scores<T>(tiles + (t - first) % kRing * kBuffer, q, places);
        wide_mask(s, joined(valid_of(t - first)), mine - t * kTile, now);
        // The reference is 2^kLift below the largest score so far.
        float top = s[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
        top = fmaxf(fmaxf(top, other_half(top)) * scale2 - T::kLift, st.top);
        if (t > first) {
          const float by = st.top == -INFINITY ? 0.0f : exp2_fast(st.top - top);
          st.sum *= by;
          // (block by block from where the loop has them, and back: left alone, the compiler moves them all, at every tile)
#pragma unroll
          for (int b = 0; b < Wide::kBlocks; ++b) {
            asm volatile("" : "+a"(st.o[b]));
            st.o[b] *= by;
            asm volatile("" : "+a"(st.o[b]));
          }
        }
        st.top = top;
#pragma unroll
        for (int i = 0; i < 8; ++i) w.take<T>(s, i, scale2, st.top == -INFINITY ? 0.0f : st.top);
      }
      const float ref = st.top == -INFINITY ? 0.0f : st.top;
      // the first tile is taken as it is (there may be nothing to see in it, or no numbers)
      bool again = true;
#pragma unroll 1
      for (; t < last; ++t) {
        // a head without a reference has to get one where it sees anything, weights that have outgrown it another
        // (no other one helps a sum that is no number)
        if (!again && __any((!(w.sum <= Wide::most<T>()) || (st.top == -INFINITY && mine > t * kTile)) && st.sum == st.sum))
          break;
        again = false;
        st.sum += w.sum;
        const int n = t - first;
        const u32x4 bits = valid_of(n + 1);  // of the tile after this one: there since the barrier before
        // Tile t + 1 has arrived (the next may be under way), and all waves are done with
        // tile t - 1, whose place is the next copy's. (Behind the last tile zeros are copied.)
        wait_copies_but<Wide::kCopies>();
        __syncthreads();
        uint32_t there;
        wide_step<T>(st.o, w, q, tiles + n % kRing * kBuffer, tiles + (n + 1) % kRing * kBuffer,
                     tiles + (n + kAheadTiles) % kRing * kBuffer, tokens, page, t + kAheadTiles, there, joined(bits),
                     mine - (t + 1) * kTile, places, ref, scale2, wave, now);
        if (now == 0) masks[(n + kAheadTiles) % kRing][wave] = there;
      }
      // what is done with the sums next is no reason to have them elsewhere in the loop
#pragma unroll
      for (int b = 0; b < Wide::kBlocks; ++b) asm volatile("" : "+a"(st.o[b]));
      if (t >= last) break;
    }
    st.sum += other_half(st.sum);
  }
  done(st);
  wait_copies();  // before the tiles' space is taken for something else
}

}  // namespace
}  // namespace dsatopk_serve

#endif  // DSATOPK_WIDE_TILES_H_
