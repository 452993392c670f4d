// append_cache.hip - a step's new tokens into the paged caches
// (dsatopk_append_latent and dsatopk_append_index in include/dsatopk.h).
//
// The rotary part of a vector is 32 pairs (a, b), turned by the angles of the
// token's position, cos and sin of which come from a table:
//
//   a' = a cos - b sin,   b' = a sin + b cos
//
// A latent vector's other elements are normalised by their root mean square,
// x / sqrt(mean x^2 + eps) * w; an indexer key is normalised as a whole, (x -
// mean) / sqrt(var + eps) * w + b, before its first 64 elements are turned.
// With 8-bit keys and queries, y becomes e4m3(y / s), s = max |y| / 448, and a
// query's s goes into its head's weight.
//
// Everything is read and written once, 16 bytes a lane. A vector of 8n elements
// is n neighbouring lanes' (8 for a rotary part), so that sums and
// maxima stay inside a row of 16 lanes, or a wave; a lane has up to four loads
// in flight, of four tokens, or of four heads of one token, which share the
// angles. The tokens' workgroups come first in the launch, those of the
// queries behind them. fp32 throughout, one rounding at the end.
//
// Long steps move memory as fast as a large copy does: 14 k tokens with the
// rotary parts of 128 heads 98 us (490 MB, 5.0 TB/s), 15 k tokens with 64 heads of
// indexer queries to 8 bits 69 us (374 MB, 5.4 TB/s; a copy 4.85). 128 single tokens take 5.6
// and 4.5 us, which are one dependent chain of loads and the launch.

#include <initializer_list>

#include "serve_common.h"

namespace dsatopk_serve {
namespace {

constexpr int kRope = 64, kRopeLanes = kRope / 8;
constexpr int kBlock = 256;
constexpr int kRun = 4;  // tokens (heads) a lane takes at once

// What both calls know of the tokens and of where their vectors go.
struct Tokens {
  const int32_t* slots;
  const int32_t* row_lens;
  const float* angles;  // [positions, angle_row]: 32 cosines, 32 sines
  int64_t angle_row;
  int32_t tokens, positions, page_bits;
  int64_t num_pages;
  char* cache;
  int64_t page, token;  // bytes
};

struct LatentParams {
  Tokens t;
  const char* x;
  int64_t x_row;  // bytes, as all of these
  const float* weight;
  float eps;
  char* out;
  int64_t out_row;
  const char* q;
  int64_t q_row, q_head;
  char* q_out;
  int64_t q_out_row, q_out_head;
  int32_t heads, runs;  // runs: of kRun heads, a token
  uint32_t token_groups;
};

struct IndexParams {
  Tokens t;
  const char* x;
  int64_t x_row;
  const float* weight;
  const float* bias;
  float eps;
  float* scales;
  int64_t scale_page;  // floats
  const char* q;
  int64_t q_row, q_head;
  char* q_out;
  int64_t q_out_row, q_out_head;
  const float* weights;
  int64_t weights_row;
  float* weights_out;
  int64_t weights_out_row;
  int32_t heads, runs;
  uint32_t token_groups;
};

struct Eight {
  float v[8];
};

template <class T>
__device__ __forceinline__ Eight widen(u32x4 x) {
  Eight e;
#pragma unroll
  for (int i = 0; i < 4; ++i) T::unpack(x[i], e.v[2 * i], e.v[2 * i + 1]);
  return e;
}

template <class T>
__device__ __forceinline__ u32x4 narrow(const Eight& e) {
  return u32x4{T::pack(e.v[0], e.v[1]), T::pack(e.v[2], e.v[3]), T::pack(e.v[4], e.v[5]),
               T::pack(e.v[6], e.v[7])};
}

// Eight floats, rounded to e4m3 (nearest even).
__device__ __forceinline__ u32x2 narrow8(const Eight& e) {
  u32x2 w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int low = __builtin_amdgcn_cvt_pk_fp8_f32(e.v[4 * i], e.v[4 * i + 1], 0, false);
    w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(e.v[4 * i + 2], e.v[4 * i + 3], low, true);
  }
  return w;
}

// A lane's value from another lane of its row of 16.
template <int kControl>
__device__ __forceinline__ float from_lane(float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), kControl, 0xf, 0xf, false));
}
constexpr int kSwap1 = 0xb1, kSwap2 = 0x4e, kReverse4 = 0x1b, kMirror8 = 0x141, kMirror16 = 0x140;

// f over kLanes neighbouring lanes, the same in all of them.
template <int kLanes, class F>
__device__ __forceinline__ float over_lanes(float x, F f) {
  static_assert(kLanes == 8 || kLanes == 16 || kLanes == 32 || kLanes == 64, "a vector's lanes");
  x = f(x, from_lane<kSwap1>(x));
  x = f(x, from_lane<kSwap2>(x));
  x = f(x, from_lane<kMirror8>(x));
  if constexpr (kLanes > 8) x = f(x, from_lane<kMirror16>(x));
  if constexpr (kLanes > 16) x = f(x, __shfl_xor(x, 16));
  if constexpr (kLanes > 32) x = f(x, __shfl_xor(x, 32));
  return x;
}
template <int kLanes>
__device__ __forceinline__ float sum_lanes(float x) {
  return over_lanes<kLanes>(x, [](float a, float b) { return a + b; });
}
template <int kLanes>
__device__ __forceinline__ float max_lanes(float x) {
  return over_lanes<kLanes>(x, [](float a, float b) { return fmaxf(a, b); });
}

// Cosines and sines that lane `chunk` of a rotary part's 8 needs: of its four
// pairs if they are neighbours, else of the eight that it has one side of.
// Without a position elements stay as they are (turned by nothing, one beside an infinite one
// would be NaN).
template <bool kNear>
struct Turn {
  static constexpr int kN = kNear ? 4 : 8;
  bool there;
  float cos[kN], sin[kN];

  __device__ __forceinline__ Turn(const Tokens& t, int32_t position, int chunk)
      : there(position >= 0 && position < t.positions) {
    const float* at = t.angles + (there ? position : 0) * t.angle_row + (kNear ? 4 * chunk : 8 * (chunk & 3));
#pragma unroll
    for (int i = 0; i < kN; i += 4) {
      f32x4 c = {}, s = {};
      if (there) {
        c = *reinterpret_cast<const f32x4*>(at + i);
        s = *reinterpret_cast<const f32x4*>(at + kRope / 2 + i);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        cos[i + j] = c[j];
        sin[i + j] = s[j];
      }
    }
    if (!kNear && chunk < 4) {
#pragma unroll
      for (int i = 0; i < kN; ++i) sin[i] = -sin[i];
    }
  }

  // All 8 lanes of the rotary part are there.
  __device__ __forceinline__ void operator()(Eight& e) const {
    if constexpr (kNear) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = e.v[2 * i], b = e.v[2 * i + 1];
        e.v[2 * i] = there ? a * cos[i] - b * sin[i] : a;
        e.v[2 * i + 1] = there ? a * sin[i] + b * cos[i] : b;
      }
    } else {
      // the other side of the pairs is four lanes away: mirrored in 8, then in 4
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float other = from_lane<kReverse4>(from_lane<kMirror8>(e.v[i]));
        e.v[i] = there ? e.v[i] * cos[i] + other * sin[i] : e.v[i];
      }
    }
  }
};

// Where token i's cache entry is, or null: no slot, a page that the cache does
// not have, no position in the angles' table.
__device__ __forceinline__ char* entry_of(const Tokens& t, int32_t slot, int32_t position) {
  const int64_t page = slot >> t.page_bits;
  if (slot < 0 || page >= t.num_pages || position < 0 || position >= t.positions) return nullptr;
  return t.cache + page * t.page + (slot & ((1 << t.page_bits) - 1)) * t.token;
}

__device__ __forceinline__ void store16(char* to, u32x4 v) { *reinterpret_cast<u32x4*>(to) = v; }

template <class T, int kLatent, bool kNear>
__global__ __launch_bounds__(kBlock) void append_latent_kernel(LatentParams p) {
  const int tid = threadIdx.x;
  if (blockIdx.x >= p.token_groups) {
    // queries: 8 lanes take the rotary parts of kRun heads of a token
    const int chunk = tid % kRopeLanes;
    const int64_t item = (int64_t)(blockIdx.x - p.token_groups) * (kBlock / kRopeLanes) + tid / kRopeLanes;
    const int32_t token = (int32_t)(item / p.runs), head = (int32_t)(item % p.runs) * kRun;
    if (token >= p.t.tokens) return;
    const Turn<kNear> turn(p.t, p.t.row_lens[token] - 1, chunk);
    const char* q = p.q + token * p.q_row + head * p.q_head + chunk * 16;
    char* to = p.q_out + token * p.q_out_row + head * p.q_out_head + chunk * 16;
    u32x4 x[kRun];
#pragma unroll
    for (int i = 0; i < kRun; ++i)
      if (head + i < p.heads) x[i] = load16(q + i * p.q_head);
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      if (head + i >= p.heads) continue;
      Eight e = widen<T>(x[i]);
      turn(e);
      store16(to + i * p.q_out_head, narrow<T>(e));
    }
    return;
  }

  // tokens: kRun for each set of kLanes lanes of a wave, one after the other
  constexpr int kLanes = kLatent / 8, kSets = 64 / kLanes;
  const int lane = tid & 63, at = lane % kLanes;
  const int32_t first = ((int32_t)blockIdx.x * (kBlock / 64) + (tid >> 6)) * kRun * kSets;
  if (first >= p.t.tokens) return;
  u32x4 x[kRun];
  char* to[kRun];
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    const int32_t token = first + i * kSets + lane / kLanes;
    to[i] = nullptr;
    x[i] = u32x4{};
    if (token < p.t.tokens) {
      to[i] = entry_of(p.t, p.t.slots[token], p.t.row_lens[token] - 1);
      if (to[i] || p.out) x[i] = load16(p.x + token * p.x_row + at * 16);
    }
  }
  // the rotary parts of the same tokens: 8 lanes for each
  constexpr int kTurned = kRun * kSets;  // at most 8
  const int32_t mine = first + lane / kRopeLanes;
  const bool turns = lane / kRopeLanes < kTurned && mine < p.t.tokens;
  const int chunk = lane % kRopeLanes;
  u32x4 rope = {};
  char* rope_to = nullptr;
  int32_t position = -1;
  if (turns) {
    position = p.t.row_lens[mine] - 1;
    rope_to = entry_of(p.t, p.t.slots[mine], position);
    if (rope_to || p.out) rope = load16(p.x + mine * p.x_row + kLatent * 2 + chunk * 16);
  }
  Eight w;
  if (p.weight) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p.weight + at * 8);
    const f32x4 b = *reinterpret_cast<const f32x4*>(p.weight + at * 8 + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w.v[j] = a[j];
      w.v[4 + j] = b[j];
    }
  }
  if (turns) {
    const Turn<kNear> turn(p.t, position, chunk);
    Eight e = widen<T>(rope);
    turn(e);
    const u32x4 v = narrow<T>(e);
    if (rope_to) store16(rope_to + kLatent * 2 + chunk * 16, v);
    if (p.out) store16(p.out + mine * p.out_row + kLatent * 2 + chunk * 16, v);
  }
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    u32x4 v = x[i];
    if (p.weight) {
      Eight e = widen<T>(v);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(e.v[j], e.v[j], sum);
      const float by = 1.0f / sqrtf(sum_lanes<kLanes>(sum) * (1.0f / kLatent) + p.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) e.v[j] *= by * w.v[j];
      v = narrow<T>(e);
    }
    const int32_t token = first + i * kSets + lane / kLanes;
    if (to[i]) store16(to[i] + at * 16, v);
    if (p.out && token < p.t.tokens) store16(p.out + token * p.out_row + at * 16, v);
  }
}

// The largest element that a scale is taken from is at least this: the scale
// and its inverse stay normal numbers, and a vector of zeros is zeros.
constexpr float kLeast = 0x1p-100f;
constexpr float kMost8 = 448.0f;

// y in 8 bits, its lanes' scale in `scale`.
template <int kLanes>
__device__ __forceinline__ u32x2 eight_bits(Eight e, float& scale) {
  float most = kLeast;
#pragma unroll
  for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(e.v[j]));
  most = max_lanes<kLanes>(most);
  scale = most * (1.0f / kMost8);
  const float by = kMost8 / most;
#pragma unroll
  for (int j = 0; j < 8; ++j) e.v[j] *= by;
  return narrow8(e);
}

template <class T, int kDim, bool kNear, bool kEight>
__global__ __launch_bounds__(kBlock) void append_index_kernel(IndexParams p) {
  constexpr int kLanes = kDim / 8, kSets = kBlock / kLanes;
  constexpr int kOut = kEight ? 8 : 16;  // bytes of a lane's result
  const int tid = threadIdx.x, at = tid % kLanes;
  const bool turns = at < kRopeLanes;
  if (blockIdx.x >= p.token_groups) {
    // queries: kLanes lanes take kRun heads of a token
    const int64_t item = (int64_t)(blockIdx.x - p.token_groups) * kSets + tid / kLanes;
    const int32_t token = (int32_t)(item / p.runs), head = (int32_t)(item % p.runs) * kRun;
    if (token >= p.t.tokens) return;
    const Turn<kNear> turn(p.t, turns ? p.t.row_lens[token] - 1 : -1, at);
    const char* q = p.q + token * p.q_row + head * p.q_head + at * 16;
    char* to = p.q_out + token * p.q_out_row + head * p.q_out_head + at * kOut;
    u32x4 x[kRun];
    float weight[kRun];
#pragma unroll
    for (int i = 0; i < kRun; ++i)
      if (head + i < p.heads) {
        x[i] = load16(q + i * p.q_head);
        if (kEight && at == 0) weight[i] = p.weights[token * p.weights_row + head + i];
      }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      if (head + i >= p.heads) continue;
      Eight e = widen<T>(x[i]);
      turn(e);
      if constexpr (kEight) {
        float scale;
        *reinterpret_cast<u32x2*>(to + i * p.q_out_head) = eight_bits<kLanes>(e, scale);
        if (at == 0) p.weights_out[token * p.weights_out_row + head + i] = weight[i] * scale;
      } else {
        store16(to + i * p.q_out_head, narrow<T>(e));
      }
    }
    return;
  }

  const int32_t token = (int32_t)blockIdx.x * kSets + tid / kLanes;
  if (token >= p.t.tokens) return;
  const int32_t slot = p.t.slots[token], position = p.t.row_lens[token] - 1;
  char* to = entry_of(p.t, slot, position);
  if (!to) return;
  Eight e = widen<T>(load16(p.x + token * p.x_row + at * 16));
  const Turn<kNear> turn(p.t, turns ? position : -1, at);
  if (p.weight) {
    Eight w, b;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const f32x4 u = *reinterpret_cast<const f32x4*>(p.weight + at * 8 + i);
      const f32x4 v = *reinterpret_cast<const f32x4*>(p.bias + at * 8 + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w.v[i + j] = u[j];
        b.v[i + j] = v[j];
      }
    }
    float sum = 0.0f, squares = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += e.v[j];
    const float mean = sum_lanes<kLanes>(sum) * (1.0f / kDim);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      e.v[j] -= mean;
      squares = fmaf(e.v[j], e.v[j], squares);
    }
    const float by = 1.0f / sqrtf(sum_lanes<kLanes>(squares) * (1.0f / kDim) + p.eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) e.v[j] = fmaf(e.v[j] * by, w.v[j], b.v[j]);
  }
  turn(e);
  if constexpr (kEight) {
    float scale;
    *reinterpret_cast<u32x2*>(to + at * 8) = eight_bits<kLanes>(e, scale);
    if (at == 0) {
      const int64_t page = slot >> p.t.page_bits;
      p.scales[page * p.scale_page + (slot & ((1 << p.t.page_bits) - 1))] = scale;
    }
  } else {
    store16(to + at * 16, narrow<T>(e));
  }
}

bool bad_strides(std::initializer_list<int64_t> strides) {
  for (const int64_t s : strides)
    if (s < 0) return true;
  return false;
}
bool off16(std::initializer_list<int64_t> elements, int each) {
  for (const int64_t s : elements)
    if (s % each) return true;
  return false;
}

// Checks and fills what both calls know of the tokens. `size`: bytes of a cache element.
int check_tokens(Tokens& t, const int32_t* slots, const int32_t* row_lens, int32_t tokens,
                 const float* angles, int64_t angle_row, int32_t positions, int32_t rope, float eps,
                 int32_t type, void* cache, int64_t num_pages, int64_t page_stride,
                 int64_t token_stride, int32_t page_size, int size) {
  if (tokens < 0 || tokens > (1 << 30) || positions < 0 || rope != kRope || angle_row < kRope || !(eps >= 0.0f) ||
      !(eps < INFINITY) || (type != DSATOPK_BF16 && type != DSATOPK_FP16) || num_pages < 0 ||
      page_stride < 0 || token_stride < 0 || !pow2(page_size) || page_size > (1 << 20))
    return DSATOPK_ERR_INVALID_ARG;
  if (tokens == 0) return DSATOPK_OK;
  if (!slots || !row_lens || (positions && !angles) || (num_pages && !cache))
    return DSATOPK_ERR_INVALID_ARG;
  if (!aligned16(angles) || angle_row % 4 || !aligned16(cache) ||
      off16({page_stride, token_stride}, 16 / size))
    return DSATOPK_ERR_ALIGNMENT;
  t.slots = slots;
  t.row_lens = row_lens;
  t.angles = angles;
  t.angle_row = angle_row;
  t.tokens = tokens;
  t.positions = positions;
  t.page_bits = log2_of(page_size);
  t.num_pages = num_pages;
  t.cache = static_cast<char*>(cache);
  t.page = page_stride * size;
  t.token = token_stride * size;
  return DSATOPK_OK;
}

// Workgroups of the queries: `sets` in each, of kRun heads of a token.
int64_t query_groups(int32_t tokens, int32_t heads, int32_t& runs, int sets) {
  runs = (heads + kRun - 1) / kRun;
  return ((int64_t)tokens * runs + sets - 1) / sets;
}

template <class T, int kLatent>
int launch_latent(const LatentParams& p, bool near, unsigned groups, void* stream) {
  return near ? launch(append_latent_kernel<T, kLatent, true>, dim3(groups), dim3(kBlock), p, stream)
              : launch(append_latent_kernel<T, kLatent, false>, dim3(groups), dim3(kBlock), p, stream);
}

template <class T, int kDim>
int launch_index(const IndexParams& p, bool near, bool eight, unsigned groups, void* stream) {
  const dim3 grid(groups), block(kBlock);
  return eight ? near ? launch(append_index_kernel<T, kDim, true, true>, grid, block, p, stream)
                      : launch(append_index_kernel<T, kDim, false, true>, grid, block, p, stream)
         : near ? launch(append_index_kernel<T, kDim, true, false>, grid, block, p, stream)
                : launch(append_index_kernel<T, kDim, false, false>, grid, block, p, stream);
}

}  // namespace
}  // namespace dsatopk_serve

using namespace dsatopk_serve;

extern "C" int dsatopk_append_latent(
    const void* latent, int64_t latent_stride, const int32_t* slots, const int32_t* row_lens,
    int32_t num_tokens, const float* cos_sin, int64_t cos_sin_stride, int32_t num_positions,
    int32_t interleaved, const float* weight, float eps, int32_t type, int32_t latent_dim,
    int32_t rope_dim, void* cache, int64_t num_pages, int64_t page_stride, int64_t token_stride,
    int32_t page_size, void* out, int64_t out_stride, const void* q_rope, int64_t q_row_stride,
    int64_t q_head_stride, void* q_out, int64_t q_out_row_stride, int64_t q_out_head_stride,
    int32_t num_heads, void* stream) {
  LatentParams p{};
  // what the call has no use for is not looked at
  if (!out) out_stride = 0;
  if (num_heads == 0) {
    q_rope = q_out = nullptr;
    q_row_stride = q_head_stride = q_out_row_stride = q_out_head_stride = 0;
  }
  if ((latent_dim != 256 && latent_dim != 512) || num_heads < 0 || num_heads > 1024 ||
      bad_strides({latent_stride, out_stride, q_row_stride, q_head_stride, q_out_row_stride,
                   q_out_head_stride}))
    return DSATOPK_ERR_INVALID_ARG;
  const int st = check_tokens(p.t, slots, row_lens, num_tokens, cos_sin, cos_sin_stride, num_positions,
                              rope_dim, eps, type, cache, num_pages, page_stride, token_stride,
                              page_size, 2);
  if (st != DSATOPK_OK || num_tokens == 0) return st;
  if (!latent || (num_heads && (!q_rope || !q_out))) return DSATOPK_ERR_INVALID_ARG;
  if (!aligned16(latent) || !aligned16(weight) || !aligned16(out) || !aligned16(q_rope) ||
      !aligned16(q_out) ||
      off16({latent_stride, out_stride, q_row_stride, q_head_stride, q_out_row_stride,
             q_out_head_stride}, 8))
    return DSATOPK_ERR_ALIGNMENT;
  p.x = static_cast<const char*>(latent);
  p.x_row = latent_stride * 2;
  p.weight = weight;
  p.eps = eps;
  p.out = static_cast<char*>(out);
  p.out_row = out_stride * 2;
  p.q = static_cast<const char*>(q_rope);
  p.q_row = q_row_stride * 2;
  p.q_head = q_head_stride * 2;
  p.q_out = static_cast<char*>(q_out);
  p.q_out_row = q_out_row_stride * 2;
  p.q_out_head = q_out_head_stride * 2;
  p.heads = num_heads;
  const int each = (kBlock / 64) * kRun * (512 / latent_dim);
  const int64_t tokens = ((int64_t)num_tokens + each - 1) / each;
  const int64_t queries = query_groups(num_tokens, num_heads, p.runs, kBlock / kRopeLanes);
  if (tokens + queries > INT32_MAX) return DSATOPK_ERR_INVALID_ARG;
  p.token_groups = (uint32_t)tokens;
  const unsigned groups = (unsigned)(tokens + queries);
  const bool near = interleaved != 0;
  if (type == DSATOPK_BF16)
    return latent_dim == 256 ? launch_latent<Bf16, 256>(p, near, groups, stream)
                             : launch_latent<Bf16, 512>(p, near, groups, stream);
  return latent_dim == 256 ? launch_latent<Fp16, 256>(p, near, groups, stream)
                           : launch_latent<Fp16, 512>(p, near, groups, stream);
}

extern "C" int dsatopk_append_index(
    const void* keys, int64_t key_stride, const int32_t* slots, const int32_t* row_lens,
    int32_t num_tokens, const float* cos_sin, int64_t cos_sin_stride, int32_t num_positions,
    int32_t rope_dim, int32_t interleaved, const float* weight, const float* bias, float eps,
    int32_t type, int32_t head_dim, void* index_keys, int32_t index_type, int64_t num_pages,
    int64_t page_stride, int64_t token_stride, int32_t page_size, float* key_scales,
    int64_t scale_page_stride, const void* q, int64_t q_row_stride, int64_t q_head_stride,
    void* q_out, int64_t q_out_row_stride, int64_t q_out_head_stride, const float* weights,
    int64_t weight_stride, float* weights_out, int64_t weight_out_stride, int32_t num_heads,
    void* stream) {
  IndexParams p{};
  const bool eight = index_type == DSATOPK_FP8;
  // what the call has no use for is not looked at
  if (num_heads == 0) {
    q = q_out = nullptr;
    q_row_stride = q_head_stride = q_out_row_stride = q_out_head_stride = 0;
  }
  if (!eight) {
    key_scales = nullptr;
    scale_page_stride = 0;
  }
  if (!eight || num_heads == 0) {
    weights = weights_out = nullptr;
    weight_stride = weight_out_stride = 0;
  }
  if ((head_dim != 64 && head_dim != 128) || num_heads < 0 || num_heads > 128 ||
      (!eight && index_type != type) || (weight == nullptr) != (bias == nullptr) ||
      bad_strides({key_stride, scale_page_stride, q_row_stride, q_head_stride, q_out_row_stride,
                   q_out_head_stride, weight_stride, weight_out_stride}))
    return DSATOPK_ERR_INVALID_ARG;
  const int size = eight ? 1 : 2;
  const int st = check_tokens(p.t, slots, row_lens, num_tokens, cos_sin, cos_sin_stride, num_positions,
                              rope_dim, eps, type, index_keys, num_pages, page_stride, token_stride,
                              page_size, size);
  if (st != DSATOPK_OK || num_tokens == 0) return st;
  if (!keys || (eight && num_pages && !key_scales) || (num_heads && (!q || !q_out)) ||
      (num_heads && eight && (!weights || !weights_out)))
    return DSATOPK_ERR_INVALID_ARG;
  if (!aligned16(keys) || !aligned16(weight) || !aligned16(bias) || !aligned16(q) ||
      !aligned16(q_out) || !aligned4(key_scales) || !aligned4(weights) || !aligned4(weights_out) ||
      off16({key_stride, q_row_stride, q_head_stride}, 8) ||
      off16({q_out_row_stride, q_out_head_stride}, 16 / size))
    return DSATOPK_ERR_ALIGNMENT;
  p.x = static_cast<const char*>(keys);
  p.x_row = key_stride * 2;
  p.weight = weight;
  p.bias = bias;
  p.eps = eps;
  p.scales = key_scales;
  p.scale_page = scale_page_stride;
  p.q = static_cast<const char*>(q);
  p.q_row = q_row_stride * 2;
  p.q_head = q_head_stride * 2;
  p.q_out = static_cast<char*>(q_out);
  p.q_out_row = q_out_row_stride * size;
  p.q_out_head = q_out_head_stride * size;
  p.weights = weights;
  p.weights_row = weight_stride;
  p.weights_out = weights_out;
  p.weights_out_row = weight_out_stride;
  p.heads = num_heads;
  const int sets = kBlock / (head_dim / 8);
  const int64_t tokens = ((int64_t)num_tokens + sets - 1) / sets;
  const int64_t queries = query_groups(num_tokens, num_heads, p.runs, sets);
  if (tokens + queries > INT32_MAX) return DSATOPK_ERR_INVALID_ARG;
  p.token_groups = (uint32_t)tokens;
  const unsigned groups = (unsigned)(tokens + queries);
  const bool near = interleaved != 0;
  if (type == DSATOPK_BF16)
    return head_dim == 64 ? launch_index<Bf16, 64>(p, near, eight, groups, stream)
                          : launch_index<Bf16, 128>(p, near, eight, groups, stream);
  return head_dim == 64 ? launch_index<Fp16, 64>(p, near, eight, groups, stream)
                        : launch_index<Fp16, 128>(p, near, eight, groups, stream);
}
