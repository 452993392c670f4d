// page_maps.hip - the pages and cache slots of a serving step, from its
// request lengths (dsatopk_page_maps in include/dsatopk.h).
//
// Request r holds len_r tokens after the step, new_r of them new, in pages
// of p tokens: it held ceil((len_r - new_r) / p) pages and needs
// ceil(len_r / p). With first_r = sum over i < r of the pages taken and
// start_r = sum over i < r of new_i, new token t = start_r + i of request r
// sits at position q = len_r - new_r + i, in the request's page q / p:
// table[r][q / p] if it was held, else free[first_r + q / p - held_r]. The
// token with q % p == 0 is the only one that opens its page, so it writes
// the table entry; nobody reads an entry that the call writes.
//
// One launch: every workgroup takes kTokens tokens, kPer consecutive ones a
// thread, and computes the running sums over the requests itself, kRequests
// at a time in LDS, up to those of its tokens. A second launch that waited for shared sums would cost more
// than the lengths' re-reading from L2 (8 bytes a request and workgroup).
// 128 requests of one new token: 4.7 us on the GPU, latency alone; half a
// million tokens of 256 requests: 7.5 us (0.8 TB/s), where the running sums and the
// search in front of each thread's four tokens take most.

#include "serve_common.h"

namespace dsatopk_serve {
namespace {

constexpr int kBlock = 256;
constexpr int kPer = 4;                    // requests and tokens a thread
constexpr int kRequests = kBlock * kPer;   // requests a pass
constexpr int kTokens = kBlock * kPer;     // tokens a workgroup

struct MapParams {
  const int32_t* seq_lens;
  const int32_t* new_lens;
  int32_t* table;
  int64_t table_stride;
  const int32_t* free_pages;
  int32_t requests, width, page_bits, num_free, num_tokens;
  int32_t* token_starts;
  int32_t* slots;
  int32_t* table_rows;
  int32_t* row_lens;
  int32_t* counts;
  bool wide;  // 16-byte stores fit slots, table_rows and row_lens
};

// Four consecutive tokens' values, those from `n` on left out.
__device__ __forceinline__ void store4(int32_t* to, const int32_t (&v)[kPer], int n, bool wide) {
  if (wide && n == kPer) {
    *reinterpret_cast<int4*>(to) = int4{v[0], v[1], v[2], v[3]};
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (j < n) to[j] = v[j];
  }
}

// Inclusive sums over a wave's lanes.
__device__ __forceinline__ int32_t wave_sum(int32_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

__global__ __launch_bounds__(kBlock) void page_maps_kernel(MapParams p) {
  __shared__ int32_t start[kRequests + 1];  // first token of each request of the pass
  __shared__ int32_t first[kRequests];      // first free page of each
  __shared__ int32_t before[kRequests];     // tokens that each held
  __shared__ int32_t sums[2][kBlock / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int32_t t0 = (int32_t)blockIdx.x * kTokens;
  const int32_t t1 = t0 + kTokens < p.num_tokens ? t0 + kTokens : p.num_tokens;
  const int32_t page = 1 << p.page_bits;
  const bool leads = blockIdx.x == 0;  // writes what there is one of
  int32_t tokens = 0, pages = 0;       // of the passes so far

  for (int32_t r0 = 0; r0 < p.requests; r0 += kRequests) {
    int32_t nw[kPer], pg[kPer], had[kPer], n = 0, g = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int32_t r = r0 + tid * kPer + j;
      nw[j] = pg[j] = had[j] = 0;
      if (r < p.requests) {
        const int32_t len = max(p.seq_lens[r], 0);
        nw[j] = p.new_lens ? min(max(p.new_lens[r], 0), len) : min(1, len);
        had[j] = len - nw[j];
        // pages up to the end, less those up to the last held token
        pg[j] = (int32_t)(((int64_t)len + page - 1) >> p.page_bits) -
                (int32_t)(((int64_t)had[j] + page - 1) >> p.page_bits);
      }
      n += nw[j];
      g += pg[j];
    }
    const int32_t ns = wave_sum(n), gs = wave_sum(g);
    if (lane == 63) {
      sums[0][wave] = ns;
      sums[1][wave] = gs;
    }
    __syncthreads();
    int32_t nb = tokens + ns - n, gb = pages + gs - g;
#pragma unroll
    for (int w = 0; w < kBlock / 64; ++w) {
      const int32_t a = sums[0][w], b = sums[1][w];
      if (w < wave) {
        nb += a;
        gb += b;
      }
      tokens += a;
      pages += b;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      start[tid * kPer + j] = nb;
      first[tid * kPer + j] = gb;
      before[tid * kPer + j] = had[j];
      const int32_t r = r0 + tid * kPer + j;
      if (leads && r < p.requests) p.token_starts[r] = nb;
      nb += nw[j];
      gb += pg[j];
    }
    if (tid == 0) start[kRequests] = tokens;
    __syncthreads();

    // This thread's tokens of these requests: a search for the first one's
    // request, steps from there for the others.
    const int32_t a = max(t0 + tid * kPer, start[0]);
    const int32_t b = min(min(t0 + (tid + 1) * kPer, t1), tokens);
    if (a < b) {
      int lo = 0, hi = min(kRequests, p.requests - r0);  // start[lo] <= a < start[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= a)
          lo = mid;
        else
          hi = mid;
      }
      int32_t slot[kPer], row[kPer], pos[kPer], entry[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        entry[j] = -1;
        if (a + j >= b) continue;
        while (start[lo + 1] <= a + j) ++lo;
        row[j] = r0 + lo;
        pos[j] = before[lo] + (a + j - start[lo]);
        const int32_t held = (int32_t)(((int64_t)before[lo] + page - 1) >> p.page_bits);
        const int32_t at = pos[j] >> p.page_bits;
        if (at >= p.width) continue;
        if (at < held) {
          entry[j] = p.table[row[j] * p.table_stride + at];
        } else {
          const int64_t f = (int64_t)first[lo] + (at - held);
          if (f < p.num_free) entry[j] = p.free_pages[f];
        }
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (a + j >= b) continue;
        const int32_t in = pos[j] & (page - 1);
        const int32_t at = pos[j] >> p.page_bits;
        if (in == 0 && at < p.width) p.table[row[j] * p.table_stride + at] = entry[j];
        const int64_t full = ((int64_t)entry[j] << p.page_bits) + in;
        slot[j] = entry[j] < 0 || full > INT32_MAX ? -1 : (int32_t)full;
        ++pos[j];
      }
      const bool wide = p.wide && (a & 3) == 0;
      store4(p.slots + a, slot, b - a, wide);
      store4(p.table_rows + a, row, b - a, wide);
      store4(p.row_lens + a, pos, b - a, wide);
    }
    if (!leads && tokens >= t1) return;
    __syncthreads();
  }
  // rows past the step's tokens: no slot, an empty window
  for (int32_t t = max(t0, tokens) + tid; t < t1; t += kBlock) {
    p.slots[t] = -1;
    p.table_rows[t] = 0;
    p.row_lens[t] = 0;
  }
  if (leads && tid == 0) {
    p.token_starts[p.requests] = tokens;
    p.counts[0] = tokens;
    p.counts[1] = pages;
  }
}

}  // namespace
}  // namespace dsatopk_serve

using namespace dsatopk_serve;

extern "C" int dsatopk_page_maps(const int32_t* seq_lens, const int32_t* new_lens,
                                 int32_t num_requests, int32_t* page_table,
                                 int64_t page_table_stride, int32_t page_table_width,
                                 int32_t page_size, const int32_t* free_pages, int32_t num_free,
                                 int32_t num_tokens, int32_t* token_starts, int32_t* slots,
                                 int32_t* table_rows, int32_t* row_lens, int32_t* counts,
                                 void* stream) {
  if (num_requests < 0 || num_free < 0 || num_tokens < 0 || num_tokens > (1 << 30) || page_table_width < 0 ||
      page_table_stride < page_table_width || !pow2(page_size) || page_size > (1 << 20))
    return DSATOPK_ERR_INVALID_ARG;
  if (!token_starts || !counts || (num_requests && !seq_lens) ||
      (num_requests && page_table_width && !page_table) ||
      (num_free && !free_pages) || (num_tokens && (!slots || !table_rows || !row_lens)))
    return DSATOPK_ERR_INVALID_ARG;
  MapParams p{};
  p.seq_lens = seq_lens;
  p.new_lens = new_lens;
  p.table = page_table;
  p.table_stride = page_table_stride;
  p.free_pages = free_pages;
  p.requests = num_requests;
  p.width = page_table_width;
  p.page_bits = log2_of(page_size);
  p.num_free = num_free;
  p.num_tokens = num_tokens;
  p.token_starts = token_starts;
  p.slots = slots;
  p.table_rows = table_rows;
  p.row_lens = row_lens;
  p.counts = counts;
  p.wide = aligned16(slots) && aligned16(table_rows) && aligned16(row_lens);
  const int64_t groups = ((int64_t)num_tokens + kTokens - 1) / kTokens;
  return launch(page_maps_kernel, dim3((unsigned)(groups < 1 ? 1 : groups)), dim3(kBlock), p,
                stream);
}
