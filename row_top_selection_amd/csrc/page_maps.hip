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
// One launch: every workgroup takes kTokens tokens and computes the running
// sums over the requests itself, kRequests at a time in LDS, up to those of
// its tokens. A second launch that waited for shared sums would cost more
// than the lengths' re-reading from L2 (8 bytes a request and workgroup).

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
};

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
  __shared__ int32_t sums[2][kBlock / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int32_t t0 = (int32_t)blockIdx.x * kTokens;
  const int32_t t1 = t0 + kTokens < p.num_tokens ? t0 + kTokens : p.num_tokens;
  const int32_t page = 1 << p.page_bits;
  const bool leads = blockIdx.x == 0;  // writes what there is one of
  int32_t tokens = 0, pages = 0;       // of the passes so far

  for (int32_t r0 = 0; r0 < p.requests; r0 += kRequests) {
    int32_t nw[kPer], pg[kPer], n = 0, g = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int32_t r = r0 + tid * kPer + j;
      nw[j] = pg[j] = 0;
      if (r < p.requests) {
        const int32_t len = max(p.seq_lens[r], 0);
        nw[j] = p.new_lens ? min(max(p.new_lens[r], 0), len) : min(1, len);
        // pages up to the end, less those up to the last held token
        pg[j] = (int32_t)(((int64_t)len + page - 1) >> p.page_bits) -
                (int32_t)(((int64_t)len - nw[j] + page - 1) >> p.page_bits);
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
      const int32_t r = r0 + tid * kPer + j;
      if (leads && r < p.requests) p.token_starts[r] = nb;
      nb += nw[j];
      gb += pg[j];
    }
    if (tid == 0) start[kRequests] = tokens;
    __syncthreads();

    // this workgroup's tokens of these requests
    const int32_t a = max(t0, start[0]), b = min(t1, tokens);
    for (int32_t t = a + tid; t < b; t += kBlock) {
      int lo = 0, hi = kRequests;  // start[lo] <= t < start[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= t)
          lo = mid;
        else
          hi = mid;
      }
      const int32_t r = r0 + lo;
      const int32_t len = max(p.seq_lens[r], 0);
      const int32_t fresh = p.new_lens ? min(max(p.new_lens[r], 0), len) : min(1, len);
      const int32_t pos = len - fresh + (t - start[lo]);
      const int32_t held = (int32_t)(((int64_t)len - fresh + page - 1) >> p.page_bits);
      const int32_t at = pos >> p.page_bits;
      int32_t entry = -1;
      if (at < p.width) {
        int32_t* e = p.table + r * p.table_stride + at;
        if (at < held) {
          entry = *e;
        } else {
          const int64_t f = (int64_t)first[lo] + (at - held);
          if (f < p.num_free) entry = p.free_pages[f];
          if ((pos & (page - 1)) == 0) *e = entry;
        }
      }
      const int64_t slot = ((int64_t)entry << p.page_bits) + (pos & (page - 1));
      p.slots[t] = entry < 0 || slot > INT32_MAX ? -1 : (int32_t)slot;
      p.table_rows[t] = r;
      p.row_lens[t] = pos + 1;
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
  if (num_requests < 0 || num_free < 0 || num_tokens < 0 || page_table_width < 0 ||
      page_table_stride < page_table_width || !pow2(page_size) || page_size > (1 << 20))
    return DSATOPK_ERR_INVALID_ARG;
  if (!token_starts || !counts || (num_requests && (!seq_lens || !page_table)) ||
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
  const int64_t groups = ((int64_t)num_tokens + kTokens - 1) / kTokens;
  return launch(page_maps_kernel, dim3((unsigned)(groups < 1 ? 1 : groups)), dim3(kBlock), p,
                stream);
}
