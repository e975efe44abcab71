// paged_plan.cu -- block tables, slot map and page spans of a step, from the
// requests' lengths (rtp_paged_plan).
//
// Per request b with `old` tokens (0 if it is released first) and n new ones:
//   have = ceil(old / ps), want = ceil((old + n) / ps), need = want - have,
//   off  = sum of the needs before it,
//   admitted  <=>  want fits the table, its tokens fit max_tokens, and need == 0
//                  or off + need <= free pages,
//   page have + j of its table = free_pages[free - 1 - off - j]   (a stack),
//   slot of position x = table[x / ps] * ps + x % ps.
// Three running sums over the requests (tokens, pages, spans), then
// independent writes.  What bounds it is latency: one CTA scans 1024 requests
// at a time; with few tokens the same CTA writes everything (one launch), with
// many a second kernel spreads the writes over the SMs.
#include <algorithm>

#include "paged.cuh"

namespace rtp {
namespace {

struct PlanParams {
  int32_t B, ps_shift, row_tokens, width, max_tokens, max_spans, free_cap;
  const int32_t* seq_lens;
  const int32_t* n_new;
  const uint8_t* release;
  int32_t* table;
  int64_t table_stride;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* seq_lens_out;
  int32_t* cu_new;
  int32_t* slot_map;
  int4* spans;
  int32_t* free_count_out;
  int32_t* admitted;
  int4* info;      // two per request, written for the fill kernel
  int32_t* head;   // {free pages after release, tokens, spans}
};

// What the writes of one request need.
struct Req {
  int64_t old;
  int32_t n, have, off, cu, span0, top;  // top: free pages once releases are back
  int32_t ok;                            // admitted
};

__device__ __forceinline__ int32_t popped(const PlanParams& p, const Req& r, int32_t j) {
  const int32_t i = r.top - 1 - r.off - j;
  return i >= 0 && i < p.free_cap ? p.free_pages[i] : -1;
}

// Physical page of column c of an admitted request: its own table below `have`
// (those entries do not change here), the free stack from there on.
__device__ __forceinline__ int32_t page_of(const PlanParams& p, const int32_t* row, const Req& r,
                                           int32_t c) {
  return c < r.have ? row[c] : popped(p, r, c - r.have);
}

// Slot of new token t of an admitted request.
__device__ __forceinline__ int32_t slot_of(const PlanParams& p, int b, const Req& r, int32_t t) {
  const int32_t* row = p.table + (int64_t)b * p.table_stride;
  const int64_t x = r.old + t;
  const int64_t slot = ((int64_t)page_of(p, row, r, (int32_t)(x >> p.ps_shift)) << p.ps_shift) +
                       (x & ((1 << p.ps_shift) - 1));
  return slot >= 0 && slot <= INT32_MAX ? (int32_t)slot : -1;
}

// Span of table column c of an admitted request.
__device__ __forceinline__ int4 span_of(const PlanParams& p, int b, const Req& r, int32_t c) {
  const int64_t lo = (int64_t)c << p.ps_shift;
  const int32_t rows = (int32_t)min((int64_t)1 << p.ps_shift, r.old + r.n - lo);
  const int32_t fresh = (int32_t)max((int64_t)0, r.old - lo);
  return make_int4(page_of(p, p.table + (int64_t)b * p.table_stride, r, c), rows, fresh,
                   (int32_t)(r.cu + lo + fresh - r.old));
}

// Table entries, slots and spans of one request; threads i, i + step, ...  The
// tokens of a refused one stay in the packed batch, without slots.
__device__ __forceinline__ void fill_request(const PlanParams& p, int b, const Req& r, int i,
                                             int step) {
  // the entries of the batch that are the request's and get no slot
  const int64_t slots_end =
      min((int64_t)r.cu + (p.row_tokens > 0 ? p.row_tokens : r.n), (int64_t)p.max_tokens);
  for (int64_t t = (int64_t)r.cu + (r.ok ? r.n : 0) + i; t < slots_end; t += step) p.slot_map[t] = -1;
  if (!r.ok) return;
  int32_t* row = p.table + (int64_t)b * p.table_stride;
  const int32_t want = (int32_t)((r.old + r.n + (1 << p.ps_shift) - 1) >> p.ps_shift);
  for (int32_t c = r.have + i; c < want; c += step) row[c] = popped(p, r, c - r.have);
  for (int32_t t = i; t < r.n; t += step) p.slot_map[r.cu + t] = slot_of(p, b, r, t);
  if (r.n > 0) {
    const int32_t first = (int32_t)(r.old >> p.ps_shift);
    for (int32_t c = first + i; c < want; c += step) {
      const int32_t at = r.span0 + c - first;
      if (at < p.max_spans) p.spans[at] = span_of(p, b, r, c);
    }
  }
}

__device__ __forceinline__ void pad_tail(const PlanParams& p, int64_t tokens, int64_t spans, int i,
                                         int step) {
  for (int64_t t = tokens + i; t < p.max_tokens; t += step) p.slot_map[t] = -1;
  for (int64_t t = spans + i; t < p.max_spans; t += step) p.spans[t] = make_int4(-1, 0, 0, 0);
}

constexpr int kPlanThreads = 1024;
constexpr int kPlanOneLaunch = 1024;  // tokens

// Inclusive block scan; *total gets the sum over the block.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int64_t w = lane < n_warps ? warp_sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int64_t before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return v + (warp ? before : 0);
}

// The requests of a one-launch plan, in shared memory.
struct PlanSmem {
  int32_t old[kPlanThreads], n[kPlanThreads], have[kPlanThreads], off[kPlanThreads];
  int32_t cu[kPlanThreads], span0[kPlanThreads], ok[kPlanThreads];
};

// The last of the first B entries of an ascending array that is <= x (x >= at[0]).
__device__ __forceinline__ int last_at(const int32_t* at, int B, int64_t x) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (at[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// FILL (B <= threads): the same CTA then writes everything: a request's thread its one
// or two tokens, or, where a request has more, a thread a token, a span, a page at a
// time, whose request it finds by bisection (64 requests, one token each: 3.3 us
// against 4.3 by bisection).
template <bool FILL>
__global__ void __launch_bounds__(kPlanThreads) plan_scan_kernel(const PlanParams p) {
  griddep_wait();
  __shared__ int64_t sums[32];
  extern __shared__ __align__(16) unsigned char plan_smem[];
  PlanSmem& sm = *reinterpret_cast<PlanSmem*>(plan_smem);
  const int tid = threadIdx.x, lane = tid & 31, n_thr = blockDim.x;
  const int ps = 1 << p.ps_shift;
  int64_t top = max(0, min(*p.free_count, p.free_cap));

  if (p.release != nullptr) {  // pages of released requests go back first, in request order
    for (int b0 = 0; b0 < p.B; b0 += n_thr) {
      const int b = b0 + tid;
      int64_t back = 0;
      if (b < p.B && p.release[b])
        back = min((int64_t)p.width, ((int64_t)max(0, p.seq_lens[b]) + ps - 1) >> p.ps_shift);
      int64_t all;
      const int64_t at = top + block_scan(back, sums, &all) - back;
      uint32_t todo = __ballot_sync(0xffffffffu, back > 0);
      while (todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const int64_t n = __shfl_sync(0xffffffffu, back, src);
        const int64_t to = __shfl_sync(0xffffffffu, at, src);
        const int32_t* row = p.table + (int64_t)(b - lane + src) * p.table_stride;
        for (int64_t j = lane; j < n; j += 32)
          if (to + j < p.free_cap) p.free_pages[to + j] = row[j];
      }
      top = min(top + all, (int64_t)p.free_cap);
    }
    __syncthreads();  // the stack is read from here on
  }

  int64_t tokens = 0, pages = 0, spans = 0;  // sums over the requests before this chunk
  int64_t taken = 0;
  bool wide = false;
  for (int b0 = 0; b0 < p.B; b0 += n_thr) {
    const int b = b0 + tid;
    const bool live = b < p.B;
    Req r = {};
    r.top = (int32_t)top;
    if (live) {
      r.old = p.release != nullptr && p.release[b] ? 0 : max(0, p.seq_lens[b]);
      r.n = max(0, p.n_new[b]);
    }
    const int64_t have = (r.old + ps - 1) >> p.ps_shift;
    const int64_t want = (r.old + r.n + ps - 1) >> p.ps_shift;
    int64_t all;
    int64_t cu = tokens + block_scan(r.n, sums, &all) - r.n;
    int64_t cu_end = cu + r.n;
    tokens += all;
    bool fits = live && want <= p.width;
    if (p.row_tokens > 0) {  // a padded batch: every request has a row of its own
      cu = (int64_t)b * p.row_tokens;
      cu_end = cu + p.row_tokens;
      fits = fits && r.n <= p.row_tokens;
    }
    fits = fits && cu + r.n <= p.max_tokens;
    const int64_t need = fits ? want - have : 0;
    const int64_t upto = pages + block_scan(need, sums, &all);
    pages += all;
    const bool ok = fits && (need == 0 || upto <= top);
    const int64_t first = r.old >> p.ps_shift;
    const int64_t n_span = ok && r.n > 0 ? want - first : 0;
    const int64_t span_end = spans + block_scan(n_span, sums, &all);
    spans += all;
    block_scan(ok ? need : 0, sums, &all);
    taken += all;
    // off only matters where pages are taken, and there it is below top
    r.have = (int32_t)min(have, (int64_t)p.width);
    r.off = (int32_t)min(upto - need, (int64_t)INT32_MAX);
    r.cu = (int32_t)min(cu, (int64_t)INT32_MAX);
    r.span0 = (int32_t)min(span_end - n_span, (int64_t)INT32_MAX);
    r.ok = ok ? 1 : 0;
    if (live) {
      p.cu_new[b + 1] = (int32_t)min(cu_end, (int64_t)INT32_MAX);
      p.admitted[b] = r.ok;
      p.seq_lens_out[b] = (int32_t)(r.old + (ok ? r.n : 0));
      if (FILL) {
        sm.old[b] = (int32_t)r.old;
        sm.n[b] = r.n;
        sm.have[b] = r.have;
        sm.off[b] = r.off;
        sm.cu[b] = r.cu;
        sm.span0[b] = r.span0;
        sm.ok[b] = r.ok;
        // a token or two: the request's own thread writes them
        const int32_t slots = p.row_tokens > 0 ? p.row_tokens : r.n;
        wide = slots > 2;
        if (!wide && slots > 0) fill_request(p, b, r, 0, 1);
      } else {
        p.info[2 * b] = make_int4((int32_t)r.old, r.n, r.have, r.off);
        p.info[2 * b + 1] = make_int4(r.cu, r.span0, r.ok, 0);
      }
    }
  }
  if (p.row_tokens > 0) tokens = (int64_t)p.B * p.row_tokens;
  if (tid == 0) {
    p.cu_new[0] = 0;
    *p.free_count_out = (int32_t)(top - taken);
    if (!FILL) {
      p.head[0] = (int32_t)top;
      p.head[1] = (int32_t)min(tokens, (int64_t)INT32_MAX);
      p.head[2] = (int32_t)min(spans, (int64_t)INT32_MAX);
    }
  }
  if (!FILL) return;

  if (!__syncthreads_or(wide)) {
    pad_tail(p, tokens, spans, tid, n_thr);
    return;
  }
  auto request = [&](int b) {
    Req r;
    r.old = sm.old[b];
    r.n = sm.n[b];
    r.have = sm.have[b];
    r.off = sm.off[b];
    r.cu = sm.cu[b];
    r.span0 = sm.span0[b];
    r.ok = sm.ok[b];
    r.top = (int32_t)top;
    return r;
  };
  for (int t = tid; t < p.max_tokens; t += n_thr) {
    int32_t slot = -1;
    if (t < tokens) {
      const int b = last_at(sm.cu, p.B, t);
      const Req r = request(b);
      if (r.ok && t - r.cu < r.n) slot = slot_of(p, b, r, t - r.cu);
    }
    p.slot_map[t] = slot;
  }
  for (int i = tid; i < p.max_spans; i += n_thr) {
    int4 sp = make_int4(-1, 0, 0, 0);
    if (i < spans) {
      const int b = last_at(sm.span0, p.B, i);
      const Req r = request(b);
      sp = span_of(p, b, r, (int32_t)(r.old >> p.ps_shift) + i - r.span0);
    }
    p.spans[i] = sp;
  }
  for (int64_t j = tid; j < taken; j += n_thr) {
    const int b = last_at(sm.off, p.B, j);
    const Req r = request(b);
    const int32_t at = (int32_t)j - r.off;
    p.table[(int64_t)b * p.table_stride + r.have + at] = popped(p, r, at);
  }
}

constexpr int kFillThreads = 256;

// CTAs (b, y): the writes of request b, in steps over y; row b == B pads the tails.
__global__ void __launch_bounds__(kFillThreads) plan_fill_kernel(const PlanParams p) {
  griddep_wait();
  const int b = blockIdx.x;
  const int i = blockIdx.y * kFillThreads + threadIdx.x, step = gridDim.y * kFillThreads;
  if (b == p.B) {
    pad_tail(p, p.head[1], p.head[2], i, step);
    return;
  }
  const int4 a = p.info[2 * b], c = p.info[2 * b + 1];
  if (a.y == 0 && p.row_tokens == 0) return;
  Req r;
  r.old = a.x;
  r.n = a.y;
  r.have = a.z;
  r.off = a.w;
  r.cu = c.x;
  r.span0 = c.y;
  r.ok = c.z;
  r.top = p.head[0];
  fill_request(p, b, r, i, step);
}

}  // namespace

size_t paged_plan_ws(int32_t B) { return align_up(kStatusBytes + 256 + (size_t)B * 32, 256); }

}  // namespace rtp

using namespace rtp;

extern "C" rtp_status rtp_paged_plan(int32_t B, int32_t page_size, int32_t row_tokens,
                                     const int32_t* seq_lens, const int32_t* n_new, const uint8_t* release,
                                     int32_t* block_table, int64_t table_stride,
                                     int32_t table_width, int32_t* free_pages, int32_t free_cap,
                                     const int32_t* free_count, int32_t max_tokens,
                                     int32_t max_spans, int32_t* seq_lens_out, int32_t* cu_new,
                                     int32_t* slot_map, int32_t* spans, int32_t* free_count_out,
                                     int32_t* admitted, void* ws, size_t ws_bytes,
                                     rtp_stream_t stream) {
  if (B < 0 || row_tokens < 0 || table_width < 0 || table_stride < table_width || free_cap < 0 || max_tokens < 0 ||
      max_spans < 0)
    return RTP_ERR_INVALID_ARG;
  rtp_status st = check_page_size(page_size);
  if (st != RTP_OK) return st;
  if ((int64_t)table_width * page_size > kMaxTokens) return RTP_ERR_UNSUPPORTED;
  if (B == 0) return RTP_OK;
  if (seq_lens == nullptr || n_new == nullptr || (block_table == nullptr && table_width > 0) ||
      (free_pages == nullptr && free_cap > 0) || free_count == nullptr ||
      seq_lens_out == nullptr || cu_new == nullptr || (slot_map == nullptr && max_tokens > 0) ||
      (spans == nullptr && max_spans > 0) || free_count_out == nullptr || admitted == nullptr)
    return RTP_ERR_INVALID_ARG;
  if (!aligned16(spans) || !aligned16(ws)) return RTP_ERR_ALIGNMENT;
  if (ws == nullptr || ws_bytes < paged_plan_ws(B)) return RTP_ERR_WORKSPACE_TOO_SMALL;
  char* w = static_cast<char*>(ws) + kStatusBytes;
  PlanParams p = {B, log2_exact(page_size), row_tokens, table_width, max_tokens, max_spans, free_cap, seq_lens,
                  n_new, release, block_table, table_stride, free_pages, free_count, seq_lens_out,
                  cu_new, slot_map, reinterpret_cast<int4*>(spans), free_count_out, admitted,
                  reinterpret_cast<int4*>(w + 256), reinterpret_cast<int32_t*>(w)};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // Few tokens of up to 1024 requests: one launch, with a thread for each token or
  // request; beyond that a second kernel over all SMs.  64 requests: 300 tokens 4.4 us
  // against 4.8 (5.5 against 7.2 from Python), 1000 tokens 6.3 against 5.0 (6.4, 7.3),
  // 5000 tokens 9.3 against 5.0.
  if (B <= kPlanThreads && max_tokens <= kPlanOneLaunch) {
    const int most = std::max(B, std::min(max_tokens, kPlanThreads));
    TraceScope tr("plan_scan", s);
    return check_cuda(launch_dependent(plan_scan_kernel<true>, dim3(1), dim3((most + 31) / 32 * 32),
                                       sizeof(PlanSmem), s, p));
  }
  const int threads = B >= kPlanThreads ? kPlanThreads : (B + 31) / 32 * 32;
  {
    TraceScope tr("plan_scan", s);
    if ((st = check_cuda(launch_dependent(plan_scan_kernel<false>, dim3(1), dim3(threads), 0, s,
                                          p))) != RTP_OK)
      return st;
  }
  // about four CTAs per SM over all requests, none with less than a step of tokens; one
  // at least: without tokens too the spans are padded
  const int64_t most = ((int64_t)max_tokens + kFillThreads - 1) / kFillThreads;
  const int y = (int)std::max<int64_t>(1, std::min((592 + (int64_t)B) / (B + (int64_t)1), most));
  TraceScope tr("plan_fill", s);
  return check_cuda(
      launch_dependent(plan_fill_kernel, dim3((unsigned)B + 1u, y), dim3(kFillThreads), 0, s, p));
}
