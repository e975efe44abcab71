// paged_write.cu -- new K/V rows into pages: by a slot map (rtp_paged_kv_write),
// or by page spans with the touched pages' bounds refreshed in the same pass
// (rtp_paged_kv_append).
//
// Stored value: the bf16 row itself, or e4m3(x / scale[head]), divided in fp32
// and rounded once to nearest even (saturating at 448).
//
// Bounds of a page and retrieval kv head, over its stored rows k_r (8-bit rows
// without their scale), per dimension d:
//   lo_d = min_r k_rd, hi_d = max_r k_rd, a = max_d max(|lo_d|, |hi_d|),
//   s = a * (1/127) (fp32),  hi8_d = min(127, ceil(hi_d / s)),
//   lo8_d = max(-127, floor(lo_d / s)),
// so s * lo8 <= k <= s * hi8 up to one rounding of the division.  s = 0 (and
// zero bounds) for an all-zero page, s = inf (and zero bounds) for one that
// holds an infinity or a NaN.  They depend on the page's rows alone, not on how
// they came there.  Bound by HBM: each row is read once and written once; old
// rows are read only where a page was part-filled, and only for K.
#include "paged.cuh"

namespace rtp {
namespace {

struct WriteParams {
  const uint16_t* k; int64_t k_st;  // row t at k + t * k_st, heads of 128 contiguous
  const uint16_t* v; int64_t v_st;
  PageAddr kp, vp;
  const float* k_scale;
  const float* v_scale;
  int32_t T, Hkv, ps_shift, n_pages;
  const int32_t* slot_map;
  const int4* spans;
  int32_t n_spans;
  int8_t* bounds;          // [n_pages][n_rkv][2][128]
  float* bound_scale;      // [n_pages][n_rkv]
  int32_t n_rkv;
  int16_t rank[kMaxHeads]; // kv head -> rank among the retrieval kv heads, -1 local
};

// Eight values (16 bytes of bf16) as eight e4m3 bytes.
__device__ __forceinline__ uint2 quantise8(const uint4& w, float scale) {
  float x[8];
  unpack8(w, x);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = x[i] / scale;
  uint2 r;
  r.x = f32x2_to_e4m3x2(x[0], x[1]) | ((uint32_t)f32x2_to_e4m3x2(x[2], x[3]) << 16);
  r.y = f32x2_to_e4m3x2(x[4], x[5]) | ((uint32_t)f32x2_to_e4m3x2(x[6], x[7]) << 16);
  return r;
}

constexpr int kWriteThreads = 256;

// Thread: one 16-byte chunk of one row of K and V.  A row's chunks (16 per
// head) are consecutive threads.
template <bool E4M3>
__global__ void __launch_bounds__(kWriteThreads) kv_write_kernel(const WriteParams p) {
  griddep_wait();
  const int64_t e = (int64_t)blockIdx.x * kWriteThreads + threadIdx.x;
  const int per_row = p.Hkv * 16;
  const int64_t t = e / per_row;
  if (t >= p.T) return;
  const int c = (int)(e - t * per_row), h = c >> 4, ch = c & 15;
  const int32_t slot = p.slot_map[t];
  if (slot < 0 || (slot >> p.ps_shift) >= p.n_pages) return;
  const int64_t page = slot >> p.ps_shift, row = slot & ((1 << p.ps_shift) - 1);
  const uint4 kw = *reinterpret_cast<const uint4*>(p.k + t * p.k_st + c * 8);
  const uint4 vw = *reinterpret_cast<const uint4*>(p.v + t * p.v_st + c * 8);
  uint8_t* ko = p.kp.ptr + page * p.kp.page + row * p.kp.row + h * p.kp.head;
  uint8_t* vo = p.vp.ptr + page * p.vp.page + row * p.vp.row + h * p.vp.head;
  if (E4M3) {
    const float ks = p.k_scale ? p.k_scale[h] : 1.f, vs = p.v_scale ? p.v_scale[h] : 1.f;
    *reinterpret_cast<uint2*>(ko + ch * 8) = quantise8(kw, ks);
    *reinterpret_cast<uint2*>(vo + ch * 8) = quantise8(vw, vs);
  } else {
    *reinterpret_cast<uint4*>(ko + ch * 16) = kw;
    *reinterpret_cast<uint4*>(vo + ch * 16) = vw;
  }
}

constexpr int kAppendThreads = 128;

// CTA: one span (page) and kv head; 16 threads a row, 8 rows at a time.  Each
// thread keeps the running bounds of its eight dimensions.
template <bool E4M3>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const WriteParams p) {
  griddep_wait();
  const int h = blockIdx.x % p.Hkv;
  const int4 sp = p.spans[blockIdx.x / p.Hkv];  // {page, rows, fresh, token}
  const int ps = 1 << p.ps_shift;
  if (sp.x < 0 || sp.x >= p.n_pages) return;
  const int rows = min(sp.y, ps), fresh = max(sp.z, 0);
  const int tid = threadIdx.x, ch = tid & 15, r0 = tid >> 4;
  const int rank = p.rank[h];
  uint8_t* kb = p.kp.ptr + sp.x * p.kp.page + h * p.kp.head;
  uint8_t* vb = p.vp.ptr + sp.x * p.vp.page + h * p.vp.head;
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = INFINITY;
    hi[i] = -INFINITY;
  }
  bool odd = false;  // an infinity or a NaN among the rows
  auto take = [&](const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = fminf(lo[i], x[i]);
      hi[i] = fmaxf(hi[i], x[i]);
      odd |= !(fabsf(x[i]) < INFINITY);
    }
  };
  if (rank >= 0) {  // rows that were there
#pragma unroll 4
    for (int r = r0; r < min(fresh, rows); r += 8) {
      float x[8];
      if (E4M3)
        unpack8(*reinterpret_cast<const uint2*>(kb + r * p.kp.row + ch * 8), x);
      else
        unpack8(*reinterpret_cast<const uint4*>(kb + r * p.kp.row + ch * 16), x);
      take(x);
    }
  }
  const float ks = E4M3 && p.k_scale ? p.k_scale[h] : 1.f;
  const float vs = E4M3 && p.v_scale ? p.v_scale[h] : 1.f;
#pragma unroll 4
  for (int r = fresh + r0; r < rows; r += 8) {
    const int64_t t = (int64_t)sp.w + r - fresh;
    if (t < 0 || t >= p.T) continue;
    const uint4 kw = *reinterpret_cast<const uint4*>(p.k + t * p.k_st + h * kD + ch * 8);
    const uint4 vw = *reinterpret_cast<const uint4*>(p.v + t * p.v_st + h * kD + ch * 8);
    float x[8];
    if (E4M3) {
      const uint2 kq = quantise8(kw, ks);
      *reinterpret_cast<uint2*>(kb + r * p.kp.row + ch * 8) = kq;
      *reinterpret_cast<uint2*>(vb + r * p.vp.row + ch * 8) = quantise8(vw, vs);
      unpack8(kq, x);
    } else {
      *reinterpret_cast<uint4*>(kb + r * p.kp.row + ch * 16) = kw;
      *reinterpret_cast<uint4*>(vb + r * p.vp.row + ch * 16) = vw;
      unpack8(kw, x);
    }
    if (rank >= 0) take(x);
  }
  if (rank < 0) return;

  // join the 8 row groups: lanes l and l ^ 16, then the four warps
  __shared__ float slo[4][kD], shi[4][kD];
  __shared__ float samax[4];
  const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = fminf(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], 16));
    hi[i] = fmaxf(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], 16));
    if (lane < 16) {
      slo[warp][ch * 8 + i] = lo[i];
      shi[warp][ch * 8 + i] = hi[i];
    }
  }
  const bool any_odd = __syncthreads_or(odd);
  // one dimension per thread
  float l = slo[0][tid], u = shi[0][tid];
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    l = fminf(l, slo[w][tid]);
    u = fmaxf(u, shi[w][tid]);
  }
  float a = warp_max(fmaxf(fabsf(l), fabsf(u)));
  if (lane == 0) samax[warp] = a;
  __syncthreads();
  a = fmaxf(fmaxf(samax[0], samax[1]), fmaxf(samax[2], samax[3]));
  // a page without rows has l = inf, u = -inf: no bounds either
  const bool empty = rows <= 0;
  float s = any_odd ? INFINITY : (empty ? 0.f : a * kInv127);
  int8_t l8 = 0, u8 = 0;
  if (s > 0.f && s < INFINITY) {
    u8 = (int8_t)fminf(fmaxf(ceilf(u / s), -127.f), 127.f);
    l8 = (int8_t)fminf(fmaxf(floorf(l / s), -127.f), 127.f);
  }
  const int64_t at = (int64_t)sp.x * p.n_rkv + rank;
  p.bounds[at * 2 * kD + tid] = l8;
  p.bounds[at * 2 * kD + kD + tid] = u8;
  if (tid == 0) p.bound_scale[at] = s;
}

rtp_status check_rows(int32_t T, int32_t Hkv, const void* x, int64_t stride) {
  if (x == nullptr) return RTP_ERR_INVALID_ARG;
  if (stride < (int64_t)Hkv * kD) return RTP_ERR_INVALID_ARG;
  if (!aligned16(x) || (stride * 2) % 16) return RTP_ERR_ALIGNMENT;
  return RTP_OK;
}

void fill_write(WriteParams* p, int32_t T, int32_t Hkv, const void* k, int64_t k_stride,
                const void* v, int64_t v_stride, const rtp_pages& kp, const rtp_pages& vp,
                const float* k_scale, const float* v_scale) {
  memset(p, 0, sizeof(*p));
  p->k = static_cast<const uint16_t*>(k);
  p->k_st = k_stride;
  p->v = static_cast<const uint16_t*>(v);
  p->v_st = v_stride;
  p->kp = page_addr(kp);
  p->vp = page_addr(vp);
  p->k_scale = k_scale;
  p->v_scale = v_scale;
  p->T = T;
  p->Hkv = Hkv;
  p->ps_shift = log2_exact(kp.page_size);
  p->n_pages = kp.n_pages;
}

}  // namespace
}  // namespace rtp

using namespace rtp;

extern "C" rtp_status rtp_paged_kv_write(int32_t T, int32_t Hkv, const void* k, int64_t k_stride,
                                         const void* v, int64_t v_stride, const int32_t* slot_map,
                                         rtp_pages k_pages, rtp_pages v_pages,
                                         const float* k_scale, const float* v_scale,
                                         rtp_stream_t stream) {
  if (T < 0 || Hkv < 1) return RTP_ERR_INVALID_ARG;
  if (Hkv > kMaxHeads) return RTP_ERR_UNSUPPORTED;
  rtp_status st = check_cache(k_pages, v_pages, k_scale, v_scale);
  if (st != RTP_OK) return st;
  if (T == 0) return RTP_OK;
  if ((st = check_rows(T, Hkv, k, k_stride)) != RTP_OK) return st;
  if ((st = check_rows(T, Hkv, v, v_stride)) != RTP_OK) return st;
  if (slot_map == nullptr) return RTP_ERR_INVALID_ARG;
  WriteParams p;
  fill_write(&p, T, Hkv, k, k_stride, v, v_stride, k_pages, v_pages, k_scale, v_scale);
  p.slot_map = slot_map;
  const int64_t n = (int64_t)T * Hkv * 16;
  const int64_t blocks = (n + kWriteThreads - 1) / kWriteThreads;
  if (blocks > INT32_MAX) return RTP_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  TraceScope tr("kv_write", s);
  return check_cuda(launch_dependent(k_pages.type == RTP_KV_E4M3 ? kv_write_kernel<true>
                                                                 : kv_write_kernel<false>,
                                     dim3((unsigned)blocks), dim3(kWriteThreads), 0, s, p));
}

extern "C" rtp_status rtp_paged_kv_append(int32_t T, int32_t Hkv, const uint8_t* kv_role,
                                          const void* k, int64_t k_stride, const void* v,
                                          int64_t v_stride, const int32_t* spans, int32_t n_spans,
                                          rtp_pages k_pages, rtp_pages v_pages,
                                          const float* k_scale, const float* v_scale,
                                          int8_t* bounds, float* bound_scale,
                                          rtp_stream_t stream) {
  if (T < 0 || n_spans < 0) return RTP_ERR_INVALID_ARG;
  PagedHeads ph;
  rtp_status st = make_paged_heads(Hkv, Hkv, kv_role, &ph);
  if (st != RTP_OK) return st;
  if ((st = check_cache(k_pages, v_pages, k_scale, v_scale)) != RTP_OK) return st;
  if (T == 0 || n_spans == 0) return RTP_OK;
  if ((st = check_rows(T, Hkv, k, k_stride)) != RTP_OK) return st;
  if ((st = check_rows(T, Hkv, v, v_stride)) != RTP_OK) return st;
  if (spans == nullptr || (ph.n_rkv > 0 && (bounds == nullptr || bound_scale == nullptr)))
    return RTP_ERR_INVALID_ARG;
  if (!aligned16(spans) || !aligned16(bounds)) return RTP_ERR_ALIGNMENT;
  WriteParams p;
  fill_write(&p, T, Hkv, k, k_stride, v, v_stride, k_pages, v_pages, k_scale, v_scale);
  p.spans = reinterpret_cast<const int4*>(spans);
  p.n_spans = n_spans;
  p.bounds = bounds;
  p.bound_scale = bound_scale;
  p.n_rkv = ph.n_rkv;
  for (int g = 0; g < Hkv; ++g) p.rank[g] = -1;
  for (int i = 0; i < ph.n_rkv; ++i) p.rank[ph.head[i]] = (int16_t)i;
  const int64_t blocks = (int64_t)n_spans * Hkv;
  if (blocks > INT32_MAX) return RTP_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  TraceScope tr("kv_append", s);
  return check_cuda(launch_dependent(k_pages.type == RTP_KV_E4M3 ? kv_append_kernel<true>
                                                                 : kv_append_kernel<false>,
                                     dim3((unsigned)blocks), dim3(kAppendThreads), 0, s, p));
}
