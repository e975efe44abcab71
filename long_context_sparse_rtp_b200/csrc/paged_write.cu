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

// e4m3(x / scale) for one scale and many x without a division each: the fp32
// quotient lies between x * lo and x * hi, lo and hi = (1 / scale) (1 -+ 2^-21) (the
// reciprocal, its factor, the products and the quotient are each off by at most
// 2^-24 of themselves), so where both round to the same e4m3 value that is the
// quotient's; the others, next to the middle of two e4m3 values, are divided.  A
// power of two as scale is exact: lo = hi.  With sixteen divisions a thread the
// write of 20 K tokens of 8 heads took 29 us.
struct Divider {
  float scale, lo, hi;
  bool always;  // divide all: the reciprocal is not a normal number
  __device__ __forceinline__ explicit Divider(float s) : scale(s) {
    const float inv = 1.f / s;
    const uint32_t b = __float_as_uint(s), e = (b >> 23) & 0xFF;
    always = e < 2 || e > 252;
    const bool exact = (b & 0x7FFFFFu) == 0u;
    lo = exact ? inv : inv * (1.f - 0x1p-21f);
    hi = exact ? inv : inv * (1.f + 0x1p-21f);
  }
};

__device__ __forceinline__ uint2 pack_e4m3(const float (&q)[8]) {
  return make_uint2(f32x2_to_e4m3x2(q[0], q[1]) | ((uint32_t)f32x2_to_e4m3x2(q[2], q[3]) << 16),
                    f32x2_to_e4m3x2(q[4], q[5]) | ((uint32_t)f32x2_to_e4m3x2(q[6], q[7]) << 16));
}

// Eight values (16 bytes of bf16) as eight e4m3 bytes.
__device__ __forceinline__ uint2 quantise8(const uint4& w, const Divider& d) {
  float x[8], lo[8], hi[8];
  unpack8(w, x);
  const unsigned long long dl = f2_pack(d.lo, d.lo), dh = f2_pack(d.hi, d.hi);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const unsigned long long v = f2_pack(x[i], x[i + 1]);
    f2_unpack(f2_mul(v, dl), lo[i], lo[i + 1]);
    f2_unpack(f2_mul(v, dh), hi[i], hi[i + 1]);
  }
  uint2 r = pack_e4m3(lo);
  const uint2 up = pack_e4m3(hi);
  if (r.x != up.x || r.y != up.y || d.always) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] / d.scale;
    r = pack_e4m3(x);
  }
  return r;
}

constexpr int kWriteThreads = 128;  // 256 threads 23.5 us where these take 21.7 (20 K tokens, 8 bits)
constexpr int kWriteRows = 2;       // tokens a thread has in flight (1 or 4: 25 us)

// A CTA takes kWriteRows times as many tokens as its threads hold rows of 16-byte
// chunks (16 a head); a thread keeps its chunk of the row.
template <bool E4M3>
__global__ void __launch_bounds__(kWriteThreads) kv_write_kernel(const WriteParams p,
                                                                 const int rows) {
  griddep_wait();
  const int per_row = p.Hkv * 16;
  const int r = per_row >= kWriteThreads ? 0 : threadIdx.x / per_row;
  if (r >= rows) return;
  const int64_t t0 = (int64_t)blockIdx.x * rows * kWriteRows + r;
  for (int c = threadIdx.x - r * per_row; c < per_row; c += kWriteThreads) {
    const int h = c >> 4, ch = c & 15;
    int32_t slot[kWriteRows];
    uint4 kw[kWriteRows], vw[kWriteRows];
#pragma unroll
    for (int i = 0; i < kWriteRows; ++i) {
      const int64_t t = t0 + i * rows;
      slot[i] = t < p.T ? p.slot_map[t] : -1;
      if (t < p.T) {
        kw[i] = *reinterpret_cast<const uint4*>(p.k + t * p.k_st + c * 8);
        vw[i] = *reinterpret_cast<const uint4*>(p.v + t * p.v_st + c * 8);
      }
    }
    const Divider kd(E4M3 && p.k_scale ? p.k_scale[h] : 1.f);
    const Divider vd(E4M3 && p.v_scale ? p.v_scale[h] : 1.f);
#pragma unroll
    for (int i = 0; i < kWriteRows; ++i) {
      const int64_t page = slot[i] >> p.ps_shift, row = slot[i] & ((1 << p.ps_shift) - 1);
      if (slot[i] < 0 || page >= p.n_pages) continue;
      uint8_t* ko = p.kp.ptr + page * p.kp.page + row * p.kp.row + h * p.kp.head;
      uint8_t* vo = p.vp.ptr + page * p.vp.page + row * p.vp.row + h * p.vp.head;
      if (E4M3) {
        *reinterpret_cast<uint2*>(ko + ch * 8) = quantise8(kw[i], kd);
        *reinterpret_cast<uint2*>(vo + ch * 8) = quantise8(vw[i], vd);
      } else {
        *reinterpret_cast<uint4*>(ko + ch * 16) = kw[i];
        *reinterpret_cast<uint4*>(vo + ch * 16) = vw[i];
      }
    }
  }
}

constexpr int kAppendThreads = 128;

// CTA: one span (page) and kv head; 16 threads a row, 8 rows at a time.  Each
// thread keeps the running bounds of its eight dimensions.  Ten CTAs an SM with two
// rows in flight suit 8 bits (26 K tokens of 8 heads, pages of 16: 50 us with four
// rows and the registers they take, 39 so), nine with four bf16.
template <bool E4M3>
__global__ void __launch_bounds__(kAppendThreads, E4M3 ? 10 : 9)
    kv_append_kernel(const WriteParams p) {
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
  const Divider kd(E4M3 && p.k_scale ? p.k_scale[h] : 1.f);
  const Divider vd(E4M3 && p.v_scale ? p.v_scale[h] : 1.f);
#pragma unroll (E4M3 ? 2 : 4)
  for (int r = fresh + r0; r < rows; r += 8) {
    const int64_t t = (int64_t)sp.w + r - fresh;
    if (t < 0 || t >= p.T) continue;
    const uint4 kw = *reinterpret_cast<const uint4*>(p.k + t * p.k_st + h * kD + ch * 8);
    const uint4 vw = *reinterpret_cast<const uint4*>(p.v + t * p.v_st + h * kD + ch * 8);
    float x[8];
    if (E4M3) {
      const uint2 kq = quantise8(kw, kd);
      *reinterpret_cast<uint2*>(kb + r * p.kp.row + ch * 8) = kq;
      *reinterpret_cast<uint2*>(vb + r * p.vp.row + ch * 8) = quantise8(vw, vd);
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
  const int rows = Hkv * 16 >= kWriteThreads ? 1 : kWriteThreads / (Hkv * 16);
  const int blocks = (int)(((int64_t)T + rows * kWriteRows - 1) / (rows * kWriteRows));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  TraceScope tr("kv_write", s);
  return check_cuda(launch_dependent(k_pages.type == RTP_KV_E4M3 ? kv_write_kernel<true>
                                                                 : kv_write_kernel<false>,
                                     dim3((unsigned)blocks), dim3(kWriteThreads), 0, s, p, rows));
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
  if (T == 0) return RTP_OK;
  if ((st = check_rows(T, Hkv, k, k_stride)) != RTP_OK) return st;
  if ((st = check_rows(T, Hkv, v, v_stride)) != RTP_OK) return st;
  if (n_spans == 0) return RTP_OK;
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
