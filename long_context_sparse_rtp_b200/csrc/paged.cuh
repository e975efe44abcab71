// paged.cuh -- what the paged-cache kernels share: page addressing, head order,
// 8-bit conversions and host-side checks.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "rtp_host.h"

namespace rtp {

constexpr float kInv127 = 1.f / 127.f;  // 8-bit steps of bounds and queries
constexpr int kGroup = 16;  // keys a warp takes at once: every page holds whole groups
constexpr int64_t kMaxTokens = 1 << 30;  // positions a block table may cover: counts fit 32 bits

// K or V pages as a kernel addresses them: strides in bytes.
struct PageAddr {
  uint8_t* ptr;
  int64_t page, row, head;
};

// kv heads with the retrieval ones first, each kind in increasing order.
struct PagedHeads {
  int32_t Hkv, G, n_rkv;
  int16_t head[kMaxHeads];
};

// launch_dependent with clusters of `csize` CTAs along x.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_dependent_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block,
                                            int csize, size_t smem, cudaStream_t s,
                                            Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)csize;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

inline int page_elt_size(int32_t type) { return type == RTP_KV_BF16 ? 2 : 1; }

inline PageAddr page_addr(const rtp_pages& p) {
  const int64_t e = page_elt_size(p.type);
  return {static_cast<uint8_t*>(p.ptr), p.stride_page * e, p.stride_row * e, p.stride_head * e};
}

inline int log2_exact(int32_t x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

inline rtp_status check_page_size(int32_t ps) {
  return ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256 ? RTP_OK : RTP_ERR_UNSUPPORTED;
}

inline rtp_status check_pages(const rtp_pages& p) {
  if (p.ptr == nullptr || p.n_pages < 1) return RTP_ERR_INVALID_ARG;
  if (p.type != RTP_KV_BF16 && p.type != RTP_KV_E4M3) return RTP_ERR_UNSUPPORTED;
  const rtp_status st = check_page_size(p.page_size);
  if (st != RTP_OK) return st;
  if ((int64_t)p.n_pages * p.page_size > INT32_MAX) return RTP_ERR_UNSUPPORTED;
  if (p.stride_page < kD || p.stride_row < kD || p.stride_head < kD) return RTP_ERR_INVALID_ARG;
  const int e = page_elt_size(p.type);
  if (!aligned16(p.ptr) || (p.stride_page * e) % 16 || (p.stride_row * e) % 16 ||
      (p.stride_head * e) % 16)
    return RTP_ERR_ALIGNMENT;
  return RTP_OK;
}

// K and V pages of one cache: same count, page size and type; scales only for 8 bits.
inline rtp_status check_cache(const rtp_pages& k, const rtp_pages& v, const float* k_scale,
                              const float* v_scale) {
  rtp_status st = check_pages(k);
  if (st != RTP_OK) return st;
  if ((st = check_pages(v)) != RTP_OK) return st;
  if (k.n_pages != v.n_pages || k.page_size != v.page_size || k.type != v.type)
    return RTP_ERR_INVALID_ARG;
  if (k.type == RTP_KV_BF16 && (k_scale != nullptr || v_scale != nullptr))
    return RTP_ERR_INVALID_ARG;
  return RTP_OK;
}

inline rtp_status make_paged_heads(int32_t H, int32_t Hkv, const uint8_t* kv_role, PagedHeads* ph) {
  if (kv_role == nullptr || H < 1 || Hkv < 1 || H % Hkv != 0) return RTP_ERR_INVALID_ARG;
  if (H > kMaxHeads || H / Hkv > 16) return RTP_ERR_UNSUPPORTED;
  ph->Hkv = Hkv;
  ph->G = H / Hkv;
  ph->n_rkv = 0;
  for (int g = 0; g < Hkv; ++g) {
    if (kv_role[g] > 1) return RTP_ERR_INVALID_ARG;
    if (kv_role[g]) ph->head[ph->n_rkv++] = (int16_t)g;
  }
  int n = ph->n_rkv;
  for (int g = 0; g < Hkv; ++g)
    if (!kv_role[g]) ph->head[n++] = (int16_t)g;
  return RTP_OK;
}

// Two e4m3 values (low byte first) as two fp16 values: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(r) : "h"(v));
  return r;
}

// Two fp32 values as two e4m3 values, nearest even, saturating at 448.
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight bf16 values of a 16-byte word as fp32.
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x);
  x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z);
  x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
}

// Eight e4m3 values of an 8-byte word as fp32.
__device__ __forceinline__ void unpack8(const uint2& w, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = e4m3x2_to_f16x2((uint16_t)((i < 2 ? w.x : w.y) >> (16 * (i & 1))));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

}  // namespace rtp
