// paged_select.cu -- the pages a decode token's retrieval heads attend to
// (rtp_paged_block_select).
//
// Score of page p for query head h, in whole numbers:
//   a_h = max_d |q_hd|,  sq_h = a_h * (1/127),  q8_hd = rint(q_hd / sq_h),
//   I(h, p) = sum_d max(q8_hd lo8_pd, q8_hd hi8_pd)
//           = sum_d min(q8_hd, 0) lo8_pd + max(q8_hd, 0) hi8_pd,
//   score = float(I) * (sq_h * s_p), and the largest over a kv head's G heads.
// |I| <= 128 * 127 * 127 < 2^24, so I is exact in the 32-bit sums of the integer
// tensor-core products and in fp32: every order of summation gives the same
// score, and the selection (score descending, index ascending) is the same on
// every run.  With sq * [lo8, hi8] * s_p bounding the page's keys, the score
// bounds every q . k of the page up to the rounding of q.
//
// paged_score_kernel reads the bounds once (2 x 128 bytes and a scale a page,
// straight into fragments: bound by HBM); paged_topn_kernel finds the n-th
// largest key of a row bit by bit with the row's keys in registers, and writes
// the kept pages in order.
#include "paged.cuh"

namespace rtp {
namespace {

struct SelectParams {
  const uint16_t* q; int64_t q_sb;
  const int8_t* bounds;       // [n_pages][n_rkv][2][128]
  const float* bound_scale;   // [n_pages][n_rkv]
  const int32_t* table; int64_t table_stride;
  const int32_t* seq_lens;
  uint32_t* keys;             // [B][n_rkv][width]: ordered score keys
  int32_t* sel;               // [B][n_rkv][n_sel]
  int32_t* count;             // [B][n_rkv]
  int32_t n_pages, width, ps_shift, G, n_rkv, n_sel, n_first, n_recent;
  int16_t head[kMaxHeads];
};

__device__ __forceinline__ int blocks_of(const SelectParams& p, int b) {
  const int64_t len = max(0, p.seq_lens[b]);
  return (int)min((int64_t)p.width, (len + (1 << p.ps_shift) - 1) >> p.ps_shift);
}

// D(16x8) += A(16x32 s8, row) * B(32x8 s8, col), 32-bit sums.
__device__ __forceinline__ void mma_s8(int32_t (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int kScoreThreads = 256;
constexpr int kScoreSteps = 2;                                    // 8-page steps per warp
constexpr int kScorePages = kScoreSteps * 8 * kScoreThreads / 32;  // pages of a CTA

__global__ void __launch_bounds__(kScoreThreads) paged_score_kernel(const SelectParams p) {
  griddep_wait();
  const int row = blockIdx.y, b = row / p.n_rkv, rk = row % p.n_rkv;
  const int nb = blocks_of(p, b);
  const int p0 = blockIdx.x * kScorePages;
  if (p0 >= nb || nb <= p.n_sel) return;  // a row that keeps every page needs no scores
  __shared__ __align__(16) int8_t qn[16][kD], qp[16][kD];
  __shared__ float sq[16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;

  // this warp's pages first: their loads overlap the query's
  const int32_t* tab = p.table + (int64_t)b * p.table_stride;
  uint4 w[kScoreSteps][4];
  float sp[kScoreSteps];
#pragma unroll
  for (int s = 0; s < kScoreSteps; ++s) {
    const int pg = p0 + (warp * kScoreSteps + s) * 8 + g;
    const int32_t phys = pg < nb ? tab[pg] : -1;
    const bool ok = phys >= 0 && phys < p.n_pages;
    const int64_t at = ok ? (int64_t)phys * p.n_rkv + rk : 0;
    sp[s] = ok ? p.bound_scale[at] : -1.f;  // negative: no such page
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[s][j] = ok ? *reinterpret_cast<const uint4*>(p.bounds + at * 2 * kD + j * 64 + t * 16)
                   : make_uint4(0, 0, 0, 0);
  }

  // the G query heads in 8 bits, split by sign; a warp takes heads warp and warp + 8
  for (int h = warp; h < 16; h += kScoreThreads / 32) {
    uint32_t neg = 0, pos = 0;
    float s = 0.f;
    if (h < p.G) {
      const uint2 x2 = *reinterpret_cast<const uint2*>(
          p.q + b * p.q_sb + (int64_t)(p.head[rk] * p.G + h) * kD + lane * 4);
      const float x[4] = {bf16_lo(x2.x), bf16_hi(x2.x), bf16_lo(x2.y), bf16_hi(x2.y)};
      bool odd = false;
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a = fmaxf(a, fabsf(x[i]));
        odd |= !(fabsf(x[i]) < INFINITY);
      }
      a = warp_max(a);
      s = __any_sync(0xffffffffu, odd) ? 0.f : a * kInv127;
      if (s > 0.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int v = (int)fminf(fmaxf(rintf(x[i] / s), -127.f), 127.f);
          neg |= (uint32_t)(min(v, 0) & 0xFF) << (8 * i);
          pos |= (uint32_t)(max(v, 0) & 0xFF) << (8 * i);
        }
      }
    }
    *reinterpret_cast<uint32_t*>(&qn[h][lane * 4]) = neg;
    *reinterpret_cast<uint32_t*>(&qp[h][lane * 4]) = pos;
    if (lane == 0) sq[h] = s;
  }
  __syncthreads();

  // A word i of a thread's 16-byte chunk j pairs with word i of its page's chunk
  // j: the order of the 256 products is the thread's, the same for A and B
  int32_t acc[kScoreSteps][4] = {};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int8_t(*src)[kD] = j < 2 ? qn : qp;
    const uint4 lo = *reinterpret_cast<const uint4*>(&src[g][(j & 1) * 64 + t * 16]);
    const uint4 hi = *reinterpret_cast<const uint4*>(&src[g + 8][(j & 1) * 64 + t * 16]);
    const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y}, a1[4] = {lo.z, hi.z, lo.w, hi.w};
#pragma unroll
    for (int s = 0; s < kScoreSteps; ++s) {
      mma_s8(acc[s], a0, w[s][j].x, w[s][j].y);
      mma_s8(acc[s], a1, w[s][j].z, w[s][j].w);
    }
  }
  const float q0 = sq[g], q1 = sq[g + 8];
#pragma unroll
  for (int s = 0; s < kScoreSteps; ++s) {
    float best[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float spp = __shfl_sync(0xffffffffu, sp[s], 4 * (2 * t + e));
      float x = -INFINITY;
      if (spp >= INFINITY) {
        x = INFINITY;
      } else if (spp >= 0.f) {  // the product of two scales stays finite
        if (g < p.G) x = (float)acc[s][e] * fminf(q0 * spp, 3.402823466e38f);
        if (g + 8 < p.G) x = fmaxf(x, (float)acc[s][2 + e] * fminf(q1 * spp, 3.402823466e38f));
      }
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
      best[e] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
    }
    const int pg = p0 + (warp * kScoreSteps + s) * 8 + 2 * t;
    if (g < 2) {
      const int pe = pg + g;
      if (pe < nb) {
        const bool forced = pe < p.n_first || pe >= nb - p.n_recent;
        const float x = forced ? INFINITY : (g ? best[1] : best[0]);
        p.keys[(int64_t)row * p.width + pe] = score_key(x + 0.f);  // -0 and 0 are one score
      }
    }
  }
}

// Sum over the block of a per-thread count; `sums` holds two buffers in turn.
template <int WARPS>
__device__ __forceinline__ int block_count(int v, int (*sums)[32], int& turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = __reduce_add_sync(0xffffffffu, v);
  if (lane == 0) sums[turn][warp] = v;
  __syncthreads();
  const int all = __reduce_add_sync(0xffffffffu, lane < WARPS ? sums[turn][lane] : 0);
  turn ^= 1;
  return all;
}

// One CTA per row.  E > 0: thread i of warp w holds keys w * 32 E + 32 e + lane;
// E == 0 (longer rows): the keys are read again from L2 on every pass.
template <int WARPS, int E>
__global__ void __launch_bounds__(WARPS * 32) paged_topn_kernel(const SelectParams p) {
  griddep_wait();
  __shared__ int sums[2][32];
  __shared__ int base_gt[32], base_eq[32];
  const int row = blockIdx.x, b = row / p.n_rkv;
  const int nb = blocks_of(p, b), n = p.n_sel;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* sel = p.sel + (int64_t)row * n;
  if (tid == 0) p.count[row] = min(nb, n);
  if (nb <= n) {
    for (int i = tid; i < n; i += WARPS * 32) sel[i] = i < nb ? i : -1;
    return;
  }
  const uint32_t* keys = p.keys + (int64_t)row * p.width;
  const int steps = E > 0 ? E : (nb + WARPS * 32 - 1) / (WARPS * 32);
  const int w0 = warp * 32 * steps + lane;  // this thread's first key
  uint32_t kreg[E > 0 ? E : 1];
  if (E > 0) {
#pragma unroll
    for (int e = 0; e < E; ++e) kreg[e] = w0 + 32 * e < nb ? keys[w0 + 32 * e] : 0u;
  }
  auto key_at = [&](int e) -> uint32_t {
    if (E > 0) return kreg[E > 0 ? e : 0];
    return w0 + 32 * e < nb ? keys[w0 + 32 * e] : 0u;
  };
  // the largest T with at least n keys >= T; a real key is never 0 (-inf maps above it)
  uint32_t T = 0;
  int turn = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t c = T | (1u << bit);
    int cnt = 0;
#pragma unroll
    for (int e = 0; e < steps; ++e) cnt += key_at(e) >= c;
    if (block_count<WARPS>(cnt, sums, turn) >= n) T = c;
  }
  // keys above T all stay; of those equal to T the first ones
  int gt = 0, eq = 0;
#pragma unroll
  for (int e = 0; e < steps; ++e) {
    const uint32_t k = key_at(e);
    gt += k > T;
    eq += k == T;
  }
  const int wg = __reduce_add_sync(0xffffffffu, gt), we = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    base_gt[warp] = wg;
    base_eq[warp] = we;
  }
  __syncthreads();
  int bg = 0, be = 0, all_gt = 0;
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) {
      bg += base_gt[w];
      be += base_eq[w];
    }
    all_gt += base_gt[w];
  }
  const int need = n - all_gt;
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll
  for (int e = 0; e < steps; ++e) {
    const uint32_t k = key_at(e);
    const uint32_t mg = __ballot_sync(0xffffffffu, k > T), me = __ballot_sync(0xffffffffu, k == T);
    const int eq_before = be + __popc(me & below);
    const bool keep = k > T || (k == T && eq_before < need);
    if (keep) sel[bg + __popc(mg & below) + min(eq_before, need)] = w0 + 32 * e;
    bg += __popc(mg);
    be += __popc(me);
  }
}

}  // namespace

size_t paged_select_ws(int32_t rows, int32_t width) {
  return align_up(kStatusBytes + (size_t)rows * width * 4, 256);
}

}  // namespace rtp

using namespace rtp;

extern "C" rtp_status rtp_paged_block_select(
    int32_t B, int32_t H, int32_t Hkv, const uint8_t* kv_role, const void* q, int64_t q_stride,
    const int8_t* bounds, const float* bound_scale, int32_t n_pages, int32_t page_size,
    const int32_t* block_table, int64_t table_stride, int32_t table_width,
    const int32_t* seq_lens, int32_t n_sel, int32_t n_first, int32_t n_recent, int32_t* sel,
    int32_t* sel_count, void* ws, size_t ws_bytes, rtp_stream_t stream) {
  PagedHeads ph;
  rtp_status st = make_paged_heads(H, Hkv, kv_role, &ph);
  if (st != RTP_OK) return st;
  if ((st = check_page_size(page_size)) != RTP_OK) return st;
  if (B < 0 || n_pages < 1 || table_width < 1 || table_stride < table_width || n_sel < 1 ||
      n_first < 0 || n_recent < 0 || n_first > n_sel - n_recent)
    return RTP_ERR_INVALID_ARG;
  if ((int64_t)table_width * page_size > kMaxTokens) return RTP_ERR_UNSUPPORTED;
  const int64_t rows = (int64_t)B * ph.n_rkv;
  if (rows == 0) return RTP_OK;
  if (rows > 65535) return RTP_ERR_UNSUPPORTED;
  if (q == nullptr || bounds == nullptr || bound_scale == nullptr || block_table == nullptr ||
      seq_lens == nullptr || sel == nullptr || sel_count == nullptr)
    return RTP_ERR_INVALID_ARG;
  if (q_stride < (int64_t)H * kD) return RTP_ERR_INVALID_ARG;
  if (!aligned16(q) || (q_stride * 2) % 16 || !aligned16(bounds) || !aligned16(ws))
    return RTP_ERR_ALIGNMENT;
  if (ws == nullptr || ws_bytes < paged_select_ws((int32_t)rows, table_width))
    return RTP_ERR_WORKSPACE_TOO_SMALL;
  SelectParams p;
  memset(&p, 0, sizeof(p));
  p.q = static_cast<const uint16_t*>(q);
  p.q_sb = q_stride;
  p.bounds = bounds;
  p.bound_scale = bound_scale;
  p.table = block_table;
  p.table_stride = table_stride;
  p.seq_lens = seq_lens;
  p.keys = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + kStatusBytes);
  p.sel = sel;
  p.count = sel_count;
  p.n_pages = n_pages;
  p.width = table_width;
  p.ps_shift = log2_exact(page_size);
  p.G = ph.G;
  p.n_rkv = ph.n_rkv;
  p.n_sel = n_sel;
  p.n_first = n_first;
  p.n_recent = n_recent;
  memcpy(p.head, ph.head, sizeof(p.head));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (table_width > n_sel) {
    TraceScope tr("paged_score", s);
    const dim3 grid((table_width + kScorePages - 1) / kScorePages, (unsigned)rows);
    if ((st = check_cuda(launch_dependent(paged_score_kernel, grid, dim3(kScoreThreads), 0, s,
                                          p))) != RTP_OK)
      return st;
  }
  // the smallest CTA whose registers hold the row
  TraceScope tr("paged_topn", s);
  const dim3 grid((unsigned)rows);
  if (table_width <= 8 * 32 * 4)
    return check_cuda(launch_dependent(paged_topn_kernel<8, 4>, grid, dim3(256), 0, s, p));
  if (table_width <= 32 * 32 * 4)
    return check_cuda(launch_dependent(paged_topn_kernel<32, 4>, grid, dim3(1024), 0, s, p));
  if (table_width <= 32 * 32 * 16)
    return check_cuda(launch_dependent(paged_topn_kernel<32, 16>, grid, dim3(1024), 0, s, p));
  return check_cuda(launch_dependent(paged_topn_kernel<32, 0>, grid, dim3(1024), 0, s, p));
}
