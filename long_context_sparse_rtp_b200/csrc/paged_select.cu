// paged_select.cu -- the pages a decode token's retrieval heads attend to
// (rtp_paged_block_select).
//
// Score of page p for query head h, in whole numbers:
//   a_h = max_d |q_hd|,  sq_h = a_h * (1/127),  q8_hd = rint(q_hd / sq_h),
//   I(h, p) = sum_d max(q8_hd lo8_pd, q8_hd hi8_pd)
//           = sum_d min(q8_hd, 0) lo8_pd + max(q8_hd, 0) hi8_pd,
//   score = float(I) * (sq_h * s_p), and the largest over a kv head's G heads.
// |I| <= 128 * 127 * 127 < 2^24: with 8-bit values in fp16 and fp32 sums the
// tensor-core products give I exactly, whatever the order of summation, so the
// selection (score descending, index ascending) is the same on every run.
// (The integer form of those products is far slower here: 96 rows of up to 2048
// pages took 20 us with it, 16 without, traced.)  With s_p * [lo8, hi8] bounding the
// page's keys, the score bounds every q . k of the page up to the rounding of q.
//
// paged_score_kernel reads the bounds once (2 x 128 bytes and a scale a page,
// straight into fragments: bound by HBM); paged_topn_kernel finds the n-th
// largest key of a row with the row's keys in registers, and writes the kept
// pages in order.
#include <algorithm>

#include "paged.cuh"

namespace rtp {
namespace {

// The score of an ordered key (score_key's inverse).
__device__ __forceinline__ float key_score(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// Key of a page that is always kept: above +inf's, which any number of pages may have.
constexpr uint32_t kForcedKey = 0xFFFFFFFFu;

struct SelectParams {
  const uint16_t* q; int64_t q_sb;
  const int8_t* bounds;       // [n_pages][n_rkv][2][128]
  const float* bound_scale;   // [n_pages][n_rkv]
  const int32_t* table; int64_t table_stride;
  const int32_t* seq_lens;
  uint32_t* keys;             // [B][n_rkv][pitch]: ordered score keys
  int32_t* sel;               // [B][n_rkv][n_sel]
  int32_t* count;             // [B][n_rkv]
  int32_t n_pages, width, pitch, ps_shift, G, n_rkv, n_sel, n_first, n_recent;
  int16_t head[kMaxHeads];
};

__device__ __forceinline__ int blocks_of(const SelectParams& p, int b) {
  const int64_t len = max(0, p.seq_lens[b]);
  return (int)min((int64_t)p.width, (len + (1 << p.ps_shift) - 1) >> p.ps_shift);
}

// D(16x8) += A(16x16 fp16, row) * B(16x8 fp16, col), fp32 sums.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four signed bytes as fp16, the first two in lo, the others in hi: exact (a byte
// + 128 is the low mantissa of 1024 + byte + 128).
__device__ __forceinline__ void s8x4_to_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
  const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
  x ^= 0x80808080u;
  lo = __byte_perm(x, 0x64646464u, 0x4140);
  hi = __byte_perm(x, 0x64646464u, 0x4342);
  const __half2 l = __hsub2(*reinterpret_cast<__half2*>(&lo), off);
  const __half2 h = __hsub2(*reinterpret_cast<__half2*>(&hi), off);
  lo = *reinterpret_cast<const uint32_t*>(&l);
  hi = *reinterpret_cast<const uint32_t*>(&h);
}

constexpr int kQRow = kD + 4;  // fp16 elements: eight bytes of padding keep reads on all banks

template <int NT>
struct ScoreSmem {
  __align__(16) uint16_t q8[2][NT * 8][kQRow];  // min(q8, 0) and max(q8, 0) as fp16
  float sq[NT * 8];
};

// Scores pages [p0, p_end) of row (b, rk), nb pages long, by a CTA of WARPS warps, 16
// pages a warp at once: out(page, key) for each.  NT: tiles of 8 heads.
template <int NT, int WARPS, typename Out>
__device__ __forceinline__ void score_pages(const SelectParams& p, ScoreSmem<NT>& sm, int b, int rk,
                                            int nb, int p0, int p_end, Out out) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int32_t* tab = p.table + (int64_t)b * p.table_stride;

  // this lane's pages: g and g + 8 of the warp's 16
  int32_t phys[2];
  uint4 w[2][4];
  float sp[2];
  auto locate = [&](int first) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int pg = first + warp * 16 + s * 8 + g;
      phys[s] = pg < p_end ? tab[pg] : -1;
    }
  };
  auto load = [&]() {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const bool ok = phys[s] >= 0 && phys[s] < p.n_pages;
      const int64_t at = ok ? (int64_t)phys[s] * p.n_rkv + rk : 0;
      sp[s] = ok ? p.bound_scale[at] : -1.f;  // negative: no such page
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[s][j] = ok ? *reinterpret_cast<const uint4*>(p.bounds + at * 2 * kD + j * 64 + t * 16)
                     : make_uint4(0, 0, 0, 0);
    }
  };
  locate(p0);

  // the G query heads in 8-bit steps, split by sign, a warp a head
  for (int h = warp; h < NT * 8; h += WARPS) {
    float x[4] = {0.f, 0.f, 0.f, 0.f}, s = 0.f;
    if (h < p.G) {
      const uint2 x2 = *reinterpret_cast<const uint2*>(
          p.q + b * p.q_sb + (int64_t)(p.head[rk] * p.G + h) * kD + lane * 4);
      x[0] = bf16_lo(x2.x); x[1] = bf16_hi(x2.x);
      x[2] = bf16_lo(x2.y); x[3] = bf16_hi(x2.y);
    }
    if (h == warp) load();  // the pages' loads overlap the rest of this
    bool odd = false;
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a = fmaxf(a, fabsf(x[i]));
      odd |= !(fabsf(x[i]) < INFINITY);
    }
    a = warp_max(a);
    s = __any_sync(0xffffffffu, odd) ? 0.f : a * kInv127;
    uint16_t neg[4], pos[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = s > 0.f ? fminf(fmaxf(rintf(x[i] / s), -127.f), 127.f) : 0.f;
      neg[i] = __half_as_ushort(__float2half_rn(fminf(v, 0.f)));
      pos[i] = __half_as_ushort(__float2half_rn(fmaxf(v, 0.f)));
    }
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      *reinterpret_cast<uint32_t*>(&sm.q8[0][h][lane * 4 + i]) = neg[i] | ((uint32_t)neg[i + 1] << 16);
      *reinterpret_cast<uint32_t*>(&sm.q8[1][h][lane * 4 + i]) = pos[i] | ((uint32_t)pos[i + 1] << 16);
    }
    if (lane == 0) sm.sq[h] = s;
  }
  if (warp >= NT * 8) load();
  __syncthreads();
  float sqv[NT][2];  // heads 8 nt + 2 t + {0, 1}
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    sqv[nt][0] = sm.sq[nt * 8 + 2 * t];
    sqv[nt][1] = sm.sq[nt * 8 + 2 * t + 1];
  }

  for (;;) {
    const int next = p0 + 16 * WARPS;
    locate(next);  // the next round's table entries arrive during this one
    // 16 products of 16 dimensions: word u of the lane's chunk j is its four
    // elements of product 4 j + u, the same dimensions of the query
    float acc[NT][4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x0[4] = {w[0][j].x, w[0][j].y, w[0][j].z, w[0][j].w};
      const uint32_t x1[4] = {w[1][j].x, w[1][j].y, w[1][j].z, w[1][j].w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t a0, a1, a2, a3;
        s8x4_to_f16(x0[u], a0, a2);
        s8x4_to_f16(x1[u], a1, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 q = *reinterpret_cast<const uint2*>(
              &sm.q8[j >> 1][nt * 8 + g][(j & 1) * 64 + t * 16 + u * 4]);
          mma_f16(acc[nt], a0, a1, a2, a3, q.x, q.y);
        }
      }
    }
    const float spv[2] = {sp[0], sp[1]};
    if (next < p_end) load();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float x = -INFINITY;
      if (spv[s] >= INFINITY) {
        x = INFINITY;
      } else if (spv[s] >= 0.f) {  // the product of two scales stays finite
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (nt * 8 + 2 * t + c < p.G)
              x = fmaxf(x, acc[nt][2 * s + c] * fminf(sqv[nt][c] * spv[s], 3.402823466e38f));
      }
      x = quad_max(x);
      const int pe = p0 + warp * 16 + s * 8 + g;
      if (t == 0 && pe < p_end) {
        const bool forced = pe < p.n_first || pe >= nb - p.n_recent;
        out(pe, forced ? kForcedKey : score_key(x + 0.f));  // -0 and 0 are one score
      }
    }
    if (next >= p_end) return;
    p0 = next;
  }
}

constexpr int kScoreThreads = 256;
constexpr int kScorePages = 16 * kScoreThreads / 32;  // pages of a CTA at once

// CTA (x, row): `rounds` blocks of kScorePages pages of a row.
template <int NT>
__global__ void __launch_bounds__(kScoreThreads) paged_score_kernel(const SelectParams p,
                                                                    const int rounds) {
  griddep_wait();
  __shared__ ScoreSmem<NT> sm;
  const int row = blockIdx.y, b = row / p.n_rkv, rk = row % p.n_rkv;
  const int nb = blocks_of(p, b);
  const int p0 = blockIdx.x * rounds * kScorePages;
  const int p_end = min(nb, p0 + rounds * kScorePages);
  if (p0 >= p_end || nb <= p.n_sel) return;  // a row that keeps every page needs no scores
  uint32_t* keys = p.keys + (int64_t)row * p.pitch;
  score_pages<NT, kScoreThreads / 32>(p, sm, b, rk, nb, p0, p_end,
                                      [&](int i, uint32_t k) { keys[i] = k; });
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

// Inclusive scan over the block.
__device__ __forceinline__ int block_scan(int v, int* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  return v + __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0);
}

constexpr int kOneWarps = 16;  // of a CTA that scores and selects
constexpr int kOneKeys = 4;    // keys of its threads
constexpr int kTopBins = 2048;
constexpr int kTopCand = 1024;

// One CTA per row; a thread has E consecutive keys in registers, or, E == 0 (longer
// rows), reads its share again from L2 on every pass.
//
// The n-th largest key: 2046 equal bins over the row's finite scores, one for
// those at +inf and the pages always kept, and one for -inf; the bin that holds it is found by a scan of the
// counts, and its few keys are ranked against one another.  The bin is a
// non-decreasing function of the score however its arithmetic rounds, so the
// result is exact.  A bin of more than 1024 keys (mass ties) is settled bit by
// bit instead.  Bound by latency: a kernel of 2048 pages takes 2.5 us beyond a
// launch.
//
// NT > 0 (short rows): the CTA scores its row itself first, in tiles of 8 heads, with
// the keys in shared memory: one kernel.
template <int WARPS, int E, int NT>
__global__ void __launch_bounds__(WARPS * 32) paged_topn_kernel(const SelectParams p) {
  constexpr int kThreads = WARPS * 32;
  constexpr int kHeld = NT > 0 ? kThreads * E : 4;
  __shared__ ScoreSmem<(NT > 0 ? NT : 1)> score;
  __shared__ __align__(16) uint32_t held[kHeld];
  __shared__ int sums[2][32], scan1[32], scan2[32];
  __shared__ float wlo[32], whi[32];
  __shared__ int hist[kTopBins];
  __shared__ __align__(16) uint32_t cand[kTopCand];
  __shared__ int n_cand, bin_at, bin_above;
  __shared__ uint32_t cut;
  const int row = blockIdx.x, b = row / p.n_rkv, n = p.n_sel;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kTopBins; i += kThreads) hist[i] = 0;
  if (tid == 0) n_cand = 0;
  griddep_wait();
  const int nb = blocks_of(p, b);
  int32_t* sel = p.sel + (int64_t)row * n;
  if (tid == 0) p.count[row] = min(nb, n);
  if (nb <= n) {
    for (int i = tid; i < n; i += kThreads) sel[i] = i < nb ? i : -1;
    return;
  }
  const uint32_t* keys = NT > 0 ? held : p.keys + (int64_t)row * p.pitch;
  if constexpr (NT > 0) {
    score_pages<NT, WARPS>(p, score, b, row % p.n_rkv, nb, 0, nb,
                           [&](int i, uint32_t k) { held[i] = k; });
    __syncthreads();
  }
  // keys of a thread: whole uint4s, an odd number of them in the longer rows (at 128 bytes
  // from thread to thread 32000 pages took 30 us, 40000 26)
  const int per = E > 0 ? E : (((nb + kThreads - 1) / kThreads + 3) & ~3) | 4;
  const int k0 = tid * per;
  auto load4 = [&](int e, uint32_t (&k)[4]) {  // keys k0 + e ..; 0 behind the last (-inf is above)
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (k0 + e < nb) w = *reinterpret_cast<const uint4*>(keys + k0 + e);
    k[0] = w.x;
    k[1] = k0 + e + 1 < nb ? w.y : 0u;
    k[2] = k0 + e + 2 < nb ? w.z : 0u;
    k[3] = k0 + e + 3 < nb ? w.w : 0u;
  };
  uint32_t kreg[E > 0 ? E / 4 : 1][4];
  if constexpr (E > 0) {
#pragma unroll
    for (int e = 0; e < E / 4; ++e) load4(4 * e, kreg[e]);
  }
  auto each = [&](auto f) {  // f(e, key e of this thread)
    if constexpr (E > 0) {
#pragma unroll
      for (int e = 0; e < E; ++e) f(e, kreg[e / 4][e & 3]);
    } else {
      for (int e = 0; e < per; e += 4) {
        uint32_t k[4];
        load4(e, k);
#pragma unroll
        for (int i = 0; i < 4; ++i) f(e + i, k[i]);
      }
    }
  };

  // range of the finite scores
  const uint32_t key_pinf = score_key(INFINITY), key_ninf = score_key(-INFINITY);
  uint32_t kmin = 0xFFFFFFFFu, kmax = 0u;
  each([&](int, uint32_t k) {
    const bool finite = k > key_ninf && k < key_pinf;
    kmin = min(kmin, finite ? k : 0xFFFFFFFFu);
    kmax = max(kmax, finite ? k : 0u);
  });
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  if (lane == 0) {
    wlo[warp] = __uint_as_float(kmin);
    whi[warp] = __uint_as_float(kmax);
  }
  __syncthreads();
  kmin = __reduce_min_sync(0xffffffffu, lane < WARPS ? __float_as_uint(wlo[lane]) : 0xFFFFFFFFu);
  kmax = __reduce_max_sync(0xffffffffu, lane < WARPS ? __float_as_uint(whi[lane]) : 0u);
  const bool some = kmin <= kmax;
  const float half_lo = some ? 0.5f * key_score(kmin) : 0.f;  // halves: no overflow
  const float range = some ? 0.5f * key_score(kmax) - half_lo : 0.f;
  const float scale = range > 0.f ? fminf((kTopBins - 3) / range, 3.402823466e38f) : 0.f;
  auto bin_of = [&](uint32_t k) -> int {
    const int mid = 1 + (int)fminf((0.5f * key_score(k) - half_lo) * scale, (float)(kTopBins - 3));
    return k >= key_pinf ? kTopBins - 1 : k <= key_ninf ? 0 : mid;
  };
  uint32_t bins[E > 0 ? E / 2 : 1] = {};  // two to a register
  each([&](int e, uint32_t k) {
    const int at = bin_of(k);
    if constexpr (E > 0) bins[e / 2] = e & 1 ? bins[e / 2] | (uint32_t)at << 16 : (uint32_t)at;
    if (k) atomicAdd(&hist[at], 1);
  });
  __syncthreads();

  // the bin that holds the n-th largest: a thread has kTopBins / kThreads bins
  constexpr int kOwn = kTopBins / kThreads;
  int own = 0;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) own += hist[tid * kOwn + i];
  int above = nb - block_scan(own, scan1);  // keys in the bins of higher threads
  if (above < n && n <= above + own) {
#pragma unroll
    for (int i = kOwn - 1; i >= 0; --i) {
      const int c = hist[tid * kOwn + i];
      if (above < n && n <= above + c) {
        bin_at = tid * kOwn + i;
        bin_above = above;
      }
      above += c;
    }
  }
  __syncthreads();
  const int bin = bin_at, among = n - bin_above, in_bin = hist[bin];
  uint32_t T = 0;
  if (in_bin <= kTopCand) {
    each([&](int e, uint32_t k) {
      int at;
      if constexpr (E > 0)
        at = (bins[e / 2] >> (16 * (e & 1))) & 0xFFFF;
      else
        at = bin_of(k);
      if (k && at == bin) cand[atomicAdd(&n_cand, 1)] = k;
    });
    __syncthreads();
    for (int i = tid; i < in_bin; i += kThreads) {
      const uint32_t k = cand[i];
      int gt = 0, ge = 0;
      for (int j = 0; j < in_bin; ++j) {
        gt += cand[j] > k;
        ge += cand[j] >= k;
      }
      if (gt < among && among <= ge) cut = k;  // equal keys store the same value
    }
    __syncthreads();
    T = cut;
  } else {
    int turn = 0;  // the largest T with at least n keys >= T
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t c = T | (1u << bit);
      int cnt = 0;
      each([&](int, uint32_t k) { cnt += k >= c; });
      if (block_count<WARPS>(cnt, sums, turn) >= n) T = c;
    }
  }
  // keys above T all stay; of those equal to T the first ones
  int gt = 0, eq = 0;
  each([&](int, uint32_t k) {
    gt += k > T;
    eq += k == T;
  });
  int gt_at = block_scan(gt, scan2) - gt;
  __syncthreads();
  int eq_at = block_scan(eq, scan1) - eq;
  __shared__ int all_gt;
  if (tid == kThreads - 1) all_gt = gt_at + gt;
  __syncthreads();
  const int need = n - all_gt;
  each([&](int e, uint32_t k) {
    const bool above_cut = k > T, at_cut = k == T;
    if (above_cut || (at_cut && eq_at < need)) sel[gt_at + min(eq_at, need)] = k0 + e;
    gt_at += above_cut;
    eq_at += at_cut;
  });
}

}  // namespace

inline int32_t select_pitch(int32_t width) { return (width + 3) & ~3; }  // whole uint4s a row

size_t paged_select_ws(int64_t rows, int32_t width) {
  return align_up(kStatusBytes + (size_t)rows * select_pitch(width) * 4, 256);
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
  if (ws == nullptr || ws_bytes < paged_select_ws(rows, table_width))
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
  p.pitch = select_pitch(table_width);
  p.ps_shift = log2_exact(page_size);
  p.G = ph.G;
  p.n_rkv = ph.n_rkv;
  p.n_sel = n_sel;
  p.n_first = n_first;
  p.n_recent = n_recent;
  memcpy(p.head, ph.head, sizeof(p.head));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)rows);
  // A round of pages (256) for a CTA: one kernel, 5.5 us against 7.1.  A second round
  // takes the gain back, unless the rows fill the GPU: 96 rows of 1000 pages 10.7 us
  // against 12.1, 256 rows of 2000 29.6 against 38.5.
  const int64_t rounds_one = std::max<int64_t>(1, std::min<int64_t>(8, rows / 24));
  if (table_width <= 16 * kOneWarps * rounds_one) {
    static_assert(16 * kOneWarps * 8 <= kOneWarps * 32 * kOneKeys, "eight rounds' keys fit");
    TraceScope tr("paged_topn", s);
    return check_cuda(launch_dependent(ph.G <= 8 ? paged_topn_kernel<kOneWarps, kOneKeys, 1>
                                                 : paged_topn_kernel<kOneWarps, kOneKeys, 2>,
                                       grid, dim3(kOneWarps * 32), 0, s, p));
  }
  if (table_width > n_sel) {
    TraceScope tr("paged_score", s);
    // one block of pages a CTA while the GPU has room for that (eight CTAs an SM),
    // else several, which reuse the CTA's query and overlap their loads
    const int64_t blocks = (table_width + kScorePages - 1) / kScorePages;
    const int rounds = (int)std::min<int64_t>(8, (blocks * rows + 8 * 148 - 1) / (8 * 148));
    const dim3 blocks2((unsigned)((blocks + rounds - 1) / rounds), (unsigned)rows);
    if ((st = check_cuda(launch_dependent(ph.G <= 8 ? paged_score_kernel<1> : paged_score_kernel<2>,
                                          blocks2, dim3(kScoreThreads), 0, s, p, rounds))) != RTP_OK)
      return st;
  }
  // the smallest CTA whose registers hold the row
  TraceScope tr("paged_topn", s);
  if (table_width <= 16 * 32 * 8)
    return check_cuda(launch_dependent(paged_topn_kernel<16, 8, 0>, grid, dim3(512), 0, s, p));
  if (table_width <= 32 * 32 * 16)
    return check_cuda(launch_dependent(paged_topn_kernel<32, 16, 0>, grid, dim3(1024), 0, s, p));
  return check_cuda(launch_dependent(paged_topn_kernel<32, 0, 0>, grid, dim3(1024), 0, s, p));
}
