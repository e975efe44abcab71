// paged_attn.cu -- attention of one new token per request over a paged KV cache
// (rtp_paged_attn_decode).
//
//   o_h = sum_j softmax_j(scale * q_h . k_j) v_j
// over the request's keys: every key (retrieval heads), the keys of the listed
// pages (retrieval heads with a selection), or sinks and window (local heads).
// One pass with a running maximum and sum.  Short rows (a request's kv head is a
// row) are split over a cluster each and joined there; otherwise requests of all
// lengths share the GPU evenly: the tiles of 64 keys of every row stand in one
// line, and each CTA takes an equal run of them.  A row that one CTA covers is
// written by it; one that several cover leaves partial results (m, l, o), which a
// second kernel joins in CTA order.
//
// Within a tile each warp has a group of 16 keys, which lies in one
// page, and its own ring of shared-memory stages filled by cp.async: no barrier
// inside a run of tiles.  The tensor-core products are K Q^T (16 keys by 8 heads)
// and V^T P^T (16 dimensions by 8 heads), P^T passing between them by an 8x8
// transpose in registers: G <= 8 heads cost half the products, exponentials and
// accumulators of a form with the heads as 16 rows (8 requests of 128K, 8-bit, all
// heads: 240 us with heads as rows, 164 so; bf16, 64 ragged requests up to 8K: 113
// and 98, before the later steps).  Bound by HBM: G flops a byte of bf16 K/V, 2 G of
// 8-bit.  Three stages a warp, two CTAs an SM (bf16) or three (8 bits), keep 128 and 96 KB
// an SM in flight; two stages and three CTAs are as fast for bf16, four CTAs or six stages
// slower for 8 bits (167-177 us).
//
// Rounding: scores, maxima, sums and outputs in fp32; row sums are taken of P before its
// rounding to the 16-bit type of the P V product.  Beside bf16 rows that is bf16, and P
// goes into two products: cut off to bf16, and the remainder, rounded (off by 2^-15 of P
// at most) and not below 2^-20 P: a V of infinity takes part in both, and neither may be
// zero there.  In one product (2^-8) the outputs were 0.0023 from 64 bits where their own
// rounding to bf16 makes 0.0017; the second one takes the tensor pipe from 9 to 14 % (64
// requests up to 8K 89.3 -> 89.5 us, 8 x 128K mixed 92.6 -> 93.0).  Beside 8-bit rows it
// is fp16, whose values hold theirs exactly, in one product: 2^-11 (2^-33 of the largest
// P, where it is subnormal) leaves the outputs at 0.0017, and a second product took 8 x
// 128K from 164.5 to 171.4 us.
// Beside 8-bit rows q is held in fp16, shifted by a power of two to a maximum in
// [2^14, 2^15): exact but for elements under 2^-28 of the head's largest.
#include <cooperative_groups.h>

#include <algorithm>

#include "paged.cuh"

namespace rtp {
namespace {

// A row that several CTAs share, and the line's share of a CTA.
struct SplitRow {
  int64_t first;      // where its tiles start on the line
  int64_t chunk;
  int32_t row, tiles; // row -1: none
  int32_t pad[2];
};

struct PagedAttnParams {
  const uint16_t* q; int64_t q_sb;
  uint16_t* o; int64_t o_sb;
  float* lse;                     // [B][H] or null
  PageAddr kp, vp;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table; int64_t table_stride;
  const int32_t* seq_lens;
  const int32_t* sel;             // [B][n_rkv][n_sel]
  const int32_t* sel_count;       // [B][n_rkv]
  float* part;                    // [CTAs][2][G][kPartRow]
  SplitRow* split;                // per CTA: the row that starts in it and goes on in the next
  float scale_log2;
  int32_t B, G, Hkv, n_rkv, H, n_pages, width, ps_shift, window, n_sink, n_sel;
  int16_t head[kMaxHeads];
};

constexpr int kAttnWarps = 4;  // of a CTA of the split over all CTAs; a tile is a group each
constexpr int kAttnThreads = kAttnWarps * 32;

// Tokens of request b, as far as its table can hold them.
__device__ __forceinline__ int paged_len(const PagedAttnParams& p, int b) {
  return (int)min((int64_t)max(0, p.seq_lens[b]), (int64_t)p.width << p.ps_shift);
}

// Groups of 16 keys that hold the sinks and the window of a local head: sink
// groups [0, n0), then groups from w0 on.
struct LocalRange {
  int n0, w0, total, win_lo;
};
__device__ __forceinline__ LocalRange local_range(const PagedAttnParams& p, int len) {
  LocalRange r;
  const int ng = (len + kGroup - 1) / kGroup;
  r.win_lo = max(0, len - p.window);
  r.n0 = (min(p.n_sink, len) + kGroup - 1) / kGroup;
  r.w0 = max(r.n0, r.win_lo / kGroup);
  r.total = r.n0 + max(0, ng - r.w0);
  return r;
}

template <bool SEL>
__device__ __forceinline__ int row_groups(const PagedAttnParams& p, int b, int i, int len) {
  if (i >= p.n_rkv) return local_range(p, len).total;
  if (SEL)
    return len > 0 ? max(0, min(p.sel_count[b * p.n_rkv + i], p.n_sel)) << (p.ps_shift - 4) : 0;
  return (len + kGroup - 1) / kGroup;
}
__device__ __forceinline__ int tiles_of(int groups) { return (groups + kAttnWarps - 1) / kAttnWarps; }

// What a row takes of the line of all rows' tiles: kRowCost more than its tiles, ahead
// of them, for starting and ending its run, so that a CTA gets fewer keys where it
// gets many short rows (17 requests up to 5044 tokens, 5 of 8 kv heads with a window
// of 12: 26.9 us without, 17.2 so).
constexpr int kRowCost = 5;
constexpr int kMinChunk = 6;  // of the line, a CTA's least share
__device__ __forceinline__ int cost_of(int groups) {
  return groups > 0 ? tiles_of(groups) + kRowCost : 0;
}

template <bool SEL>
__device__ __forceinline__ int64_t request_cost(const PagedAttnParams& p, int b) {
  const int len = paged_len(p, b);
  int64_t n = 0;
  if (p.Hkv > p.n_rkv) n = (int64_t)(p.Hkv - p.n_rkv) * cost_of(row_groups<SEL>(p, b, p.n_rkv, len));
  if (SEL) {
    for (int i = 0; i < p.n_rkv; ++i) n += cost_of(row_groups<SEL>(p, b, i, len));
  } else if (p.n_rkv > 0) {
    n += (int64_t)p.n_rkv * cost_of(row_groups<SEL>(p, b, 0, len));
  }
  return n;
}

__device__ __forceinline__ void mma16816_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float ex2(float x) {  // 2^x, relative error under 2^-22
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}

// The 8x8 16-bit matrix held one row per quad, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
  return r;
}

// The reference m of P = 2^(x - m) moves only when a score exceeds it by more
// than 2^kGrow, so most groups need one vote instead of a reduction.  In fp16 P
// is held as 2^kShift p: at most 2^(kGrow + kShift) = 2^14, and subnormal only
// under 2^-22 of the reference.
constexpr float kGrow = 6.f;
template <bool E4M3>
constexpr float kShift = E4M3 ? 8.f : 0.f;
constexpr float kNoRef = -3.0e38f;  // no key seen: any score moves it

// One warp's stages.  K rows: bf16 swizzled by row & 7 (ldmatrix), 8-bit by
// (row & 1) << 2; V rows: bf16 by row & 7, 8-bit by ((row >> 1) & 3) << 1: each
// makes the eight 16-byte reads of a quarter warp fall on different banks.
template <bool E4M3>
struct WarpStages {
  static constexpr int kRow = E4M3 ? kD : 2 * kD;  // bytes
  static constexpr int kStages = 3;
  static constexpr int kCtasPerSm = E4M3 ? 3 : 2;
  uint8_t k[kStages][kGroup][kRow];
  uint8_t v[kStages][kGroup][kRow];
};

template <bool E4M3, int WARPS>
struct AttnSmem {
  WarpStages<E4M3> w[WARPS];  // a finished run's partial outputs reuse each warp's stages
  float wm[WARPS][16], wl[WARPS][16];
  int64_t sums[WARPS], first;
  int req;
};
// A finished run's outputs in a warp's stages: rows of heads, padded so that the
// quads' stores fall on different banks.
template <bool E4M3>
constexpr int kOutRow = E4M3 ? 148 : 132;
template <bool E4M3>
__device__ __forceinline__ int out_at(int r, int d) {
  return r * kOutRow<E4M3> + d + (E4M3 ? 2 * (d >> 4) : 0);
}
static_assert(sizeof(WarpStages<true>) >= 16 * kOutRow<true> * 4, "partials fit a warp's stages");
static_assert(sizeof(WarpStages<false>) >= 16 * kOutRow<false> * 4, "partials fit a warp's stages");

// Where a run's results go: o and lse, or a partial.
__device__ __forceinline__ void store_final(const PagedAttnParams& p, int b, int g, int r, int d,
                                            float m, float l, float o) {
  const int h = g * p.G + r;
  const float vs = p.v_scale ? p.v_scale[g] : 1.f;
  const float x = l > 0.f || l != l ? o / l * vs : 0.f;
  p.o[b * p.o_sb + (int64_t)h * kD + d] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
  if (d == 0 && p.lse != nullptr)
    p.lse[(int64_t)b * p.H + h] = l > 0.f || l != l ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// Tiles [t0, t0 + n_run) of row i of request b by this CTA: leaves each warp's
// maximum, sum and outputs in shared memory, after a barrier.  NT: tiles of 8 query
// heads (1 for G <= 8).
template <bool E4M3, bool SEL, int NT, int WARPS>
__device__ __forceinline__ void attend_run(const PagedAttnParams& p, AttnSmem<E4M3, WARPS>& sm,
                                           int b, int i, int len, int groups, int t0, int n_run) {
  constexpr int kRow = WarpStages<E4M3>::kRow, kStages = WarpStages<E4M3>::kStages;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int head = p.head[i];
  const LocalRange lr = local_range(p, len);
  const bool local = i >= p.n_rkv;
  uint8_t* const kst = &sm.w[warp].k[0][0][0];
  uint8_t* const vst = &sm.w[warp].v[0][0][0];
  constexpr int kStageBytes = kGroup * kRow;
  constexpr int kChunks = kRow / 16, kRows = 32 / kChunks;  // 16-byte chunks a row; rows a step
  const int lr_ = lane / kChunks, lc = lane % kChunks;      // this lane's row of a step and chunk
  const int64_t k_lane = lr_ * p.kp.row + lc * 16, v_lane = lr_ * p.vp.row + lc * 16;

  // ---- this warp's groups: tile tt of the run is group WARPS (t0 + tt) + warp
  const int32_t* tab = p.table + (int64_t)b * p.table_stride;
  const int32_t* sl = SEL ? p.sel + ((int64_t)b * p.n_rkv + (local ? 0 : i)) * p.n_sel : nullptr;
  // Each lane looks one tile's group up, 32 tiles at once: its physical page (-1
  // where there is none), and its first row in the page with the keys that count
  // (bit r of the low half: key r of the group).
  auto locate = [&](int first, int& page, uint32_t& rows) {
    const int tt = first + lane, gi = WARPS * (t0 + tt) + warp;
    page = -1;
    rows = 0;
    if (tt >= n_run || gi >= groups) return;
    int key0 = gi * kGroup;
    if (local) {
      key0 = (gi < lr.n0 ? gi : lr.w0 + gi - lr.n0) * kGroup;
    } else if (SEL) {
      const int per = p.ps_shift - 4;
      const int lp = sl[gi >> per];
      if (lp < 0 || lp >= p.width) return;
      key0 = (lp << p.ps_shift) + (gi & ((1 << per) - 1)) * kGroup;
    }
    if (key0 >= len) return;
    page = tab[key0 >> p.ps_shift];
    uint32_t mask = len - key0 >= kGroup ? 0xFFFFu : (1u << (len - key0)) - 1u;
    if (local) {
      const int below = p.n_sink - key0, from = lr.win_lo - key0;  // j < n_sink or j >= win_lo
      const uint32_t sink = below >= kGroup ? 0xFFFFu : (below > 0 ? (1u << below) - 1u : 0u);
      const uint32_t win = from <= 0 ? 0xFFFFu : (from < kGroup ? 0xFFFFu << from : 0u);
      mask &= sink | win;
    }
    rows = ((uint32_t)(key0 & ((1 << p.ps_shift) - 1)) << 16) | mask;
  };
  const uint8_t* const khead = p.kp.ptr + head * p.kp.head + k_lane;
  const uint8_t* const vhead = p.vp.ptr + head * p.vp.head + v_lane;
  int page_now, page_next = -1;
  uint32_t rows_now, rows_next = 0;
  locate(0, page_now, rows_now);
  // Starts the loads of tile j (in order); returns its key mask.
  auto issue = [&](int j, int st) -> uint32_t {
    if (j >= n_run) return 0;
    if ((j & 31) == 0 && j > 0) {
      page_now = page_next;
      rows_now = rows_next;
    }
    if ((j & 31) == 16) locate((j & ~31) + 32, page_next, rows_next);  // arrives in time
    const int page = __shfl_sync(0xffffffffu, page_now, j & 31);
    const uint32_t rows = __shfl_sync(0xffffffffu, rows_now, j & 31);
    const uint32_t mask = page >= 0 && page < p.n_pages ? rows & 0xFFFFu : 0u;
    if (mask == 0) return 0;  // nothing to load and nothing read
    const int row_in = rows >> 16;
    const uint8_t* kb = khead + (int64_t)page * p.kp.page + row_in * p.kp.row;
    const uint8_t* vb = vhead + (int64_t)page * p.vp.page + row_in * p.vp.row;
    const uint32_t ks = smem_u32(kst + st * kStageBytes), vs = smem_u32(vst + st * kStageBytes);
#pragma unroll
    for (int u = 0; u < kGroup / kRows; ++u) {
      const int r = u * kRows + lr_;
      const bool ok = (mask >> r) & 1u;  // other rows become zeros and are not read
      const int ck = E4M3 ? lc ^ ((r & 1) << 2) : lc ^ (r & 7);
      const int cv = E4M3 ? lc ^ (((r >> 1) & 3) << 1) : lc ^ (r & 7);
      cp_async16(ks + r * kRow + ck * 16, kb, ok);
      cp_async16(vs + r * kRow + cv * 16, vb, ok);
      kb += kRows * p.kp.row;
      vb += kRows * p.vp.row;
    }
    return mask;
  };

  uint32_t masks[kStages - 1];  // of the tiles in flight
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    masks[s] = issue(s, s);
    cp_async_commit();
  }

  // ---- query heads nt * 8 + g as product operands (columns; keys are the rows)
  uint32_t qb[NT][8][2];
  float ms[NT][2];  // score multipliers of this thread's columns, heads nt * 8 + 2 t + {0, 1}
  {
    const uint16_t* q = p.q + b * p.q_sb + (int64_t)head * p.G * kD;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = nt * 8 + g;
          // 8-bit rows are read 16 bytes a thread: product 4 j + u takes dimensions
          // 64 j + 16 t + 4 u + {0, 1 | 2, 3}
          const int d = E4M3 ? 64 * (kk >> 2) + 16 * t + 4 * (kk & 3) + 2 * e
                             : 16 * kk + 8 * e + 2 * t;
          qb[nt][kk][e] = r < p.G ? *reinterpret_cast<const uint32_t*>(q + r * kD + d) : 0u;
        }
      ms[nt][0] = ms[nt][1] = p.scale_log2;
      if (E4M3) {
        float a = 0.f;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            a = fmaxf(a, fmaxf(fabsf(bf16_lo(qb[nt][kk][e])), fabsf(bf16_hi(qb[nt][kk][e]))));
        a = quad_max(a);
        int ex = (int)((__float_as_uint(a) >> 23) & 0xFF) - 127;
        ex = a > 0.f ? max(-100, min(ex, 127)) : 14;
        // k_scale's sign goes into q and its size into the multiplier, which stays above zero
        // (masked scores are -inf before it, maxima are taken before it): where it would be
        // smaller than a normal number, scores under 2^31 times that are 0 to fp32 either way
        const float ks = p.k_scale ? p.k_scale[head] : 1.f;
        float up = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
        up = ks < 0.f ? -up : up;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            qb[nt][kk][e] = pack_f16x2(bf16_lo(qb[nt][kk][e]) * up, bf16_hi(qb[nt][kk][e]) * up);
        float down = p.scale_log2 * fabsf(ks) * __uint_as_float((uint32_t)(ex - 14 + 127) << 23);
        down = down < 0x1p-126f ? 0x1p-126f : down;
        if (!(fabsf(ks) < INFINITY)) down = __uint_as_float(0x7FC00000u);  // NaN: so are its keys
        ms[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t);
        ms[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
      }
    }
  }

  // o: 8 tiles of 16 dimensions (rows) x 8 heads (columns)
  float oacc[NT][8][4];
  float nref[NT][2], lsum[NT][2];  // kShift - m, and this thread's share of the sum
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int d = 0; d < 8; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) oacc[nt][d][e] = 0.f;
    nref[nt][0] = nref[nt][1] = -kNoRef;
    lsum[nt][0] = lsum[nt][1] = 0.f;
  }

  int st = 0, st_in = kStages - 1;  // stage of this tile, and of the one to load
#pragma unroll 1
  for (int tt = 0; tt < n_run; ++tt) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    const uint32_t mask = masks[0];
#pragma unroll
    for (int m = 0; m + 2 < kStages; ++m) masks[m] = masks[m + 1];
    masks[kStages - 2] = issue(tt + kStages - 1, st_in);
    cp_async_commit();
    const uint8_t* kt = kst + st * kStageBytes;
    const uint8_t* vt = vst + st * kStageBytes;
    st = st == kStages - 1 ? 0 : st + 1;
    st_in = st_in == kStages - 1 ? 0 : st_in + 1;
    if (mask == 0u) continue;

    // S: 16 keys (rows) x 8 heads; this thread has keys g and g + 8
    float s[NT][4] = {}, s2[NT][4] = {};  // two chains of products: half the latency
    if (E4M3) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint8_t* at = kt + g * kRow + ((4 * j + t) ^ ((g & 1) << 2)) * 16;
        const uint4 w0 = *reinterpret_cast<const uint4*>(at);
        const uint4 w1 = *reinterpret_cast<const uint4*>(at + 8 * kRow);
        const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t a[4] = {
              e4m3x2_to_f16x2((uint16_t)x0[u]), e4m3x2_to_f16x2((uint16_t)x1[u]),
              e4m3x2_to_f16x2((uint16_t)(x0[u] >> 16)), e4m3x2_to_f16x2((uint16_t)(x1[u] >> 16))};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816_f16(u & 1 ? s2[nt] : s[nt], a, qb[nt][4 * j + u][0], qb[nt][4 * j + u][1]);
        }
      }
    } else {
      const int r = lane & 15;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        uint32_t a[4];
        ldmatrix_x4(a, smem_u32(kt + r * kRow + (((2 * kk + (lane >> 4)) ^ (r & 7)) << 4)));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma16816(kk & 1 ? s2[nt] : s[nt], a, qb[nt][kk][0], qb[nt][kk][1], kk & 1 ? s2[nt] : s[nt]);
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] += s2[nt][e];
    if (mask != 0xFFFFu) {
      const bool ok0 = (mask >> g) & 1u, ok1 = (mask >> (g + 8)) & 1u;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // the multipliers are positive
        if (!ok0) s[nt][0] = s[nt][1] = -INFINITY;
        if (!ok1) s[nt][2] = s[nt][3] = -INFINITY;
      }
    }
    float y[NT][4];
    bool grow = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y[nt][e] = fmaf(s[nt][e], ms[nt][e & 1], nref[nt][e & 1]);
        grow |= y[nt][e] > kGrow + kShift<E4M3>;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float m = fmaxf(s[nt][c], s[nt][2 + c]) * ms[nt][c];
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
          const float to = fminf(nref[nt][c], kShift<E4M3> - m);
          const float alpha = ex2(to - nref[nt][c]);
          nref[nt][c] = to;
          lsum[nt][c] *= alpha;
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            oacc[nt][d][c] *= alpha;
            oacc[nt][d][2 + c] *= alpha;
          }
          y[nt][c] = fmaf(s[nt][c], ms[nt][c], to);
          y[nt][2 + c] = fmaf(s[nt][2 + c], ms[nt][c], to);
        }
    }
    uint32_t pb[NT][2], pl[NT][2];  // P; beside bf16 rows the remainder of its rounding too
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float pr[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) pr[e] = ex2(y[nt][e]);
      lsum[nt][0] += pr[0] + pr[2];
      lsum[nt][1] += pr[1] + pr[3];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float p0 = pr[2 * c], p1 = pr[2 * c + 1];
        if (E4M3) {
          pb[nt][c] = transpose8x8(pack_f16x2(p0, p1));
        } else {
          const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
          const float r0 = p0 - __uint_as_float(u0 & 0xFFFF0000u);
          const float r1 = p1 - __uint_as_float(u1 & 0xFFFF0000u);
          pb[nt][c] = transpose8x8(__byte_perm(u0, u1, 0x7632));
          pl[nt][c] = transpose8x8(pack_bf16x2(fmaxf(r0, p0 * 0x1p-20f), fmaxf(r1, p1 * 0x1p-20f)));
        }
      }
    }
    if (E4M3) {
      // the thread's keys 2t, 2t+1, 2t+8, 2t+9, dimensions 16 g .. 16 g + 15:
      // product d takes dimensions 16 n + 2 d (its row n) and 16 n + 2 d + 1 (n + 8)
      uint4 w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        w[u] = *reinterpret_cast<const uint4*>(vt + (2 * t + (u & 1) + 8 * (u >> 1)) * kRow +
                                               ((g ^ (t << 1)) << 4));
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          x[u] = c == 0 ? w[u].x : c == 1 ? w[u].y : c == 2 ? w[u].z : w[u].w;
#pragma unroll
        for (int hlf = 0; hlf < 2; ++hlf) {
          const uint32_t sel = hlf ? 0x7362u : 0x5140u;
          const uint32_t lo = __byte_perm(x[0], x[1], sel), hi = __byte_perm(x[2], x[3], sel);
          const uint32_t a[4] = {
              e4m3x2_to_f16x2((uint16_t)lo), e4m3x2_to_f16x2((uint16_t)(lo >> 16)),
              e4m3x2_to_f16x2((uint16_t)hi), e4m3x2_to_f16x2((uint16_t)(hi >> 16))};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816_f16(oacc[nt][2 * c + hlf], a, pb[nt][0], pb[nt][1]);
        }
      }
    } else {
      const int r = (lane & 7) + 8 * (lane >> 4);  // matrices: keys lo, dims lo | dims hi; keys hi ...
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        uint32_t a[4];
        ldmatrix_x4_trans(
            a, smem_u32(vt + r * kRow + (((2 * d + ((lane >> 3) & 1)) ^ (r & 7)) << 4)));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816(oacc[nt][d], a, pb[nt][0], pb[nt][1], oacc[nt][d]);
          mma16816(oacc[nt][d], a, pl[nt][0], pl[nt][1], oacc[nt][d]);
        }
      }
    }
  }
  cp_async_wait<0>();
  __syncwarp();

  // ---- join the four warps; each leaves its rows in its own (now idle) stages
  float* wo = reinterpret_cast<float*>(kst);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float l = lsum[nt][c];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      const int r = nt * 8 + 2 * t + c;
      if (r < p.G) {
        if (g == 0) {
          sm.wm[warp][r] = nref[nt][c] == -kNoRef ? -INFINITY : kShift<E4M3> - nref[nt][c];
          sm.wl[warp][r] = l;
        }
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          if (E4M3) {
            *reinterpret_cast<float2*>(wo + out_at<true>(r, 16 * g + 2 * d)) =
                make_float2(oacc[nt][d][c], oacc[nt][d][2 + c]);
          } else {
            wo[out_at<false>(r, 16 * d + g)] = oacc[nt][d][c];
            wo[out_at<false>(r, 16 * d + g + 8)] = oacc[nt][d][2 + c];
          }
        }
      }
    }
  __syncthreads();
}

// A finished run's result for one query head and dimension: the warps' joined.
template <bool E4M3, int WARPS>
__device__ __forceinline__ void join_warps(const AttnSmem<E4M3, WARPS>& sm, int r, int d, float& M,
                                           float& l, float& o) {
  M = -INFINITY;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sm.wm[w][r]);
  o = l = 0.f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    // a warp that saw no key has l = 0 and o = 0; a NaN score leaves NaN in l and o
    const float f = ex2(sm.wm[w][r] - (M == -INFINITY ? 0.f : M) - kShift<E4M3>);
    const float fw = sm.wm[w][r] == -INFINITY && sm.wl[w][r] == sm.wl[w][r] ? 0.f : f;
    o += fw * reinterpret_cast<const float*>(&sm.w[w].k[0][0][0])[out_at<E4M3>(r, d)];
    l += fw * sm.wl[w][r];
  }
}

template <bool E4M3, bool SEL, int NT>
__global__ void __launch_bounds__(kAttnThreads, WarpStages<E4M3>::kCtasPerSm)
    paged_attn_kernel(const PagedAttnParams p) {
  griddep_wait();
  extern __shared__ __align__(128) unsigned char smem_raw[];
  AttnSmem<E4M3, kAttnWarps>& sm = *reinterpret_cast<AttnSmem<E4M3, kAttnWarps>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ---- this CTA's share of the line
  auto scan = [&](int64_t v, int64_t& all) {  // exclusive over the CTA
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sm.sums[warp] = x;
    __syncthreads();
    int64_t before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
      if (w < warp) before += sm.sums[w];
      all += sm.sums[w];
    }
    return before + x - v;
  };
  int64_t W = 0, mine = 0, before = 0;  // the first 128 requests' sums stay in registers
  for (int b0 = 0; b0 < p.B; b0 += kAttnThreads) {
    int64_t all;
    const int64_t n = b0 + tid < p.B ? request_cost<SEL>(p, b0 + tid) : 0;
    const int64_t at = scan(n, all);
    if (b0 == 0) {
      mine = n;
      before = at;
    }
    W += all;
  }
  const int64_t chunk = max((int64_t)kMinChunk, (W + gridDim.x - 1) / gridDim.x);
  if (tid == 0) p.split[blockIdx.x].row = -1;
  int64_t pos = (int64_t)blockIdx.x * chunk;
  const int64_t end = min(W, pos + chunk);
  if (pos >= end) return;
  for (int64_t b0 = 0, run = 0; b0 < p.B && run <= pos; b0 += kAttnThreads) {
    const int b = (int)b0 + tid;
    int64_t n = mine, at = before, all = 0;
    if (p.B > kAttnThreads) {
      n = b < p.B ? request_cost<SEL>(p, b) : 0;
      at = run + scan(n, all);
    }
    if (at <= pos && pos < at + n) {
      sm.req = b;
      sm.first = at;
    }
    run += all;
  }
  __syncthreads();
  int b = sm.req, i = 0;
  int len = paged_len(p, b);
  int64_t row0 = sm.first;  // where row (b, i) starts on the line
  const int64_t start = pos;

  while (pos < end) {
    // ---- the row at `pos`
    int groups = row_groups<SEL>(p, b, i, len);
    while (row0 + cost_of(groups) <= pos) {
      row0 += cost_of(groups);
      if (++i == p.Hkv) {
        i = 0;
        len = paged_len(p, ++b);
      }
      groups = row_groups<SEL>(p, b, i, len);
    }
    const int head = p.head[i];
    const int tiles = tiles_of(groups);
    const int64_t tile0 = row0 + kRowCost;  // its first tile
    const int t0 = (int)max((int64_t)0, pos - tile0);
    const int t1 = (int)max((int64_t)0, min((int64_t)tiles, end - tile0));
    pos = min(end, tile0 + tiles);
    if (t1 <= t0) continue;  // only the row's own cost
    if (t0 == 0 && t1 < tiles && tid == 0)
      p.split[blockIdx.x] = {tile0, chunk, b * p.Hkv + i, tiles, {0, 0}};

    attend_run<E4M3, SEL, NT, kAttnWarps>(p, sm, b, i, len, groups, t0, t1 - t0);
    const bool whole = t0 == 0 && t1 == tiles;
    float* part =
        p.part + ((int64_t)blockIdx.x * 2 + (tile0 + t0 == start ? 0 : 1)) * p.G * kPartRow;
#pragma unroll 4
    for (int r = 0; r < p.G; ++r) {
      float M, l, o;
      join_warps(sm, r, tid, M, l, o);
      if (whole) {
        store_final(p, b, head, r, tid, M, l, o);
      } else {
        part[r * kPartRow + 4 + tid] = o;
        if (tid == 0) {
          part[r * kPartRow] = M;
          part[r * kPartRow + 1] = l;
        }
      }
    }
    __syncthreads();
  }
}

// The same for short rows, without a second kernel: a cluster of up to 16 CTAs
// takes a row, each an equal run of its tiles, and joins them through distributed
// shared memory in rank order.
//
// MAXC: 8, or 16 (a larger loop over the CTAs' parts, which costs every size).
template <bool E4M3, bool SEL, int NT, int MAXC, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, WARPS > kAttnWarps ? 1 : WarpStages<E4M3>::kCtasPerSm)
    paged_attn_short_kernel(const PagedAttnParams p, const int csize) {
  griddep_wait();
  namespace cg = cooperative_groups;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  AttnSmem<E4M3, WARPS>& sm = *reinterpret_cast<AttnSmem<E4M3, WARPS>*>(smem_raw);
  __shared__ __align__(16) float part[16][kPartRow];  // m, l, pad, o of this CTA's run
  const cg::cluster_group cluster = cg::this_cluster();
  const int row = blockIdx.x / csize, rank = blockIdx.x % csize;
  const int b = row / p.Hkv, i = row % p.Hkv;
  // every 128 threads have the dimensions of one query head
  constexpr int kParts = WARPS / 4;
  const int part_of = threadIdx.x >> 7, tid = threadIdx.x & 127;
  const int len = paged_len(p, b), groups = row_groups<SEL>(p, b, i, len);
  const int tiles = (groups + WARPS - 1) / WARPS;
  const int t0 = (int)((int64_t)tiles * rank / csize);
  attend_run<E4M3, SEL, NT, WARPS>(p, sm, b, i, len, groups, t0,
                                   (int)((int64_t)tiles * (rank + 1) / csize) - t0);
#pragma unroll 4
  for (int r = part_of; r < p.G; r += kParts) {
    float M, l, o;
    join_warps(sm, r, tid, M, l, o);
    if (csize == 1) {
      store_final(p, b, p.head[i], r, tid, M, l, o);
      continue;
    }
    part[r][4 + tid] = o;
    if (tid == 0) {
      part[r][0] = M;
      part[r][1] = l;
    }
  }
  if (csize == 1) return;
  cluster.sync();
  for (int r = rank + part_of * csize; r < p.G; r += csize * kParts) {
    float m[MAXC], l[MAXC], o[MAXC], M = -INFINITY;
#pragma unroll
    for (int c = 0; c < MAXC; ++c) {
      if (c >= csize) continue;
      const float* x = cluster.map_shared_rank(&part[r][0], c);
      m[c] = x[0];
      l[c] = x[1];
      o[c] = x[4 + tid];
      M = fmaxf(M, m[c]);
    }
    const float m0 = M == -INFINITY ? 0.f : M;
    float ls = 0.f, os = 0.f;
#pragma unroll
    for (int c = 0; c < MAXC; ++c) {
      if (c >= csize) continue;
      const float f = m[c] == -INFINITY && l[c] == l[c] ? 0.f : ex2(m[c] - m0);
      ls += f * l[c];
      os += f * o[c];
    }
    store_final(p, b, p.head[i], r, tid, M, ls, os);
  }
  cluster.sync();  // no CTA leaves while another reads its part
}

// Joins the partials of the rows that several CTAs share, in CTA order; rows without
// keys get zeros (lse -inf).  A CTA for query head blockIdx.y of
//  - ROWS: row blockIdx.x, whose first CTA it looks for (few rows: as many warps as
//    there are partials for);
//  - else, x < ctas: the row that starts in CTA x's share and goes on, if there is
//    one; the CTAs behind look through 128 rows each for those without keys.
// Each warp sums an equal part of the partials, lane i dimensions 4 i .. 4 i + 3.
template <bool SEL, bool ROWS>
__global__ void __launch_bounds__(ROWS ? 512 : 128) paged_join_kernel(const PagedAttnParams p,
                                                                      const int ctas) {
  griddep_wait();
  constexpr int kThreads = ROWS ? 512 : 128, kWarps = kThreads / 32;
  const int r = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][kD];
  __shared__ int found;
  int64_t c0 = blockIdx.x;
  if (ROWS) {
    const int row = blockIdx.x, b = row / p.Hkv, i = row % p.Hkv;
    if (tid == 0) found = -1;
    __syncthreads();
    for (int c = tid; c < ctas; c += kThreads)
      if (p.split[c].row == row) found = c;
    const bool none = row_groups<SEL>(p, b, i, paged_len(p, b)) == 0;
    if (none && tid < kD) store_final(p, b, p.head[i], r, tid, -INFINITY, 0.f, 0.f);
    __syncthreads();
    c0 = found;
    if (c0 < 0) return;  // no keys, or one CTA wrote it
  } else if (blockIdx.x >= ctas) {
    const int row0 = ((int)blockIdx.x - ctas) * 128, mine = row0 + tid;
    const bool none = mine < p.B * p.Hkv &&
                      row_groups<SEL>(p, mine / p.Hkv, mine % p.Hkv, paged_len(p, mine / p.Hkv)) == 0;
    if (!__syncthreads_or(none)) return;
    uint32_t* set = reinterpret_cast<uint32_t*>(sm_m);  // 128 bits
    const uint32_t m = __ballot_sync(0xffffffffu, none);
    if (lane == 0) set[warp] = m;
    __syncthreads();
    for (int k = 0; k < 128; ++k)
      if ((set[k >> 5] >> (k & 31)) & 1u)
        store_final(p, (row0 + k) / p.Hkv, p.head[(row0 + k) % p.Hkv], r, tid, -INFINITY, 0.f, 0.f);
    return;
  }
  const SplitRow sp = p.split[c0];
  if (sp.row < 0) return;
  const int b = sp.row / p.Hkv, i = sp.row % p.Hkv;
  const int n = (int)((sp.first + sp.tiles - 1) / sp.chunk - c0 + 1);
  // the first CTA's part is its second one unless the row's tiles start its share
  const int64_t stride = (int64_t)p.G * kPartRow;
  auto at = [&](int s) {
    return p.part + ((c0 + s) * 2 + (s == 0 && sp.first != c0 * sp.chunk ? 1 : 0)) * stride +
           r * kPartRow;
  };
  float M = -INFINITY;
  for (int s = tid; s < n; s += kThreads) M = fmaxf(M, __ldcg(at(s)));
  M = warp_max(M);
  if (lane == 0) sm_m[warp] = M;
  __syncthreads();
  M = warp_max(sm_m[lane % kWarps]);
  const float m0 = M == -INFINITY ? 0.f : M;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  const int s0 = (int)((int64_t)n * warp / kWarps), s1 = (int)((int64_t)n * (warp + 1) / kWarps);
#pragma unroll 8
  for (int s = s0; s < s1; ++s) {
    const float* x = at(s);
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(x));
    const float4 v = __ldcg(reinterpret_cast<const float4*>(x + 4 + 4 * lane));
    const float f = ml.x == -INFINITY && ml.y == ml.y ? 0.f : exp2f(ml.x - m0);
    l += f * ml.y;
    acc.x += f * v.x;
    acc.y += f * v.y;
    acc.z += f * v.z;
    acc.w += f * v.w;
  }
  reinterpret_cast<float4*>(sm_o[warp])[lane] = acc;
  if (lane == 0) sm_l[warp] = l;
  __syncthreads();
  if (tid >= kD) return;
  float o = 0.f;
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    o += sm_o[w][tid];
    l += sm_l[w];
  }
  store_final(p, b, p.head[i], r, tid, M, l, o);
}

constexpr int kSms = 148;
constexpr int kMaxAttnCtas = 3 * kSms;

// CTAs of a row's cluster (as many as fit on the GPU at once), 0 for the split over
// all CTAs.  max_tiles: the longest row's, as far as the host can tell, which is what the
// block table can hold; the times below are of tables as wide as their longest request
// (one request of 517 tokens 5.5 us, in a table of 2048 pages of 16, which is split over
// all CTAs, 9.8; 24 requests up to 2000 15.9 in either).
//  - Clusters need their CTAs within one of the GPU's eight groups of SMs: 128 SMs'
//    worth of clusters run at once (36 clusters of 8 at two CTAs an SM take two waves,
//    12.0 against 7.4 us).
//  - Up to 16 tiles (1024 keys) a CTA a cluster saves the second kernel and the search
//    for the run's row: 32 rows of 2000 keys 10.1 us against 12.0 (bf16).  Beyond, one
//    long request among short ones would leave most CTAs idle: with 8 of 32 rows longer
//    than the others (131072 keys against 4100) 133 us against 94.  8-bit tiles have
//    half the bytes: there 32 a CTA, where the clusters fill half the GPU or more (64
//    ragged rows up to 6000 keys: 18.9 against 29.8 us).
//  - A few tiles are one CTA's (100 keys: 4.0 us, a cluster 5.1).
//  - Rows that fill the GPU need no cluster: a CTA each, the next one starting where one
//    ends, as long as the rows are not so long against their number that the last ones
//    decide (800 rows of up to 500 keys 27.5 us against 44.2, of 4000 239 against 256,
//    but 400 rows of 1 to 8000 keys 144 against 139).
//  - Sixteen, with an SM for each CTA, suit the longer of few rows (4 rows: 4000 keys 8.5
//    us, 9.0 with eight; 16000 keys 11.4, 16.0 over all CTAs), but start more slowly.
inline int short_cluster(int64_t rows, int max_tiles, int per_sm, bool e4m3) {
  if (rows * 16 <= kSms && max_tiles > 64) return max_tiles <= 256 ? 16 : 0;
  const int slots = per_sm * 128;
  int c = max_tiles <= 4 ? 1 : 8;
  while (c > 1 && rows * c > slots) c >>= 1;
  if (c == 1 && max_tiles * (int64_t)(per_sm * kSms) <= rows * (e4m3 ? 64 : 48)) return 1;
  const int most = e4m3 && rows * c * 2 >= slots ? 32 : 16;
  return rows * c <= per_sm * kSms && max_tiles <= most * c ? c : 0;
}

template <bool E4M3, bool SEL, int NT, int MAXC, int WARPS>
rtp_status launch_short(const PagedAttnParams& p, int c, cudaStream_t s) {
  const size_t smem = sizeof(AttnSmem<E4M3, WARPS>);
  auto* kernel = paged_attn_short_kernel<E4M3, SEL, NT, MAXC, WARPS>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
          cudaSuccess ||
      (MAXC > 8 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                        1) != cudaSuccess))
    return RTP_ERR_CUDA;
  TraceScope tr("paged_attn", s);
  return check_cuda(launch_dependent_cluster(kernel, dim3(p.B * p.Hkv * c), dim3(WARPS * 32), c,
                                             smem, s, p, c));
}

template <bool E4M3, bool SEL, int NT>
rtp_status launch(const PagedAttnParams& p, int max_tiles, cudaStream_t s) {
  const size_t smem = sizeof(AttnSmem<E4M3, kAttnWarps>);
  constexpr int per_sm = WarpStages<E4M3>::kCtasPerSm, ctas = per_sm * kSms;
  static_assert(ctas <= kMaxAttnCtas, "the workspace holds every CTA's partials");
  const int64_t rows = (int64_t)p.B * p.Hkv;
  const int c = short_cluster(rows, max_tiles, per_sm, E4M3);
  if (c > 0) {
    // the longer of very few rows: eight warps a CTA hide more of a group's latency (4 rows
    // of 16000 keys 11.6 us against 13.3)
    if (c > 8)
      return rows * c <= 64 ? launch_short<E4M3, SEL, NT, 16, 8>(p, c, s)
                            : launch_short<E4M3, SEL, NT, 16, 4>(p, c, s);
    return launch_short<E4M3, SEL, NT, 8, 4>(p, c, s);
  }
  auto* kernel = paged_attn_kernel<E4M3, SEL, NT>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
      cudaSuccess)
    return RTP_ERR_CUDA;
  rtp_status st;
  {
    TraceScope tr("paged_attn", s);
    if ((st = check_cuda(launch_dependent(kernel, dim3(ctas), dim3(kAttnThreads), smem, s, p))) !=
        RTP_OK)
      return st;
  }
  TraceScope tr("paged_join", s);
  if (rows <= ctas / 4)
    return check_cuda(launch_dependent(paged_join_kernel<SEL, true>, dim3((unsigned)rows, p.G),
                                       dim3(512), 0, s, p, ctas));
  return check_cuda(launch_dependent(paged_join_kernel<SEL, false>,
                                     dim3((unsigned)(ctas + (rows + 127) / 128), p.G), dim3(128), 0,
                                     s, p, ctas));
}

template <bool E4M3, bool SEL>
rtp_status launch(const PagedAttnParams& p, int max_tiles, cudaStream_t s) {
  return p.G <= 8 ? launch<E4M3, SEL, 1>(p, max_tiles, s) : launch<E4M3, SEL, 2>(p, max_tiles, s);
}

struct AttnWs {
  size_t split, part, total;
};
AttnWs attn_ws(int32_t G) {
  AttnWs w;
  w.split = kStatusBytes;
  w.part = align_up(w.split + (size_t)kMaxAttnCtas * sizeof(SplitRow), 256);
  w.total = align_up(w.part + (size_t)kMaxAttnCtas * 2 * G * kPartRow * 4, 256);
  return w;
}

}  // namespace

size_t paged_plan_ws(int32_t B);
size_t paged_select_ws(int64_t rows, int32_t width);

}  // namespace rtp

using namespace rtp;

extern "C" size_t rtp_paged_workspace_size(rtp_paged_op op, int32_t B, int32_t H, int32_t Hkv,
                                           const uint8_t* kv_role, int32_t table_width) {
  if (B < 0 || table_width < 0) return kStatusBytes;
  if (op == RTP_PAGED_PLAN) return paged_plan_ws(B);
  PagedHeads ph;
  if (make_paged_heads(H, Hkv, kv_role, &ph) != RTP_OK) return kStatusBytes;
  if (op == RTP_PAGED_SELECT) return paged_select_ws((int64_t)B * ph.n_rkv, table_width);
  if (op == RTP_PAGED_ATTN) return attn_ws(ph.G).total;
  return kStatusBytes;
}

extern "C" rtp_status rtp_paged_attn_decode(
    int32_t B, int32_t H, int32_t Hkv, const uint8_t* kv_role, int32_t window, int32_t n_sink,
    const void* q, int64_t q_stride, rtp_pages k_pages, rtp_pages v_pages, const float* k_scale,
    const float* v_scale, const int32_t* block_table, int64_t table_stride, int32_t table_width,
    const int32_t* seq_lens, const int32_t* sel, const int32_t* sel_count, int32_t n_sel,
    float softmax_scale, void* o, int64_t o_stride, float* lse, void* ws, size_t ws_bytes,
    rtp_stream_t stream) {
  PagedHeads ph;
  rtp_status st = make_paged_heads(H, Hkv, kv_role, &ph);
  if (st != RTP_OK) return st;
  if (B < 0 || table_width < 1 || table_stride < table_width) return RTP_ERR_INVALID_ARG;
  if (ph.n_rkv < Hkv && (window < 1 || n_sink < 0)) return RTP_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || !isfinite(softmax_scale)) return RTP_ERR_INVALID_ARG;
  if ((sel == nullptr) != (sel_count == nullptr) || (sel != nullptr && n_sel < 1))
    return RTP_ERR_INVALID_ARG;
  if ((st = check_cache(k_pages, v_pages, k_scale, v_scale)) != RTP_OK) return st;
  if ((int64_t)table_width * k_pages.page_size > kMaxTokens) return RTP_ERR_UNSUPPORTED;
  if (sel != nullptr && (int64_t)n_sel * k_pages.page_size > kMaxTokens) return RTP_ERR_UNSUPPORTED;
  if (B == 0) return RTP_OK;
  if ((int64_t)B * Hkv > INT32_MAX / 4) return RTP_ERR_UNSUPPORTED;
  if (q == nullptr || o == nullptr || block_table == nullptr || seq_lens == nullptr)
    return RTP_ERR_INVALID_ARG;
  if (q_stride < (int64_t)H * kD || o_stride < (int64_t)H * kD) return RTP_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || (q_stride * 2) % 16 || (o_stride * 2) % 16 ||
      !aligned16(ws))
    return RTP_ERR_ALIGNMENT;
  const AttnWs L = attn_ws(ph.G);
  if (ws == nullptr || ws_bytes < L.total) return RTP_ERR_WORKSPACE_TOO_SMALL;
  PagedAttnParams p;
  memset(&p, 0, sizeof(p));
  p.q = static_cast<const uint16_t*>(q);
  p.q_sb = q_stride;
  p.o = static_cast<uint16_t*>(o);
  p.o_sb = o_stride;
  p.lse = lse;
  p.kp = page_addr(k_pages);
  p.vp = page_addr(v_pages);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.table = block_table;
  p.table_stride = table_stride;
  p.seq_lens = seq_lens;
  p.sel = sel;
  p.sel_count = sel_count;
  p.split = reinterpret_cast<SplitRow*>(static_cast<char*>(ws) + L.split);
  p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + L.part);
  p.scale_log2 = softmax_scale * kLog2e;
  p.B = B;
  p.G = ph.G;
  p.Hkv = Hkv;
  p.n_rkv = ph.n_rkv;
  p.H = H;
  p.n_pages = k_pages.n_pages;
  p.width = table_width;
  p.ps_shift = log2_exact(k_pages.page_size);
  p.window = window;
  p.n_sink = n_sink;
  p.n_sel = n_sel;
  memcpy(p.head, ph.head, sizeof(p.head));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // the longest row's tiles, as far as the host can tell
  const int64_t most = (int64_t)table_width * k_pages.page_size;
  int64_t keys = 0;
  if (ph.n_rkv > 0) keys = sel ? (int64_t)n_sel * k_pages.page_size : most;
  if (ph.n_rkv < Hkv) keys = std::max(keys, std::min(most, (int64_t)window + n_sink + 3 * kGroup));
  const int max_tiles = (int)((keys + kAttnWarps * kGroup - 1) / (kAttnWarps * kGroup));
  if (k_pages.type == RTP_KV_E4M3)
    return sel ? launch<true, true>(p, max_tiles, s) : launch<true, false>(p, max_tiles, s);
  return sel ? launch<false, true>(p, max_tiles, s) : launch<false, false>(p, max_tiles, s);
}
