// asp_attend_flat.cu -- step 4 with equal shares of rows per CTA: attention over a cache
// held in 8 bits, and attention that also sums each token's weight (8-bit and bf16 caches).
//
// With x_gj = q_g . k_j log2(e) / sqrt(d) over the attended rows j of a unit (sequence, KV
// head):  m = ceil(max x), l = sum 2^(x - m), out = sum 2^(x - m) v_j / l; the weight sums
// are acc_j += sum_g 2^(x - m) / l.  Bound by HBM: each row's K and V are read once.
//
//  * The 16-row tiles of all units, by the lengths on the device, are cut into equal
//    contiguous ranges, one per CTA: ragged batches balance whatever their lengths.  A unit
//    shared by CTAs leaves a partial (m, l, M, unnormalised output) per CTA in the workspace
//    and finish_kernel joins them.  With few rows per unit a CTA takes a whole unit instead
//    and nothing is joined.
//  * A warp owns every 8th tile of its CTA's range and a ring of two stages: rows come in
//    by 16-byte cp.async, swizzled so that the fragment loads below meet no bank twice.
//  * S^T[head x row] = Q . K^T and O^T[channel x head] = V^T . P by mma.m16n8k16.  A pair of
//    codes becomes an fp16x2 operand register exactly; V's pairs run along the rows, taken
//    by a byte permute from two rows' words, so nothing is transposed through shared memory.
//    Heads fill 8 of the 16 rows of Q's fragments; for an fp32 query the other 8 hold the
//    second fp16 part.  The accumulator of S^T is already the operand P.
//  * K's scale multiplies the fp32 logits.  V's scale s = mant * 2^e multiplies the weight
//    before it is rounded to fp16: w = 2^(x + e - M + 14) mant with M = ceil(max(x + e)),
//    an integer like m, so rescaling is exact and no pair of scales leaves fp16's range.
//    A weight keeps 11 bits (a second fp16 part, 22, for an fp32 query) down to 2^-28 of
//    the largest.
#include "asp_internal.h"
#include "asp_kv8.cuh"

namespace asp {
namespace {

constexpr int kTile = 16;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 2;
constexpr int kWBias = 14;      // the largest weight is below 2^15 before its rounding to fp16
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kNone = 0xffffffffu;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct FlatParams {
  const void* q;
  int q_f32;
  int n_q_heads, G;
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  int block_shift, blocks_per_row;
  int units, n_kv, t_max, page_size, max_pages, n_pages;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* idx;
  const int32_t* count;
  int C;
  const int32_t* tail_begin;
  int max_tail;
  int whole;
  float* part_o;      // [2 ctas][G][d]
  float* part_ml;     // [2 ctas][G][4]: m, l, M
  int4* info;         // [units]: first CTA, last CTA, slot of the first
  float* stat;        // [units][G][2]: m, 1 / l of units one CTA holds (accumulate)
  float* logits;      // [units][G][row_stride] (accumulate)
  int row_stride;
  float* acc;
  void* out;
  int out_f32;
  float* lse;
  float qscale;       // log2(e) / sqrt(d)
};

struct UnitRows {
  int n_sel, tb, T, n_rows;
};

__device__ __forceinline__ UnitRows unit_rows(const FlatParams& p, int unit, bool flag) {
  UnitRows r;
  const int b = unit / p.n_kv;
  const int T = p.seq_lens ? __ldg(p.seq_lens + b) : p.t_max;
  r.T = T < 0 ? 0 : (T > p.t_max ? p.t_max : T);
  const int n = p.C > 0 ? __ldg(p.count + unit) : 0;
  r.n_sel = n < 0 ? 0 : (n > p.C ? p.C : n);
  r.tb = r.T;
  if (p.tail_begin) {
    const int tb = __ldg(p.tail_begin + b);
    r.tb = tb < 0 ? 0 : (tb > r.T ? r.T : tb);
  }
  int tail = r.T - r.tb;
  if (tail > p.max_tail) {
    if (flag) flag_status(ASP_DEV_TAIL_LIMIT);
    tail = p.max_tail;
  }
  r.n_rows = r.n_sel + tail;
  return r;
}
// A unit without rows keeps one (empty) tile, so that some CTA writes its output.
__device__ __forceinline__ int unit_tiles(const UnitRows& r) { return r.n_rows > 0 ? (r.n_rows + kTile - 1) / kTile : 1; }

__device__ __forceinline__ int range_start(int c, int total, int n) { return (int)((long long)c * total / n); }
__device__ __forceinline__ int range_owner(int i, int total, int n) { return (int)((((long long)i + 1) * n - 1) / total); }

// Operand formats.  kEB: bytes of a value.
template <typename CT>
struct Fmt {   // 8-bit codes, fp16 products
  static constexpr int kEB = 1;
  static constexpr bool kScaled = true;
  __device__ __forceinline__ static void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
  __device__ __forceinline__ static uint32_t pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ __forceinline__ static float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
};
template <>
struct Fmt<__nv_bfloat16> {
  static constexpr int kEB = 2;
  static constexpr bool kScaled = false;
  __device__ __forceinline__ static void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
  __device__ __forceinline__ static uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ __forceinline__ static float2 unpack(uint32_t w) { return bf16x2_to_float2(w); }
};

// Stage: K rows, V rows (swizzled 16-byte chunks), then K and V scales and the row mask.
template <typename CT, int D>
struct Stage {
  static constexpr int ROW = D * Fmt<CT>::kEB;      // bytes of a row
  static constexpr int CH = ROW / 16;               // its chunks
  static constexpr int HALF = kTile * ROW;
  static constexpr int SCALES = 2 * HALF;           // 16 + 16 floats
  static constexpr int MASK = SCALES + (Fmt<CT>::kScaled ? 2 * kTile * 4 : 0);
  static constexpr int BYTES = MASK + 16;
  // The fragment loads of a quarter (half) warp fall in distinct banks: K's touch rows g,
  // g + 1 at 4 chunks, V's the rows 2t at the chunks of two (four) lanes g.
  __device__ __forceinline__ static int k_swz(int r) { return CH >= 8 ? (r & 1) << 2 : 0; }
  __device__ __forceinline__ static int v_swz(int r) {
    if constexpr (CH == 16) return ((r >> 1) & 1) | (((r >> 2) & 1) << 2);
    else if constexpr (CH == 8) return ((r >> 1) & 3) << 1;
    else return ((r >> 1) & 1) << 1;
  }
};

constexpr int mo_stride(int D) { return D + 4; }
template <typename CT, int D>
constexpr size_t flat_smem(int G) {
  return (size_t)kWarps * kStages * Stage<CT, D>::BYTES + (size_t)kWarps * G * mo_stride(D) * 4 + (size_t)kWarps * G * 4 * 4;
}

// QP: parts of the query (8-bit caches: 1 for bf16, 2 for fp32; bf16 caches: 1 or 3).
template <typename CT, int D, int QP, bool ACC>
__global__ void __launch_bounds__(kThreads, sizeof(CT) == 1 ? 2 : 1) attend_flat_kernel(FlatParams p) {
  using F = Fmt<CT>;
  using S = Stage<CT, D>;
  constexpr int KS = D / 16;                 // k-steps of the logits
  constexpr int MT = D / 16;                 // m-tiles of the output
  constexpr bool WSPLIT = !F::kScaled || QP > 1;   // weights in two parts

  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int run_pre[kThreads + 1];
  __shared__ int scan[33];
  __shared__ int s_first[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int G = p.G;
  uint8_t* const ring = smem + (size_t)warp * kStages * S::BYTES;
  float* const mo = reinterpret_cast<float*>(smem + (size_t)kWarps * kStages * S::BYTES);   // [warp][G][D + 4]
  float* const mml = mo + (size_t)kWarps * G * mo_stride(D);                                // [warp][G][4]

  pdl_wait();

  // ---- this CTA's range of tiles
  int t0, t1, total, u0, tl0;
  int N = gridDim.x;
  const int cta = blockIdx.x;
  if (p.whole) {
    u0 = cta;
    tl0 = 0;
    t0 = 0;
    t1 = total = unit_tiles(unit_rows(p, u0, threadIdx.x == 0));
  } else {
    const int per = (p.units + kThreads - 1) / kThreads;   // units of a thread's run
    cta_prefix_sum(kThreads, run_pre, [&](int i) {
      int n = 0;
      for (int u = i * per; u < min(p.units, (i + 1) * per); ++u) n += unit_tiles(unit_rows(p, u, cta == 0));
      return n;
    }, scan);
    total = run_pre[kThreads];
    N = min(N, (total + kWarps - 1) / kWarps);   // a tile per warp, and no CTA without tiles
    if (cta >= N) return;
    t0 = range_start(cta, total, N);
    t1 = range_start(cta + 1, total, N);
    if (run_pre[threadIdx.x] <= t0 && t0 < run_pre[threadIdx.x + 1]) {
      int u = threadIdx.x * per, left = t0 - run_pre[threadIdx.x];
      for (;;) {
        const int n = unit_tiles(unit_rows(p, u, false));
        if (left < n) break;
        left -= n;
        ++u;
      }
      s_first[0] = u;
      s_first[1] = left;
    }
    __syncthreads();
    u0 = s_first[0];
    tl0 = s_first[1];
  }
  const int ntl = t1 - t0;
  const int my_n = ntl > warp ? (ntl - warp + kWarps - 1) / kWarps : 0;   // this warp's tiles

  // ---- producer side of the warp: its tiles in order, one position ahead of the copies
  int pu = u0, ptl = tl0 + warp;
  UnitRows pr = unit_rows(p, pu, false);
  int pn = unit_tiles(pr);
  int pj = 0;                // tiles whose index has been requested
  int raw = 0, r_unit = 0, r_tl = 0;
  UnitRows rr = pr;
  auto fetch = [&]() {       // position and raw index of the next tile
    if (pj >= my_n) return;
    while (ptl >= pn) {
      ptl -= pn;
      pr = unit_rows(p, ++pu, false);
      pn = unit_tiles(pr);
    }
    r_unit = pu;
    r_tl = ptl;
    rr = pr;
    const int r = ptl * kTile + (lane & 15);
    raw = r < pr.n_sel ? __ldg(p.idx + (size_t)pu * p.C + r) : 0;
    ptl += kWarps;
    ++pj;
  };
  int issued = 0;
  auto issue = [&]() {       // the fetched tile into the next stage (an empty group past the end)
    if (issued < my_n) {
      uint8_t* const st = ring + (issued % kStages) * S::BYTES;
      const int b = r_unit / p.n_kv, h = r_unit - b * p.n_kv;
      const int r = r_tl * kTile + (lane & 15);
      uint32_t row = kNone, srow = 0;
      int tok = -1;
      if (r < rr.n_sel) {
        tok = raw;
        if (tok < 0 || tok >= rr.T) {
          if (lane < 16) flag_status(ASP_DEV_BAD_INDEX);
          tok = -1;
        } else if (tok >= rr.tb) {
          tok = -1;   // covered by the tail
        }
      } else if (r < rr.n_rows) {
        tok = rr.tb + (r - rr.n_sel);
      }
      if (tok >= 0) {
        if (p.page_size == 0) {
          row = (uint32_t)((size_t)r_unit * p.t_max + tok);
          if (F::kScaled) srow = (uint32_t)((size_t)r_unit * p.blocks_per_row + (tok >> p.block_shift));
        } else {
          const int page = __ldg(p.page_table + (size_t)b * p.max_pages + tok / p.page_size);
          if (page < 0 || page >= p.n_pages) {
            if (lane < 16) flag_status(ASP_DEV_BAD_PAGE);
          } else {
            const int in = tok % p.page_size;
            row = (uint32_t)(((size_t)page * p.n_kv + h) * p.page_size + in);
            if (F::kScaled) srow = (uint32_t)(((size_t)page * p.n_kv + h) * p.blocks_per_row + (in >> p.block_shift));
          }
        }
      }
      const uint32_t vm = __ballot_sync(0xffffffffu, row != kNone) & 0xffffu;
      const uint32_t base = smem_u32(st);
      constexpr int RPI = 32 / S::CH;   // rows per warp instruction
      const int ch = lane % S::CH;
#pragma unroll
      for (int i = 0; i < 32 / RPI; ++i) {
        const int ri = RPI * i + lane / S::CH;     // 0-15 K rows, 16-31 V rows
        const uint32_t src = __shfl_sync(0xffffffffu, row, ri & 15);
        const bool ok = src != kNone;
        const int sw = ch ^ (ri < 16 ? S::k_swz(ri) : S::v_swz(ri & 15));
        const uint8_t* from = (ri < 16 ? p.k : p.v) + (ok ? (size_t)src * S::ROW + ch * 16 : 0);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(base + ri * S::ROW + sw * 16), "l"(from),
                     "r"(ok ? 16 : 0)
                     : "memory");
      }
      if constexpr (F::kScaled) {
        const float* from = (lane < 16 ? p.k_scale : p.v_scale) + (row != kNone ? srow : 0u);
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(base + S::SCALES + lane * 4), "l"(from),
                     "r"(row != kNone ? 4 : 0)
                     : "memory");
      }
      if (lane == 0) *reinterpret_cast<uint32_t*>(st + S::MASK) = vm;
      ++issued;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) {
    fetch();
    issue();
  }
  fetch();

  // ---- query fragments: row g is head g (part 0), row g + 8 its second part
  constexpr int QR = QP == 1 ? 2 : (QP == 2 ? 4 : 6);   // registers per k-step
  uint32_t qa[KS][QR];
  float qfac = p.qscale;     // of head g
  // channel of (k-step ks, element c): the order in which K's chunks arrive
  auto chan = [&](int ks, int c) -> int {
    if constexpr (F::kEB == 1) return (ks >> 2) * 64 + t * 16 + (ks & 3) * 4 + c;
    else return (ks >> 1) * 32 + t * 8 + (ks & 1) * 4 + c;
  };
  auto load_q = [&](int unit) {
    const int b = unit / p.n_kv, h = unit - b * p.n_kv;
    const size_t off = ((size_t)b * p.n_q_heads + h * G + g) * D;
    auto at = [&](int ch) -> float {
      if (g >= G) return 0.f;
      return p.q_f32 ? static_cast<const float*>(p.q)[off + ch]
                     : __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[off + ch]);
    };
    float up = 1.f;
    if constexpr (F::kScaled) {   // largest channel to [2^14, 2^15)
      uint32_t amax = 0u;
      bool bad = false;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int c = 0; c < 4; ++c) amax = max(amax, finite_abs(at(chan(ks, c)), bad));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      int e = (int)(amax >> 23) - 127;
      e = e < -112 ? -112 : e;
      up = exp2i(14 - e);
      qfac = exp2i(e - 14) * p.qscale;
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      float x[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = at(chan(ks, c)) * up;
#pragma unroll
      for (int part = 0; part < QP; ++part) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t w = F::pack(x[2 * c], x[2 * c + 1]);
          const float2 y = F::unpack(w);
          x[2 * c] -= y.x;
          x[2 * c + 1] -= y.y;
          qa[ks][2 * part + c] = w;
        }
      }
    }
  };
  load_q(u0);

  // ---- consumer side
  int j = 0;                 // this warp's next tile
  int seg_t0 = t0 - tl0;     // where the current unit's tiles begin in the flattened order
  for (int u = u0;; ++u) {
    const UnitRows ur = unit_rows(p, u, false);
    const int un = unit_tiles(ur);
    const int seg_end = min(t1, seg_t0 + un);
    const int kend = seg_end - t0 - warp;
    const int jend = kend > 0 ? (kend + kWarps - 1) / kWarps : 0;
    float o[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m = -INFINITY, M = -INFINITY, l = 0.f;   // of head g; l: this lane's share
#pragma unroll 1
    for (; j < jend; ++j) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();
      const uint8_t* const st = ring + (j % kStages) * S::BYTES;
      const uint32_t vm = *reinterpret_cast<const uint32_t*>(st + S::MASK);
      // logits: n-tile 0 = rows 0-7, n-tile 1 = rows 8-15
      float sc[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
        const int r = nt * 8 + g;
        const uint8_t* const krow = st + r * S::ROW;
        const int sw = S::k_swz(r);
#pragma unroll
        for (int i = 0; i < S::CH / 4; ++i) {
          const uint4 w4 = *reinterpret_cast<const uint4*>(krow + (((4 * i + t) ^ sw) * 16));
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
          if constexpr (F::kEB == 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int ks = 4 * i + e;
              const uint32_t x = CT::prep(w[e]);
              const uint32_t b0 = CT::pair(x, 0), b1 = CT::pair(x, 1);
              if constexpr (QP == 1) F::mma(sc[nt], qa[ks][0], 0u, qa[ks][1], 0u, b0, b1);
              else F::mma(sc[nt], qa[ks][0], qa[ks][2], qa[ks][1], qa[ks][3], b0, b1);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int ks = 2 * i + e;
              if constexpr (QP == 1) {
                F::mma(sc[nt], qa[ks][0], 0u, qa[ks][1], 0u, w[2 * e], w[2 * e + 1]);
              } else {
                F::mma(sc[nt], qa[ks][0], qa[ks][2], qa[ks][1], qa[ks][3], w[2 * e], w[2 * e + 1]);
                F::mma(sc[nt], qa[ks][4], 0u, qa[ks][5], 0u, w[2 * e], w[2 * e + 1]);
              }
            }
          }
        }
      }
      // softmax of head g over the lane's rows 2t, 2t+1, 8+2t, 9+2t
      float x[4] = {sc[0][0], sc[0][1], sc[1][0], sc[1][1]};
      if constexpr (QP > 1) {
        x[0] += sc[0][2];
        x[1] += sc[0][3];
        x[2] += sc[1][2];
        x[3] += sc[1][3];
      }
      int ve[4];
      float vmant[4];
      if constexpr (F::kScaled) {
        const float2* const ksc = reinterpret_cast<const float2*>(st + S::SCALES);
        const float2 k0 = ksc[t], k1 = ksc[4 + t], v0 = ksc[8 + t], v1 = ksc[12 + t];
        x[0] *= k0.x * qfac;
        x[1] *= k0.y * qfac;
        x[2] *= k1.x * qfac;
        x[3] *= k1.y * qfac;
        const float vs[4] = {v0.x, v0.y, v1.x, v1.y};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t bits = __float_as_uint(vs[e]);
          ve[e] = (int)(bits >> 23) - 127;
          vmant[e] = __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] *= qfac;
      }
      bool ok[4];
      float mx = -INFINITY, Mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ok[e] = (vm >> (2 * t + (e & 1) + (e >> 1) * 8)) & 1u;
        if (!ok[e]) x[e] = -INFINITY;
        mx = fmaxf(mx, x[e]);
        if constexpr (F::kScaled) Mx = fmaxf(Mx, x[e] + (float)ve[e]);
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if constexpr (F::kScaled) {
        Mx = fmaxf(Mx, __shfl_xor_sync(0xffffffffu, Mx, 1));
        Mx = fmaxf(Mx, __shfl_xor_sync(0xffffffffu, Mx, 2));
      }
      if constexpr (ACC) {
        if (g < G) {
          const int tl = t0 + warp + j * kWarps - seg_t0;   // tile of the unit
          float* const lg = p.logits + ((size_t)u * G + g) * p.row_stride + tl * kTile + 2 * t;
          *reinterpret_cast<float2*>(lg) = make_float2(x[0], x[1]);
          *reinterpret_cast<float2*>(lg + 8) = make_float2(x[2], x[3]);
        }
      }
      const float mn = fmaxf(m, ceilf(mx));
      const float lcorr = mn == -INFINITY ? 1.f : ex2(m - mn);
      float pr4[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) pr4[e] = ok[e] ? ex2(x[e] - mn) : 0.f;
      l = l * lcorr + ((pr4[0] + pr4[1]) + (pr4[2] + pr4[3]));
      m = mn;
      float w4[4], ocorr;
      if constexpr (F::kScaled) {
        const float Mn = fmaxf(M, ceilf(Mx));
        ocorr = Mn == -INFINITY ? 1.f : ex2(M - Mn);
        M = Mn;
#pragma unroll
        for (int e = 0; e < 4; ++e) w4[e] = ok[e] ? ex2(x[e] + ((float)(ve[e] + kWBias) - Mn)) * vmant[e] : 0.f;
      } else {
        ocorr = lcorr;
#pragma unroll
        for (int e = 0; e < 4; ++e) w4[e] = pr4[e];
      }
      if (__any_sync(0xffffffffu, ocorr != 1.f)) {
        const float c0 = __shfl_sync(0xffffffffu, ocorr, 8 * t), c1 = __shfl_sync(0xffffffffu, ocorr, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          o[i][0] *= c0;
          o[i][1] *= c1;
          o[i][2] *= c0;
          o[i][3] *= c1;
        }
      }
      const uint32_t b0 = F::pack(w4[0], w4[1]), b1 = F::pack(w4[2], w4[3]);
      uint32_t l0 = 0u, l1 = 0u;
      if constexpr (WSPLIT) {
        const float2 h0 = F::unpack(b0), h1 = F::unpack(b1);
        l0 = F::pack(w4[0] - h0.x, w4[1] - h0.y);
        l1 = F::pack(w4[2] - h1.x, w4[3] - h1.y);
      }
      // O^T += V^T . P: lane g holds a run of channels of the rows 2t, 2t+1, 8+2t, 9+2t
      const uint8_t* const vb = st + S::HALF;
      constexpr int CPG = D / 8;                       // channels per lane
      constexpr int WPR = CPG * F::kEB / 4;            // words of them per row
      uint32_t vw[4][WPR];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 2 * t + (e & 1) + (e >> 1) * 8;
        const uint8_t* const vrow = vb + r * S::ROW;
        const int sw = S::v_swz(r);
        if constexpr (WPR == 2) {
          const uint2 y = *reinterpret_cast<const uint2*>(vrow + (((g >> 1) ^ sw) * 16) + (g & 1) * 8);
          vw[e][0] = y.x;
          vw[e][1] = y.y;
        } else {
#pragma unroll
          for (int c = 0; c < WPR / 4; ++c) {
            const uint4 y = *reinterpret_cast<const uint4*>(vrow + (((WPR / 4 * g + c) ^ sw) * 16));
            vw[e][4 * c] = y.x;
            vw[e][4 * c + 1] = y.y;
            vw[e][4 * c + 2] = y.z;
            vw[e][4 * c + 3] = y.w;
          }
        }
      }
      auto pv = [&](int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
        F::mma(o[i], a0, a1, a2, a3, b0, b1);
        if constexpr (WSPLIT) F::mma(o[i], a0, a1, a2, a3, l0, l1);
      };
#pragma unroll
      for (int w = 0; w < WPR; ++w) {
        if constexpr (F::kEB == 1) {   // 4 channels: m-tiles 2w and 2w + 1
          const uint32_t e0 = CT::prep(__byte_perm(vw[0][w], vw[1][w], 0x5140));
          const uint32_t e1 = CT::prep(__byte_perm(vw[0][w], vw[1][w], 0x7362));
          const uint32_t f0 = CT::prep(__byte_perm(vw[2][w], vw[3][w], 0x5140));
          const uint32_t f1 = CT::prep(__byte_perm(vw[2][w], vw[3][w], 0x7362));
          pv(2 * w, CT::pair(e0, 0), CT::pair(e0, 1), CT::pair(f0, 0), CT::pair(f0, 1));
          pv(2 * w + 1, CT::pair(e1, 0), CT::pair(e1, 1), CT::pair(f1, 0), CT::pair(f1, 1));
        } else {                       // 2 channels: m-tile w
          pv(w, __byte_perm(vw[0][w], vw[1][w], 0x5410), __byte_perm(vw[0][w], vw[1][w], 0x7632),
             __byte_perm(vw[2][w], vw[3][w], 0x5410), __byte_perm(vw[2][w], vw[3][w], 0x7632));
        }
      }
      __syncwarp();
      issue();
      fetch();
    }
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if constexpr (!F::kScaled) M = m;

    // ---- the warps' results of this unit meet in shared memory; position 16 i + 2 g + e of
    // a head's row is channel (D / 8) g + 2 i + e
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (2 * t < G)
        *reinterpret_cast<float2*>(mo + ((size_t)warp * G + 2 * t) * mo_stride(D) + 16 * i + 2 * g) =
            make_float2(o[i][0], o[i][2]);
      if (2 * t + 1 < G)
        *reinterpret_cast<float2*>(mo + ((size_t)warp * G + 2 * t + 1) * mo_stride(D) + 16 * i + 2 * g) =
            make_float2(o[i][1], o[i][3]);
    }
    if (g < G && t == 0) {
      float* const ml = mml + (warp * G + g) * 4;
      ml[0] = m;
      ml[1] = l;
      ml[2] = M;
    }
    __syncthreads();
    const bool last = seg_end >= t1;
    if (!last) load_q(u + 1);
    const bool starts = seg_t0 >= t0, ends = seg_t0 + un <= t1;
    const bool alone = starts && ends;
    const int slot = 2 * cta + (u == u0 ? 0 : 1);
    if (!p.whole && starts && threadIdx.x == 0)
      p.info[u] = make_int4(cta, ends ? cta : range_owner(seg_t0 + un - 1, total, N), slot, 0);
    const int b = u / p.n_kv, h = u - b * p.n_kv;
    for (int e = threadIdx.x; e < G * D; e += kThreads) {
      const int gg = e / D, pos = e - gg * D;
      const int c = (D / 8) * ((pos & 15) >> 1) + 2 * (pos >> 4) + (pos & 1);
      float mm = -INFINITY, MM = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        mm = fmaxf(mm, mml[(w * G + gg) * 4]);
        MM = fmaxf(MM, mml[(w * G + gg) * 4 + 2]);
      }
      float L = 0.f, O = 0.f;
      if (mm != -INFINITY) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float* const ml = mml + (w * G + gg) * 4;
          if (ml[0] == -INFINITY) continue;
          L += ml[1] * ex2(ml[0] - mm);
          O += mo[((size_t)w * G + gg) * mo_stride(D) + pos] * ex2(ml[2] - MM);
        }
      }
      const size_t bh = (size_t)b * p.n_q_heads + h * G + gg;
      if (alone) {
        const float scale = F::kScaled ? ex2(MM - mm - (float)kWBias) : 1.f;
        const float y = mm == -INFINITY ? 0.f : O / L * scale;
        if (p.out_f32) static_cast<float*>(p.out)[bh * D + c] = y;
        else static_cast<__nv_bfloat16*>(p.out)[bh * D + c] = __float2bfloat16_rn(y);
        if (pos == 0) {
          if (p.lse) p.lse[bh] = mm == -INFINITY ? -INFINITY : mm * kLn2 + logf(L);
          if constexpr (ACC) {
            p.stat[((size_t)u * G + gg) * 2] = mm;
            p.stat[((size_t)u * G + gg) * 2 + 1] = mm == -INFINITY ? 0.f : 1.f / L;
          }
        }
      } else {
        p.part_o[((size_t)slot * G + gg) * D + c] = O;
        if (pos == 0) {
          float* const ml = p.part_ml + ((size_t)slot * G + gg) * 4;
          ml[0] = mm;
          ml[1] = L;
          ml[2] = MM;
        }
      }
    }
    if constexpr (ACC) {
      if (p.whole) {   // this CTA holds every logit of the unit: the weights right away
        __syncthreads();
        for (int r = threadIdx.x; r < ur.n_rows; r += kThreads) {
          float w = 0.f;
          bool any = false;
          for (int gg = 0; gg < G; ++gg) {
            const float xv = p.logits[((size_t)u * G + gg) * p.row_stride + r];
            if (xv == -INFINITY) continue;
            any = true;
            w += ex2(xv - p.stat[((size_t)u * G + gg) * 2]) * p.stat[((size_t)u * G + gg) * 2 + 1];
          }
          if (!any) continue;
          const int tok = r < ur.n_sel ? p.idx[(size_t)u * p.C + r] : ur.tb + (r - ur.n_sel);
          atomicAdd(p.acc + (size_t)u * p.t_max + tok, w);
        }
      }
    }
    if (last) break;
    __syncthreads();
    seg_t0 += un;
  }
}

// Joins the units that several CTAs share (one CTA per unit) and, for ACC, adds the weights
// of the unit's rows (blockIdx.y: chunks of kAccRows rows).
constexpr int kAccRows = 1024;

template <int D, bool ACC>
__global__ void __launch_bounds__(kThreads) finish_kernel(FlatParams p, float bias) {
  __shared__ float s_m[8], s_il[8];
  const int u = blockIdx.x, G = p.G;
  pdl_wait();
  const int4 in = p.info[u];
  const int n = in.y - in.x + 1;   // CTAs of the unit
  auto slot_of = [&](int i) -> int { return i == 0 ? in.z : 2 * (in.x + i); };
  const bool shared = n > 1;
  if (ACC && blockIdx.y * kAccRows >= p.row_stride) return;
  UnitRows ur;
  if constexpr (ACC) {
    ur = unit_rows(p, u, false);
    if (blockIdx.y > 0 && (int)blockIdx.y * kAccRows >= ur.n_rows) return;
  }
  if (shared && blockIdx.y == 0) {
    const int b = u / p.n_kv, h = u - b * p.n_kv;
    for (int e = threadIdx.x; e < G * D; e += kThreads) {
      const int gg = e / D, c = e - gg * D;
      float mm = -INFINITY, MM = -INFINITY;
      for (int i = 0; i < n; ++i) {
        const float* const ml = p.part_ml + ((size_t)slot_of(i) * G + gg) * 4;
        mm = fmaxf(mm, ml[0]);
        MM = fmaxf(MM, ml[2]);
      }
      float L = 0.f, O = 0.f;
      if (mm != -INFINITY) {
        for (int i = 0; i < n; ++i) {
          const float* const ml = p.part_ml + ((size_t)slot_of(i) * G + gg) * 4;
          if (ml[0] == -INFINITY) continue;
          L += ml[1] * ex2(ml[0] - mm);
          O += p.part_o[((size_t)slot_of(i) * G + gg) * D + c] * ex2(ml[2] - MM);
        }
      }
      const size_t bh = (size_t)b * p.n_q_heads + h * G + gg;
      const float y = mm == -INFINITY ? 0.f : O / L * ex2(MM - mm - bias);
      if (p.out_f32) static_cast<float*>(p.out)[bh * D + c] = y;
      else static_cast<__nv_bfloat16*>(p.out)[bh * D + c] = __float2bfloat16_rn(y);
      if (c == 0 && p.lse) p.lse[bh] = mm == -INFINITY ? -INFINITY : mm * kLn2 + logf(L);
    }
  }
  if constexpr (ACC) {
    if (threadIdx.x < G) {
      const int gg = threadIdx.x;
      float mm = -INFINITY, L = 0.f;
      if (shared) {
        for (int i = 0; i < n; ++i) mm = fmaxf(mm, p.part_ml[((size_t)slot_of(i) * G + gg) * 4]);
        if (mm != -INFINITY)
          for (int i = 0; i < n; ++i) {
            const float* const ml = p.part_ml + ((size_t)slot_of(i) * G + gg) * 4;
            if (ml[0] != -INFINITY) L += ml[1] * ex2(ml[0] - mm);
          }
        s_m[gg] = mm;
        s_il[gg] = mm == -INFINITY ? 0.f : 1.f / L;
      } else {
        s_m[gg] = p.stat[((size_t)u * G + gg) * 2];
        s_il[gg] = p.stat[((size_t)u * G + gg) * 2 + 1];
      }
    }
    __syncthreads();
    const int r1 = min(ur.n_rows, ((int)blockIdx.y + 1) * kAccRows);
    for (int r = blockIdx.y * kAccRows + threadIdx.x; r < r1; r += kThreads) {
      float w = 0.f;
      bool any = false;
      for (int gg = 0; gg < G; ++gg) {
        const float xv = p.logits[((size_t)u * G + gg) * p.row_stride + r];
        if (xv == -INFINITY) continue;   // a row that was not attended
        any = true;
        w += ex2(xv - s_m[gg]) * s_il[gg];
      }
      if (!any) continue;
      const int tok = r < ur.n_sel ? p.idx[(size_t)u * p.C + r] : ur.tb + (r - ur.n_sel);
      atomicAdd(p.acc + (size_t)u * p.t_max + tok, w);
    }
  }
}

// acc from the logits (base 2) of attend_kernel and the final lse.
__global__ void __launch_bounds__(kThreads) accumulate_kernel(FlatParams p) {
  __shared__ float s_l[8];
  const int u = blockIdx.x, G = p.G;
  const int b = u / p.n_kv, h = u - b * p.n_kv;
  pdl_wait();
  const UnitRows ur = unit_rows(p, u, false);
  if ((int)blockIdx.y * kAccRows >= ur.n_rows) return;
  if (threadIdx.x < G) s_l[threadIdx.x] = p.lse[(size_t)b * p.n_q_heads + h * G + threadIdx.x];
  __syncthreads();
  const int r1 = min(ur.n_rows, ((int)blockIdx.y + 1) * kAccRows);
  for (int r = blockIdx.y * kAccRows + threadIdx.x; r < r1; r += kThreads) {
    float w = 0.f;
    bool any = false;
    for (int gg = 0; gg < G; ++gg) {
      const float xv = p.logits[((size_t)u * G + gg) * p.row_stride + r];
      if (xv == -INFINITY) continue;
      any = true;
      w += expf(xv * kLn2 - s_l[gg]);
    }
    if (!any) continue;
    const int tok = r < ur.n_sel ? p.idx[(size_t)u * p.C + r] : ur.tb + (r - ur.n_sel);
    atomicAdd(p.acc + (size_t)u * p.t_max + tok, w);
  }
}

template <typename CT, int D, int QP, bool ACC>
cudaError_t launch_flat_t(const FlatParams& p, int ctas, int chunks, cudaStream_t s) {
  auto kern = attend_flat_kernel<CT, D, QP, ACC>;
  const size_t smem = flat_smem<CT, D>(p.G);
  if (prepare_kernel((const void*)kern, smem, kThreads) < 1) return cudaErrorInvalidConfiguration;
  cudaError_t e = launch_pdl(kern, dim3(ctas), dim3(kThreads), smem, s, p);
  if (e != cudaSuccess || p.whole) return e;
  return launch_pdl(finish_kernel<D, ACC>, dim3(p.units, ACC ? chunks : 1), dim3(kThreads), 0, s, p,
                    Fmt<CT>::kScaled ? (float)kWBias : 0.f);
}

template <typename CT, int QP, bool ACC>
cudaError_t launch_flat_d(const FlatParams& p, int D, int ctas, int chunks, cudaStream_t s) {
  return D == 64 ? launch_flat_t<CT, 64, QP, ACC>(p, ctas, chunks, s) : launch_flat_t<CT, 128, QP, ACC>(p, ctas, chunks, s);
}

template <typename CT>
cudaError_t launch_flat_8(const FlatParams& p, int D, int ctas, int chunks, cudaStream_t s) {
  if (p.logits)
    return p.q_f32 ? launch_flat_d<CT, 2, true>(p, D, ctas, chunks, s) : launch_flat_d<CT, 1, true>(p, D, ctas, chunks, s);
  return p.q_f32 ? launch_flat_d<CT, 2, false>(p, D, ctas, chunks, s) : launch_flat_d<CT, 1, false>(p, D, ctas, chunks, s);
}

FlatParams flat_params(const void* q, int q_f32, int n_q_heads, const KvView& kv, const int32_t* idx,
                       const int32_t* count, int C, const int32_t* tail_begin, int max_tail) {
  FlatParams p = {};
  p.q = q;
  p.q_f32 = q_f32;
  p.n_q_heads = n_q_heads;
  p.G = n_q_heads / kv.n_kv;
  p.k = static_cast<const uint8_t*>(kv.k);
  p.v = static_cast<const uint8_t*>(kv.v);
  p.k_scale = kv.k_scale;
  p.v_scale = kv.v_scale;
  p.block_shift = kv.block_shift;
  p.blocks_per_row = kv.blocks_per_row;
  p.units = kv.batch * kv.n_kv;
  p.n_kv = kv.n_kv;
  p.t_max = kv.t_max;
  p.page_size = kv.page_size;
  p.max_pages = kv.max_pages;
  p.n_pages = kv.n_pages;
  p.page_table = kv.page_table;
  p.seq_lens = kv.seq_lens;
  p.idx = idx;
  p.count = count;
  p.C = C;
  p.tail_begin = tail_begin;
  p.max_tail = tail_begin ? max_tail : 0;
  p.qscale = kLog2e / sqrtf((float)kv.head_dim);
  return p;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

// A unit of at most kWholeRows rows stays whole: joining costs a second launch.
constexpr int kWholeRows = 256;
constexpr int kFlatSms = 148;

FlatPlan flat_plan(int batch, int n_q_heads, int n_kv_heads, int head_dim, int C, int max_tail, bool kv8,
                   bool accumulate, int ctas_per_sm) {
  FlatPlan pl = {};
  const long rows = (long)C + (max_tail > 0 ? max_tail : 0);
  const long units = (long)batch * n_kv_heads;
  const int G = n_q_heads / n_kv_heads;
  const long tiles = units * ((rows + kTile - 1) / kTile);
  long ctas = (tiles + kWarps - 1) / kWarps;
  const long most = (long)kFlatSms * (ctas_per_sm > 0 ? ctas_per_sm : (kv8 ? 2 : 1));
  pl.whole = rows <= kWholeRows ? 1 : 0;
  pl.ctas = (int)(pl.whole ? units : (ctas < most ? (ctas < 1 ? 1 : ctas) : most));
  pl.row_stride = accumulate ? (int)((rows + kTile - 1) / kTile * kTile) : 0;
  size_t at = 0;
  pl.part_off = at;
  if (!pl.whole) at += round256((size_t)2 * pl.ctas * G * head_dim * 4) + round256((size_t)2 * pl.ctas * G * 16);
  pl.info_off = at;
  if (!pl.whole) at += round256((size_t)units * 16);
  pl.logits_off = at;
  if (accumulate) at += round256((size_t)units * G * 8) + round256((size_t)units * G * pl.row_stride * 4);
  pl.workspace_bytes = at;
  return pl;
}

cudaError_t launch_attend_flat(const void* q, int q_f32, int n_q_heads, const KvView& kv, const int32_t* idx,
                               const int32_t* count, int C, const int32_t* tail_begin, int max_tail, void* out,
                               float* lse, float* acc, void* workspace, const FlatPlan& pl, cudaStream_t s) {
  FlatParams p = flat_params(q, q_f32, n_q_heads, kv, idx, count, C, tail_begin, max_tail);
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  p.whole = pl.whole;
  if (!pl.whole) {
    p.part_o = reinterpret_cast<float*>(ws + pl.part_off);
    p.part_ml = reinterpret_cast<float*>(ws + pl.part_off + round256((size_t)2 * pl.ctas * p.G * kv.head_dim * 4));
    p.info = reinterpret_cast<int4*>(ws + pl.info_off);
  }
  if (acc) {
    p.stat = reinterpret_cast<float*>(ws + pl.logits_off);
    p.logits = reinterpret_cast<float*>(ws + pl.logits_off + round256((size_t)p.units * p.G * 8));
    p.row_stride = pl.row_stride;
    p.acc = acc;
  }
  p.out = out;
  p.out_f32 = kv.kv8 ? q_f32 : 0;
  p.lse = lse;
  const int chunks = pl.row_stride > 0 ? (pl.row_stride + kAccRows - 1) / kAccRows : 1;
  if (kv.kv8 == 1) return launch_flat_8<CodeE4M3>(p, kv.head_dim, pl.ctas, chunks, s);
  if (kv.kv8 == 2) return launch_flat_8<CodeI8>(p, kv.head_dim, pl.ctas, chunks, s);
  return q_f32 ? launch_flat_d<__nv_bfloat16, 3, true>(p, kv.head_dim, pl.ctas, chunks, s)
               : launch_flat_d<__nv_bfloat16, 1, true>(p, kv.head_dim, pl.ctas, chunks, s);
}

cudaError_t launch_accumulate(const float* logits, int row_stride, const float* lse, int n_q_heads, const KvView& kv,
                              const int32_t* idx, const int32_t* count, int C, const int32_t* tail_begin, int max_tail,
                              float* acc, cudaStream_t s) {
  FlatParams p = flat_params(nullptr, 1, n_q_heads, kv, idx, count, C, tail_begin, max_tail);
  p.logits = const_cast<float*>(logits);
  p.row_stride = row_stride;
  p.lse = const_cast<float*>(lse);
  p.acc = acc;
  return launch_pdl(accumulate_kernel, dim3(p.units, (row_stride + kAccRows - 1) / kAccRows), dim3(kThreads), 0, s, p);
}

ASP_STATUS_READER(read_status_attend_flat)

}  // namespace asp
