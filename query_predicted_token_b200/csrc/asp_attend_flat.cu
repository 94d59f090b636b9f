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
//  * A warp owns every W-th tile of its CTA's range and a ring of two stages, and fetches for
//    itself in three steps that each have a whole tile's work to arrive in: the raw indices,
//    then the pages, then the rows by 16-byte cp.async, swizzled so that the fragment loads
//    below meet no bank twice.  (Three producer warps for twelve consumers took 196 us where
//    this takes about 100: a tile's fetch is a quarter of its instructions, and three warps
//    issue them too slowly.)
//  * S[row x head] = K . Q^T and O^T[channel x head] = V^T . P by mma.m16n8k16.  A pair of codes
//    becomes an fp16x2 operand register exactly; V's pairs run along the rows, taken by a
//    byte permute from two rows' words, so V is not transposed through shared memory; P is, in
//    registers, by movmatrix.  An fp32 query has a second fp16 part, one more product each.
//  * K's scale multiplies the fp32 logits.  V's scale s = mant * 2^e multiplies the weight
//    before it is rounded to fp16: w = 2^((x - m) + e - R + 14) mant with R = ceil(max((x - m) +
//    e)).  Only R, m's distance from the maximum of x + e and so at most 127 either way, meets
//    the exponents: they hold at any finite logit, whatever the spacing of floats there is.  m
//    and R are integers, so rescaling is exact and no pair of scales leaves fp16's range.
//    A weight keeps 11 bits (a second fp16 part, 22, for an fp32 query) down to 2^-28 of
//    the largest.  A second part for a bf16 query as well would not show behind the output's own
//    rounding to 8 bits (1.65e-3 against 1.64e-3 from the 64-bit result) and costs 6 to 14 %:
//    8 x 32768 tokens 110.6 against 104.4 us, 2048 of each of 64 sequences 83.9 against 73.7.
#include "asp_internal.h"
#include "asp_kv8.cuh"

namespace asp {
namespace {

constexpr int kTile = 16;
constexpr int kWarps = 8;                  // of a CTA
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 2;
constexpr int kMinTiles = 8;               // of a CTA's range
constexpr int kFlatSms = 148;
constexpr int kMaxCtas = 2 * kFlatSms;     // of a launch that cuts units
constexpr int kFinThreads = 256;           // finish_kernel, accumulate_kernel
constexpr int kWBias = 14;      // the largest weight is below 2^15 before its rounding to fp16
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kNone = 0xffffffffu;
constexpr float kLowest = -3.402823466e38f;   // a maximum before any row: finite, so that no difference is inf - inf
constexpr float kNoRows = -1024.f;            // R before any row: below any row's

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct FlatParams {
  const void* q;
  int q_f32;
  int q_aligned;         // q on a 16-byte boundary
  int n_q_heads, G;
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  int block_shift, blocks_per_row;
  int units, n_kv, t_max, page_size, max_pages, n_pages;
  uint32_t page_magic;   // 2^32 / (page_size / 16), rounded up; 0 for pages of 16
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* idx;
  const int32_t* count;
  int C;
  const int32_t* tail_begin;
  int max_tail;
  int whole;
  float* part_o;      // [2 ctas][G][d]
  float* part_ml;     // [2 ctas][G][4]: m, l, R
  int4* info;         // [units]: first CTA, last CTA, slot of the first
  float* stat;        // [units][G][2]: m, 1 / l (accumulate; of attend_flat_kernel, where one CTA holds the unit)
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
  static constexpr int kCtas = 2;                // per SM
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
  static constexpr int kCtas = 1;
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

static_assert(kFlatSms * Fmt<CodeE4M3>::kCtas <= kMaxCtas && kFlatSms * Fmt<__nv_bfloat16>::kCtas <= kMaxCtas, "join");

// Stage: K rows, V rows (16-byte chunks, chunk c of row r at c ^ swz(r)), then K and V scales
// and the row mask.  The loads of a quarter warp (half warp for 8-byte loads) fall in
// distinct banks: K's touch rows g and g + 1 at the chunks 2t, V's the rows 2t at the chunks
// of two lanes g (64-byte rows: K's both halves of a row pair; V's meet twice).
template <typename CT, int D>
struct Stage {
  static constexpr int ROW = D * Fmt<CT>::kEB;      // bytes of a row
  static constexpr int CH = ROW / 16;               // its chunks
  static constexpr int HALF = kTile * ROW;
  static constexpr int SCALES = 2 * HALF;           // 16 + 16 floats
  static constexpr int MASK = SCALES + (Fmt<CT>::kScaled ? 2 * kTile * 4 : 0);
  static constexpr int BYTES = MASK + 16;
  static constexpr bool SMALL = CH == 4;
  __device__ __forceinline__ static constexpr int swz(int r) { return SMALL ? ((r >> 1) & 1) << 1 : r & 7; }
  // chunk of K that lane t takes in load i
  __device__ __forceinline__ static constexpr int k_chunk(int i, int t) {
    return SMALL ? t : 2 * t + (i & 1) + 8 * (i >> 1);
  }
  // channel of element e of m-tile i at lane g, and of element c of k-step ks at lane t
  __device__ __forceinline__ static constexpr int v_chan(int i, int g, int e) {
    return Fmt<CT>::kEB == 1 ? (D / 8) * g + 2 * i + e : (i >> 2) * 64 + 8 * g + 2 * (i & 3) + e;
  }
  __device__ __forceinline__ static constexpr int k_chan(int ks, int t, int c) {
    return Fmt<CT>::kEB == 1 ? 16 * k_chunk(ks >> 2, t) + 4 * (ks & 3) + c : 8 * k_chunk(ks >> 1, t) + 4 * (ks & 1) + c;
  }
};

__host__ __device__ constexpr int mo_stride(int D) { return D + 4; }
template <typename CT, int D>
constexpr size_t flat_smem(int G) {
  return (size_t)kWarps * (kStages * Stage<CT, D>::BYTES + G * (mo_stride(D) + 4) * 4);
}

// The logits of rows r .. r + 3 (r a multiple of 4), one vector per head; rows past the unit's
// and rows that were not attended hold -inf.
constexpr int kAccRows = 4 * kFinThreads;   // of a CTA of finish_kernel
static_assert(kMaxAccumulateRows == 65535L * kAccRows, "the sums' grid");

struct RowLogits {
  float4 x[8];
  int tok[4];          // -1: not a row
  bool run;            // four tokens that follow one another, on a 16-byte boundary of acc
};

__device__ __forceinline__ void load_logits(const FlatParams& p, int u, const UnitRows& ur, int r, RowLogits& q) {
  q.run = false;
#pragma unroll
  for (int k = 0; k < 4; ++k) q.tok[k] = -1;
  if (r >= ur.n_rows) return;
#pragma unroll
  for (int gg = 0; gg < 8; ++gg)
    if (gg < p.G) q.x[gg] = *reinterpret_cast<const float4*>(p.logits + ((size_t)u * p.G + gg) * p.row_stride + r);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (r + k < ur.n_rows)
      q.tok[k] = r + k < ur.n_sel ? p.idx[(size_t)u * p.C + r + k] : ur.tb + (r + k - ur.n_sel);
  q.run = r >= ur.n_sel && r + 3 < ur.n_rows &&
          (reinterpret_cast<uintptr_t>(p.acc + (size_t)u * p.t_max + q.tok[0]) & 15) == 0;
}

// acc of those rows: the weights of the group's heads, each from its logit by `weight`.  A row
// whose logits are -inf in every head was not attended (or has no weight); one head's can overflow
// to it alone.
template <typename W>
__device__ __forceinline__ void add_weights(const FlatParams& p, int u, const RowLogits& q, W weight) {
  float w[4] = {0.f, 0.f, 0.f, 0.f};
  bool has[4];
  if (q.tok[0] < 0) return;              // past the unit's rows
#pragma unroll
  for (int k = 0; k < 4; ++k) has[k] = (k == 0 ? q.x[0].x : k == 1 ? q.x[0].y : k == 2 ? q.x[0].z : q.x[0].w) != -INFINITY;
  if (!(has[0] && has[1] && has[2] && has[3])) {   // rare: the other heads
#pragma unroll
    for (int gg = 1; gg < 8; ++gg)
      if (gg < p.G) {
        has[0] |= q.x[gg].x != -INFINITY;
        has[1] |= q.x[gg].y != -INFINITY;
        has[2] |= q.x[gg].z != -INFINITY;
        has[3] |= q.x[gg].w != -INFINITY;
      }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) has[k] = has[k] && q.tok[k] >= 0;
#pragma unroll
  for (int gg = 0; gg < 8; ++gg)
    if (gg < p.G) {
      w[0] += weight(gg, q.x[gg].x);
      w[1] += weight(gg, q.x[gg].y);
      w[2] += weight(gg, q.x[gg].z);
      w[3] += weight(gg, q.x[gg].w);
    }
  float* const acc = p.acc + (size_t)u * p.t_max;
  if (q.run && has[0] && has[1] && has[2] && has[3]) {
    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(acc + q.tok[0]), "f"(w[0]), "f"(w[1]), "f"(w[2]),
                 "f"(w[3])
                 : "memory");
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (has[k]) atomicAdd(acc + q.tok[k], w[k]);
}

// Barrier 1 of the CTA: the joiner of a unit waits, the other warps only arrive.
__device__ __forceinline__ void joiner_wait() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }
__device__ __forceinline__ void joiner_arrive() { asm volatile("bar.arrive 1, %0;" ::"n"(kThreads) : "memory"); }

// Transposes an 8x8 matrix of 16-bit values held two per lane.
__device__ __forceinline__ uint32_t movm(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// QP: parts of the query (8-bit caches: 1 for bf16, 2 for fp32; bf16 caches: 1 or 3).
template <typename CT, int D, int QP, bool ACC>
__global__ void __launch_bounds__(kThreads, Fmt<CT>::kCtas) attend_flat_kernel(FlatParams p) {
  using F = Fmt<CT>;
  using S = Stage<CT, D>;
  constexpr int W = kWarps, THREADS = kThreads;
  constexpr int KS = D / 16;                 // k-steps of the logits
  constexpr int MT = D / 16;                 // m-tiles of the output
  constexpr bool WSPLIT = !F::kScaled || QP > 1;   // weights in two parts

  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int run_pre[THREADS + 1];
  __shared__ int scan[33];
  __shared__ int s_first[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int G = p.G;
  uint8_t* const ring = smem + (size_t)warp * kStages * S::BYTES;
  float* const mo = reinterpret_cast<float*>(smem + (size_t)W * kStages * S::BYTES);   // [warp][G][D + 4]
  float* const mml = mo + (size_t)W * G * mo_stride(D);                                // [warp][G][4]

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
    const int per = (p.units + THREADS - 1) / THREADS;   // units of a thread's run
    cta_prefix_sum(THREADS, run_pre, [&](int i) {
      int n = 0;
      for (int u = i * per; u < min(p.units, (i + 1) * per); ++u) n += unit_tiles(unit_rows(p, u, cta == 0));
      return n;
    }, scan);
    total = run_pre[THREADS];
    N = min(N, (total + kMinTiles - 1) / kMinTiles);   // no CTA without tiles
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
  const int my_n = ntl > warp ? (ntl - warp + W - 1) / W : 0;   // this warp's tiles

  // ---- fetching: request() the tile's position and raw indices; resolve() its tokens and
  // their pages; issue() the copies
  int pu = u0, pb = u0 / p.n_kv, ph = u0 - pb * p.n_kv, ptl = tl0 + warp;
  UnitRows pr = unit_rows(p, pu, false);
  int pn = unit_tiles(pr);
  const int rr = lane & 15;
  int asked = 0, a_tl = 0, raw = 0;
  auto request = [&]() {
    if (asked >= my_n) return;
    while (ptl >= pn) {
      ptl -= pn;
      ++pu;
      if (++ph == p.n_kv) {
        ph = 0;
        ++pb;
      }
      pr = unit_rows(p, pu, false);
      pn = unit_tiles(pr);
    }
    a_tl = ptl;
    if (a_tl * kTile < pr.n_sel) {
      const int r = a_tl * kTile + rr;
      raw = r < pr.n_sel ? __ldg(p.idx + (size_t)pu * p.C + r) : 0;
    }
    ptl += W;
    ++asked;
  };
  // this lane's row of the resolved tile: contiguous, its row and scale; paged, its page and
  // the row in it
  uint32_t b_row = kNone, b_srow = 0;
  int b_page = 0, b_h = 0, resolved = 0;
  bool b_run = false;        // 16 rows that follow one another in memory
  auto resolve = [&]() {
    if (resolved >= my_n) return;
    ++resolved;
    const int r0 = a_tl * kTile, r = r0 + rr;
    int tok = -1;
    if (r < pr.n_sel) {
      tok = raw;
      if (tok < 0 || tok >= pr.T) {
        if (lane < 16) flag_status(ASP_DEV_BAD_INDEX);
        tok = -1;
      } else if (tok >= pr.tb) {
        tok = -1;   // covered by the tail
      }
    } else if (r < pr.n_rows) {
      tok = pr.tb + (r - pr.n_sel);
    }
    b_run = r0 >= pr.n_sel && r0 + kTile <= pr.n_rows &&
            (p.page_size == 0 || ((pr.tb + r0 - pr.n_sel) & (kTile - 1)) == 0);
    b_row = kNone;
    if (p.page_size == 0) {
      if (tok >= 0) {
        b_row = (uint32_t)((size_t)pu * p.t_max + tok);
        if (F::kScaled) b_srow = (uint32_t)((size_t)pu * p.blocks_per_row + (tok >> p.block_shift));
      }
    } else if (tok >= 0) {   // tok / page_size: pages are 16 m tokens, m <= 16, and tok / 16 < 2^27
      const uint32_t t16 = (uint32_t)tok >> 4;
      const uint32_t lp = p.page_magic ? __umulhi(t16, p.page_magic) : t16;
      b_page = __ldg(p.page_table + (size_t)pb * p.max_pages + lp);
      b_row = (uint32_t)tok - lp * (uint32_t)p.page_size;
      b_h = ph;
    }
  };
  int issued = 0;
  const int lr = lane / S::CH, lc = lane % S::CH;
  auto issue = [&]() {       // an empty group past the end
    if (issued < my_n) {
      uint8_t* const st = ring + (issued % kStages) * S::BYTES;
      uint32_t row = b_row, srow = b_srow;
      if (p.page_size && row != kNone) {
        if (b_page < 0 || b_page >= p.n_pages) {
          if (lane < 16) flag_status(ASP_DEV_BAD_PAGE);
          row = kNone;
        } else {
          const size_t head = (size_t)b_page * p.n_kv + b_h;
          if (F::kScaled) srow = (uint32_t)(head * p.blocks_per_row + (row >> p.block_shift));
          row = (uint32_t)(head * p.page_size + row);
        }
      }
      const uint32_t vm = __ballot_sync(0xffffffffu, row != kNone) & 0xffffu;
      if (vm) {
        constexpr int RPI = 32 / S::CH;   // rows per warp instruction
        const uint32_t base = smem_u32(st);
        auto copy = [&](int i, const uint8_t* kf, const uint8_t* vf) {
          const int ri = RPI * i + lr;
          const uint32_t dst = base + ri * S::ROW + ((lc ^ S::swz(ri)) * 16);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(kf) : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + S::HALF), "l"(vf) : "memory");
        };
        if (b_run && vm == 0xffffu) {
          const uint32_t row0 = __shfl_sync(0xffffffffu, row, 0);
          const size_t off = (size_t)row0 * S::ROW + lane * 16;
          const uint8_t* const kf = p.k + off;
          const uint8_t* const vf = p.v + off;
#pragma unroll
          for (int i = 0; i < kTile / RPI; ++i) copy(i, kf + i * 512, vf + i * 512);
        } else {
          // a row that is not read repeats one that is: its weight is zero, and nothing that
          // was not written meets it
          const int first = __ffs(vm) - 1;
          const uint32_t fr = __shfl_sync(0xffffffffu, row, first), fs = __shfl_sync(0xffffffffu, srow, first);
          if (row == kNone) {
            row = fr;
            srow = fs;
          }
#pragma unroll
          for (int i = 0; i < kTile / RPI; ++i) {
            const uint32_t src = __shfl_sync(0xffffffffu, row, RPI * i + lr);
            const size_t off = (size_t)src * S::ROW + lc * 16;
            copy(i, p.k + off, p.v + off);
          }
        }
        if constexpr (F::kScaled) {
          const float* from = (lane < 16 ? p.k_scale : p.v_scale) + srow;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(base + S::SCALES + lane * 4), "l"(from)
                       : "memory");
        }
      }
      if (lane == 0) *reinterpret_cast<uint32_t*>(st + S::MASK) = vm;
      ++issued;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // ---- query fragments: column g is head g
  uint32_t qa[KS][2 * QP];
  float qfac[2] = {p.qscale, p.qscale};     // of heads 2t and 2t + 1
  auto load_q = [&](int unit) {
    const int b = unit / p.n_kv, h = unit - b * p.n_kv;
    const size_t off = ((size_t)b * p.n_q_heads + h * G + (g < G ? g : 0)) * D;
    float4 q4[KS];   // all loads before any use
    if (p.q_f32) {
      const float* const src = static_cast<const float*>(p.q) + off;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const float* const s4 = src + S::k_chan(ks, t, 0);
        q4[ks] = p.q_aligned ? __ldg(reinterpret_cast<const float4*>(s4)) : make_float4(s4[0], s4[1], s4[2], s4[3]);
      }
    } else {
      const __nv_bfloat16* const src = static_cast<const __nv_bfloat16*>(p.q) + off;
      uint2 w[KS];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const __nv_bfloat16* const s4 = src + S::k_chan(ks, t, 0);
        if (p.q_aligned) {
          w[ks] = __ldg(reinterpret_cast<const uint2*>(s4));
        } else {
          const unsigned short* const us = reinterpret_cast<const unsigned short*>(s4);
          w[ks] = make_uint2((uint32_t)us[0] | ((uint32_t)us[1] << 16), (uint32_t)us[2] | ((uint32_t)us[3] << 16));
        }
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const float2 lo = bf16x2_to_float2(w[ks].x), hi = bf16x2_to_float2(w[ks].y);
        q4[ks] = make_float4(lo.x, lo.y, hi.x, hi.y);
      }
    }
    if (g >= G) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) q4[ks] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float up = 1.f;
    if constexpr (F::kScaled) {   // largest channel to [2^14, 2^15)
      uint32_t amax = 0u;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        amax = max(max(amax, max(finite_abs(q4[ks].x), finite_abs(q4[ks].y))),
                   max(finite_abs(q4[ks].z), finite_abs(q4[ks].w)));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      int e = (int)(amax >> 23) - 127;
      e = e < -112 ? -112 : e;
      up = exp2i(14 - e);
      const float f = exp2i(e - 14) * p.qscale;
      qfac[0] = __shfl_sync(0xffffffffu, f, 8 * t);
      qfac[1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      float x[4] = {q4[ks].x * up, q4[ks].y * up, q4[ks].z * up, q4[ks].w * up};
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
  request();
  load_q(u0);      // while the first indices arrive
  resolve();
  request();
#pragma unroll
  for (int s = 0; s < kStages; ++s) {
    issue();
    resolve();
    request();
  }

  // ---- the tiles of each unit in turn
  int j = 0;                 // this warp's next tile
  int seg = 0;               // units so far
  int seg_t0 = t0 - tl0;     // where the current unit's tiles begin in the flattened order
  for (int u = u0;; ++u) {
    const UnitRows ur = unit_rows(p, u, false);
    const int un = unit_tiles(ur);
    const int seg_end = min(t1, seg_t0 + un);
    const int kend = seg_end - t0 - warp;
    const int jend = kend > 0 ? (kend + W - 1) / W : 0;
    float o[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    // of heads 2t and 2t + 1; l: this lane's share
    float m[2] = {kLowest, kLowest}, R[2] = {kNoRows, kNoRows}, l[2] = {0.f, 0.f};
#pragma unroll 1
    for (; j < jend; ++j) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();
      const uint8_t* const st = ring + (j % kStages) * S::BYTES;
      const uint32_t vm = *reinterpret_cast<const uint32_t*>(st + S::MASK);
      float* lg = nullptr;   // logits of head 2t, row g
      if constexpr (ACC) lg = p.logits + ((size_t)u * G + 2 * t) * p.row_stride + (t0 + warp + j * W - seg_t0) * kTile + g;
      if (vm) {
        // x[2 r + e]: logit of row g + 8 r and head 2t + e
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        const uint8_t* const k0 = st + g * S::ROW;   // rows g and g + 8 are swizzled alike
#pragma unroll
        for (int i = 0; i < S::CH / 4; ++i) {
          const int at = (S::k_chunk(i, t) ^ S::swz(g)) * 16;
          const uint4 y0 = *reinterpret_cast<const uint4*>(k0 + at);
          const uint4 y1 = *reinterpret_cast<const uint4*>(k0 + 8 * S::ROW + at);
          const uint32_t w0[4] = {y0.x, y0.y, y0.z, y0.w}, w1[4] = {y1.x, y1.y, y1.z, y1.w};
          if constexpr (F::kEB == 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int ks = 4 * i + e;
              const uint32_t z0 = CT::prep(w0[e]), z1 = CT::prep(w1[e]);
              const uint32_t a0 = CT::pair(z0, 0), a1 = CT::pair(z1, 0), a2 = CT::pair(z0, 1), a3 = CT::pair(z1, 1);
#pragma unroll
              for (int part = 0; part < QP; ++part) F::mma(x, a0, a1, a2, a3, qa[ks][2 * part], qa[ks][2 * part + 1]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int ks = 2 * i + e;
#pragma unroll
              for (int part = 0; part < QP; ++part)
                F::mma(x, w0[2 * e], w1[2 * e], w0[2 * e + 1], w1[2 * e + 1], qa[ks][2 * part], qa[ks][2 * part + 1]);
            }
          }
        }
        float ve[2], vmant[2];   // V's scale of rows g and g + 8: exponent and fraction
        if constexpr (F::kScaled) {
          const float* const ksc = reinterpret_cast<const float*>(st + S::SCALES);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float k = ksc[8 * r + g];
            x[2 * r] *= k * qfac[0];
            x[2 * r + 1] *= k * qfac[1];
            const uint32_t bits = __float_as_uint(ksc[16 + 8 * r + g]);
            ve[r] = __uint_as_float((bits >> 23) | 0x4b000000u) - 8388735.f;   // 2^23 + 127
            vmant[r] = __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] *= qfac[0];
        }
        if (vm != 0xffffu) {
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (!((vm >> (g + 8 * r)) & 1u)) x[2 * r] = x[2 * r + 1] = -INFINITY;
        }
        if constexpr (ACC) {
          if (2 * t < G) {
            lg[0] = x[0];
            lg[8] = x[2];
          }
          if (2 * t + 1 < G) {
            lg[p.row_stride] = x[1];
            lg[p.row_stride + 8] = x[3];
          }
        }
        // dx: x - m; a: exponents of the weights, at most 14 where R holds; the maxima are raised
        // only when a row of the tile passes them
        float dx[4], a[4];
        const float mx[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
        bool up = mx[0] > m[0] || mx[1] > m[1];
        auto exponents = [&]() {
#pragma unroll
          for (int e = 0; e < 4; ++e) dx[e] = x[e] - m[e & 1];
          if constexpr (F::kScaled) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float off = (float)kWBias - R[e];   // integers below 2^12: exact
              a[e] = dx[e] + (ve[0] + off);
              a[2 + e] = dx[2 + e] + (ve[1] + off);
            }
          }
        };
        exponents();
        if constexpr (F::kScaled) up |= fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])) > (float)kWBias;
        if (__any_sync(0xffffffffu, up)) {
          float corr[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mr = mx[e];
            mr = fmaxf(mr, __shfl_xor_sync(0xffffffffu, mr, 4));
            mr = fmaxf(mr, __shfl_xor_sync(0xffffffffu, mr, 8));
            mr = fmaxf(mr, __shfl_xor_sync(0xffffffffu, mr, 16));
            const float mn = fmaxf(m[e], ceilf(mr));
            const float down = m[e] - mn;   // exact, or so far that what was there counts for nothing
            corr[e] = ex2(down);
            l[e] *= corr[e];
            m[e] = mn;
            if constexpr (F::kScaled) {
              float Rr = fmaxf((x[e] - mn) + ve[0], (x[2 + e] - mn) + ve[1]);
              Rr = fmaxf(Rr, __shfl_xor_sync(0xffffffffu, Rr, 4));
              Rr = fmaxf(Rr, __shfl_xor_sync(0xffffffffu, Rr, 8));
              Rr = fmaxf(Rr, __shfl_xor_sync(0xffffffffu, Rr, 16));
              const float was = R[e] + down;   // R of the rows so far, from the new m
              R[e] = fmaxf(fmaxf(was, ceilf(Rr)), kNoRows);
              corr[e] = ex2(was - R[e]);
            }
          }
          exponents();
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            o[i][0] *= corr[0];
            o[i][1] *= corr[1];
            o[i][2] *= corr[0];
            o[i][3] *= corr[1];
          }
        }
        float w4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w4[e] = ex2(dx[e]);
        l[0] += w4[0] + w4[2];
        l[1] += w4[1] + w4[3];
        if constexpr (F::kScaled) {
#pragma unroll
          for (int e = 0; e < 4; ++e) w4[e] = ex2(a[e]) * vmant[e >> 1];
        }
        const uint32_t h0 = F::pack(w4[0], w4[1]), h1 = F::pack(w4[2], w4[3]);
        const uint32_t b0 = movm(h0), b1 = movm(h1);   // rows 2t, 2t + 1 (+ 8) of head g
        uint32_t l0 = 0u, l1 = 0u;
        if constexpr (WSPLIT) {
          const float2 f0 = F::unpack(h0), f1 = F::unpack(h1);
          l0 = movm(F::pack(w4[0] - f0.x, w4[1] - f0.y));
          l1 = movm(F::pack(w4[2] - f1.x, w4[3] - f1.y));
        }
        // O^T += V^T . P: lane g holds a run of channels of the rows 2t, 2t+1, 8+2t, 9+2t
        const uint8_t* const vb = st + S::HALF;
        constexpr int WPR = (D / 8) * F::kEB / 4;        // words of them per row
        uint32_t vw[4][WPR];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 2 * t + (e & 1) + (e >> 1) * 8;
          const uint8_t* const vrow = vb + r * S::ROW;
          if constexpr (WPR == 2) {
            const uint2 y = *reinterpret_cast<const uint2*>(vrow + (((g >> 1) ^ S::swz(r)) * 16) + (g & 1) * 8);
            vw[e][0] = y.x;
            vw[e][1] = y.y;
          } else {
#pragma unroll
            for (int c = 0; c < WPR / 4; ++c) {
              const uint4 y = *reinterpret_cast<const uint4*>(vrow + (((g + 8 * c) ^ S::swz(r)) * 16));
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
      } else if constexpr (ACC) {
        if (2 * t < G) lg[0] = lg[8] = -INFINITY;
        if (2 * t + 1 < G) lg[p.row_stride] = lg[p.row_stride + 8] = -INFINITY;
      }
      __syncwarp();
      issue();
      resolve();
      request();
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 4);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 8);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 16);
      if constexpr (!F::kScaled) R[e] = 0.f;
    }

    // ---- the warps' results of this unit meet in shared memory (position 16 i + 2 g + e of a
    // head's row is channel v_chan(i, g, e)), and one warp, another for each unit, joins them
    // while the others go on with the next unit.  Barrier 1: the results are there.  Every warp,
    // the last joiner too, meets the others before the buffer is written again: a warp that
    // did not could arrive at a barrier's phase before the one meant for it.
    const int joiner = seg % W;
    if (seg > 0) __syncthreads();
    if (g == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (2 * t + e < G)
          *reinterpret_cast<float4*>(mml + (warp * G + 2 * t + e) * 4) = make_float4(m[e], l[e], R[e], 0.f);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (2 * t + e < G) {
        float* const row = mo + ((size_t)warp * G + 2 * t + e) * mo_stride(D) + 2 * g;
#pragma unroll
        for (int i = 0; i < MT; ++i) *reinterpret_cast<float2*>(row + 16 * i) = make_float2(o[i][e], o[i][2 + e]);
      }
    }
    const bool last = seg_end >= t1;
    __syncwarp();
    if (warp != joiner) {
      joiner_arrive();
    } else {
      joiner_wait();
      const bool starts = seg_t0 >= t0, ends = seg_t0 + un <= t1;
      const bool alone = starts && ends;
      const int slot = 2 * cta + (u == u0 ? 0 : 1);
      if (!p.whole && starts && lane == 0)
        p.info[u] = make_int4(cta, ends ? cta : range_owner(seg_t0 + un - 1, total, N), slot, 0);
      const int b = u / p.n_kv, h = u - b * p.n_kv;
      for (int gg = 0; gg < G; ++gg) {
        // lane w: warp w's statistics of the head and the factor of its output (l = 0, o = 0
        // for a warp without rows)
        float4 ml = make_float4(kLowest, 0.f, kNoRows, 0.f);
        if (lane < W) ml = *reinterpret_cast<const float4*>(mml + (lane * G + gg) * 4);
        float mm = ml.x;
#pragma unroll
        for (int sh = W / 2; sh; sh >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, sh));
        mm = __shfl_sync(0xffffffffu, mm, 0);
        const float rw = ml.z + (ml.x - mm);   // the warp's R from the common m
        float RR = fmaxf(rw, kNoRows);
#pragma unroll
        for (int sh = W / 2; sh; sh >>= 1) RR = fmaxf(RR, __shfl_xor_sync(0xffffffffu, RR, sh));
        RR = __shfl_sync(0xffffffffu, RR, 0);
        const float fw = ex2(rw - RR);
        float L = ml.y * ex2(ml.x - mm);
#pragma unroll
        for (int sh = W / 2; sh; sh >>= 1) L += __shfl_xor_sync(0xffffffffu, L, sh);
        L = __shfl_sync(0xffffffffu, L, 0);
        float f[W];
#pragma unroll
        for (int w = 0; w < W; ++w) f[w] = __shfl_sync(0xffffffffu, fw, w);
        const float scale = L == 0.f ? 0.f : ex2(RR - (F::kScaled ? (float)kWBias : 0.f)) / L;
        const size_t bh = (size_t)b * p.n_q_heads + h * G + gg;
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {   // two channels per lane
          const int pos = 64 * k + 2 * lane;
          const int c = S::v_chan(pos >> 4, (pos & 15) >> 1, 0);
          float2 O = make_float2(0.f, 0.f);
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const float2 x = *reinterpret_cast<const float2*>(mo + ((size_t)w * G + gg) * mo_stride(D) + pos);
            O.x += x.x * f[w];
            O.y += x.y * f[w];
          }
          if (alone) {
            if (L == 0.f) O = make_float2(0.f, 0.f);
            else O = make_float2(O.x * scale, O.y * scale);
            if (p.out_f32) {
              static_cast<float*>(p.out)[bh * D + c] = O.x;
              static_cast<float*>(p.out)[bh * D + c + 1] = O.y;
            } else {
              static_cast<__nv_bfloat16*>(p.out)[bh * D + c] = __float2bfloat16_rn(O.x);
              static_cast<__nv_bfloat16*>(p.out)[bh * D + c + 1] = __float2bfloat16_rn(O.y);
            }
          } else {
            *reinterpret_cast<float2*>(p.part_o + ((size_t)slot * G + gg) * D + c) = O;
          }
        }
        if (lane == 0) {
          if (!alone) {
            *reinterpret_cast<float4*>(p.part_ml + ((size_t)slot * G + gg) * 4) = make_float4(mm, L, RR, 0.f);
          } else {
            if (p.lse) p.lse[bh] = L == 0.f ? -INFINITY : mm * kLn2 + logf(L);
            if constexpr (ACC) {
              p.stat[((size_t)u * G + gg) * 2] = mm;
              p.stat[((size_t)u * G + gg) * 2 + 1] = L == 0.f ? 0.f : 1.f / L;
            }
          }
        }
      }
    }
    if constexpr (ACC) {
      if (p.whole) {   // this CTA holds every logit of the unit: the weights right away
        __syncthreads();
        const float* const stat = p.stat + (size_t)u * G * 2;
        for (int r = threadIdx.x; r < ur.n_rows; r += THREADS) {   // few rows: one at a time, in few registers
          const float* const x = p.logits + (size_t)u * G * p.row_stride + r;
          float w = 0.f;
          bool has = false;        // as in add_weights
#pragma unroll 1
          for (int gg = 0; gg < G; ++gg) {
            const float xv = x[(size_t)gg * p.row_stride];
            has |= xv != -INFINITY;
            w += ex2(xv - stat[2 * gg]) * stat[2 * gg + 1];
          }
          if (!has) continue;
          const int tok = r < ur.n_sel ? p.idx[(size_t)u * p.C + r] : ur.tb + (r - ur.n_sel);
          atomicAdd(p.acc + (size_t)u * p.t_max + tok, w);
        }
      }
    }
    if (last) break;
    load_q(u + 1);
    seg_t0 += un;
    ++seg;
  }
}

// Joins the units that several CTAs share (one CTA per unit) and, for ACC, adds the weights
// of the unit's rows (blockIdx.y: chunks of kAccRows rows).
template <int D, bool ACC>
__global__ void __launch_bounds__(kFinThreads) finish_kernel(FlatParams p, float bias) {
  __shared__ float2 fac[8][kMaxCtas];      // of a CTA's output: its m and R, then its weight
  __shared__ float s_m[8], s_l[8], s_R[8];
  __shared__ float4 red[kFinThreads];
  const int u = blockIdx.x, G = p.G, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  const int4 in = p.info[u];
  const int n = in.y - in.x + 1;           // CTAs of the unit
  const bool join = n > 1 && blockIdx.y == 0;
  if (!ACC && !join) return;
  UnitRows ur;
  if constexpr (ACC) {
    ur = unit_rows(p, u, false);
    if (!join && (int)blockIdx.y * kAccRows >= ur.n_rows) return;
  }
  RowLogits rows;   // requested ahead of the statistics
  if constexpr (ACC) load_logits(p, u, ur, blockIdx.y * kAccRows + 4 * threadIdx.x, rows);
  auto slot_of = [&](int i) -> int { return i == 0 ? in.z : 2 * (in.x + i); };
  if (warp < G) {   // warp gg: statistics of head gg
    if (n > 1) {
      float mm = kLowest, RR = kNoRows, L = 0.f;
      for (int i = lane; i < n; i += 32) {
        const float4 ml = *reinterpret_cast<const float4*>(p.part_ml + ((size_t)slot_of(i) * G + warp) * 4);
        fac[warp][i] = make_float2(ml.x, ml.z);
        const float mn = fmaxf(mm, ml.x);
        RR = fmaxf(RR + (mm - mn), ml.z + (ml.x - mn));
        L = L * ex2(mm - mn) + ml.y * ex2(ml.x - mn);
        mm = mn;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, mm, o), l2 = __shfl_xor_sync(0xffffffffu, L, o);
        const float r2 = __shfl_xor_sync(0xffffffffu, RR, o);
        const float mn = fmaxf(mm, m2);
        RR = fmaxf(RR + (mm - mn), r2 + (m2 - mn));
        L = L * ex2(mm - mn) + l2 * ex2(m2 - mn);
        mm = mn;
      }
      RR = fmaxf(RR, kNoRows);
      for (int i = lane; i < n; i += 32) {
        const float2 f = fac[warp][i];
        fac[warp][i].x = ex2((f.y + (f.x - mm)) - RR);
      }
      if (lane == 0) {
        s_m[warp] = mm;
        s_l[warp] = L;
        s_R[warp] = RR;
      }
    } else if (lane == 0) {
      s_m[warp] = p.stat[((size_t)u * G + warp) * 2];
      s_l[warp] = p.stat[((size_t)u * G + warp) * 2 + 1];   // 1 / l
    }
  }
  __syncthreads();
  if (join) {   // four channels per thread; groups of threads take every ngrp-th CTA's output
    const int cols = G * D / 4, ngrp = kFinThreads / cols;
    const int col = threadIdx.x % cols, grp = threadIdx.x / cols;
    const int gg = 4 * col / D, c = 4 * col - gg * D;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = grp; i < n; i += ngrp) {
      const float4 x = *reinterpret_cast<const float4*>(p.part_o + ((size_t)slot_of(i) * G + gg) * D + c);
      const float f = fac[gg][i].x;
      a.x += x.x * f;
      a.y += x.y * f;
      a.z += x.z * f;
      a.w += x.w * f;
    }
    red[threadIdx.x] = a;
    __syncthreads();
    if (grp == 0) {
      for (int k = 1; k < ngrp; ++k) {
        const float4 x = red[k * cols + col];
        a.x += x.x;
        a.y += x.y;
        a.z += x.z;
        a.w += x.w;
      }
      const int b = u / p.n_kv, h = u - b * p.n_kv;
      const size_t bh = (size_t)b * p.n_q_heads + h * G + gg;
      const float L = s_l[gg], mm = s_m[gg];
      const float f = ex2(s_R[gg] - bias);
      const float y[4] = {a.x / L * f, a.y / L * f, a.z / L * f, a.w / L * f};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = L == 0.f ? 0.f : y[e];
        if (p.out_f32) static_cast<float*>(p.out)[bh * D + c + e] = v;
        else static_cast<__nv_bfloat16*>(p.out)[bh * D + c + e] = __float2bfloat16_rn(v);
      }
      if (c == 0 && p.lse) p.lse[bh] = L == 0.f ? -INFINITY : mm * kLn2 + logf(L);
    }
  }
  if constexpr (ACC) {
    __syncthreads();
    if (n > 1 && threadIdx.x < G) s_l[threadIdx.x] = s_l[threadIdx.x] == 0.f ? 0.f : 1.f / s_l[threadIdx.x];
    __syncthreads();
    add_weights(p, u, rows, [&](int gg, float xv) { return ex2(xv - s_m[gg]) * s_l[gg]; });
  }
}

// acc from the logits (base 2) and statistics of attend_kernel: the weights come from x - m as
// the output's do, so that they sum to the group's heads at any size of the logits (from the
// lse, a rounded sum of logit and logarithm, they would be off by |lse| 2^-24 relative).
__global__ void __launch_bounds__(kFinThreads) accumulate_kernel(FlatParams p) {
  __shared__ float s_m[8], s_l[8];
  const int u = blockIdx.x, G = p.G;
  pdl_wait();
  const UnitRows ur = unit_rows(p, u, false);
  if ((int)blockIdx.y * kAccRows >= ur.n_rows) return;
  RowLogits rows;
  load_logits(p, u, ur, blockIdx.y * kAccRows + 4 * threadIdx.x, rows);
  if (threadIdx.x < G) {
    s_m[threadIdx.x] = p.stat[((size_t)u * G + threadIdx.x) * 2];
    s_l[threadIdx.x] = p.stat[((size_t)u * G + threadIdx.x) * 2 + 1];
  }
  __syncthreads();
  add_weights(p, u, rows, [&](int gg, float xv) { return ex2(xv - s_m[gg]) * s_l[gg]; });
}

template <typename CT, int D, int QP, bool ACC>
cudaError_t launch_flat_t(const FlatParams& p, int ctas, int chunks, cudaStream_t s) {
  auto kern = attend_flat_kernel<CT, D, QP, ACC>;
  const size_t smem = flat_smem<CT, D>(p.G);
  if (prepare_kernel((const void*)kern, smem, kThreads) < 1) return cudaErrorInvalidConfiguration;
  cudaError_t e = launch_pdl(kern, dim3(ctas), dim3(kThreads), smem, s, p);
  if (e != cudaSuccess || p.whole) return e;
  return launch_pdl(finish_kernel<D, ACC>, dim3(p.units, ACC ? chunks : 1), dim3(kFinThreads), 0, s, p,
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
  p.q_aligned = (reinterpret_cast<uintptr_t>(q) & 15) == 0;
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
  const int m16 = kv.page_size / 16;
  p.page_magic = m16 > 1 ? (uint32_t)(((1ull << 32) + m16 - 1) / m16) : 0u;
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

// A unit of at most kWholeRows rows stays whole: four tiles per warp cost no more than joining
// the shares of several CTAs in a second launch, however few units there are.  E4M3, d = 128,
// group 4, bf16 query, call times in us, whole against shared (the timer's step is 2 us):
//   rows       1 to 8 units      128 units         512 units
//    256       12.3 / 14 to 16   14.3 / 18.4       26.6 / 32.8
//    512       16.4 / 16.4       16.4 / 24.6       32.8 / 36.9
//    768       18.4 / 16.4       18.4 / 26.6       38.9 / 43.0
//   2048       26 to 29 / 18     28.7 / 32.8       67.6 / 69.6
// 512 is where whole units stop losing for few units; with an fp32 query or sums it is the same.
constexpr int kWholeRows = 512;

FlatPlan flat_plan(int batch, int n_q_heads, int n_kv_heads, int head_dim, int C, int max_tail, bool kv8,
                   bool accumulate, int ctas_per_sm) {
  FlatPlan pl = {};
  const long rows = (long)C + (max_tail > 0 ? max_tail : 0);
  const long units = (long)batch * n_kv_heads;
  const int G = n_q_heads / n_kv_heads;
  const long tiles = units * ((rows + kTile - 1) / kTile);
  const long ctas = (tiles + kMinTiles - 1) / kMinTiles;
  // beside the key scan in the decode step: one CTA per SM.  At d = 64 it shares the SM with a
  // CTA of the scan; at d = 128 the two do not fit (286 KB of shared memory), and one is faster
  // all the same: 94 us against 98 to 102 with two for a step at 8 x 32768, E4M3
  const long most = (long)kFlatSms * (ctas_per_sm > 0 ? ctas_per_sm : (kv8 ? Fmt<CodeE4M3>::kCtas : 1));
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

cudaError_t launch_accumulate(const float* logits, int row_stride, const float* stat, int n_q_heads, const KvView& kv,
                              const int32_t* idx, const int32_t* count, int C, const int32_t* tail_begin, int max_tail,
                              float* acc, cudaStream_t s) {
  FlatParams p = flat_params(nullptr, 1, n_q_heads, kv, idx, count, C, tail_begin, max_tail);
  p.logits = const_cast<float*>(logits);
  p.row_stride = row_stride;
  p.stat = const_cast<float*>(stat);
  p.acc = acc;
  return launch_pdl(accumulate_kernel, dim3(p.units, (row_stride + kAccRows - 1) / kAccRows), dim3(kFinThreads), 0, s, p);
}

ASP_STATUS_READER(read_status_attend_flat)

}  // namespace asp
