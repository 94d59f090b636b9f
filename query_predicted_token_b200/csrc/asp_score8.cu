// asp_score8.cu -- step 2 over keys held in 8 bits.
//
// scores[b, h, j] = max_g (qpred[b, h*G+g] . code_j) * scale_j / sqrt(d): one read of every
// key row (128 + 4 / scale_block bytes for d = 128) and 4 bytes written, bound by HBM.
//
// The warps of a CTA take the 64-row steps of its contiguous range in turn.  Each has a ring of
// three stages, filled by one bulk copy (TMA, 1-D) per 16-row tile, which never crosses a page,
// counted on an mbarrier; page numbers come for eight steps at a time, one tile per lane, the
// next eight ahead of their use.  The copies bound it: a call over 269 MB takes 53 us with E4M3
// codes and 57 with integers, and 53 with no arithmetic at all (rings of 12 or 16 warps with the
// same bytes in flight: 56 to 60).
// Lane (g, t) = (lane / 4, lane % 4) reads 16-byte pieces of rows g and g + 8 of a 16-row tile
// from shared memory, which are its operand A; the order in which channels meet the k index
// is the same for both operands and otherwise free.  (Rows loaded straight into registers, two
// steps of them, spilled and waited: 112 us for 312 MB of integers.)
// Every wait is bounded (ASP_DEV_WAIT_LIMIT).
//
// E4M3 codes are widened to fp16 (exact) for m16n8k16; the query, scaled by a power of two so
// that its largest channel lies in [2^14, 2^15), is split into two fp16 parts (22 bits) in
// neighbouring columns of B: 4 query heads are one n-tile of 8.  Integer codes are A as they
// lie in memory, for m16n8k32 on integers: the query as a 23-bit integer of its largest
// channel, in three 8-bit digits, one n-tile each.  Either way every product and every sum of
// digits is exact; widening integer codes to fp16 instead takes 5 instructions per 4 codes.
// The maximum over a group's heads keeps a NaN: a head that is not finite must not vanish behind
// the others.
#include <type_traits>

#include "asp_internal.h"
#include "asp_kv8.cuh"

namespace asp {
namespace {

constexpr int kTiles = 4;      // 16-row tiles of a warp's step
constexpr int kRows = 16 * kTiles;
constexpr int kWarps = 8;      // of the SM's one CTA

struct Score8Params {
  const float* qpred;
  int n_q_heads, G;
  const uint8_t* k;
  const float* k_scale;
  int block_shift, blocks_per_row;
  int batch, n_kv, t_max, page_size, max_pages, n_pages;
  uint32_t page_magic;   // 2^32 / (page_size / 16), rounded up; 0 for pages of 16
  const int32_t* page_table;
  const int32_t* seq_lens;
  float* scores;
  int32_t* hist;
  float scale;
  int stages;          // of a warp's ring
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first product of a sum: the accumulator starts at zero.
__device__ __forceinline__ void mma_f16_0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_s8_0(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
}

// The query is read twice, for its largest channel and for its parts, so that only one piece of
// it is in registers at a time beside the rows in flight.
__device__ __forceinline__ void ld_query(const float* p, float (&x)[4]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) asm volatile("ld.global.f32 %0, [%1];" : "=f"(x[c]) : "l"(p + c));
}

// Piece l of rows g and g + 8 of the two tiles at st.
template <int D>
__device__ __forceinline__ void load_rows(const uint8_t* st, int g, int t, int l, uint32_t (&w)[2][2][4]) {
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint4 y = *reinterpret_cast<const uint4*>(st + (16 * u + 8 * e + g) * D + (t * (D / 64) + l) * 16);
      w[u][e][0] = y.x;
      w[u][e][1] = y.y;
      w[u][e][2] = y.z;
      w[u][e][3] = y.w;
    }
}

// Operand B of one group: NT n-tiles.  load() fills it for group (b, h); scores() turns rows g
// and g + 8 of two tiles (their products interleaved: each is a chain) into the group's maxima
// over this lane's heads.
template <typename CT, int D, int NT>
struct Query;

template <int D, int NT>
struct Query<CodeE4M3, D, NT> {   // NT = 1 for up to 4 heads, 2 for 8; column g of n-tile nt: part g & 1 of head 4 nt + g / 2
  static constexpr int LD = D / 64;     // 16-byte pieces of a row per lane
  uint32_t b[NT][4 * LD][2];
  float fac[NT];   // of head 4 nt + t: undoes the power of two, times 1 / sqrt(d)

  __device__ __forceinline__ void load(const Score8Params& p, int bi, int h, int g, int t) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int head = 4 * nt + (g >> 1);
      const bool has = head < p.G;
      const float* const src = p.qpred + ((size_t)bi * p.n_q_heads + h * p.G + (has ? head : 0)) * D + t * 16 * LD;
      uint32_t amax = 0u;
#pragma unroll
      for (int i = 0; i < 4 * LD; ++i) {
        float x[4];
        ld_query(src + 4 * i, x);
#pragma unroll
        for (int c = 0; c < 4; ++c) amax = max(amax, finite_abs(x[c]));
      }
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      int e = (int)(amax >> 23) - 127;
      e = e < -112 ? -112 : e;             // the factors stay normal
      const float up = exp2i(14 - e);
      fac[nt] = __shfl_sync(0xffffffffu, exp2i(e - 14) * p.scale, 8 * t);   // lane 8 t has g / 2 = t
#pragma unroll
      for (int i = 0; i < 4 * LD; ++i) {
        float x[4], w[4];
        ld_query(src + 4 * i, x);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float v = has ? x[c] * up : 0.f, hi = __half2float(__float2half_rn(v));
          w[c] = (g & 1) ? v - hi : hi;
        }
        const __half2 lo2 = __floats2half2_rn(w[0], w[1]), hi2 = __floats2half2_rn(w[2], w[3]);
        b[nt][i][0] = *reinterpret_cast<const uint32_t*>(&lo2);
        b[nt][i][1] = *reinterpret_cast<const uint32_t*>(&hi2);
      }
    }
  }
  __device__ __forceinline__ void scores(const Score8Params& p, const uint8_t* st, int g, int t, float (&best)[2][2]) const {
    float acc[2][NT][4];
#pragma unroll
    for (int l = 0; l < LD; ++l) {
      uint32_t w[2][2][4];   // [tile][row g, row g + 8]
      load_rows<D>(st, g, t, l, w);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t a0 = CodeE4M3::pair(w[u][0][j], 0), a1 = CodeE4M3::pair(w[u][1][j], 0);
          const uint32_t a2 = CodeE4M3::pair(w[u][0][j], 1), a3 = CodeE4M3::pair(w[u][1][j], 1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (l == 0 && j == 0) mma_f16_0(acc[u][nt], a0, a1, a2, a3, b[nt][0][0], b[nt][0][1]);
            else mma_f16(acc[u][nt], a0, a1, a2, a3, b[nt][4 * l + j][0], b[nt][4 * l + j][1]);
          }
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        best[u][e] = t < p.G ? (acc[u][0][2 * e] + acc[u][0][2 * e + 1]) * fac[0] : -INFINITY;
        if constexpr (NT == 2) best[u][e] = max_nan(best[u][e], (acc[u][1][2 * e] + acc[u][1][2 * e + 1]) * fac[1]);
      }
  }
};

template <int D, int NT>
struct Query<CodeI8, D, NT> {     // NT = 3: column g of n-tile n is digit n (highest first) of head g
  static_assert(NT == 3, "three digits");
  static constexpr int LD = D / 64;
  uint32_t b[3][2 * LD][2];
  float fac[2];    // of heads 2 t and 2 t + 1

  __device__ __forceinline__ void load(const Score8Params& p, int bi, int h, int g, int t) {
    const bool has = g < p.G;
    const float* const src = p.qpred + ((size_t)bi * p.n_q_heads + h * p.G + (has ? g : 0)) * D + t * 16 * LD;
    uint32_t amax = 0u;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4 * LD; ++i) {
      float x[4];
      ld_query(src + 4 * i, x);
#pragma unroll
      for (int c = 0; c < 4; ++c) amax = max(amax, finite_abs(x[c], bad));
    }
    bad = bad && has;
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    int e = (int)(amax >> 23) - 127;
    e = e < -105 ? -105 : e;
    const float up = exp2i(21 - e);        // |q| up < 2^22
    const bool any_bad = __any_sync(0xffffffffu, bad);
    // an infinite or NaN channel has no digits: the head's scores become NaN
    const uint32_t bads = any_bad ? __ballot_sync(0xffffffffu, bad) : 0u;
    const float f = ((bads >> (4 * g)) & 15u) ? __uint_as_float(0x7fc00000u) : exp2i(e - 21) * p.scale;
    fac[0] = __shfl_sync(0xffffffffu, f, 8 * t);
    fac[1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
    for (int i = 0; i < 4 * LD; ++i) {     // word i: 4 channels; k-step i / 2, register i & 1
      uint32_t d[3] = {0u, 0u, 0u};
      float x[4];
      ld_query(src + 4 * i, x);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int q = has ? __float2int_rn(x[c] * up) : 0;
        const int d2 = ((q + 128) & 255) - 128, q1 = (q - d2) >> 8;
        const int d1 = ((q1 + 128) & 255) - 128, d0 = (q1 - d1) >> 8;   // |d0| <= 64
        d[0] |= ((uint32_t)d0 & 255u) << (8 * c);
        d[1] |= ((uint32_t)d1 & 255u) << (8 * c);
        d[2] |= ((uint32_t)d2 & 255u) << (8 * c);
      }
#pragma unroll
      for (int n = 0; n < 3; ++n) b[n][i >> 1][i & 1] = d[n];
    }
  }
  __device__ __forceinline__ void scores(const Score8Params& p, const uint8_t* st, int g, int t, float (&best)[2][2]) const {
    int acc[2][3][4];
#pragma unroll
    for (int l = 0; l < LD; ++l) {
      uint32_t w[2][2][4];
      load_rows<D>(st, g, t, l, w);
#pragma unroll
      for (int j = 0; j < 4; j += 2)
#pragma unroll
        for (int n = 0; n < 3; ++n)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int ks = 2 * l + j / 2;
            if (ks == 0) mma_s8_0(acc[u][n], w[u][0][j], w[u][1][j], w[u][0][j + 1], w[u][1][j + 1], b[n][ks][0], b[n][ks][1]);
            else mma_s8(acc[u][n], w[u][0][j], w[u][1][j], w[u][0][j + 1], w[u][1][j + 1], b[n][ks][0], b[n][ks][1]);
          }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e) {        // |acc| < 2^22: the lower two digits stay below 2^31
        float v[2];
#pragma unroll
        for (int c = 0; c < 2; ++c)
          v[c] = fmaf((float)acc[u][0][2 * e + c], 65536.f,
                      (float)(acc[u][1][2 * e + c] * 256 + acc[u][2][2 * e + c])) * fac[c];
        best[u][e] = 2 * t + 1 < p.G ? max_nan(v[0], v[1]) : (2 * t < p.G ? v[0] : -INFINITY);
      }
  }
};

template <int D>
struct Ring {                          // of a warp
  static constexpr int STAGES = 3;                   // at most; two where a large batch's lengths need the room
  static constexpr int ROWS = kRows * D;             // bytes of a step's rows
  static constexpr int BYTES = ROWS + 16;            // and where its tiles' scales lie
};

template <typename CT, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, 1) score8_kernel(Score8Params p) {
  using R = Ring<D>;
  const int S = p.stages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int scratch[33];
  __shared__ uint64_t bars_all[kWarps * R::STAGES];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* const ring = smem + (size_t)warp * S * R::BYTES;
  uint64_t* const bars = bars_all + warp * S;
  int* const pre = reinterpret_cast<int*>(smem + (size_t)kWarps * S * R::BYTES);
  int* const lens = pre + p.batch + 1;
  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&bars[s], 1);
    mbar_init_fence();
  }
  __syncwarp();

  pdl_wait();
  pdl_trigger();
  for (int b = threadIdx.x; b < p.batch; b += blockDim.x) {
    const int T = p.seq_lens ? p.seq_lens[b] : p.t_max;
    lens[b] = T < 0 ? 0 : (T > p.t_max ? p.t_max : T);
  }
  __syncthreads();
  cta_prefix_sum(p.batch, pre, [&](int b) { return ((lens[b] + kRows - 1) / kRows) * p.n_kv; }, scratch);

  const int total = pre[p.batch];
  // a CTA's steps follow one another and its warps take them in turn, so that it streams one
  // region (a range per warp instead: 56 us even without any arithmetic)
  const int i0 = (int)((long long)blockIdx.x * total / gridDim.x) + warp;
  const int i1 = (int)((long long)(blockIdx.x + 1) * total / gridDim.x);
  const int n = i1 > i0 ? (i1 - i0 + kWarps - 1) / kWarps : 0;
  if (n == 0) return;

  struct Cursor {
    int b, h, blk, nblk, T;
  };
  auto advance = [&](Cursor& c) {      // the warp's next step
    c.blk += kWarps;
    while (c.blk >= c.nblk) {
      c.blk -= c.nblk;
      if (++c.h == p.n_kv) {
        c.h = 0;
        do { ++c.b; } while (c.b < p.batch && pre[c.b + 1] == pre[c.b]);
        if (c.b >= p.batch) break;
        c.T = lens[c.b];
        c.nblk = (pre[c.b + 1] - pre[c.b]) / p.n_kv;
      }
    }
  };
  Cursor ic;                           // the next step to request
  {
    int lo = 0, hi = p.batch;          // pre[lo] <= i0 < pre[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= i0) lo = mid; else hi = mid;
    }
    ic.b = lo;
    ic.T = lens[lo];
    ic.nblk = (pre[lo + 1] - pre[lo]) / p.n_kv;
    const int r = i0 - pre[lo];
    ic.h = r / ic.nblk;
    ic.blk = r - ic.h * ic.nblk;
  }
  Cursor cc = ic;

  // The window: the warp's next eight steps of unit (w_b, w_h), lane l holding the row (first
  // row of the tile in k; page checked) and the scale's place for tile l % 4 of step l / 4.  The
  // next one's page numbers are requested when a window opens.
  int w_b = -1, w_h = -1, w_pos = 0, n_page = 0;
  uint32_t w_row = 0, w_srow = 0;
  constexpr int W_TILES = 8 * kWarps * kTiles;            // tiles from a window to the next
  const int l_tile = (lane / kTiles) * kWarps * kTiles + lane % kTiles;
  auto page_at = [&](const Cursor& c, int tile) -> int {   // page number of this lane's tile
    if (p.page_size == 0 || tile * 16 >= c.T) return 0;
    const uint32_t lp = p.page_magic ? __umulhi((uint32_t)tile, p.page_magic) : (uint32_t)tile;
    return __ldg(p.page_table + (size_t)c.b * p.max_pages + lp);
  };
  auto place = [&](const Cursor& c, int tile, int page, uint32_t& row, uint32_t& srow) {
    if (p.page_size == 0) {
      const uint32_t unit = (uint32_t)c.b * (uint32_t)p.n_kv + (uint32_t)c.h;
      const int j = min(tile * 16, c.T - 1);
      row = unit * (uint32_t)p.t_max + (uint32_t)j;
      srow = unit * (uint32_t)p.blocks_per_row + ((uint32_t)j >> p.block_shift);
    } else {
      if (page < 0 || page >= p.n_pages) {
        flag_status(ASP_DEV_BAD_PAGE);
        page = 0;                      // keeps the byte count; the rows' scores are not meaningful
      }
      const uint32_t lp = p.page_magic ? __umulhi((uint32_t)tile, p.page_magic) : (uint32_t)tile;
      const uint32_t in = (uint32_t)tile * 16u - lp * (uint32_t)p.page_size;
      const uint32_t head = (uint32_t)page * (uint32_t)p.n_kv + (uint32_t)c.h;
      row = head * (uint32_t)p.page_size + in;
      srow = head * (uint32_t)p.blocks_per_row + (in >> p.block_shift);
    }
  };
  const uint64_t policy = l2_evict_first_policy();
  auto issue = [&](int slot) {
    const int t0 = ic.blk * kTiles;
    if (ic.b != w_b || ic.h != w_h || w_pos == 8) {
      const bool next = ic.b == w_b && ic.h == w_h;
      w_b = ic.b;
      w_h = ic.h;
      w_pos = 0;
      place(ic, t0 + l_tile, next ? n_page : page_at(ic, t0 + l_tile), w_row, w_srow);
      n_page = page_at(ic, t0 + W_TILES + l_tile);
    }
    // lanes 0-3: a tile each
    const int u = lane & (kTiles - 1);
    const uint32_t r = __shfl_sync(0xffffffffu, w_row, w_pos * kTiles + u);
    const uint32_t sr = __shfl_sync(0xffffffffu, w_srow, w_pos * kTiles + u);
    ++w_pos;
    uint8_t* const st = ring + slot * R::BYTES;
    const int rows = ic.T - t0 * 16;   // > 0
    if (lane == 0) {
      fence_proxy_async_smem();        // the stage was read: those reads before the copies' writes
      mbar_arrive_expect_tx(&bars[slot], (uint32_t)(p.page_size ? min(kRows, (rows + 15) & ~15) : min(kRows, rows)) * D);
    }
    __syncwarp();
    if (lane < kTiles) {
      reinterpret_cast<uint32_t*>(st + R::ROWS)[lane] = sr;
      const int have = rows - 16 * lane;
      if (have > 0)
        bulk_g2s_hint(st + 16 * lane * D, p.k + (size_t)r * D, (uint32_t)(p.page_size ? 16 : min(16, have)) * D, &bars[slot],
                      policy);
    }
    __syncwarp();
    advance(ic);
  };

  int issued = 0;
  for (; issued < S && issued < n; ++issued) issue(issued);
  Query<CT, D, NT> q;
  int qb = -1, qh = -1;
  bool ok = true;
  // lane l: the scale of tile l % 4 of the next step, requested a step ahead
  auto scale_of = [&](int slot) -> float {
    return __ldg(p.k_scale + reinterpret_cast<const uint32_t*>(ring + slot * R::BYTES + R::ROWS)[lane % kTiles]);
  };
  float n_scale = scale_of(0);
#pragma unroll 1
  for (int i = 0, slot = 0, phase = 0; i < n; ++i) {
    if (cc.b != qb || cc.h != qh) {
      qb = cc.b;
      qh = cc.h;
      q.load(p, qb, qh, g, t);
    }
    ok = __all_sync(0xffffffffu, mbar_wait(&bars[slot], (uint32_t)phase));
    if (!ok) break;
    const uint8_t* const st = ring + slot * R::BYTES;
    const float sc = n_scale;
    if (i + 1 < n) n_scale = scale_of(slot + 1 == S ? 0 : slot + 1);
    float best[kTiles][2];   // [tile][row g, row g + 8] over this lane's heads
#pragma unroll
    for (int u = 0; u < kTiles; u += 2) {   // rows past the end hold an earlier step's: their scores are not written
      float two[2][2];
      q.scores(p, st + 16 * u * D, g, t, two);
      best[u][0] = two[0][0];
      best[u][1] = two[0][1];
      best[u + 1][0] = two[1][0];
      best[u + 1][1] = two[1][1];
    }
    float scale[kTiles / 2];              // of the row whose maximum the lane ends with
#pragma unroll
    for (int u = 0; u < kTiles; u += 2) scale[u / 2] = __shfl_sync(0xffffffffu, sc, u + (t >> 1));
    __syncwarp();
    if (issued < n) {
      issue(slot);
      ++issued;
    }
    const size_t row = (size_t)qb * p.n_kv + qh;
#pragma unroll
    for (int u = 0; u < kTiles; u += 2) {
      // maximum over the four lanes of a row: each lane ends with one of the four rows
      const bool up2 = t & 2, up1 = t & 1;
      float v0 = up2 ? best[u + 1][0] : best[u][0], v1 = up2 ? best[u + 1][1] : best[u][1];
      v0 = max_nan(v0, __shfl_xor_sync(0xffffffffu, up2 ? best[u][0] : best[u + 1][0], 2));
      v1 = max_nan(v1, __shfl_xor_sync(0xffffffffu, up2 ? best[u][1] : best[u + 1][1], 2));
      const float m = max_nan(up1 ? v1 : v0, __shfl_xor_sync(0xffffffffu, up1 ? v0 : v1, 1)) * scale[u / 2];
      const int j = cc.blk * kRows + 16 * u + (t >> 1) * 16 + (t & 1) * 8 + g;
      const bool has = j < cc.T;
      if (has) p.scores[row * p.t_max + j] = m;
      if (p.hist) {   // first radix pass of the selection
        const uint32_t dig = order_key(m) >> kTopShift;
        const uint32_t hm = __ballot_sync(0xffffffffu, has);
        if (has) {
          const uint32_t peers = __match_any_sync(hm, dig);
          if (lane == __ffs(peers) - 1) atomicAdd(p.hist + row * kTopBins + dig, __popc(peers));
        }
      }
    }
    advance(cc);
    if (++slot == S) {
      slot = 0;
      phase ^= 1;
    }
  }
  if (!ok) {   // a wait ran out: give the copies in flight a bounded chance to land
    for (int i = max(0, issued - S); i < issued; ++i) mbar_wait(&bars[i % S], (uint32_t)(i / S) & 1u);
  }
}

template <typename CT, int D, int NT>
cudaError_t launch_t(Score8Params p, cudaStream_t s) {
  auto kern = score8_kernel<CT, D, NT>;
  const size_t stage = (size_t)kWarps * Ring<D>::BYTES, lens = (2 * (size_t)p.batch + 1) * 4;
  constexpr size_t kRoom = 224 * 1024;   // of the 227 KB a CTA may have; the rest holds the barriers
  p.stages = Ring<D>::STAGES * stage + lens <= kRoom ? Ring<D>::STAGES : 2;
  const size_t smem = p.stages * stage + lens;
  if (prepare_kernel((const void*)kern, smem, kWarps * 32) < 1) return cudaErrorInvalidConfiguration;
  return launch_pdl(kern, dim3(sm_count()), dim3(kWarps * 32), smem, s, p);
}

template <typename CT>
cudaError_t dispatch(const Score8Params& p, int D, cudaStream_t s) {
  if constexpr (std::is_same<CT, CodeI8>::value) {
    return D == 64 ? launch_t<CT, 64, 3>(p, s) : launch_t<CT, 128, 3>(p, s);
  } else {
    if (D == 64) return p.G == 8 ? launch_t<CT, 64, 2>(p, s) : launch_t<CT, 64, 1>(p, s);
    return p.G == 8 ? launch_t<CT, 128, 2>(p, s) : launch_t<CT, 128, 1>(p, s);
  }
}

}  // namespace

cudaError_t launch_score8(const float* qpred, int n_q_heads, const KvView& kv, float* scores, cudaStream_t s,
                          int32_t* hist) {
  Score8Params p;
  p.qpred = qpred;
  p.n_q_heads = n_q_heads;
  p.G = n_q_heads / kv.n_kv;
  p.k = static_cast<const uint8_t*>(kv.k);
  p.k_scale = kv.k_scale;
  p.block_shift = kv.block_shift;
  p.blocks_per_row = kv.blocks_per_row;
  p.batch = kv.batch;
  p.n_kv = kv.n_kv;
  p.t_max = kv.t_max;
  p.page_size = kv.page_size;
  p.max_pages = kv.max_pages;
  p.n_pages = kv.n_pages;
  const int m16 = kv.page_size / 16;
  p.page_magic = m16 > 1 ? (uint32_t)(((1ull << 32) + m16 - 1) / m16) : 0u;
  p.page_table = kv.page_table;
  p.seq_lens = kv.seq_lens;
  p.scores = scores;
  p.hist = hist;
  p.scale = 1.0f / sqrtf((float)kv.head_dim);
  return kv.kv8 == 1 ? dispatch<CodeE4M3>(p, kv.head_dim, s) : dispatch<CodeI8>(p, kv.head_dim, s);
}

ASP_STATUS_READER(read_status_score8)

}  // namespace asp
