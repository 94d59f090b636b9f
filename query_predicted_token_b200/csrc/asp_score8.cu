// asp_score8.cu -- step 2 over keys held in 8 bits.
//
// scores[b, h, j] = max_g (qpred[b, h*G+g] . code_j) * scale_j / sqrt(d): one read of every
// key row (128 + 4 / scale_block bytes for d = 128) and 4 bytes written, bound by HBM.
//
// A warp takes 32 rows at a time from global memory straight into the registers that feed
// mma.m16n8k16: lane (g, t) = (lane / 4, lane % 4) loads 16-byte pieces of rows g and g + 8
// of a 16-row tile, which are its A fragments once each pair of codes is widened to fp16
// (exact); the order in which channels meet the k index is the same for both operands and
// otherwise free.  Every lane has the next 32 rows' loads in flight while it computes.
// The query, scaled by a power of two so that its largest channel lies in [2^14, 2^15), is
// split into two fp16 parts (22 bits) that fill neighbouring columns of B: 4 query heads
// are one n-tile of 8.  Every product is exact in the fp32 accumulator.
#include "asp_internal.h"
#include "asp_kv8.cuh"

namespace asp {
namespace {

constexpr int kRows = 32;      // rows of a warp's step: two 16-row tiles
constexpr int kWarps = 8;

struct Score8Params {
  const float* qpred;
  int n_q_heads, G;
  const uint8_t* k;
  const float* k_scale;
  int block_shift, blocks_per_row;
  int batch, n_kv, t_max, page_size, max_pages, n_pages;
  const int32_t* page_table;
  const int32_t* seq_lens;
  float* scores;
  int32_t* hist;
  float scale;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Read once: no line of it is kept in L1.
__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <typename CT, int D, int NT>   // NT: n-tiles of 4 query heads (G <= 4: 1, G = 8: 2)
__global__ void __launch_bounds__(kWarps * 32, 2) score8_kernel(Score8Params p) {
  constexpr int LD = D / 64;           // 16-byte pieces of a row per lane
  extern __shared__ int pre[];
  __shared__ int scratch[33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  int* const lens = pre + p.batch + 1;

  pdl_wait();
  pdl_trigger();
  for (int b = threadIdx.x; b < p.batch; b += blockDim.x) {
    const int T = p.seq_lens ? p.seq_lens[b] : p.t_max;
    lens[b] = T < 0 ? 0 : (T > p.t_max ? p.t_max : T);
  }
  __syncthreads();
  cta_prefix_sum(p.batch, pre, [&](int b) { return ((lens[b] + kRows - 1) / kRows) * p.n_kv; }, scratch);

  const int total = pre[p.batch];
  const int nw = gridDim.x * kWarps, gw = blockIdx.x * kWarps + warp;
  const int i0 = (int)((long long)gw * total / nw), i1 = (int)((long long)(gw + 1) * total / nw);
  if (i0 >= i1) return;

  struct Cursor {
    int b, h, blk, nblk, T;
  };
  auto advance = [&](Cursor& c) {
    if (++c.blk == c.nblk) {
      c.blk = 0;
      if (++c.h == p.n_kv) {
        c.h = 0;
        do { ++c.b; } while (c.b < p.batch && pre[c.b + 1] == pre[c.b]);
        if (c.b < p.batch) {
          c.T = lens[c.b];
          c.nblk = (pre[c.b + 1] - pre[c.b]) / p.n_kv;
        }
      }
    }
  };
  Cursor ic;
  {
    int lo = 0, hi = p.batch;   // pre[lo] <= i0 < pre[hi]
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

  int pt_b = -1, pt_base = 0, pt_val = -1, pt_next = -1;   // table window: entry pt_base + lane of row pt_b

  uint4 kreg[2][2][LD];   // [tile][row g, row g + 8]: the rows in flight
  float ks[2];
  auto load = [&](const Cursor& c) {
    const int j0 = c.blk * kRows;
    if (p.page_size) {
      const int lp = j0 / p.page_size, lpe = (j0 + 16) / p.page_size;
      if (c.b != pt_b || lp < pt_base || lpe >= pt_base + 32) {
        if (c.b == pt_b && lp == pt_base + 32) {
          pt_val = pt_next;
        } else {
          pt_val = lp + lane < p.max_pages ? __ldg(p.page_table + (size_t)c.b * p.max_pages + lp + lane) : -1;
        }
        pt_b = c.b;
        pt_base = lp;
        pt_next = lp + 32 + lane < p.max_pages ? __ldg(p.page_table + (size_t)c.b * p.max_pages + lp + 32 + lane) : -1;
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int j = j0 + 16 * u;
      size_t row, sidx;
      bool ok = j < c.T;   // uniform over the warp
      if (p.page_size == 0) {
        const size_t unit = (size_t)c.b * p.n_kv + c.h;
        row = unit * p.t_max + j;
        sidx = unit * p.blocks_per_row + (j >> p.block_shift);
      } else {
        const int lp = j / p.page_size, r = j - lp * p.page_size;
        const int page = __shfl_sync(0xffffffffu, pt_val, (lp - pt_base) & 31);
        if (ok && (page < 0 || page >= p.n_pages)) {
          if (lane == 0) flag_status(ASP_DEV_BAD_PAGE);
          ok = false;   // zeros: the rows' scores are not meaningful
        }
        const size_t ph = (size_t)page * p.n_kv + c.h;
        row = ph * p.page_size + r;
        sidx = ph * p.blocks_per_row + (r >> p.block_shift);
      }
      ks[u] = ok ? __ldg(p.k_scale + sidx) : 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint8_t* src = p.k + (row + g + 8 * e) * D + t * 16;
        const bool has = ok && j + g + 8 * e < c.T;
#pragma unroll
        for (int i = 0; i < LD; ++i) kreg[u][e][i] = has ? ld_stream(src + 64 * i) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  };

  // query fragments of the group: column g of n-tile nt is part g & 1 of head 4 nt + g / 2
  uint32_t qb[NT][4 * LD][2];
  float fac[NT];   // of head 4 nt + t: undoes the power of two, times 1 / sqrt(d)
  auto load_q = [&](int b, int h) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int head = 4 * nt + (g >> 1);
      float4 x[4 * LD];
      uint32_t amax = 0u;
#pragma unroll
      for (int i = 0; i < 4 * LD; ++i) {
        const float* src = p.qpred + ((size_t)b * p.n_q_heads + h * p.G + head) * D + (i >> 2) * 64 + t * 16 + (i & 3) * 4;
        x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (head < p.G) x[i] = make_float4(src[0], src[1], src[2], src[3]);
        bool bad = false;
        amax = max(max(amax, finite_abs(x[i].x, bad)), max(finite_abs(x[i].y, bad), max(finite_abs(x[i].z, bad),
                                                                                          finite_abs(x[i].w, bad))));
      }
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // up: 2^(14 - exponent), within the normal range (a query below 2^-112 keeps fewer bits)
      int e = (int)(amax >> 23) - 127;
      e = e < -112 ? -112 : e;
      const float up = exp2i(14 - e);
      const float f = exp2i(e - 14 < -126 ? -126 : e - 14) * p.scale;
      fac[nt] = __shfl_sync(0xffffffffu, f, 8 * t);   // lane 8 t has g / 2 = t
#pragma unroll
      for (int i = 0; i < 4 * LD; ++i) {
        const float v[4] = {x[i].x * up, x[i].y * up, x[i].z * up, x[i].w * up};
        float w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float hi = __half2float(__float2half_rn(v[c]));
          w[c] = (g & 1) ? v[c] - hi : hi;
        }
        const __half2 lo2 = __floats2half2_rn(w[0], w[1]), hi2 = __floats2half2_rn(w[2], w[3]);
        qb[nt][i][0] = *reinterpret_cast<const uint32_t*>(&lo2);
        qb[nt][i][1] = *reinterpret_cast<const uint32_t*>(&hi2);
      }
    }
  };

  load(ic);
  advance(ic);
  int qu = -1;
#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
    if (cc.b * p.n_kv + cc.h != qu) {
      qu = cc.b * p.n_kv + cc.h;
      load_q(cc.b, cc.h);
    }
    uint4 kc[2][2][LD];
    const float sc[2] = {ks[0], ks[1]};
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int l = 0; l < LD; ++l) kc[u][e][l] = kreg[u][e][l];
    if (i + 1 < i1) {
      load(ic);
      advance(ic);
    }
    float best[2][2];   // [tile][row g, row g + 8] of head t (then t + 4)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float acc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
      for (int l = 0; l < LD; ++l) {
        const uint32_t w0[4] = {kc[u][0][l].x, kc[u][0][l].y, kc[u][0][l].z, kc[u][0][l].w};
        const uint32_t w1[4] = {kc[u][1][l].x, kc[u][1][l].y, kc[u][1][l].z, kc[u][1][l].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x0 = CT::prep(w0[j]), x1 = CT::prep(w1[j]);
          const uint32_t a0 = CT::pair(x0, 0), a2 = CT::pair(x0, 1), a1 = CT::pair(x1, 0), a3 = CT::pair(x1, 1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt], a0, a1, a2, a3, qb[nt][4 * l + j][0], qb[nt][4 * l + j][1]);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float m = t < p.G ? (acc[0][2 * e] + acc[0][2 * e + 1]) * fac[0] : -INFINITY;
        if constexpr (NT == 2) m = fmaxf(m, (acc[1][2 * e] + acc[1][2 * e + 1]) * fac[1]);
        best[u][e] = m;
      }
    }
    // maximum over the four lanes of a row: each lane ends with one of the four rows
    const bool up2 = t & 2, up1 = t & 1;
    float v0 = up2 ? best[1][0] : best[0][0], v1 = up2 ? best[1][1] : best[0][1];
    v0 = fmaxf(v0, __shfl_xor_sync(0xffffffffu, up2 ? best[0][0] : best[1][0], 2));
    v1 = fmaxf(v1, __shfl_xor_sync(0xffffffffu, up2 ? best[0][1] : best[1][1], 2));
    const float m = fmaxf(up1 ? v1 : v0, __shfl_xor_sync(0xffffffffu, up1 ? v0 : v1, 1)) * (up2 ? sc[1] : sc[0]);
    const int j = cc.blk * kRows + (t >> 1) * 16 + (t & 1) * 8 + g;
    const bool has = j < cc.T;
    if (has) p.scores[(size_t)qu * p.t_max + j] = m;
    if (p.hist) {   // first radix pass of the selection
      const uint32_t dig = order_key(m) >> kTopShift;
      const uint32_t hm = __ballot_sync(0xffffffffu, has);
      if (has) {
        const uint32_t peers = __match_any_sync(hm, dig);
        if (lane == __ffs(peers) - 1) atomicAdd(p.hist + (size_t)qu * kTopBins + dig, __popc(peers));
      }
    }
    advance(cc);
  }
}

template <typename CT, int D, int NT>
cudaError_t launch_t(const Score8Params& p, cudaStream_t s) {
  auto kern = score8_kernel<CT, D, NT>;
  const size_t smem = (2 * (size_t)p.batch + 1) * 4;
  const int per_sm = prepare_kernel((const void*)kern, smem, kWarps * 32);
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  return launch_pdl(kern, dim3(sm_count() * (per_sm < 2 ? per_sm : 2)), dim3(kWarps * 32), smem, s, p);
}

template <typename CT>
cudaError_t dispatch(const Score8Params& p, int D, cudaStream_t s) {
  if (D == 64) return p.G == 8 ? launch_t<CT, 64, 2>(p, s) : launch_t<CT, 64, 1>(p, s);
  return p.G == 8 ? launch_t<CT, 128, 2>(p, s) : launch_t<CT, 128, 1>(p, s);
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
  p.page_table = kv.page_table;
  p.seq_lens = kv.seq_lens;
  p.scores = scores;
  p.hist = hist;
  p.scale = 1.0f / sqrtf((float)kv.head_dim);
  return kv.kv8 == 1 ? dispatch<CodeE4M3>(p, kv.head_dim, s) : dispatch<CodeI8>(p, kv.head_dim, s);
}

ASP_STATUS_READER(read_status_score8)

}  // namespace asp
