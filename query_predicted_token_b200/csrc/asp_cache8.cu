// asp_cache8.cu -- filling, reading back and appending to a KV cache held in 8 bits.
//
// Block of scale_block tokens of a KV head and side: s = smallest power of two >= 2^-100
// with max |x| <= qmax s, codes x / s (exact: s is a power of two) rounded to nearest even.
// All three are bound by HBM: every row is read once and written once.
#include "asp_internal.h"
#include "asp_kv8.cuh"

namespace asp {
namespace {

constexpr int kThreads = 256;

// Tokens of sequence b that the wide rows hold too; `flag`: this thread reports a longer one.
__device__ __forceinline__ int bounded_len(const KvView& kv, long long b, int n_tokens, bool flag) {
  int T = kv.seq_lens ? kv.seq_lens[b] : kv.t_max;
  T = T > kv.t_max ? kv.t_max : T;
  if (T > n_tokens) {
    if (flag) flag_status(ASP_DEV_ROW_LIMIT);
    T = n_tokens;
  }
  return T;
}

template <typename ST>
struct Vec;   // 16 bytes of source values as fp32
template <>
struct Vec<float> {
  static constexpr int N = 4;
  // running maximum of |x| as bits, infinities and NaN included; top() of it as fp32 bits
  __device__ __forceinline__ static void amax(uint32_t& m, const uint4& u) {
    m = max(max(m, max(u.x & 0x7fffffffu, u.y & 0x7fffffffu)), max(u.z & 0x7fffffffu, u.w & 0x7fffffffu));
  }
  __device__ __forceinline__ static uint32_t top(uint32_t m) { return m; }
  __device__ __forceinline__ static void get(const uint4& u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ __forceinline__ static void amax(uint32_t& m, const uint4& u) {   // two 16-bit maxima
    m = __vmaxu2(__vmaxu2(m, __vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu)),
                 __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
  }
  __device__ __forceinline__ static uint32_t top(uint32_t m) { return max(m << 16, m & 0xffff0000u); }
  __device__ __forceinline__ static void get(const uint4& u, float (&x)[8]) {
    float2 f[4];
    Elem<__nv_bfloat16>::unpack(u, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = f[i].x;
      x[2 * i + 1] = f[i].y;
    }
  }
};

// A scale block stays in the registers of TPB threads between its maximum and its codes:
// one pass over the source.  A thread keeps 8 vectors (2 KB blocks 4, 64 KB blocks 16), a CTA
// holds 256 / TPB blocks.  The grid is resident and a CTA requests its next block before it
// encodes the present one (but for 64 KB blocks, whose registers are full).
// Neighbouring CTAs take neighbouring KV heads, so that a [batch, token, head, channel]
// source, whose rows of one head lie apart, is still read in whole runs.
template <typename ST, typename CT, int D, int BL>
struct QuantLayout {
  static constexpr int N = Vec<ST>::N;
  static constexpr int VPR = D / N;                 // vectors of a row
  static constexpr int VB = BL * VPR;               // vectors of a block
  static constexpr int NV = VB < 256 ? 4 : (VB <= 8 * kThreads ? 8 : 16);
  static constexpr int TPB = VB / NV;               // threads of a block: 32 to 256
  static constexpr int BPC = kThreads / TPB;        // blocks of a CTA
  static constexpr bool AHEAD = NV <= 8;
  static constexpr int CTAS = NV > 4 ? 2 : 3;       // per SM
  static_assert(TPB >= 32 && TPB <= kThreads && TPB * NV == VB, "layout");
};

template <typename ST, typename CT, int D, int BL>
__global__ void __launch_bounds__(kThreads, QuantLayout<ST, CT, D, BL>::CTAS) quantize_kernel(KvView kv, const ST* __restrict__ k_src,
                                                            const ST* __restrict__ v_src, Strides3 st, int n_tokens,
                                                            int nb, long long items) {
  using L = QuantLayout<ST, CT, D, BL>;
  constexpr int N = L::N, VPR = L::VPR, NV = L::NV, TPB = L::TPB;
  __shared__ uint32_t wmax[2][kThreads / 32];
  const int sub = threadIdx.x / TPB, t = threadIdx.x % TPB, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const ST* const src = blockIdx.y ? v_src : k_src;
  uint8_t* const code = static_cast<uint8_t*>(const_cast<void*>(blockIdx.y ? kv.v : kv.k));
  float* const scale = blockIdx.y ? kv.v_scale : kv.k_scale;
  const long long stride = (long long)gridDim.x * L::BPC;
  // the thread's item as (sequence, block, head), moved on by the stride without divisions
  long long item = (long long)blockIdx.x * L::BPC + sub;
  int h = (int)(item % kv.n_kv), i = (int)(item / kv.n_kv % nb);
  long long b = item / kv.n_kv / nb;
  const int dh = (int)(stride % kv.n_kv), di = (int)(stride / kv.n_kv % nb);
  const long long db = stride / kv.n_kv / nb;

  struct Block {
    int rows;            // rows of the block that hold tokens (0: nothing to do)
    size_t row0, sidx;
    uint4 u[NV];
  };
  auto load = [&](Block& q) {
    q.rows = 0;
    if (item < items) {
      const int T = bounded_len(kv, b, n_tokens, i == 0 && t == 0);
      const int tok0 = i * BL;
      q.rows = T - tok0 > BL ? BL : (T > tok0 ? T - tok0 : 0);
      if (q.rows) {
        if (kv.page_size == 0) {
          q.row0 = ((size_t)b * kv.n_kv + h) * kv.t_max + tok0;
          q.sidx = ((size_t)b * kv.n_kv + h) * kv.blocks_per_row + i;
        } else {   // a block lies within one page
          const int page = kv.page_table[(size_t)b * kv.max_pages + tok0 / kv.page_size];
          if (page < 0 || page >= kv.n_pages) {
            if (t == 0) flag_status(ASP_DEV_BAD_PAGE);
            q.rows = 0;
          } else {
            const int r = tok0 % kv.page_size;
            q.row0 = ((size_t)page * kv.n_kv + h) * kv.page_size + r;
            q.sidx = ((size_t)page * kv.n_kv + h) * kv.blocks_per_row + r / BL;
          }
        }
      }
      const ST* const s0 = src + (size_t)b * st.batch + (size_t)h * st.head + (size_t)tok0 * st.token;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int vec = v * TPB + t, r = vec / VPR;
        q.u[v] = r < q.rows ? *reinterpret_cast<const uint4*>(s0 + (size_t)r * st.token + (vec % VPR) * N)
                            : make_uint4(0u, 0u, 0u, 0u);
      }
    }
    item += stride;
    h += dh;
    i += di;
    b += db;
    if (h >= kv.n_kv) {
      h -= kv.n_kv;
      ++i;
    }
    if (i >= nb) {
      i -= nb;
      ++b;
    }
  };

  Block cur, nxt;
  if (L::AHEAD) load(nxt);
  int turn = 0;
  for (long long base = (long long)blockIdx.x * L::BPC; base < items; base += stride, turn ^= 1) {
    if constexpr (L::AHEAD) {
      cur = nxt;
      load(nxt);
    } else {
      load(cur);
    }
    uint32_t amax = 0u;
    bool bad = false;
    if (cur.rows) {
#pragma unroll
      for (int v = 0; v < NV; ++v) Vec<ST>::amax(amax, cur.u[v]);
      amax = Vec<ST>::top(amax);
      if (amax >= 0x7f800000u) {   // an infinity or NaN among them: the finite ones again
        amax = 0u;
#pragma unroll 1
        for (int v = 0; v < NV; ++v) {
          uint4 u = cur.u[0];
#pragma unroll
          for (int k = 1; k < NV; ++k)
            if (k == v) u = cur.u[k];
          float x[N];
          Vec<ST>::get(u, x);
#pragma unroll
          for (int e = 0; e < N; ++e) amax = max(amax, finite_abs(x[e], bad));
        }
      }
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    if constexpr (TPB > 32) {   // two alternating arrays: one barrier per block
      if (lane == 0) wmax[turn][warp] = amax;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < TPB / 32; ++w) amax = max(amax, wmax[turn][sub * (TPB / 32) + w]);
    }
    if (!cur.rows) continue;
    if (bad) flag_status(ASP_DEV_NONFINITE);
    const int e = scale_exp<CT>(amax);
    const float inv = exp2i(-e);
    if (t == 0) scale[cur.sidx] = exp2i(e);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int vec = v * TPB + t, r = vec / VPR;
      if (r >= cur.rows) continue;
      float x[N];
      Vec<ST>::get(cur.u[v], x);
      uint32_t w[N / 4];
#pragma unroll
      for (int j = 0; j < N / 4; ++j)
        w[j] = CT::encode4(x[4 * j] * inv, x[4 * j + 1] * inv, x[4 * j + 2] * inv, x[4 * j + 3] * inv);
      uint8_t* const dst = code + (cur.row0 + r) * D + (vec % VPR) * N;
      if constexpr (N == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(dst) = w[0];
    }
  }
}

// UV (2 or 8) vectors of 8 codes (bf16 values) or 4 (fp32) per thread and turn, in the cache's row
// order: a warp's 16-byte stores of one turn follow one another.  (16 codes per thread, whose
// two stores leave gaps of 16 bytes: 280 us for 2 x 268 M codes into bf16.)
template <typename DT, int D, int UV>
struct DeqLayout {
  static constexpr int N = 16 / (int)sizeof(DT);   // codes per vector
  static constexpr int VPR = D / N;
  static constexpr int U = UV;
  static constexpr int ROWS = U * kThreads / VPR;  // tokens of a tile
};

template <typename DT, typename CT, int D, int UV>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(KvView kv, DT* __restrict__ k_dst,
                                                              DT* __restrict__ v_dst, Strides3 st, int n_tokens,
                                                              int tiles) {
  using L = DeqLayout<DT, D, UV>;
  constexpr int N = L::N, VPR = L::VPR, U = L::U, ROWS = L::ROWS;
  const uint8_t* const code = static_cast<const uint8_t*>(blockIdx.z ? kv.v : kv.k);
  const float* const scale = blockIdx.z ? kv.v_scale : kv.k_scale;
  DT* const dst = blockIdx.z ? v_dst : k_dst;
  // the units' first tiles come first: the CTAs past short sequences end the launch
  const int unit = blockIdx.x;
  for (int tile = blockIdx.y; tile < tiles; tile += gridDim.y) {
    const int b = unit / kv.n_kv, h = unit - b * kv.n_kv;
    const int T = bounded_len(kv, b, n_tokens, tile == 0 && threadIdx.x == 0);
    if (tile * ROWS >= T) continue;
    uint32_t u[U][N / 4];
    float s[U];
    bool ok[U];
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int vec = v * kThreads + threadIdx.x;
      const int tok = tile * ROWS + vec / VPR;
      ok[v] = tok < T;
      s[v] = 0.f;
#pragma unroll
      for (int j = 0; j < N / 4; ++j) u[v][j] = 0u;
      if (!ok[v]) continue;
      size_t row, sidx;
      if (kv.page_size == 0) {
        row = (size_t)unit * kv.t_max + tok;
        sidx = (size_t)unit * kv.blocks_per_row + (tok >> kv.block_shift);
      } else {
        const int page = kv.page_table[(size_t)b * kv.max_pages + tok / kv.page_size];
        if (page < 0 || page >= kv.n_pages) {
          flag_status(ASP_DEV_BAD_PAGE);
          ok[v] = false;
          continue;
        }
        const int r = tok % kv.page_size;
        row = ((size_t)page * kv.n_kv + h) * kv.page_size + r;
        sidx = ((size_t)page * kv.n_kv + h) * kv.blocks_per_row + (r >> kv.block_shift);
      }
      const uint8_t* const from = code + row * D + (vec % VPR) * N;
      if constexpr (N == 8) {
        const uint2 w = *reinterpret_cast<const uint2*>(from);
        u[v][0] = w.x;
        u[v][N / 4 - 1] = w.y;
      } else {
        u[v][0] = *reinterpret_cast<const uint32_t*>(from);
      }
      s[v] = scale[sidx];
    }
#pragma unroll
    for (int v = 0; v < U; ++v) {
      if (!ok[v]) continue;
      const int vec = v * kThreads + threadIdx.x;
      const int tok = tile * ROWS + vec / VPR;
      DT* const o = dst + (size_t)b * st.batch + (size_t)h * st.head + (size_t)tok * st.token + (vec % VPR) * N;
      float x[N];
#pragma unroll
      for (int j = 0; j < N / 4; ++j) {
        float y[4];
        decode4<CT>(u[v][j], y);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * j + e] = y[e] * s[v];
      }
      if constexpr (N == 4) {
        *reinterpret_cast<float4*>(o) = make_float4(x[0], x[1], x[2], x[3]);
      } else {
        uint32_t p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
          p[e] = *reinterpret_cast<const uint32_t*>(&y);
        }
        *reinterpret_cast<uint4*>(o) = make_uint4(p[0], p[1], p[2], p[3]);
      }
    }
  }
}

// One CTA per sequence, one warp per KV head and side at a time.  Every thread reads the
// length before any write.  The row's maximum, the block's scale and the codes are one
// warp's work; only a token that raises the scale touches the block's older rows.
constexpr int kAppendThreads = 512;

template <typename ST, typename CT, int D>
__global__ void __launch_bounds__(kAppendThreads) append8_kernel(KvView kv, const ST* __restrict__ k_new,
                                                                 const ST* __restrict__ v_new, int32_t* seq_lens,
                                                                 int32_t* tail_begin) {
  constexpr int PER = D / 32;                // channels per lane: 2 or 4
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  const int T = seq_lens[b];
  const int cap = kv.page_size ? min(kv.t_max, kv.max_pages * kv.page_size) : kv.t_max;
  bool fits = T >= 0 && T < cap;
  int page = 0;
  if (fits && kv.page_size) {
    page = kv.page_table[(size_t)b * kv.max_pages + T / kv.page_size];
    fits = page >= 0 && page < kv.n_pages;
  }
  if (!fits) {   // uniform over the CTA
    if (threadIdx.x == 0) flag_status(ASP_DEV_BAD_PAGE);
    return;
  }
  const int in_block = T & ((1 << kv.block_shift) - 1);   // older tokens of the block
  for (int hs = threadIdx.x >> 5; hs < 2 * kv.n_kv; hs += kAppendThreads / 32) {
    const int h = hs >> 1, side = hs & 1;
    const ST* const src = (side ? v_new : k_new) + ((size_t)b * kv.n_kv + h) * D + lane * PER;
    uint8_t* const code = static_cast<uint8_t*>(const_cast<void*>(side ? kv.v : kv.k));
    size_t row, sidx;
    if (kv.page_size == 0) {
      row = ((size_t)b * kv.n_kv + h) * kv.t_max + T;
      sidx = ((size_t)b * kv.n_kv + h) * kv.blocks_per_row + (T >> kv.block_shift);
    } else {
      const int r = T % kv.page_size;
      row = ((size_t)page * kv.n_kv + h) * kv.page_size + r;
      sidx = ((size_t)page * kv.n_kv + h) * kv.blocks_per_row + (r >> kv.block_shift);
    }
    float* const sp = (side ? kv.v_scale : kv.k_scale) + sidx;
    const float was = in_block ? *sp : 0.f;
    float x[PER];
    uint32_t amax = 0u;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      x[e] = Elem<ST>::load(src + e);
      amax = max(amax, finite_abs(x[e], bad));
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    if (bad) flag_status(ASP_DEV_NONFINITE);
    const int e = scale_exp<CT>(amax);
    const float need = exp2i(e);
    const bool raise = in_block && __uint_as_float(amax) > CT::kMax * was;   // the row does not fit
    // the codes: x / scale, exact for the powers of two the library writes
    float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < PER; ++j) y[j] = in_block && !raise ? x[j] / was : x[j] * exp2i(-e);
    const uint32_t w = CT::encode4(y[0], y[1], y[2], y[3]);
    uint8_t* const dst = code + row * D + lane * PER;
    if constexpr (PER == 4) *reinterpret_cast<uint32_t*>(dst) = w;
    else *reinterpret_cast<unsigned short*>(dst) = (unsigned short)w;
    if (raise) {   // the older rows again, at the new scale
      const float f = was * exp2i(-e);   // < 1
      uint32_t* const old = reinterpret_cast<uint32_t*>(code + (row - in_block) * D);
      const int words = in_block * (D / 4);
      for (int i = lane; i < words; i += 32) {
        float z[4];
        decode4<CT>(old[i], z);
        old[i] = CT::encode4(z[0] * f, z[1] * f, z[2] * f, z[3] * f);
      }
    }
    if (lane == 0 && (raise || !in_block)) *sp = need;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    if (tail_begin) tail_begin[b] = T;
    seq_lens[b] = T + 1;
  }
}

template <typename ST, typename CT, int D, int BL>
cudaError_t quantize_t(const KvView& kv, const void* k, const void* v, int n, Strides3 st, cudaStream_t s) {
  constexpr int BPC = QuantLayout<ST, CT, D, BL>::BPC;
  const int nb = (n + BL - 1) / BL;
  const long long items = (long long)kv.batch * nb * kv.n_kv;
  const long long ctas = (items + BPC - 1) / BPC;
  auto kern = quantize_kernel<ST, CT, D, BL>;
  const int per_sm = prepare_kernel((const void*)kern, 0, kThreads);
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  const long long most = ((long long)sm_count() * per_sm + 1) / 2;   // of each side
  kern<<<dim3((unsigned)(ctas < most ? ctas : most), 2), kThreads, 0, s>>>(kv, static_cast<const ST*>(k),
                                                                           static_cast<const ST*>(v), st, n, nb,
                                                                           items);
  return cudaGetLastError();
}

template <typename ST, typename CT, int D>
cudaError_t quantize_b(const KvView& kv, const void* k, const void* v, int n, Strides3 st, cudaStream_t s) {
  switch (kv.block_shift) {
    case 4: return quantize_t<ST, CT, D, 16>(kv, k, v, n, st, s);
    case 5: return quantize_t<ST, CT, D, 32>(kv, k, v, n, st, s);
    case 6: return quantize_t<ST, CT, D, 64>(kv, k, v, n, st, s);
    case 7: return quantize_t<ST, CT, D, 128>(kv, k, v, n, st, s);
    default: return cudaErrorInvalidValue;
  }
}

template <typename ST, typename CT>
cudaError_t quantize_d(const KvView& kv, const void* k, const void* v, int n, Strides3 st, cudaStream_t s) {
  return kv.head_dim == 64 ? quantize_b<ST, CT, 64>(kv, k, v, n, st, s) : quantize_b<ST, CT, 128>(kv, k, v, n, st, s);
}

template <typename DT, typename CT, int D, int UV>
cudaError_t dequantize_u(const KvView& kv, void* k, void* v, int n, Strides3 st, cudaStream_t s) {
  constexpr int ROWS = DeqLayout<DT, D, UV>::ROWS;
  const int tiles = (n + ROWS - 1) / ROWS;
  dequantize_kernel<DT, CT, D, UV><<<dim3(kv.batch * kv.n_kv, tiles < 65535 ? tiles : 65535, 2), kThreads, 0, s>>>(
      kv, static_cast<DT*>(k), static_cast<DT*>(v), st, n, tiles);
  return cudaGetLastError();
}

// Caches that would not fill the SMs with 8 vectors per thread take 2 (2 x 512 tokens, d = 64:
// 2.9 against 4.4 us).
template <typename DT, typename CT, int D>
cudaError_t dequantize_t(const KvView& kv, void* k, void* v, int n, Strides3 st, cudaStream_t s) {
  constexpr int ROWS = DeqLayout<DT, D, 8>::ROWS;
  const long long ctas = 2LL * kv.batch * kv.n_kv * ((n + ROWS - 1) / ROWS);
  return ctas < sm_count() ? dequantize_u<DT, CT, D, 2>(kv, k, v, n, st, s) : dequantize_u<DT, CT, D, 8>(kv, k, v, n, st, s);
}

template <typename DT, typename CT>
cudaError_t dequantize_d(const KvView& kv, void* k, void* v, int n, Strides3 st, cudaStream_t s) {
  return kv.head_dim == 64 ? dequantize_t<DT, CT, 64>(kv, k, v, n, st, s) : dequantize_t<DT, CT, 128>(kv, k, v, n, st, s);
}

template <typename ST, typename CT>
cudaError_t append8_d(const KvView& kv, const void* k, const void* v, int32_t* lens, int32_t* tail, cudaStream_t s) {
  if (kv.head_dim == 64)
    append8_kernel<ST, CT, 64><<<kv.batch, kAppendThreads, 0, s>>>(kv, static_cast<const ST*>(k),
                                                                   static_cast<const ST*>(v), lens, tail);
  else
    append8_kernel<ST, CT, 128><<<kv.batch, kAppendThreads, 0, s>>>(kv, static_cast<const ST*>(k),
                                                                    static_cast<const ST*>(v), lens, tail);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize(const KvView& kv, const void* k_src, const void* v_src, int src_f32, int n_tokens,
                            Strides3 st, cudaStream_t s) {
  if (kv.kv8 == 1)
    return src_f32 ? quantize_d<float, CodeE4M3>(kv, k_src, v_src, n_tokens, st, s)
                   : quantize_d<__nv_bfloat16, CodeE4M3>(kv, k_src, v_src, n_tokens, st, s);
  return src_f32 ? quantize_d<float, CodeI8>(kv, k_src, v_src, n_tokens, st, s)
                 : quantize_d<__nv_bfloat16, CodeI8>(kv, k_src, v_src, n_tokens, st, s);
}

cudaError_t launch_dequantize(const KvView& kv, void* k_dst, void* v_dst, int dst_f32, int n_tokens, Strides3 st,
                              cudaStream_t s) {
  if (kv.kv8 == 1)
    return dst_f32 ? dequantize_d<float, CodeE4M3>(kv, k_dst, v_dst, n_tokens, st, s)
                   : dequantize_d<__nv_bfloat16, CodeE4M3>(kv, k_dst, v_dst, n_tokens, st, s);
  return dst_f32 ? dequantize_d<float, CodeI8>(kv, k_dst, v_dst, n_tokens, st, s)
                 : dequantize_d<__nv_bfloat16, CodeI8>(kv, k_dst, v_dst, n_tokens, st, s);
}

cudaError_t launch_append8(const KvView& kv, const void* k_new, const void* v_new, int src_f32, int32_t* seq_lens,
                           int32_t* tail_begin, cudaStream_t s) {
  if (kv.kv8 == 1)
    return src_f32 ? append8_d<float, CodeE4M3>(kv, k_new, v_new, seq_lens, tail_begin, s)
                   : append8_d<__nv_bfloat16, CodeE4M3>(kv, k_new, v_new, seq_lens, tail_begin, s);
  return src_f32 ? append8_d<float, CodeI8>(kv, k_new, v_new, seq_lens, tail_begin, s)
                 : append8_d<__nv_bfloat16, CodeI8>(kv, k_new, v_new, seq_lens, tail_begin, s);
}

ASP_STATUS_READER(read_status_cache8)

}  // namespace asp
