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

template <typename ST>
struct Vec;   // 16 bytes of source values as fp32
template <>
struct Vec<float> {
  static constexpr int N = 4;
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
// one pass over the source.  Blocks of up to 16 KB keep 4 vectors per thread in flight
// (larger ones 8 or 16), a CTA holds 256 / TPB blocks.  Neighbouring blocks are those of
// the next KV head, so that a [batch, token, head, channel] source, whose rows of one head
// lie apart, is still read in whole runs.
template <typename ST, typename CT, int D, int BL>
__global__ void __launch_bounds__(kThreads) quantize_kernel(KvView kv, const ST* __restrict__ k_src,
                                                            const ST* __restrict__ v_src, Strides3 st, int nb,
                                                            long long items) {
  constexpr int N = Vec<ST>::N;
  constexpr int VPR = D / N;                 // vectors of a row
  constexpr int VB = BL * VPR;               // vectors of a block
  constexpr int NV = VB <= 4 * kThreads ? 4 : VB / kThreads;
  constexpr int TPB = VB / NV;               // threads of a block: 32 to 256
  constexpr int BPC = kThreads / TPB;        // blocks of a CTA
  static_assert(TPB >= 32 && TPB <= kThreads && TPB * NV == VB, "layout");
  __shared__ uint32_t wmax[2][kThreads / 32];
  const int sub = threadIdx.x / TPB, t = threadIdx.x % TPB, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const ST* const src = blockIdx.y ? v_src : k_src;
  uint8_t* const code = static_cast<uint8_t*>(const_cast<void*>(blockIdx.y ? kv.v : kv.k));
  float* const scale = blockIdx.y ? kv.v_scale : kv.k_scale;
  const int stride = gridDim.x * BPC;
  int turn = 0;
  for (long long base = (long long)blockIdx.x * BPC; base < items; base += stride, turn ^= 1) {
    const long long item = base + sub;
    const int h = (int)(item % kv.n_kv);
    const long long bi = item / kv.n_kv;
    const int i = (int)(bi % nb), b = (int)(bi / nb);
    int T = 0;
    if (item < items) {
      T = kv.seq_lens ? kv.seq_lens[b] : kv.t_max;
      T = T > kv.t_max ? kv.t_max : T;
    }
    const int tok0 = i * BL;
    bool live = tok0 < T;
    size_t row0 = 0, sidx = 0;
    if (live) {
      if (kv.page_size == 0) {
        row0 = ((size_t)b * kv.n_kv + h) * kv.t_max + tok0;
        sidx = ((size_t)b * kv.n_kv + h) * kv.blocks_per_row + i;
      } else {   // a block lies within one page
        const int page = kv.page_table[(size_t)b * kv.max_pages + tok0 / kv.page_size];
        if (page < 0 || page >= kv.n_pages) {
          if (t == 0) flag_status(ASP_DEV_BAD_PAGE);
          live = false;
        } else {
          const int r = tok0 % kv.page_size;
          row0 = ((size_t)page * kv.n_kv + h) * kv.page_size + r;
          sidx = ((size_t)page * kv.n_kv + h) * kv.blocks_per_row + r / BL;
        }
      }
    }
    uint4 u[NV];
    const ST* const s0 = src + (size_t)b * st.batch + (size_t)h * st.head;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int vec = v * TPB + t, r = vec / VPR;
      u[v] = live && tok0 + r < T
                 ? *reinterpret_cast<const uint4*>(s0 + (size_t)(tok0 + r) * st.token + (vec % VPR) * N)
                 : make_uint4(0u, 0u, 0u, 0u);
    }
    uint32_t amax = 0u;
    bool bad = false;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float x[N];
      Vec<ST>::get(u[v], x);
#pragma unroll
      for (int e = 0; e < N; ++e) amax = max(amax, finite_abs(x[e], bad));
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    if constexpr (TPB > 32) {   // two alternating arrays: one barrier per block
      if (lane == 0) wmax[turn][warp] = amax;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < TPB / 32; ++w) amax = max(amax, wmax[turn][sub * (TPB / 32) + w]);
    }
    if (!live) continue;
    if (bad) flag_status(ASP_DEV_NONFINITE);
    const int e = scale_exp<CT>(amax);
    const float inv = exp2i(-e);
    if (t == 0) scale[sidx] = exp2i(e);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int vec = v * TPB + t, r = vec / VPR;
      if (tok0 + r >= T) continue;
      float x[N];
      Vec<ST>::get(u[v], x);
      uint32_t w[N / 4];
#pragma unroll
      for (int j = 0; j < N / 4; ++j)
        w[j] = CT::encode4(x[4 * j] * inv, x[4 * j + 1] * inv, x[4 * j + 2] * inv, x[4 * j + 3] * inv);
      uint8_t* const dst = code + (row0 + r) * D + (vec % VPR) * N;
      if constexpr (N == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(dst) = w[0];
    }
  }
}

// Four vectors of 16 codes per thread and turn, in the cache's row order.
template <typename DT, typename CT, int D>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(KvView kv, DT* __restrict__ k_dst,
                                                              DT* __restrict__ v_dst, Strides3 st, int tiles) {
  constexpr int VPR = D / 16;
  constexpr int U = 4;
  constexpr int ROWS = U * kThreads / VPR;   // tokens of a tile
  const uint8_t* const code = static_cast<const uint8_t*>(blockIdx.y ? kv.v : kv.k);
  const float* const scale = blockIdx.y ? kv.v_scale : kv.k_scale;
  DT* const dst = blockIdx.y ? v_dst : k_dst;
  const long long items = (long long)kv.batch * kv.n_kv * tiles;
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const int unit = (int)(item / tiles), tile = (int)(item - (long long)unit * tiles);
    const int b = unit / kv.n_kv, h = unit - b * kv.n_kv;
    int T = kv.seq_lens ? kv.seq_lens[b] : kv.t_max;
    T = T > kv.t_max ? kv.t_max : T;
    if (tile * ROWS >= T) continue;
    uint4 u[U];
    float s[U];
    bool ok[U];
#pragma unroll
    for (int v = 0; v < U; ++v) {
      const int vec = v * kThreads + threadIdx.x;
      const int tok = tile * ROWS + vec / VPR;
      ok[v] = tok < T;
      s[v] = 0.f;
      u[v] = make_uint4(0u, 0u, 0u, 0u);
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
      u[v] = *reinterpret_cast<const uint4*>(code + row * D + (vec % VPR) * 16);
      s[v] = scale[sidx];
    }
#pragma unroll
    for (int v = 0; v < U; ++v) {
      if (!ok[v]) continue;
      const int vec = v * kThreads + threadIdx.x;
      const int tok = tile * ROWS + vec / VPR;
      DT* const o = dst + (size_t)b * st.batch + (size_t)h * st.head + (size_t)tok * st.token + (vec % VPR) * 16;
      const uint32_t w[4] = {u[v].x, u[v].y, u[v].z, u[v].w};
      float x[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float y[4];
        decode4<CT>(w[j], y);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * j + e] = y[e] * s[v];
      }
      if constexpr (sizeof(DT) == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          reinterpret_cast<float4*>(o)[j] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 y = __floats2bfloat162_rn(x[8 * j + 2 * e], x[8 * j + 2 * e + 1]);
            p[e] = *reinterpret_cast<const uint32_t*>(&y);
          }
          reinterpret_cast<uint4*>(o)[j] = make_uint4(p[0], p[1], p[2], p[3]);
        }
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
    const bool raise = in_block && need > was;
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
cudaError_t quantize_t(const KvView& kv, const void* k, const void* v, Strides3 st, cudaStream_t s) {
  constexpr int VB = BL * D / Vec<ST>::N;
  constexpr int NV = VB <= 4 * kThreads ? 4 : VB / kThreads;
  constexpr int BPC = kThreads / (VB / NV);
  const int nb = (kv.t_max + BL - 1) / BL;
  const long long items = (long long)kv.batch * nb * kv.n_kv;
  const long long ctas = (items + BPC - 1) / BPC;
  const int grid = (int)(ctas < (1 << 22) ? ctas : (1 << 22));
  quantize_kernel<ST, CT, D, BL><<<dim3(grid, 2), kThreads, 0, s>>>(kv, static_cast<const ST*>(k),
                                                                    static_cast<const ST*>(v), st, nb, items);
  return cudaGetLastError();
}

template <typename ST, typename CT, int D>
cudaError_t quantize_b(const KvView& kv, const void* k, const void* v, Strides3 st, cudaStream_t s) {
  switch (kv.block_shift) {
    case 4: return quantize_t<ST, CT, D, 16>(kv, k, v, st, s);
    case 5: return quantize_t<ST, CT, D, 32>(kv, k, v, st, s);
    case 6: return quantize_t<ST, CT, D, 64>(kv, k, v, st, s);
    case 7: return quantize_t<ST, CT, D, 128>(kv, k, v, st, s);
    default: return cudaErrorInvalidValue;
  }
}

template <typename ST, typename CT>
cudaError_t quantize_d(const KvView& kv, const void* k, const void* v, Strides3 st, cudaStream_t s) {
  return kv.head_dim == 64 ? quantize_b<ST, CT, 64>(kv, k, v, st, s) : quantize_b<ST, CT, 128>(kv, k, v, st, s);
}

template <typename DT, typename CT, int D>
cudaError_t dequantize_t(const KvView& kv, void* k, void* v, Strides3 st, cudaStream_t s) {
  constexpr int ROWS = 4 * kThreads / (D / 16);
  const int tiles = (kv.t_max + ROWS - 1) / ROWS;
  const long long items = (long long)kv.batch * kv.n_kv * tiles;
  const int grid = (int)(items < (1 << 22) ? items : (1 << 22));
  dequantize_kernel<DT, CT, D><<<dim3(grid, 2), kThreads, 0, s>>>(kv, static_cast<DT*>(k), static_cast<DT*>(v), st, tiles);
  return cudaGetLastError();
}

template <typename DT, typename CT>
cudaError_t dequantize_d(const KvView& kv, void* k, void* v, Strides3 st, cudaStream_t s) {
  return kv.head_dim == 64 ? dequantize_t<DT, CT, 64>(kv, k, v, st, s) : dequantize_t<DT, CT, 128>(kv, k, v, st, s);
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

cudaError_t launch_quantize(const KvView& kv, const void* k_src, const void* v_src, int src_f32, Strides3 st,
                            cudaStream_t s) {
  if (kv.kv8 == 1)
    return src_f32 ? quantize_d<float, CodeE4M3>(kv, k_src, v_src, st, s)
                   : quantize_d<__nv_bfloat16, CodeE4M3>(kv, k_src, v_src, st, s);
  return src_f32 ? quantize_d<float, CodeI8>(kv, k_src, v_src, st, s)
                 : quantize_d<__nv_bfloat16, CodeI8>(kv, k_src, v_src, st, s);
}

cudaError_t launch_dequantize(const KvView& kv, void* k_dst, void* v_dst, int dst_f32, Strides3 st, cudaStream_t s) {
  if (kv.kv8 == 1)
    return dst_f32 ? dequantize_d<float, CodeE4M3>(kv, k_dst, v_dst, st, s)
                   : dequantize_d<__nv_bfloat16, CodeE4M3>(kv, k_dst, v_dst, st, s);
  return dst_f32 ? dequantize_d<float, CodeI8>(kv, k_dst, v_dst, st, s)
                 : dequantize_d<__nv_bfloat16, CodeI8>(kv, k_dst, v_dst, st, s);
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
