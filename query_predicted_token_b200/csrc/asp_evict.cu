// asp_evict.cu -- eviction to a budget: the kept rows moved to the front, in place.
//
// A selection kernel chooses C tokens per row of sums, ascending, and leaves the row's length.
// Row i of the front comes from position idx[i] >= i.  One CTA takes one side (K or V) of a
// (sequence, KV head) and moves its rows in ascending chunks: a chunk's rows are all read,
// then (after a barrier) all written, and the next chunk's reads are already in flight.
// That is safe in place: a chunk writes rows below (k + 1) n, later chunks read rows at or
// above their own, and earlier chunks are read before.  Bound by HBM; each kept row is read
// and written once.  8-bit caches: the rows of a new scale block meet in a shared-memory
// maximum and are encoded again at their own scale.
#include <type_traits>

#include "asp_internal.h"
#include "asp_kv8.cuh"

namespace asp {
namespace {

constexpr int kThreads = 1024;
constexpr int kVecs = 4;                 // 16-byte vectors per thread and chunk: 64 KB
constexpr int kBlocks = 64;              // scale blocks of a chunk, at most

struct MoveParams {
  KvView kv;
  EvictArgs a;
  int32_t* seq_lens;
  uint32_t page_magic;   // 2^32 / (page_size / 16), rounded up; 0 for pages of 16
};

// ---- the choice, for rows of up to 32K sums ----------------------------------------------
//
// One CTA per row, every key in a register: thread t holds the run [t KPT, (t + 1) KPT).  The
// threshold (the C-th largest key, less the sinks and recents) is found from the top, 11, 11
// and 10 bits at a time: shared-memory counts of the digit over the keys that still match,
// and a scan of the counts; the search stops when a digit's keys are all wanted.  Then one
// scan of (above, at) counts gives every thread its output position; ties go to the lowest
// index.  The sums of the kept tokens are written from the registers, in place or not.  The
// radix select of asp_select.cu, built for rows that arrive with a histogram, took 18.5 us
// for 64 rows of 8192 sums; counting candidate thresholds bit by bit, without a histogram,
// 13 us.
constexpr int kSelThreads = 1024;
constexpr int kSelMaxKeys = 32 * kSelThreads;

// The float an order key stands for (see order_key; -0 comes back as +0).
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

template <int KPT>
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(SelectArgs a, float* acc_out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x, b = row / a.rows_per_seq, C = a.c_units;
  __shared__ int hist[kTopBins];
  __shared__ uint32_t wsum[32];
  __shared__ int res[3];
  static_assert(kTopBins == 2 * kSelThreads, "two bins per thread");
  pdl_wait();
  int T = a.seq_lens[b];
  T = T < 0 ? 0 : (T > a.t_max ? a.t_max : T);
  int32_t* const out = a.idx + (size_t)row * C;
  const float* const src = a.scores + (size_t)row * a.row_stride;
  float* const dst = acc_out + (size_t)row * a.row_stride;
  if (tid == 0) {
    a.keep_len[row] = T;
    a.count[row] = T < C ? T : C;
  }
  if (T <= C) {
    for (int i = tid; i < C; i += kSelThreads) out[i] = i < T ? i : -1;
    for (int i = tid; i < a.t_max; i += kSelThreads) dst[i] = i < T ? src[i] : 0.f;
    return;
  }
  const int i0 = tid * KPT;
  const bool vec = (a.row_stride & 3) == 0 && (reinterpret_cast<uintptr_t>(a.scores) & 15) == 0;
  uint32_t key[KPT];                     // 0 past the row and for sinks and recents
  uint32_t forced = 0u;                  // bit k: key k is a sink or a recent
  bool nan = false;
#pragma unroll
  for (int k = 0; k < KPT; k += 4) {
    const int i = i0 + k;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (vec && i < T) {   // the last vector stays inside the row
      const float4 f = *reinterpret_cast<const float4*>(src + i);
      v[0] = f.x;
      v[1] = f.y;
      v[2] = f.z;
      v[3] = f.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < T) v[e] = src[i + e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool in = i + e < T, must = in && (i + e < a.n_sink || i + e >= T - a.n_recent);
      nan |= in && isnan(v[e]);
      if (must) forced |= 1u << (k + e);
      key[k + e] = in && !must ? order_key(v[e]) : 0u;
    }
  }
  if (__syncthreads_or(nan) && tid == 0) flag_status(ASP_DEV_NAN_SCORE);

  int want = C - a.n_sink - a.n_recent;  // of the others; T > C: sinks and recents do not meet
  uint32_t th = 0u, mask = 0u;           // the bits of the threshold found so far
  if (want == 0) th = mask = 0xffffffffu;
#pragma unroll 1
  for (int shift = 21; mask != 0xffffffffu; shift = shift > 11 ? shift - 11 : 0) {   // 21, 10, 0
    const int bits = shift == 0 ? 10 : 11;
    hist[tid] = 0;
    hist[tid + kSelThreads] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KPT; ++k)
      if (key[k] != 0u && (key[k] & mask) == th) atomicAdd(&hist[(key[k] >> shift) & ((1u << bits) - 1u)], 1);
    __syncthreads();
    // this thread's two bins, highest first
    const int top = kTopBins - 1 - 2 * tid, v0 = hist[top], v1 = hist[top - 1];
    int incl = v0 + v1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) wsum[warp] = (uint32_t)incl;
    __syncthreads();
    int ws = (int)wsum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, ws, o);
      if (lane >= o) ws += y;
    }
    const int excl = __shfl_sync(0xffffffffu, ws, warp) - (int)wsum[warp] + incl - v0 - v1;   // counted keys above the bins
    if (excl < want && want <= excl + v0 + v1) {
      const bool second = excl + v0 < want;
      res[0] = second ? top - 1 : top;
      res[1] = second ? excl + v0 : excl;
      res[2] = second ? v1 : v0;
    }
    __syncthreads();
    th |= (uint32_t)res[0] << shift;
    mask |= ((1u << bits) - 1u) << shift;
    want -= res[1];
    if (res[2] == want) break;           // every key of the digit is kept
  }
  // keys that match the whole threshold found count as equal to it
  const uint32_t low = ~mask;

  // kept for certain, and at the threshold: low and high half of a word (at most 2^15 each)
  uint32_t own = (uint32_t)__popc(forced);
#pragma unroll
  for (int k = 0; k < KPT; ++k) own += key[k] > (th | low) ? 1u : (key[k] >= th ? 0x10000u : 0u);
  uint32_t incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) wsum[warp] = incl;
#pragma unroll
  for (int k = 0; k < KPT; ++k)          // their sums, before any is overwritten
    if ((forced >> k) & 1u) key[k] = __float_as_uint(src[i0 + k]);
  __syncthreads();
  uint32_t ws = wsum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, ws, o);
    if (lane >= o) ws += y;
  }
  const int need = C - (int)(__shfl_sync(0xffffffffu, ws, 31) & 0xffffu);   // ties to keep, lowest index first
  const uint32_t before = __shfl_sync(0xffffffffu, ws, warp) - wsum[warp] + incl - own;
  int gt = (int)(before & 0xffffu), eq = (int)(before >> 16);
#pragma unroll
  for (int k = 0; k < KPT; ++k) {
    const bool f = (forced >> k) & 1u, g = f || key[k] > (th | low), e = !f && !g && key[k] >= th;
    if (g || (e && eq < need)) {
      const int pos = gt + min(eq, need);
      if (pos < C) {                     // always, for sums that are no NaN
        out[pos] = i0 + k;
        dst[pos] = f ? __uint_as_float(key[k]) : key_value(key[k]);
      }
    }
    gt += g;
    eq += e;
  }
  for (int i = C + tid; i < a.t_max; i += kSelThreads) dst[i] = 0.f;
}

// ---- the move ---------------------------------------------------------------------------------

constexpr uint32_t kNone = 0xffffffffu;

// Position `tok` of the unit: its row of k / v (kNone for an invalid page) and its scale; 32
// bits, as the cache fits in device memory.  u_row, u_scale: the unit's first row and scale
// in a contiguous cache.
__device__ __forceinline__ uint32_t row_of(const MoveParams& p, uint32_t u_row, uint32_t u_scale, int b, int h, int tok,
                                           uint32_t& sidx) {
  const KvView& kv = p.kv;
  if (kv.page_size == 0) {
    sidx = u_scale + ((uint32_t)tok >> kv.block_shift);
    return u_row + (uint32_t)tok;
  }
  const uint32_t t16 = (uint32_t)tok >> 4;   // pages are 16 m tokens, m <= 16, and tok / 16 < 2^27
  const uint32_t lp = p.page_magic ? __umulhi(t16, p.page_magic) : t16;
  const int page = kv.page_table[(size_t)b * kv.max_pages + lp];
  if (page < 0 || page >= kv.n_pages) {
    flag_status(ASP_DEV_BAD_PAGE);
    return kNone;
  }
  const uint32_t in = (uint32_t)tok - lp * (uint32_t)kv.page_size;
  const uint32_t head = (uint32_t)page * (uint32_t)kv.n_kv + (uint32_t)h;
  sidx = head * (uint32_t)kv.blocks_per_row + (in >> kv.block_shift);
  return head * (uint32_t)kv.page_size + in;
}

// The sums follow their tokens (rows that evict_select_kernel does not take).
__device__ void move_sums(const MoveParams& p, int unit, int T) {
  const int n = min(p.a.C, T);
  const float* const src = p.a.acc + (size_t)unit * p.kv.t_max;
  float* const dst = p.a.acc_out + (size_t)unit * p.kv.t_max;
  const int32_t* const idx = p.a.idx + (size_t)unit * p.a.C;
  for (int base = 0; base < n; base += kVecs * kThreads) {
    float v[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int i = base + k * kThreads + threadIdx.x;
      v[k] = i < n ? src[idx[i]] : 0.f;
    }
    __syncthreads();   // acc_out may be acc: the chunk is read before it is written
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int i = base + k * kThreads + threadIdx.x;
      if (i < n) dst[i] = v[k];
    }
  }
  __syncthreads();
  for (int i = n + threadIdx.x; i < p.kv.t_max; i += kThreads) dst[i] = 0.f;
}

// CT: code type, or void for rows that only move.  ROWB: bytes of a row.
template <typename CT, int ROWB>
__global__ void __launch_bounds__(kThreads, 1) evict_move_kernel(MoveParams p) {
  constexpr bool CODES = !std::is_void<CT>::value;
  constexpr int VPR = ROWB / 16;
  constexpr int CR = kVecs * kThreads / VPR;     // rows of a chunk
  constexpr int RV = kThreads / VPR;             // rows from a thread's vector to its next
  static_assert(!CODES || CR / 16 <= kBlocks, "blocks of a chunk");
  __shared__ uint32_t bmax[3][kBlocks];
  const int unit = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const int r0 = tid / VPR, c16 = (tid % VPR) * 16;
  const KvView& kv = p.kv;
  const int b = unit / kv.n_kv, h = unit - b * kv.n_kv;
  const uint32_t u_row = (uint32_t)unit * (uint32_t)kv.t_max, u_scale = (uint32_t)unit * (uint32_t)kv.blocks_per_row;
  pdl_wait();
  const int T = p.a.keep_len[unit], C = p.a.C;
  if (blockIdx.y == 0 && h == 0 && tid == 0) p.seq_lens[b] = min(C, T);   // read by the selection alone, before
  if (blockIdx.y == 2) {
    move_sums(p, unit, T);
    return;
  }
  if (T <= C) return;
  uint8_t* const data = static_cast<uint8_t*>(const_cast<void*>(blockIdx.y ? kv.v : kv.k)) + c16;
  float* const scale = blockIdx.y ? kv.v_scale : kv.k_scale;
  const int32_t* const idx = p.a.idx + (size_t)unit * C;
  if (CODES) {
    for (int i = tid; i < 3 * kBlocks; i += kThreads) (&bmax[0][0])[i] = 0u;
    __syncthreads();
  }

  // the indices of the chunk after next, the rows of the next chunk
  int tok[kVecs];
  uint4 nxt[kVecs];
  float nsc[kVecs];
  auto ask = [&](int base) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int i = base + r0 + v * RV;
      tok[v] = i < C ? idx[i] : -1;
      if (tok[v] < i || tok[v] >= T) tok[v] = -1;   // an unspecified choice (NaN sums): nothing is read
    }
  };
  auto load = [&]() {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      nxt[v] = make_uint4(0u, 0u, 0u, 0u);
      nsc[v] = 0.f;
      if (tok[v] < 0) continue;
      uint32_t sidx = 0;
      const uint32_t row = row_of(p, u_row, u_scale, b, h, tok[v], sidx);
      if (row == kNone) continue;
      nxt[v] = *reinterpret_cast<const uint4*>(data + (size_t)row * ROWB);
      if (CODES) nsc[v] = scale[sidx];
    }
  };
  ask(0);
  load();
  ask(CR);
  int turn = 0;
  for (int base = 0; base < C; base += CR, turn = turn == 2 ? 0 : turn + 1) {
    uint4 cur[kVecs];
    float sc[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      cur[v] = nxt[v];
      sc[v] = nsc[v];
    }
    // The next chunk's loads go out ahead of this chunk's barrier and stores; they touch no
    // row, and no scale, that this chunk writes.
    if (base + CR < C) {
      load();
      ask(base + 2 * CR);
    }
    if constexpr (CODES) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        const uint4 w = cur[v];
        uint32_t m4 = __vmaxu4(__vmaxu4(CT::mag4(w.x), CT::mag4(w.y)), __vmaxu4(CT::mag4(w.z), CT::mag4(w.w)));
        m4 = __vmaxu4(m4, m4 >> 16);
        uint32_t m = max(m4 & 0xffu, (m4 >> 8) & 0xffu);
        if (m == CT::kNanMag) {   // a NaN among the codes: the others again
          m = 0u;
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint32_t c = (CT::mag4(ws[j >> 2]) >> (8 * (j & 3))) & 0xffu;
            if (c != CT::kNanMag) m = max(m, c);
          }
        }
        const float top = CT::mag_value(m) * sc[v];
        const uint32_t amax = __reduce_max_sync(0xffffffffu, __float_as_uint(top));   // a warp's rows lie in one block
        if (lane == 0) atomicMax(&bmax[turn][(r0 + v * RV) >> kv.block_shift], min(amax, 0x7f7fffffu));
      }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int r = r0 + v * RV, i = base + r;
      if (i >= C) continue;
      uint32_t sidx = 0;
      const uint32_t row = row_of(p, u_row, u_scale, b, h, i, sidx);
      if (row == kNone) continue;
      uint4 y = cur[v];
      if constexpr (CODES) {
        const int e = scale_exp<CT>(bmax[turn][r >> kv.block_shift]);
        const float f = sc[v] * exp2i(-e);
        const uint32_t fb = __float_as_uint(f);
        if (f == 1.f) {
        } else if ((fb & 0x7fffffu) == 0u && fb <= 0x47000000u) {   // a power of two up to 2^15 (or zero)
          const __half2 fh = __float2half2_rn(f);   // below 2^-24: zero, as every code then is
          y.x = CT::rescale4(y.x, fh);
          y.y = CT::rescale4(y.y, fh);
          y.z = CT::rescale4(y.z, fh);
          y.w = CT::rescale4(y.w, fh);
        } else {
          uint32_t z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x[4];
            decode4<CT>(z[j], x);
            z[j] = CT::encode4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
          }
          y = make_uint4(z[0], z[1], z[2], z[3]);
        }
        if (c16 == 0 && (r & ((1 << kv.block_shift) - 1)) == 0) scale[sidx] = exp2i(e);
      }
      *reinterpret_cast<uint4*>(data + (size_t)row * ROWB) = y;
    }
    // the maxima of the turn after next: read last a turn ago, before this turn's barrier
    if (CODES && tid < kBlocks) bmax[turn == 0 ? 2 : turn - 1][tid] = 0u;
  }
}

template <typename CT, int ROWB>
cudaError_t move_t(const MoveParams& p, bool sums, cudaStream_t s) {
  return launch_pdl(evict_move_kernel<CT, ROWB>, dim3(p.kv.batch * p.kv.n_kv, sums ? 3 : 2), dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_evict(const KvView& kv, int32_t* seq_lens, const EvictArgs& a, cudaStream_t s) {
  SelectArgs sa;
  sa.scores = a.acc;
  sa.row_stride = kv.t_max;
  sa.seq_lens = seq_lens;
  sa.t_max = kv.t_max;
  sa.rows_per_seq = kv.n_kv;
  sa.n_rows = kv.batch * kv.n_kv;
  sa.c_units = a.C;
  sa.expand = 1;
  sa.idx = a.idx;
  sa.count = a.count;
  sa.hist0 = nullptr;
  sa.n_sink = a.n_sink;
  sa.n_recent = a.n_recent;
  sa.keep_len = a.keep_len;
  cudaError_t e;
  const dim3 rows(sa.n_rows), threads(kSelThreads);
  const bool sums = kv.t_max > kSelMaxKeys;   // longer rows: keys in shared memory or read again from L2
  if (sums) e = launch_select(sa, s);
  else if (kv.t_max <= 4 * kSelThreads) e = launch_pdl(evict_select_kernel<4>, rows, threads, 0, s, sa, a.acc_out);
  else if (kv.t_max <= 8 * kSelThreads) e = launch_pdl(evict_select_kernel<8>, rows, threads, 0, s, sa, a.acc_out);
  else if (kv.t_max <= 16 * kSelThreads) e = launch_pdl(evict_select_kernel<16>, rows, threads, 0, s, sa, a.acc_out);
  else e = launch_pdl(evict_select_kernel<32>, rows, threads, 0, s, sa, a.acc_out);
  if (e != cudaSuccess) return e;
  const int m16 = kv.page_size / 16;
  const MoveParams p{kv, a, seq_lens, m16 > 1 ? (uint32_t)(((1ull << 32) + m16 - 1) / m16) : 0u};
  if (kv.kv8 == 1) return kv.head_dim == 64 ? move_t<CodeE4M3, 64>(p, sums, s) : move_t<CodeE4M3, 128>(p, sums, s);
  if (kv.kv8 == 2) return kv.head_dim == 64 ? move_t<CodeI8, 64>(p, sums, s) : move_t<CodeI8, 128>(p, sums, s);
  switch (kv.head_dim * (kv.kv_f32 ? 4 : 2)) {
    case 128: return move_t<void, 128>(p, sums, s);
    case 256: return move_t<void, 256>(p, sums, s);
    case 512: return move_t<void, 512>(p, sums, s);
    default: return cudaErrorInvalidValue;
  }
}

ASP_STATUS_READER(read_status_evict)

}  // namespace asp
