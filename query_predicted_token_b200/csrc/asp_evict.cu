// asp_evict.cu -- eviction to a budget: the kept rows moved to the front, in place.
//
// asp_select.cu has chosen C tokens per row of sums, ascending, and left the row's length.
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
};

// Position `tok` of the unit as a row of k / v; -1 for an invalid page.
__device__ __forceinline__ long long row_of(const KvView& kv, int b, int h, int tok) {
  if (kv.page_size == 0) return ((long long)b * kv.n_kv + h) * kv.t_max + tok;
  const int page = kv.page_table[(size_t)b * kv.max_pages + tok / kv.page_size];
  if (page < 0 || page >= kv.n_pages) {
    flag_status(ASP_DEV_BAD_PAGE);
    return -1;
  }
  return ((long long)page * kv.n_kv + h) * kv.page_size + tok % kv.page_size;
}
__device__ __forceinline__ size_t scale_of_row(const KvView& kv, long long row, int tok) {
  if (kv.page_size == 0) {
    const long long unit = (row - tok) / kv.t_max;
    return (size_t)unit * kv.blocks_per_row + (tok >> kv.block_shift);
  }
  const long long ph = row / kv.page_size;
  return (size_t)ph * kv.blocks_per_row + ((int)(row - ph * kv.page_size) >> kv.block_shift);
}

// The sums follow their tokens; the lengths shrink.
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
  if (threadIdx.x == 0 && unit % p.kv.n_kv == 0) p.seq_lens[unit / p.kv.n_kv] = n;
}

// CT: code type, or void for rows that only move.  ROWB: bytes of a row.
template <typename CT, int ROWB>
__global__ void __launch_bounds__(kThreads, 1) evict_move_kernel(MoveParams p) {
  constexpr bool CODES = !std::is_void<CT>::value;
  constexpr int VPR = ROWB / 16;
  constexpr int CR = kVecs * kThreads / VPR;     // rows of a chunk
  static_assert(!CODES || CR / 16 <= kBlocks, "blocks of a chunk");
  __shared__ uint32_t bmax[3][kBlocks];
  const int unit = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const KvView& kv = p.kv;
  const int b = unit / kv.n_kv, h = unit - b * kv.n_kv;
  pdl_wait();
  const int T = p.a.keep_len[unit], C = p.a.C;
  if (blockIdx.y == 2) {
    move_sums(p, unit, T);
    return;
  }
  if (T <= C) return;
  uint8_t* const data = static_cast<uint8_t*>(const_cast<void*>(blockIdx.y ? kv.v : kv.k));
  float* const scale = blockIdx.y ? kv.v_scale : kv.k_scale;
  const int32_t* const idx = p.a.idx + (size_t)unit * C;
  if (CODES) {
    for (int i = tid; i < 3 * kBlocks; i += kThreads) (&bmax[0][0])[i] = 0u;
    __syncthreads();
  }

  uint4 nxt[kVecs];
  float nsc[kVecs];
  auto load = [&](int base) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int vec = v * kThreads + tid, i = base + vec / VPR;
      nxt[v] = make_uint4(0u, 0u, 0u, 0u);
      nsc[v] = 0.f;
      if (i >= C) continue;
      const int tok = idx[i];
      if (tok < i || tok >= T) continue;   // an unspecified choice (NaN sums): nothing is read
      const long long row = row_of(kv, b, h, tok);
      if (row < 0) continue;
      nxt[v] = *reinterpret_cast<const uint4*>(data + (size_t)row * ROWB + (vec % VPR) * 16);
      if (CODES) nsc[v] = scale[scale_of_row(kv, row, tok)];
    }
  };
  load(0);
  int turn = 0;
  for (int base = 0; base < C; base += CR, turn = turn == 2 ? 0 : turn + 1) {
    uint4 cur[kVecs];
    float sc[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      cur[v] = nxt[v];
      sc[v] = nsc[v];
    }
    if constexpr (CODES) {
#pragma unroll
      for (int v = 0; v < kVecs; ++v) {
        const uint32_t w[4] = {cur[v].x, cur[v].y, cur[v].z, cur[v].w};
        uint32_t amax = 0u;
        bool bad = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x[4];
          decode4<CT>(w[j], x);
#pragma unroll
          for (int e = 0; e < 4; ++e) amax = max(amax, finite_abs(x[e] * sc[v], bad));
        }
        amax = __reduce_max_sync(0xffffffffu, amax);   // a warp's rows lie in one block
        if (lane == 0) atomicMax(&bmax[turn][((v * kThreads + tid) / VPR) >> kv.block_shift], amax);
      }
    }
    // Reads of a scale that a later chunk's block owns come before it is written: the next
    // chunk's loads go out here, ahead of this chunk's barrier and stores.
    if (base + CR < C) load(base + CR);
    __syncthreads();
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const int vec = v * kThreads + tid, r = vec / VPR, i = base + r;
      if (i >= C) continue;
      const long long row = row_of(kv, b, h, i);
      if (row < 0) continue;
      uint4 y = cur[v];
      if constexpr (CODES) {
        const int e = scale_exp<CT>(bmax[turn][r >> kv.block_shift]);
        const float inv = exp2i(-e);
        const uint32_t w[4] = {y.x, y.y, y.z, y.w};
        uint32_t z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x[4];
          decode4<CT>(w[j], x);
          z[j] = CT::encode4(x[0] * sc[v] * inv, x[1] * sc[v] * inv, x[2] * sc[v] * inv, x[3] * sc[v] * inv);
        }
        y = make_uint4(z[0], z[1], z[2], z[3]);
        if (vec % VPR == 0 && (r & ((1 << kv.block_shift) - 1)) == 0) scale[scale_of_row(kv, row, i)] = exp2i(e);
      }
      *reinterpret_cast<uint4*>(data + (size_t)row * ROWB + (vec % VPR) * 16) = y;
    }
    // the maxima of the turn after next: read last a turn ago, before this turn's barrier
    if (CODES && tid < kBlocks) bmax[turn == 0 ? 2 : turn - 1][tid] = 0u;
  }
}

template <typename CT, int ROWB>
cudaError_t move_t(const MoveParams& p, cudaStream_t s) {
  return launch_pdl(evict_move_kernel<CT, ROWB>, dim3(p.kv.batch * p.kv.n_kv, 3), dim3(kThreads), 0, s, p);
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
  cudaError_t e = launch_select(sa, s);
  if (e != cudaSuccess) return e;
  const MoveParams p{kv, a, seq_lens};
  if (kv.kv8 == 1) return kv.head_dim == 64 ? move_t<CodeE4M3, 64>(p, s) : move_t<CodeE4M3, 128>(p, s);
  if (kv.kv8 == 2) return kv.head_dim == 64 ? move_t<CodeI8, 64>(p, s) : move_t<CodeI8, 128>(p, s);
  switch (kv.head_dim * (kv.kv_f32 ? 4 : 2)) {
    case 128: return move_t<void, 128>(p, s);
    case 256: return move_t<void, 256>(p, s);
    case 512: return move_t<void, 512>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

ASP_STATUS_READER(read_status_evict)

}  // namespace asp
