// Attention of a ragged batch's new tokens over the paged latent cache on CUDA
// cores, for every storage type and shape: the fp32 configuration, the FP8
// cache, and bf16 shapes without the tensor-core kernel.
//
// One CTA per (token, head).  Its warps take the token's visible pages in
// turn, half a page (32 rows) at a time: lane r computes the score of row r,
//   s = scale log2(e) (q_lat . c + q_rope . k_R),
// the warp takes the running maximum and sum of the online softmax, and then
// accumulates O += 2^(s - m) c with the lanes across the latent columns.  The
// warps' (m, l, O) are merged through shared memory at the end, in warp
// order, so results do not depend on timing.  Rows that are not visible are
// never read.  All sums are fp32; the output is rounded once.
#pragma once

#include "chunk_plan.cuh"

namespace mla {
namespace chunk {

constexpr int kSimtWarps = 8;

struct SimtArgs {
  const void* q_lat;   // [n_tok, H] rows, `q_stride` values apart
  const void* q_rope;  // [n_tok, H] rows, `qr_stride` values apart
  const void* q_lo_lat;  // remainders of a split query, or null
  const void* q_lo_rope;
  long long q_stride, qr_stride;
  const void* pool;
  const float* row_scale;
  const int32_t* block_table;
  int max_blocks, num_blocks, bs;
  Batch q;
  int H, d_c, d_r;
  float scale_log2;
  void* o_lat;  // [n_tok, H, d_c]
  float* lse;   // [n_tok, H] or null
};

// The sequence of token t: the last b with cu_q[b] <= t (cu_q ascending).
__device__ __forceinline__ int sequence_of_token(const int32_t* cu_q, int batch, int t) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu_q[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// TQ: type of the query rows, T: cached values, TO: output; DPL: latent columns per lane.
template <typename TQ, typename T, typename TO, int DPL>
__global__ void __launch_bounds__(32 * kSimtWarps) chunk_simt_kernel(const SimtArgs a) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float sm[];  // q [row], then [warps][d_c] merged outputs
  __shared__ float wm[kSimtWarps], wl[kSimtWarps];
  const int t = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = a.d_c + a.d_r;
  if (t == 0 && h == 0)
    for (int b = threadIdx.x; b < a.q.batch; b += blockDim.x) report_sequence(a.q, b, sequence_of(a.q, b));
  const int b = sequence_of_token(a.q.cu_q, a.q.batch, t);
  const Sequence s = sequence_of(a.q, b);
  // rows behind the last sequence stay as they are
  if (t < s.t0 || t >= s.t0 + s.n) return;
  const long long qi = (long long)t * a.H + h;
  for (int d = threadIdx.x; d < row; d += blockDim.x) {
    const long long o = d < a.d_c ? qi * a.q_stride + d : qi * a.qr_stride + d - a.d_c;
    float v = Store<TQ>::ld(static_cast<const TQ*>(d < a.d_c ? a.q_lat : a.q_rope) + o);
    if (a.q_lo_lat != nullptr) v += Store<TQ>::ld(static_cast<const TQ*>(d < a.d_c ? a.q_lo_lat : a.q_lo_rope) + o);
    sm[d] = v * a.scale_log2;
  }
  __syncthreads();

  float m = -INFINITY, l = 0.f, o[DPL];
#pragma unroll
  for (int i = 0; i < DPL; ++i) o[i] = 0.f;
  const int p = s.p0 + (t - s.t0);
  // the visible rows: [0, sinks) and [w0, p], or one run from 0
  const int w0 = s.p0 < 0 ? 0 : a.q.vis.start(p);
  const int n_sink = w0 > 0 ? a.q.vis.sinks : 0;
  const int n_vis = s.p0 < 0 ? 0 : n_sink + (p + 1 - w0);
  const T* pool = static_cast<const T*>(a.pool);
  for (int base = 32 * warp; base < n_vis; base += 32 * kSimtWarps) {
    const int i = base + lane;
    const int u = i < n_sink ? i : w0 + (i - n_sink);
    const T* kv = nullptr;
    float sc = 1.f, x = -INFINITY;
    if (i < n_vis) {
      const int page = u / a.bs;
      const int phys = a.block_table[(long long)b * a.max_blocks + page];
      if (phys < 0 || phys >= a.num_blocks) {
        report(MLA_ERR_BOUNDS, 22, b, phys);
      } else {
        const long long slot = (long long)phys * a.bs + (u - page * a.bs);
        kv = pool + slot * row;
        if (a.row_scale != nullptr) sc = a.row_scale[slot];
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        int d = 0;
#pragma unroll 4
        for (; d + 4 <= row; d += 4) {
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] = fmaf(sm[d + e], Store<T>::ld(kv + d + e), acc[e]);
        }
        for (; d < row; ++d) acc[0] = fmaf(sm[d], Store<T>::ld(kv + d), acc[0]);
        x = ((acc[0] + acc[1]) + (acc[2] + acc[3])) * sc;
      }
    }
    const float m_new = fmaxf(m, warp_max(x));
    if (m_new == -INFINITY) {  // no finite score yet; the maximum passes over NaN, the sum must not
      if (__any_sync(0xffffffffu, x != x)) l = NAN;
      continue;
    }
    const float corr = exp2f(m - m_new), pw = kv != nullptr ? exp2f(x - m_new) : 0.f;
    m = m_new;
    l = l * corr + warp_sum(pw);
    const float pws = pw * sc;
#pragma unroll
    for (int k = 0; k < DPL; ++k) o[k] *= corr;
    const int rows = min(32, n_vis - base);
    for (int r = 0; r < rows; ++r) {
      const T* c = reinterpret_cast<const T*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(kv), r));
      const float w = __shfl_sync(0xffffffffu, pws, r);
      if (c == nullptr) continue;
#pragma unroll
      for (int k = 0; k < DPL; ++k) {
        const int d = lane + 32 * k;
        if (d < a.d_c) o[k] = fmaf(w, Store<T>::ld(c + d), o[k]);
      }
    }
  }

  // merge the warps
  float* om = sm + row;
  if (lane == 0) {
    wm[warp] = m;
    wl[warp] = l;
  }
#pragma unroll
  for (int k = 0; k < DPL; ++k) {
    const int d = lane + 32 * k;
    if (d < a.d_c) om[warp * a.d_c + d] = o[k];
  }
  __syncthreads();
  float M = -INFINITY, Z = 0.f, f[kSimtWarps];
#pragma unroll
  for (int w = 0; w < kSimtWarps; ++w) M = fmaxf(M, wm[w]);
#pragma unroll
  for (int w = 0; w < kSimtWarps; ++w) {
    f[w] = M == -INFINITY ? 0.f : exp2f(wm[w] - M);
    Z = fmaf(f[w], wl[w], Z);
  }
  const float inv = Z > 0.f ? 1.f / Z : (Z == 0.f ? 0.f : Z);  // a NaN sum stays NaN
  TO* out = static_cast<TO*>(a.o_lat) + qi * a.d_c;
  for (int d = threadIdx.x; d < a.d_c; d += blockDim.x) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kSimtWarps; ++w) v = fmaf(f[w], om[w * a.d_c + d], v);
    Store<TO>::st(out + d, v * inv);
  }
  if (a.lse != nullptr && threadIdx.x == 0) a.lse[qi] = Z == 0.f ? -INFINITY : M + log2f(Z);
}

}  // namespace chunk
}  // namespace mla
