// Attention of a ragged batch's new tokens over the paged latent cache on CUDA
// cores, for every storage type and shape: the fp32 configuration, the FP8
// cache, and bf16 shapes without the tensor-core kernel.
//
// One CTA per token and up to 8 heads, which share the token's cached rows.  The
// visible rows come through shared memory in tiles, read once for all heads in
// 16-byte pieces; with fewer than 8 heads several warps take a head, each its own
// blocks of 32 rows of a tile.  Lane r computes the score of row r,
//   s = scale log2(e) (q_lat . c + q_rope . k_R),
// the warp takes the running maximum and sum of the online softmax, and then
// accumulates O += 2^(s - m) c with the lanes across the latent columns.  A row
// in shared memory is an odd number of 16-byte pieces long, so that 8 lanes
// reading one piece each of their rows meet no bank twice.  The warps' (m, l, O)
// of a head are merged at the end in warp order, so results do not depend on
// timing.  Rows that are not visible are zeros there and are never read.  All
// sums are fp32; the output is rounded once.
//
// What bounds it is the latency of its dependent steps (sequence, table, rows)
// and the shared-memory reads: the fp32 shape of 91 tokens over up to 440 rows
// took 37 us with each lane reading its row from global memory word by word.
// A token is not split over its rows: one token of 4 heads in fp32 takes 14 us over
// 440 rows, 65 over 4,000 and 240 over 16,000 (the decode entry points, which split
// it, 32, 51 and 117).
#pragma once

#include "chunk_plan.cuh"
#include "sm100.cuh"

namespace mla {
namespace chunk {

using sm100::smem_u32;

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

// 16 bytes of T as floats.
template <typename T>
struct Piece16;
template <>
struct Piece16<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void get(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
  }
};
template <>
struct Piece16<bf16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void get(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  }
};
template <>
struct Piece16<__nv_fp8_e4m3> {
  static constexpr int kN = 16;
  static __device__ __forceinline__ void get(const uint4& v, float (&x)[16]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      __nv_fp8_e4m3 c;
      c.__x = (__nv_fp8_storage_t)((w[k >> 2] >> (8 * (k & 3))) & 0xFFu);
      x[k] = static_cast<float>(c);
    }
  }
};

// Shared memory of a CTA: queries fp32 [heads][pieces * kN], then the tile of rows
// (afterwards the warps' outputs).
struct SimtShape {
  int heads, splits, blocks;  // heads of a CTA, warps per head, 32-row blocks of a warp in a tile
  int pieces, stride;         // 16-byte pieces of a row, bytes between rows
  size_t q_bytes, tile_bytes;
  size_t total(int d_c) const {
    const size_t out = sizeof(float) * (size_t)kSimtWarps * d_c;
    return q_bytes + (tile_bytes > out ? tile_bytes : out);
  }
};
// Heads share a CTA, and so its rows, as far as there are CTAs enough for the
// SMs; a tile is as long as 256 rows and 96 KiB allow, for the steps between two
// tiles are all latency (91 tokens of 4 heads over up to 440 rows: 28 us in tiles of 64 rows, 17 in tiles of 256).
constexpr size_t kSimtTile = 96 * 1024;
constexpr int kSimtRows = 32 * kSimtWarps;
template <typename T>
SimtShape simt_shape(int n_tok, int H, int row, int sms) {
  SimtShape s;
  s.heads = kSimtWarps;
  while (s.heads > 1 && (s.heads / 2 >= H || (long long)n_tok * ((H + s.heads - 1) / s.heads) < sms)) s.heads /= 2;
  s.pieces = (row * (int)sizeof(T) + 15) / 16;
  s.stride = 16 * (s.pieces | 1);
  s.splits = kSimtWarps / s.heads;
  while (s.splits > 1 && (size_t)s.splits * 32 * s.stride > kSimtTile) s.splits /= 2;
  s.blocks = kSimtRows / (32 * s.splits);
  while (s.blocks > 1 && (size_t)s.blocks * s.splits * 32 * s.stride > kSimtTile) s.blocks /= 2;
  s.q_bytes = (sizeof(float) * s.heads * s.pieces * Piece16<T>::kN + 15) / 16 * 16;
  s.tile_bytes = (size_t)s.blocks * s.splits * 32 * s.stride;
  return s;
}

// TQ: type of the query rows, T: cached values, TO: output; DPL: latent columns per lane.
template <typename TQ, typename T, typename TO, int DPL>
__global__ void __launch_bounds__(32 * kSimtWarps) chunk_simt_kernel(const SimtArgs a, const SimtShape g) {
  using P = Piece16<T>;
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float wm[kSimtWarps], wl[kSimtWarps], row_sc[kSimtRows];
  __shared__ long long row_slot[kSimtRows];  // of the tile's rows: pool slot, -1 where none is visible
  float* qs = reinterpret_cast<float*>(smem);
  uint8_t* tile = smem + g.q_bytes;
  const int t = blockIdx.x, h0 = blockIdx.y * g.heads, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = a.d_c + a.d_r, q_row = g.pieces * P::kN;
  if (t == 0 && h0 == 0)
    for (int b = threadIdx.x; b < a.q.batch; b += blockDim.x) report_sequence(a.q, b, sequence_of(a.q, b));
  const int b = sequence_of_token(a.q.cu_q, a.q.batch, t);
  const Sequence s = sequence_of(a.q, b);
  // rows behind the last sequence stay as they are
  if (t < s.t0 || t >= s.t0 + s.n) return;
  const int nh = min(g.heads, a.H - h0);
  for (int i = threadIdx.x; i < nh * q_row; i += blockDim.x) {
    const int d = i % q_row;
    const long long qi = (long long)t * a.H + h0 + i / q_row;
    float v = 0.f;
    if (d < row) {
      const long long o = d < a.d_c ? qi * a.q_stride + d : qi * a.qr_stride + d - a.d_c;
      v = Store<TQ>::ld(static_cast<const TQ*>(d < a.d_c ? a.q_lat : a.q_rope) + o);
      if (a.q_lo_lat != nullptr) v += Store<TQ>::ld(static_cast<const TQ*>(d < a.d_c ? a.q_lo_lat : a.q_lo_rope) + o);
    }
    qs[i] = v * a.scale_log2;
  }
  // this warp's head and its part of a tile
  const int hl = warp % g.heads, part = warp / g.heads;
  const bool works = hl < nh && part < g.splits;
  const float* q = qs + hl * q_row;

  float m = -INFINITY, l = 0.f, o[DPL];
#pragma unroll
  for (int i = 0; i < DPL; ++i) o[i] = 0.f;
  const int p = s.p0 + (t - s.t0);
  // the visible rows: [0, sinks) and [w0, p], or one run from 0
  const int w0 = s.p0 < 0 ? 0 : a.q.vis.start(p);
  const int n_sink = w0 > 0 ? a.q.vis.sinks : 0;
  const int n_vis = s.p0 < 0 ? 0 : n_sink + (p + 1 - w0);
  const int rows = 32 * g.splits * g.blocks;
  const bool wide = ((reinterpret_cast<uintptr_t>(a.pool) | (size_t)row * sizeof(T)) & 15u) == 0;
  for (int base = 0; base < n_vis; base += rows) {
    const int n_rows = min(rows, (n_vis - base + 31) / 32 * 32);  // of this tile, in whole blocks
    __syncthreads();  // the tile before has been read
    if (threadIdx.x < n_rows) {
      const int i = base + threadIdx.x;
      long long slot = -1;
      float sc = 1.f;
      if (i < n_vis) {
        const int u = i < n_sink ? i : w0 + (i - n_sink);
        const int page = u / a.bs;
        const int phys = a.block_table[(long long)b * a.max_blocks + page];
        if (phys < 0 || phys >= a.num_blocks) {
          report(MLA_ERR_BOUNDS, 22, b, phys);
        } else {
          slot = (long long)phys * a.bs + (u - page * a.bs);
          if (a.row_scale != nullptr) sc = a.row_scale[slot];
        }
      }
      row_slot[threadIdx.x] = slot;
      row_sc[threadIdx.x] = sc;
    }
    __syncthreads();
    if (wide) {  // 8 threads a row, all pieces in flight; a row that is not seen is filled with zeros
      for (int r = threadIdx.x / 8; r < n_rows; r += 4 * kSimtWarps) {
        const long long slot = row_slot[r];
        const T* src = static_cast<const T*>(a.pool) + (slot < 0 ? 0 : slot * row);
        const uint32_t dst = smem_u32(tile + r * g.stride), bytes = slot < 0 ? 0 : 16;
        for (int c = threadIdx.x % 8; c < g.pieces; c += 8)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 16 * c), "l"(src + c * P::kN), "r"(bytes)
                       : "memory");
      }
      asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
    } else {
      for (int i = threadIdx.x; i < n_rows * q_row; i += blockDim.x) {
        const int r = i / q_row, d = i % q_row;
        const long long slot = row_slot[r];
        T v = T(0.f);
        if (slot >= 0 && d < row) v = static_cast<const T*>(a.pool)[slot * row + d];
        *reinterpret_cast<T*>(tile + r * g.stride + sizeof(T) * d) = v;
      }
    }
    __syncthreads();
    for (int k = 0; works && k < g.blocks; ++k) {
      const int r0 = 32 * (k * g.splits + part);
      if (base + r0 >= n_vis) break;
      const uint8_t* my = tile + (size_t)r0 * g.stride;
      const bool seen = row_slot[r0 + lane] >= 0;
      const float sc = row_sc[r0 + lane];
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int c = 0; c < g.pieces; ++c) {
        float x[P::kN];
        P::get(*reinterpret_cast<const uint4*>(my + lane * g.stride + 16 * c), x);
#pragma unroll
        for (int e = 0; e < P::kN; e += 4) {
          const float4 y = *reinterpret_cast<const float4*>(q + c * P::kN + e);
          acc[0] = fmaf(y.x, x[e], acc[0]);
          acc[1] = fmaf(y.y, x[e + 1], acc[1]);
          acc[2] = fmaf(y.z, x[e + 2], acc[2]);
          acc[3] = fmaf(y.w, x[e + 3], acc[3]);
        }
      }
      const float x = seen ? ((acc[0] + acc[1]) + (acc[2] + acc[3])) * sc : -INFINITY;
      const float m_new = fmaxf(m, warp_max(x));
      if (m_new == -INFINITY) {  // no finite score yet; the maximum passes over NaN, the sum must not
        if (__any_sync(0xffffffffu, x != x)) l = NAN;
        continue;
      }
      const float corr = exp2f(m - m_new), pw = seen ? exp2f(x - m_new) : 0.f;
      m = m_new;
      l = l * corr + warp_sum(pw);
      const float pws = pw * sc;
#pragma unroll
      for (int i = 0; i < DPL; ++i) o[i] *= corr;
#pragma unroll 8
      for (int r = 0; r < 32; ++r) {
        const float w = __shfl_sync(0xffffffffu, pws, r);
        const T* c = reinterpret_cast<const T*>(my + r * g.stride);
#pragma unroll
        for (int i = 0; i < DPL; ++i)
          if (lane + 32 * i < a.d_c) o[i] = fmaf(w, Store<T>::ld(c + lane + 32 * i), o[i]);
      }
    }
  }

  // merge the warps of a head
  __syncthreads();
  float* om = reinterpret_cast<float*>(tile);
  if (lane == 0) {
    wm[warp] = m;
    wl[warp] = l;
  }
#pragma unroll
  for (int k = 0; k < DPL; ++k)
    if (lane + 32 * k < a.d_c) om[warp * a.d_c + lane + 32 * k] = o[k];
  __syncthreads();
  if (!works || part > 0) return;
  const long long qi = (long long)t * a.H + h0 + hl;
  float M = -INFINITY, Z = 0.f;
  for (int w = hl; w < g.heads * g.splits; w += g.heads) M = fmaxf(M, wm[w]);
  for (int w = hl; w < g.heads * g.splits; w += g.heads) {
    const float f = M == -INFINITY ? 0.f : exp2f(wm[w] - M);
    Z = fmaf(f, wl[w], Z);
  }
  const float inv = Z == 0.f ? 0.f : 1.f / Z;  // no visible row: zero (a NaN sum stays NaN)
  TO* out = static_cast<TO*>(a.o_lat) + qi * a.d_c;
  for (int d = lane; d < a.d_c; d += 32) {
    float v = 0.f;
    for (int w = hl; w < g.heads * g.splits; w += g.heads) {
      const float f = M == -INFINITY ? 0.f : exp2f(wm[w] - M);
      v = fmaf(f, om[w * a.d_c + d], v);
    }
    Store<TO>::st(out + d, v * inv);
  }
  if (a.lse != nullptr && lane == 0) a.lse[qi] = Z == 0.f ? -INFINITY : M + log2f(Z);
}

}  // namespace chunk
}  // namespace mla
