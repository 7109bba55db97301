// Block tables, positions and slot maps of a ragged step, from the requests'
// lengths.
//
// Request b holds cached[b] rows in its pages and brings new_[b] tokens.  Its
// table has have = ceil(cached / bs) pages and needs ceil((cached + new) / bs):
// the missing ones are taken from the free list, in the order of the requests.
// With the two prefix sums over the requests
//   cu[b]    = sum of new over the requests before b
//   first[b] = sum of missing pages over the requests before b
// every output is an independent gather: page k >= have of request b is
// free[head + first[b] + k - have]; token t of request b stands at position
// cached + t - cu[b], in slot page * bs + position mod bs.
//
// Requests whose tokens or pages do not fit any more (and all behind them) get
// no tokens and no pages; both prefix sums only grow, so "fits" is a prefix of
// the requests.  With fixed_rows a request with bad entries counts as one that does
// not fit, so that nothing behind it moves; without, it is passed over.
//
// What bounds it is latency: 8 bytes read a request, 16 bytes written a token.
// One cluster of 8 CTAs, each of which makes both prefix sums for itself
// (a scan of at most 16,384 values costs less than handing them round) and
// then fills its share of the tokens: 4 us for 64 requests of a token each (one CTA
// alone the same), 4.8 for 512 of 16 (13.2), 10.3 for 64 of 1024 (66), 16 for 16,384
// of one (72), one call behind the other in a graph.  Inputs that an output may replace (the
// lengths by seq_lens, the cursor by its new value) are read by all CTAs before
// the cluster's barrier and written behind it; one launch and no workspace.
#pragma once

#include "decode_pair.cuh"

namespace mla {
namespace tables {

constexpr int kMaxBatch = 16384;  // requests of a call: two prefix sums in shared memory
constexpr int kThreads = 1024;
constexpr int kCtas = 8;

struct Args {
  int batch, bs, n_free, num_blocks, max_blocks, n_tok;
  int fixed_rows;
  uint32_t inv;  // floor(2^32 / bs), at most 2^32 - 1
  const int32_t* cached;
  const int32_t* new_;
  const int32_t* free_blocks;
  const int32_t* free_head;
  int32_t* block_table;
  int32_t* cu_q;
  int32_t* seq_lens;
  int32_t* seq_idx;
  int32_t* pos;
  long long* slots;
  int32_t* head_out;
};

// x / bs and x mod bs for 0 <= x < 2^31: x inv / 2^32 is less than 1 below x / bs,
// so one step mends it.  77,000 tokens on 8 SMs are bound by their instructions:
// 14.7 us with divisions, 12.8 with this.
struct DivMod {
  int q, r;
  __device__ __forceinline__ DivMod(int x, const Args& a) {
    q = (int)__umulhi((uint32_t)x, a.inv);
    r = x - q * a.bs;
    if (r >= a.bs) {
      ++q;
      r -= a.bs;
    }
  }
};
__device__ __forceinline__ int pages_of(int rows, const Args& a) {
  const DivMod d(rows, a);
  return d.q + (d.r != 0);
}

// Inclusive sums over the block of two values per thread (64 bits: a sum of
// lengths that do not fit may pass 31).
__device__ __forceinline__ void scan2(long long& x, long long& y, long long (*tot)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += a;
      y += b;
    }
  }
  if (lane == 31) {
    tot[warp][0] = x;
    tot[warp][1] = y;
  }
  __syncthreads();
  if (warp == 0) {
    long long a = tot[lane][0], b = tot[lane][1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long c = __shfl_up_sync(0xffffffffu, a, o), d = __shfl_up_sync(0xffffffffu, b, o);
      if (lane >= o) {
        a += c;
        b += d;
      }
    }
    tot[lane][0] = a;
    tot[lane][1] = b;
  }
  __syncthreads();
  if (warp > 0) {
    x += tot[warp - 1][0];
    y += tot[warp - 1][1];
  }
}

// The last b of [lo, hi] with sums[b] <= t, given sums[lo] <= t.
__device__ __forceinline__ int last_at_most(const int* sums, int lo, int hi, int t) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sums[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) batch_tables_kernel(const Args a) {
  extern __shared__ int sm[];
  int* cu = sm;                      // [batch + 1]
  int* first = sm + a.batch + 1;     // [batch + 1]
  int* len = sm + 2 * (a.batch + 1); // [batch] cached rows
  __shared__ long long tot[32][2];
  __shared__ int served;
  const int tid = threadIdx.x, rank = (int)sm100::cluster_ctarank(), ctas = gridDim.x;
  pdl_wait();
  pdl_trigger();

  const int cursor = *a.free_head;
  const bool bad_head = cursor < 0 || cursor > a.n_free;
  const int head = bad_head ? a.n_free : cursor;  // bad: nothing to hand out, and the cursor stays what it is
  const int avail = a.n_free - head;
  // every request's own counts, until the scan
#pragma unroll 4
  for (int b = tid; b < a.batch; b += kThreads) {
    const int c = a.cached[b], w = a.new_[b];
    const long long rows = (long long)a.max_blocks * a.bs;
    const bool bad = c < 0 || w < 0 || (long long)c + w > rows;
    len[b] = bad && !(a.fixed_rows && c >= 0 && c <= rows) ? -1 : c;
    cu[b + 1] = bad ? 0 : w;
    first[b + 1] = bad ? -1 : pages_of(c + w, a) - pages_of(c, a);
  }
  const int per = (a.batch + kThreads - 1) / kThreads | 1;  // odd: the threads' runs begin in different banks
  if (per > 1) __syncthreads();
  const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
  long long n = 0, pages = 0;
  int miss = a.batch;  // the first request of this thread's that is not served
  for (int b = b0; b < b1; ++b) {
    int taken = first[b + 1];
    if (taken < 0) {
      if (rank == 0) report(MLA_ERR_BOUNDS, 30, b, a.cached[b] < 0 ? a.cached[b] : a.new_[b]);
      if (a.fixed_rows) miss = min(miss, b);
      first[b + 1] = taken = 0;
    }
    n += cu[b + 1];
    pages += taken;
  }
  if (tid == 0) {
    served = a.batch;
    cu[0] = first[0] = 0;
    if (bad_head && rank == 0) report(MLA_ERR_BOUNDS, 33, cursor, a.n_free);
  }
  const long long own_n = n, own_p = pages;
  scan2(n, pages, tot);
  n -= own_n;
  pages -= own_p;
  for (int b = b0; b < b1; ++b) {
    n += cu[b + 1];
    pages += first[b + 1];
    if (b >= miss || n > a.n_tok || pages > avail) {
      miss = b;
      break;
    }
    cu[b + 1] = (int)n;
    first[b + 1] = (int)pages;
  }
  if (miss < a.batch) atomicMin(&served, miss);
  __syncthreads();
  const int S = served;
  if (S < a.batch) {
    // the requests from S on: nothing new (their entries may hold raw counts)
    for (int b = S + tid; b < a.batch; b += kThreads) {
      cu[b + 1] = cu[S];
      first[b + 1] = first[S];
    }
    if (tid == 0 && rank == 0) report(MLA_ERR_BOUNDS, 31, S, a.batch);
    __syncthreads();
  }
  const int total = cu[a.batch];
  sm100::cluster_sync();  // every CTA has read the lengths and the cursor

  if (rank == 0) {
    for (int b = tid; b <= a.batch; b += kThreads) {
      a.cu_q[b] = cu[b];
      if (b < a.batch) a.seq_lens[b] = len[b] < 0 ? 0 : len[b] + (cu[b + 1] - cu[b]);
    }
    if (tid == 0) *a.head_out = bad_head ? cursor : head + first[a.batch];
  }
  // new table entries: one per page taken
  const int step = ctas * kThreads, me = rank * kThreads + tid;
  for (int i = me; i < first[a.batch]; i += step) {
    const int lo = last_at_most(first, 0, a.batch - 1, i);
    const int id = a.free_blocks[head + i];
    a.block_table[(long long)lo * a.max_blocks + pages_of(len[lo], a) + i - first[lo]] = id;
    if (id < 0 || id >= a.num_blocks) report(MLA_ERR_BOUNDS, 32, lo, id);
  }
  // tokens
  for (int t = me; t < a.n_tok; t += step) {
    int b = -1, p = 0;
    long long slot = -1;
    if (t < total) {
      b = last_at_most(cu, 0, a.batch - 1, t);
      p = len[b] + t - cu[b];
      const DivMod at(p, a);
      const int id = p - at.r < len[b] ? a.block_table[(long long)b * a.max_blocks + at.q]
                                       : a.free_blocks[head + first[b] + at.q - pages_of(len[b], a)];
      if (id < 0 || id >= a.num_blocks) report(MLA_ERR_BOUNDS, 32, b, id);
      else slot = (long long)id * a.bs + at.r;
    }
    a.seq_idx[t] = b;
    a.pos[t] = p;
    a.slots[t] = slot;
  }
}

inline mla_status launch(const Args& a, cudaStream_t s) {
  const size_t smem = sizeof(int) * (3 * (size_t)a.batch + 2);
  static std::atomic<uint64_t> attr{0};
  if (smem > 46 * 1024 &&
      pairdec::set_smem_once((const void*)batch_tables_kernel, sizeof(int) * (3 * (size_t)kMaxBatch + 2), attr) != MLA_OK)
    return MLA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cfg.gridDim.x;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  note_launch();
  return cudaLaunchKernelEx(&cfg, batch_tables_kernel, a) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace tables
}  // namespace mla
