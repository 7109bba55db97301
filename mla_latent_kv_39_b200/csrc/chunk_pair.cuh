// Attention of a ragged batch's new tokens over the paged latent cache on pairs
// of SMs (tcgen05 .cta_group::2), bf16, 128 heads, 512 + 64 wide rows.
//
// For every token t and head h, over the token's visible rows u
// (chunk_plan.cuh):
//   s_u = scale (q_lat . c_u + q_rope . k_R,u),   o_lat = sum_u softmax(s)_u c_u
// in one pass with the running maximum and sum.  In the absorbed form every
// head reads the same 576-wide row, so a token is a 128-row MMA operand and a
// page serves as keys and as values.
//
// A worker is a cluster of two CTAs; CTA r holds heads [64 r, 64 r + 64) of
// one token at a time: their scores and their whole 512-wide output fill its
// tensor memory.  A tile is four items (pages) of the token:
//   scores: pair MMAs M = 128 heads, N = 256 tokens, over 9 slabs of 64
//           values; CTA r supplies items 2 r and 2 r + 1;
//   P V:    pair MMAs M = 128, N = 256 latent columns, over 16 tokens a step;
//           of column block j CTA r supplies columns 256 j + 128 r + (0..127).
// N = 256 is what keeps the tensor pipe at its rate: a pair MMA with 64 rows
// per SM takes as long for 128 columns as for 256 (measured back to back:
// 64.8 clocks either way).
//
// Every operand slab is loaded by TMA into one ring of 16 KiB slots in the
// order in which the MMAs take them:
//   K(0), K(1), V(0), K(2), V(1), ...   (9 slots for K, 2 per page for V;
//   7 slots: 8 or 9 gained under 1%, 6 and 5 cost 2 and 9%),
// and the MMAs are issued in that order by one warp: the scores of tile i + 1
// run ahead of P V of tile i, into the other of two score buffers, so the
// softmax of a tile has the time of two MMA phases.  Keys are read a second
// time as values (an L2 hit): holding them from the scores to P V would take
// two tiles of shared memory.  Two warps take the ring's slots in turn, the
// loads issued under elect.sync (under `lane == 0` a load and its barrier work
// took 420 clocks, 19 B per clock and SM).
//
// What bounds it is the bandwidth of shared memory.  A tile moves 724 KB through
// each SM's: 414 KB of operands into the MMAs, 278 KB from TMA, 32 KB of P.  At
// 128 B per clock that is 5,656 clocks; measured are 5,620 a tile, with the
// tensor pipe at 68% over a whole call (its own time is 4,352).  8 sequences of
// 64 new tokens over 1k to 4k rows (315 GFLOP) take 252 to 302 us, 1.25 to 1.04
// PFLOP/s, on a cool GPU and behind minutes of load; 1,024 new tokens of a 16k
// request (4.53 TFLOP) 3.33 to 3.70 ms, 1.36 to 1.22 PFLOP/s, at the clock that the
// power limit leaves.  In decode steps, whose pages no two tokens share, a tile takes
// 10,000 clocks (5.2 us; 3.6 TB/s over 64 pairs) with its pages in HBM and 7,800 with
// them in L2, behind 7 us of planning and output where calls follow one another, some
// 15 with the launch of a call alone.
//
// Measured and left out: pages fetched into L2 ahead (bulk and single prefetches
// cost as much as the loads they go ahead of, 54 -> 61 us on a decode step of 64
// requests; plain loads neither gain nor lose); scores two tiles ahead, the output
// kept in registers or set aside in TMEM across pieces (1 to 14% slower); four load
// warps, eight more warps for the output (2 to 6% slower).
//
// TMEM (512 columns): scores [0, 128) and [128, 256), output [256, 512).
// A pair MMA of M = 128 leaves a CTA's 64 rows in 128 lanes x N / 2 columns:
// lane l holds head 64 r + (l mod 64), lanes 0..63 the first half of the N
// columns and lanes 64..127 the second.  So the softmax thread of lane l and
// column half ch owns one item of the tile, q = 2 (l / 64) + ch.
//
// Warp roles (384 threads): warps 0..7 softmax and output, warp 8 issues the
// MMAs (leader CTA), warps 9 and 10 load the ring, warp 11 plans the tiles and
// loads the queries.
//
// Rows that are not visible never reach an MMA: a page's box is shifted so
// that they fall outside the page and arrive as zeros, or, when the range is
// cut on both sides (only a window shorter than a page does that), it is read
// through a tensor map that ends at the range's last row.
//
// A worker's range of work may begin or end inside a token.  A token that one
// worker holds whole is written to o_lat at once, rounded once to bf16; the
// pieces of the others go to the workspace in fp32 with their log2-sum-exp
// (at most two pieces a worker, so the workspace does not grow with the
// tokens) and chunk_merge_kernel joins them.
//
// Every wait gives up after a time limit, records MLA_ERR_TIMEOUT and makes
// the roles wind down.
#pragma once

#include "chunk_plan.cuh"
#include "decode_pair.cuh"

namespace mla {
namespace chunk {

using namespace sm100;

constexpr int kH = 128, kHalfH = 64, kDc = 512, kDr = 64, kRow = kDc + kDr;
constexpr int kSlabs = kRow / 64;
constexpr int kSlab = 64 * 128;  // 64 rows x 64 bf16, 128-byte swizzle
constexpr int kKvSlot = 2 * kSlab;
constexpr int kTmemS = 0, kTmemO = 256, kTmemCols = 512;
constexpr int kSoftmaxWarps = 8, kMmaWarp = 8, kLoadWarp0 = 9, kLoadWarps = 2, kPlanWarp = 11;
constexpr int kThreads = 32 * 12;
constexpr float kRescaleLog2 = 8.f;
constexpr uint16_t kBoth = 3;
constexpr int kMaxWorkers = 1024;
static_assert((kLoadWarps & (kLoadWarps - 1)) == 0, "slots are dealt to the load warps by a mask");

// Ring slots: a key slab of two pages (in split-query mode followed by the
// low part of the query's slab), or 128 value columns of one page.
template <bool kSplit>
struct Geo {
  static constexpr int kSlot = kSplit ? kKvSlot + kSlab : kKvSlot;
  static constexpr int kSlots = kSplit ? 4 : 7;
};

// A tile as the load, MMA and softmax warps of a CTA need it, planned by its
// plan warp up to kTiles ahead; one with n = 0 comes behind the last.
struct Tile {
  int n;                   // items
  int first, last, whole;  // the tile begins / ends its piece; the piece is the whole token
  int tok, slot;           // the piece's token, its place in the workspace
  int phys[kTilePages], y[kTilePages], map[kTilePages];  // per item: page, first row of the box, tensor map
  int lo[kTilePages], hi[kTilePages];                    // visible columns of its 64 scores, as the box shifts them
};
constexpr int kTiles = 4;

// What the costs come to, over a warp's sequences.
struct Sums {
  long long cost, tokens, longest;
};
template <bool kSplit>
struct Smem {
  using G = Geo<kSplit>;
  uint8_t q[kSlabs][kSlab];                  // 64 heads x 576 values, K-major slabs; first member: 1024-byte aligned
  uint8_t p[kTilePages][kSlab];              // P of the tile: per item 64 heads x 64 tokens
  uint8_t ring[G::kSlots][G::kSlot];         // the prefix sums of the cut, then the ring
  uint64_t full[G::kSlots], empty[G::kSlots];
  uint64_t q_full, q_empty, s_full[2], p_full, pv_done, fin, xbar[2], lbar, tile_full[kTiles], tile_empty[kTiles];
  Tile tile[kTiles];
  Sums sums[kThreads / 32];
  float xm[2][2][128];                       // [tile parity][column half] maximum of each lane's columns
  float xl[2][2][128];                       // [tile parity][column half] shares of a finished piece's row sums
  uint32_t tmem_base;
  int abort_flag;
};

template <bool kSplit>
constexpr size_t smem_bytes() {
  return sizeof(Smem<kSplit>) + 1024;
}
static_assert(smem_bytes<false>() <= 232448 && smem_bytes<true>() <= 232448, "over the 227 KiB per-block limit");
static_assert(kSoftmaxWarps * 3 * 4096 <= 4 * (kKvSlot + kSlab) && kSoftmaxWarps * 3 * 4096 <= 7 * kKvSlot,
              "the last output's room fits the ring");
static_assert(sizeof(long long) * (kMaxBatch + 1) <= 4 * (kKvSlot + kSlab) &&
                  sizeof(long long) * (kMaxBatch + 1) <= 7 * kKvSlot,
              "the prefix sums fit the ring");

// Workspace: per worker its two pieces (0: the rest of a token begun by an
// earlier worker, 1: the beginning of a token that a later one goes on with).
struct Layout {
  int workers;
  long long off_shares, off_lse, off_o, total;
};
inline Layout layout(int workers) {
  Layout L{};
  L.workers = workers;
  size_t o = 0;
  L.off_shares = o; o = align_up(o + sizeof(Shares) * (size_t)workers, 256);
  L.off_lse = o;   o = align_up(o + sizeof(float) * 2 * (size_t)workers * kH, 256);
  L.off_o = o;     o = align_up(o + sizeof(float) * 2 * (size_t)workers * kH * kDc, 256);
  L.total = o;
  return L;
}

struct Params {
  Batch q;
  const int32_t* block_table;
  int max_blocks, num_blocks;
  float scale_log2;
  unsigned long long wait_ns;
  int workers;
  float inv_workers;
  int single;       // a token to a worker, whatever the costs (then no merge follows)
  Shares* shares;   // what the workers hold of cut tokens
  float* part_lse;
  float* part_o;
  bf16* o_lat;
  float* lse;
};

// Tensor maps of the pool: map r - 1 ends at row r of every page.  Only windows
// shorter than a page read through any but the last.
struct PoolMaps {
  CUtensorMap end[kPage];
};
struct PoolMap {
  CUtensorMap end[1];
};

__device__ __forceinline__ uint32_t leader(const uint64_t* bar) { return mapa(smem_u32(bar), 0); }
__device__ __forceinline__ uint64_t kmajor(const void* p) { return smem_desc(smem_u32(p), 16, 1024, kSwizzle128B); }
__device__ __forceinline__ uint64_t desc_add(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One lane of a converged warp, as a predicate that the compiler knows to hold
// for a single lane: MMAs, commits and loads issued under it take their operands
// from the uniform registers.  Issued under `lane == 0` the same instructions
// went through per-lane moves: a tile of 68 MMAs with its 17 waits and commits
// took 9,002 clocks, under elect 4,354, which is the pipe's own time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}

// 2-D tile store of a shared-memory box, tracked by this thread's bulk groups.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
               "r"(smem_u32(src)), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// All lanes of a converged warp wait; the outcome is the warp's.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int where, uint64_t wns) {
  const bool ok = mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, where, wns));
}

template <bool kSplit>
__device__ __forceinline__ void set_abort(Smem<kSplit>& sm) {
  *(volatile int*)&sm.abort_flag = 1;
}
template <bool kSplit>
__device__ __forceinline__ bool aborted(Smem<kSplit>& sm) {
  return uni(*(volatile int*)&sm.abort_flag) != 0;
}

// ---------------------------------------------------------------- the cut
__device__ __forceinline__ long long shfl64(long long v, int lane) { return __shfl_sync(0xffffffffu, v, lane); }
__device__ __forceinline__ Found found_of(const Found& f, int lane) {
  Found r;
  r.at = {__shfl_sync(0xffffffffu, f.at.b, lane), __shfl_sync(0xffffffffu, f.at.j, lane),
          __shfl_sync(0xffffffffu, f.at.k, lane)};
  r.s.t0 = __shfl_sync(0xffffffffu, f.s.t0, lane);
  r.s.n = __shfl_sync(0xffffffffu, f.s.n, lane);
  r.s.p0 = __shfl_sync(0xffffffffu, f.s.p0, lane);
  r.s.state = Sequence::kFine;
  r.base = shfl64(f.base, lane);
  return r;
}

// The costs of the sequences, summed up in `C` (shared memory), a run of them to
// each of kIds threads: a warp or, with `sums`, the whole block.
template <int kIds>
__device__ __forceinline__ Cut sum_costs(const Params& p, long long* C, Sums* sums) {
  const Batch& q = p.q;
  const int id = threadIdx.x % kIds, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (q.batch + kIds - 1) / kIds, b0 = min(id * per, q.batch), b1 = min(b0 + per, q.batch);
  Cut cut{0, p.workers, p.inv_workers, 0};
  long long mine = 0, longest = 0;
  long long own = 0;  // tokens of this thread's run
  for (int b = b0; b < b1; ++b) {
    const Sequence s = sequence_of(q, b);
    if (blockIdx.x == 0) report_sequence(q, b, s);
    mine += cut.tokens(q.vis, s, s.n);
    own += s.n;
    longest = max(longest, longest_token(q.vis, s));
    C[b + 1] = mine;
  }
  long long x = mine;
  long long t = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    const long long u = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) {
      x += y;
      t += u;
    }
    longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
  }
  cut.total = shfl64(x, 31);
  long long tokens = shfl64(t, 31);
  if constexpr (kIds > 32) {
    if (lane == 0) sums[warp] = Sums{cut.total, tokens, longest};
    __syncthreads();
    cut.total = tokens = 0;
    for (int w = 0; w < kIds / 32; ++w) {
      const Sums o = sums[w];
      if (w < warp) {
        x += o.cost;
        t += o.tokens;
      }
      cut.total += o.cost;
      tokens += o.tokens;
      longest = max(longest, o.longest);
    }
  }
  long long ahead = x - mine;
  if (p.single || one_token_each(tokens, cut.total, longest, p.workers)) {
    cut.single = 1;
    cut.total = tokens;
    ahead = t - own;
    mine = 0;
    for (int b = b0; b < b1; ++b) C[b + 1] = mine += sequence_of(q, b).n;
  }
  for (int b = b0; b < b1; ++b) C[b + 1] += ahead;
  if (id == 0) C[0] = 0;
  return cut;
}

// Up to kWarpBatch sequences the plan warp does it alone while the others go to
// their roles; above, the whole block does it ahead of the roles.  A call with 16
// new tokens takes, by warp and by block, 21.8 and 23.4 us for 64 sequences, 22.5
// and 23.5 for 128, 24.2 and 23.7 for 256, 28.6 and 24.4 for 512; for 8192 of
// 100 rows 230 and 48.  Out of line, so that it does not weigh on the registers of
// what follows (inlined: 4 us more on a decode step of 100,000 rows).
constexpr int kWarpBatch = 128;
static __device__ __noinline__ Cut sum_costs_of_block(const Params& p, long long* C, Sums* sums) {
  const Cut cut = sum_costs<kThreads>(p, C, sums);
  fence_proxy_async_smem();  // the sums give way to the ring's loads
  __syncthreads();
  return cut;
}

// The two ends of this worker's range, by one warp: lane 0 looks for the one end
// and lane 1 for the other.
__device__ __forceinline__ void find_range(const Params& p, const Cut& cut, const long long* C, int worker, int lane,
                                           Found& from, Found& to) {
  const Found f = place_at(p.q, cut, C, cut.at(worker + (lane & 1)));
  from = found_of(f, 0);
  to = found_of(f, 1);
  __syncwarp();
}

// ---------------------------------------------------------------- tile records
// Record i of the ring: false if the wait ran out.  A warp that has copied what
// it needs releases it.
template <bool kSplit>
__device__ __forceinline__ bool wait_tile(Smem<kSplit>& sm, int i, uint64_t wns) {
  return warp_wait(&sm.tile_full[i % kTiles], (i / kTiles) & 1, 42, wns);
}
template <bool kSplit>
__device__ __forceinline__ void release_tile(Smem<kSplit>& sm, int i, bool one) {
  __syncwarp();
  if (one) mbar_arrive(&sm.tile_empty[i % kTiles]);
}

// ---------------------------------------------------------------- TMA producers
// Both CTAs' load warps arrive on every slot, also where a CTA has nothing to
// load (a tile of one or two items): the MMAs never run more than a ring ahead
// of either, so a phase of `empty` is always seen before the next one ends.
template <bool kSplit, typename Maps>
struct Loader {
  using G = Geo<kSplit>;
  Smem<kSplit>& sm;
  const Maps& pool;
  const CUtensorMap* qlo;
  const Params& p;
  const int me, rank;
  const bool one;  // the issuing lane
  int sl = 0, use = 0, g = 0;  // ring slot, its use, running count

  __device__ bool mine() const { return (g & (kLoadWarps - 1)) == me; }
  __device__ void step() {
    ++g;
    if (++sl == G::kSlots) {
      sl = 0;
      ++use;
    }
  }
  __device__ bool ready() {
    return use == 0 || warp_wait(&sm.empty[sl], (use - 1) & 1, 40, p.wait_ns);
  }
  // the 9 key slabs of a tile of n items of token `tok`; lane i holds item i
  __device__ bool keys(int3 it, int n, int tok) {
    const int phys[2] = {__shfl_sync(0xffffffffu, it.x, 2 * rank), __shfl_sync(0xffffffffu, it.x, 2 * rank + 1)};
    const int y[2] = {__shfl_sync(0xffffffffu, it.y, 2 * rank), __shfl_sync(0xffffffffu, it.y, 2 * rank + 1)};
    const int m[2] = {__shfl_sync(0xffffffffu, it.z, 2 * rank), __shfl_sync(0xffffffffu, it.z, 2 * rank + 1)};
#pragma unroll 1
    for (int e = 0; e < kSlabs; ++e, step()) {
      if (!mine()) continue;
      if (!ready()) return false;
      if (one) {
        const uint32_t bar = leader(&sm.full[sl]);
        if (rank == 0) mbar_arrive_expect_tx(&sm.full[sl], n * kSlab + (kSplit ? 2 * kSlab : 0));
        else mbar_arrive_remote(bar);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (2 * rank + h < n) tma_load_3d_pair(sm.ring[sl] + h * kSlab, &pool.end[m[h]], 64 * e, y[h], phys[h], bar);
        if (kSplit) tma_load_2d_pair(sm.ring[sl] + kKvSlot, qlo, 64 * e, tok * kH + kHalfH * rank, bar);
      }
      __syncwarp();
    }
    return true;
  }
  // the value columns of a tile of n items: per item two blocks of 256 columns
  __device__ bool values(int3 it, int n) {
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int phys = __shfl_sync(0xffffffffu, it.x, i), y = __shfl_sync(0xffffffffu, it.y, i),
                m = __shfl_sync(0xffffffffu, it.z, i);
#pragma unroll 1
      for (int j = 0; j < 2; ++j, step()) {
        if (!mine()) continue;
        if (!ready()) return false;
        if (one) {
          const uint32_t bar = leader(&sm.full[sl]);
          if (rank == 0) mbar_arrive_expect_tx(&sm.full[sl], 2 * kKvSlot);
          else mbar_arrive_remote(bar);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            tma_load_3d_pair(sm.ring[sl] + h * kSlab, &pool.end[m], 256 * j + 128 * rank + 64 * h, y, phys, bar);
        }
        __syncwarp();
      }
    }
    return true;
  }
};

template <bool kSplit, typename Maps>
__device__ void load_role(Smem<kSplit>& sm, const Maps& pool, const CUtensorMap* qlo, const Params& p, int me, int rank,
                          int lane) {
  Loader<kSplit, Maps> ld{sm, pool, qlo, p, me, rank, elect_one()};
  int3 prev = make_int3(0, 0, 0);
  int n_prev = 0;
  bool ok = true;
  for (int i = 0;; ++i) {
    ok = ok && wait_tile(sm, i, p.wait_ns);
    if (!ok) break;
    const Tile& t = sm.tile[i % kTiles];
    const int n = uni(t.n), tok = uni(t.tok), k = lane % kTilePages;
    const int3 it = make_int3(t.phys[k], t.y[k], t.map[k]);
    if (n == 0) break;
    release_tile(sm, i, ld.one);
    ok = ld.keys(it, n, tok) && ld.values(prev, n_prev) && !aborted(sm);
    prev = it;
    n_prev = n;
  }
  if (ok) ok = ld.values(prev, n_prev);
  if (!ok) set_abort(sm);
}

// Finds the worker's range and walks it: plans the tiles, loads a piece's
// queries once the scores of the one before are done, and, as no other warp meets
// them, writes the rows of tokens that see nothing (zeros, log-sum-exp of an
// empty set) and what the merge needs to know.
template <bool kSplit, typename Maps>
__device__ void plan_role(Smem<kSplit>& sm, const CUtensorMap* qmap, const Params& p, Cut cut, int rank, int worker,
                          int lane) {
  constexpr int kWhole = sizeof(Maps) / sizeof(CUtensorMap) - 1;
  const bool one = elect_one();
  int pieces = 0, i = 0;
  const auto slot_free = [&] {
    return i < kTiles || warp_wait(&sm.tile_empty[i % kTiles], (i / kTiles - 1) & 1, 43, p.wait_ns);
  };
  const auto give_up = [&] {  // nothing to merge
    set_abort(sm);
    if (rank == 0 && one) p.shares[worker] = Shares{-1, -1, worker, -1};
  };
  const auto load_query = [&](int tok) {
    if (one) {
      if (rank == 0) mbar_arrive_expect_tx(&sm.q_full, 2 * kSlabs * kSlab);
      for (int e = 0; e < kSlabs; ++e)
        tma_load_2d_pair(sm.q[e], qmap, 64 * e, tok * kH + kHalfH * rank, leader(&sm.q_full));
    }
    __syncwarp();
  };
  long long* C = reinterpret_cast<long long*>(sm.ring);
  if (p.q.batch <= kWarpBatch) {
    cut = sum_costs<32>(p, C, nullptr);
    __syncwarp();
  }
  Found from, to;
  find_range(p, cut, C, worker, lane, from, to);
  fence_proxy_async_smem();  // the prefix sums give way to the ring's loads
  __syncwarp();
  for (Walk w(p.q, from.at, from.s, to.at); w.valid(); w.next()) {
    const int tok = w.token(), nt = w.tiles();
    if (nt == 0) {
      const long long row = (long long)tok * kH + kHalfH * rank;
      uint4* dst = reinterpret_cast<uint4*>(p.o_lat + row * kDc);
      for (int k = lane; k < kHalfH * kDc / 8; k += 32) dst[k] = make_uint4(0, 0, 0, 0);
      if (p.lse != nullptr)
        for (int h = lane; h < kHalfH; h += 32) p.lse[row + h] = -INFINITY;
      __syncwarp();
      continue;
    }
    if (pieces == 0) load_query(tok);
    for (int t = 0; t < nt; ++t, ++i) {
      const int k0 = w.at.k + t * kTilePages, n = min(kTilePages, w.k1 - k0);
      int phys = p.num_blocks, y = 0, m = kWhole, lo = 0, hi = 0;
      if (lane < n) {
        const Item it = item_of(p.q.vis, w.position(), k0 + lane);
        phys = p.block_table[(long long)w.at.b * p.max_blocks + it.page];
        if (it.a == 0) {  // rows past the range fall behind the page's top, negative rows arrive as zeros
          y = it.b - kPage;
          lo = kPage - it.b;
          hi = kPage;
        } else {
          y = it.a;
          hi = it.b - it.a;
          if (it.b < kPage) m = it.b - 1;  // only with a map for every end, see chunk_tc_impl
        }
        if (phys < 0 || phys >= p.num_blocks) {
          if (rank == 0) report(MLA_ERR_BOUNDS, 22, w.at.b, phys);
          phys = p.num_blocks;  // outside the pool: arrives as zeros, and is not visible
          lo = hi = 0;
        }
      }
      if (!slot_free()) return give_up();
      Tile& d = sm.tile[i % kTiles];
      if (lane < kTilePages) {
        d.phys[lane] = phys;
        d.y[lane] = y;
        d.map[lane] = m;
        d.lo[lane] = lo;
        d.hi[lane] = hi;
      }
      if (one) {
        d.n = n;
        d.first = t == 0;
        d.last = t == nt - 1;
        d.whole = w.whole();
        d.tok = tok;
        d.slot = 2 * worker + (w.at.k > 0 ? 0 : 1);
      }
      __syncwarp();
      if (one) mbar_arrive(&sm.tile_full[i % kTiles]);
      __syncwarp();
      if (t == 0 && pieces++ > 0) {  // with the tile handed out, its query follows when the one before is done with
        if (!warp_wait(&sm.q_empty, (pieces - 2) & 1, 41, p.wait_ns)) return give_up();
        load_query(tok);
      }
    }
  }
  if (!slot_free()) return give_up();
  if (one) {
    sm.tile[i % kTiles].n = 0;
    mbar_arrive(&sm.tile_full[i % kTiles]);
  }
  __syncwarp();
  const Shares e = shares_of(p.q, cut, from, to, worker);
  if (rank == 0 && one) p.shares[worker] = e;
  if (e.continues < 0)  // nothing of this worker's in its first place
    for (int h = lane; h < kHalfH; h += 32) p.part_lse[2LL * worker * kH + kHalfH * rank + h] = -INFINITY;
  __syncwarp();
}

// ---------------------------------------------------------------- MMA issuer (leader CTA)
template <bool kSplit>
struct Issuer {
  using G = Geo<kSplit>;
  static constexpr uint32_t kIdS = idesc_bf16_f32(128, 256, 0, 0), kIdO = idesc_bf16_f32(128, 256, 0, 1);
  Smem<kSplit>& sm;
  const uint32_t tmem;
  const uint64_t wns;
  const bool one;  // the issuing lane
  const uint64_t qd, pd, kd, vd;
  int sl = 0, ph = 0, nq = 0;
  __device__ Issuer(Smem<kSplit>& s, uint32_t t, uint64_t w)
      : sm(s), tmem(t), wns(w), one(elect_one()), qd(kmajor(s.q)), pd(kmajor(s.p)), kd(kmajor(s.ring)),
        // values as the MN-major operand: 64-column slabs 8 KiB apart, 8-token groups 1 KiB apart
        vd(smem_desc(smem_u32(s.ring), kSlab, 1024, kSwizzle128B)) {}
  __device__ void step() {
    if (++sl == G::kSlots) {
      sl = 0;
      ph ^= 1;
    }
  }
  // what the MMAs need of a tile's record
  struct Next {
    int n;
    bool first, last;
  };
  __device__ bool look(int i, Next& t) {
    if (!wait_tile(sm, i, wns)) return false;
    const Tile& r = sm.tile[i % kTiles];
    t.n = uni(r.n);
    t.first = uni(r.first);
    t.last = uni(r.last);
    release_tile(sm, i, one);
    return true;
  }
  // The scores of tile i; on the way, with MMAs in the pipe, the record of the
  // tile behind it is read.
  __device__ bool scores(int i, bool first, bool last, Next& ahead) {
    if (first && !warp_wait(&sm.q_full, nq++ & 1, 50, wns)) return false;
    const uint32_t d = tmem + kTmemS + 128 * (i & 1);
#pragma unroll
    for (int e = 0; e < kSlabs; ++e, step()) {
      if (!warp_wait(&sm.full[sl], ph, 51, wns)) return false;
      tc_fence_after();
      if (one) {
        const uint64_t a = qd + e * (kSlab >> 4), b = kd + (uint32_t)sl * (G::kSlot >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_ss_pair(d, a + 2 * k, b + 2 * k, kIdS, (e | k) ? 1u : 0u);
        if (kSplit) {
          const uint64_t al = b + (kKvSlot >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_ss_pair(d, al + 2 * k, b + 2 * k, kIdS, 1u);
        }
        mma_commit_pair(&sm.empty[sl], kBoth);
        if (e == kSlabs - 1) {
          mma_commit_pair(&sm.s_full[i & 1], kBoth);
          if (last) mma_commit_pair(&sm.q_empty, kBoth);
        }
      }
      __syncwarp();
      if (e == kSlabs / 2 && !look(i + 1, ahead)) return false;
    }
    return true;
  }
  // P V of tile i of n items; `first`: it begins its token's output
  __device__ bool values(int i, int n, bool first) {
    if (!warp_wait(&sm.p_full, i & 1, 52, wns)) return false;
    tc_fence_after();
#pragma unroll
    for (int q = 0; q < kTilePages; ++q) {
      if (q >= n) break;
#pragma unroll
      for (int j = 0; j < 2; ++j, step()) {
        if (!warp_wait(&sm.full[sl], ph, 53, wns)) return false;
        tc_fence_after();
        if (one) {
          const uint64_t a = pd + q * (kSlab >> 4), b = vd + (uint32_t)sl * (G::kSlot >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss_pair(tmem + kTmemO + 128 * j, a + 2 * k, b + 128 * k, kIdO, (first && q == 0 && k == 0) ? 0u : 1u);
          mma_commit_pair(&sm.empty[sl], kBoth);
        }
        __syncwarp();
      }
    }
    if (one) mma_commit_pair(&sm.pv_done, kBoth);
    __syncwarp();
    return true;
  }
};

template <bool kSplit>
__device__ void mma_role(Smem<kSplit>& sm, uint32_t tmem, const Params& p) {
  Issuer<kSplit> is(sm, tmem, p.wait_ns);
  typename Issuer<kSplit>::Next t, ahead;
  int i = 0, n_prev = 0;
  bool first_prev = false, ok = is.look(0, t);
  for (; ok && t.n > 0; ++i) {
    ok = is.scores(i, t.first, t.last, ahead) && (i == 0 || is.values(i - 1, n_prev, first_prev));
    n_prev = t.n;
    first_prev = t.first;
    t = ahead;
  }
  if (ok && i > 0) ok = is.values(i - 1, n_prev, first_prev);
  if (!ok) set_abort(sm);
  if (is.one) mma_commit_pair(&sm.fin, 1);
  warp_wait(&sm.fin, 0, 54, p.wait_ns);
}

// ---------------------------------------------------------------- softmax and output
// Two floats in one register pair: one instruction for both.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <bool kSplit>
struct Softmax {
  Smem<kSplit>& sm;
  const Params& p;
  const CUtensorMap* omap;         // o_lat
  const CUtensorMap* partmap;      // the workspace's pieces
  const uint32_t tl;               // this warp's TMEM lane quarter
  const int lane, l, half, ch, head;
  const bool one;                  // the issuing lane

  // A piece whose output is in TMEM: its row sum, its maximum (in units of the
  // raw scores) and where it goes.
  struct Piece {
    float sum, m;
    int tok, slot, whole;
    __device__ float inv() const { return sum == 0.f ? 0.f : 1.f / sum; }  // no visible row: zero (a NaN sum stays NaN)
  };

  // The row sum of this thread's head from the shares of its four threads, in
  // one order for all of them.
  __device__ float row_sum(const float (&xl)[2][128]) const {
    const int l0 = l & 63;
    return (xl[0][l0] + xl[1][l0]) + (xl[0][l0 + 64] + xl[1][l0 + 64]);
  }
  __device__ void store_lse(const Piece& d) {
    if (half != 0 || ch != 0) return;
    const float lse = d.sum == 0.f ? -INFINITY : fmaf(d.m, p.scale_log2, log2f(d.sum));
    if (!d.whole) p.part_lse[(long long)d.slot * kH + head] = lse;
    else if (p.lse != nullptr) p.lse[(long long)d.tok * kH + head] = lse;
  }

  // The finished piece's output: this warp's 32 heads x 128 columns (256 ch +
  // 128 half on), a lane a head, go out through the warp's own 4 KiB of the P
  // buffer (free until this tile's P is written there) by bulk tensor stores: a
  // whole token's in bf16 to o_lat, 64 columns a pass, a part's in fp32 to the
  // workspace, 32 columns a pass.  Plain stores, a row to a lane, kept the warps
  // 2.8 us a token; here the tensor pipe computes the next tile's scores meanwhile.
  __device__ void own_free() {  // the bulk stores have read what was there
    if (one) bulk_wait_read_all();
    __syncwarp();
  }
  __device__ void put(uint8_t* own, const uint32_t (&v)[32], const CUtensorMap* map, int x, int y) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      *reinterpret_cast<uint4*>(own + lane * 128 + ((c ^ (lane & 7)) << 4)) =
          make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (one) {
      tma_store_2d(map, own, x, y);
      bulk_commit_group();
    }
    __syncwarp();
  }
  // `room`: 12 KiB more of this warp's where nothing is loaded any more (the ring,
  // behind the last piece), so that no pass waits for the one before; or null.
  __device__ void write_out(uint8_t* own, uint8_t* room, const Piece& d) {
    const float inv = d.inv();
    const int col = 256 * ch + 128 * half, row0 = head - lane;  // the warp's first head
    if (d.whole) {
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t v[32];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t a[32];
          tmem_ld32(tl + kTmemO + 128 * ch + 64 * c + 32 * e, a);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k)
            v[16 * e + k] = pack_bf16x2(__uint_as_float(a[2 * k]) * inv, __uint_as_float(a[2 * k + 1]) * inv);
        }
        if (c > 0 && room == nullptr) own_free();
        put(c > 0 && room != nullptr ? room : own, v, omap, col + 64 * c, d.tok * kH + row0);
      }
    } else {
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t v[32];
        tmem_ld32(tl + kTmemO + 128 * ch + 32 * c, v);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * inv);
        if (c > 0 && room == nullptr) own_free();
        put(c > 0 && room != nullptr ? room + (c - 1) * 4096 : own, v, partmap, col + 32 * c, d.slot * kH + row0);
      }
    }
    tc_fence_before();
  }

  __device__ bool run() {
    float m_used = -INFINITY, lsum = 0.f;
    Piece open{0.f, 0.f, 0, 0, 0};
    int i = 0;
    const int q = 2 * half + ch;                        // this warp's item of every tile
    uint8_t* own = sm.p[q] + ((l & 63) - lane) * 128;   // its 32 rows of the item's P slab
    for (;; ++i) {
      if (!wait_tile(sm, i, p.wait_ns)) return false;
      const Tile& t = sm.tile[i % kTiles];
      const int n = uni(t.n);
      if (n == 0) break;
      const bool first = uni(t.first);
      const int lo = uni(t.lo[q]), hi = uni(t.hi[q]);
      const int tok = uni(t.tok), slot = uni(t.slot), whole = uni(t.whole);
      release_tile(sm, i, one);
      if (!warp_wait(&sm.s_full[i & 1], (i >> 1) & 1, 62, p.wait_ns)) return false;
      tc_fence_after();
      float s[64];
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (hi > lo) {
        uint32_t a[32], b[32];
        const uint32_t at = tl + kTmemS + 128 * (i & 1) + 64 * ch;
        tmem_ld32(at, a);
        tmem_ld32(at + 32, b);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          s[c] = __uint_as_float(a[c]);
          s[32 + c] = __uint_as_float(b[c]);
        }
        if (hi - lo < kPage) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c < lo || c >= hi) s[c] = -INFINITY;
        }
#pragma unroll
        for (int c = 0; c < 64; ++c) mx[c & 3] = fmaxf(mx[c & 3], s[c]);
      }
      tc_fence_before();
      const bool close = first && i > 0;  // another piece's output is still in TMEM
      sm.xm[i & 1][ch][l] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      if (close) sm.xl[i & 1][ch][l] = lsum;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.xbar[i & 1]);
      if (!warp_wait(&sm.xbar[i & 1], (i >> 1) & 1, 63, p.wait_ns)) return false;
      const float m_tile = fmaxf(fmaxf(sm.xm[i & 1][0][l], sm.xm[i & 1][1][l]),
                                 fmaxf(sm.xm[i & 1][0][l ^ 64], sm.xm[i & 1][1][l ^ 64]));
      if (first) {
        if (close) open.sum = row_sum(sm.xl[i & 1]);
        open.m = m_used;
        m_used = -INFINITY;
        lsum = 0.f;
      }
      // rescale only when P could grow past 2^8: P and O are exact in the scale
      float alpha = 1.f;
      const bool rescale = (m_tile - m_used) * p.scale_log2 > kRescaleLog2;  // never from -inf to -inf (NaN)
      if (rescale) {
        alpha = exp2_fast((m_used - m_tile) * p.scale_log2);  // 0 at the piece's first finite maximum
        m_used = m_tile;
      }
      const float base = m_used == -INFINITY ? 0.f : -m_used * p.scale_log2;
      // P goes into the MMA in bf16, as the values do (both operands of an MMA have one
      // type, and one in fp32 would be read at half the rate): half a step of 2^-8 a weight, of either sign, which
      // leaves o_lat 0.0021 (rms, relative) from the exact result where rounding that
      // result alone leaves 0.0017.  The row sum takes the unrounded weights, so the
      // log-sum-exp has none of it; sums and the pieces' outputs are fp32.
      uint32_t pk[32];
      if (hi > lo) {
        const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2), base2 = pack2(base, base);
        uint64_t sum2[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          float x, y;
          unpack2(fma2(pack2(s[2 * c], s[2 * c + 1]), scale2, base2), x, y);
          x = exp2_fast(x);
          y = exp2_fast(y);
          sum2[c & 1] = add2(sum2[c & 1], pack2(x, y));
          pk[c] = pack_bf16x2(x, y);
        }
        float x, y;
        unpack2(add2(sum2[0], sum2[1]), x, y);
        lsum = fmaf(lsum, alpha, x + y);
      } else {
        lsum *= alpha;
#pragma unroll
        for (int c = 0; c < 32; ++c) pk[c] = 0;
      }

      // P V of the tile before reads P and adds to O: it must be over before
      // this tile writes P, rescales O or hands O to the next piece.
      if (i >= 1) {
        if (!warp_wait(&sm.pv_done, (i - 1) & 1, 64, p.wait_ns)) return false;
        tc_fence_after();
      }
      if (!first && __any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          const uint32_t a = tl + kTmemO + 128 * ch + 32 * c;
          tmem_ld32(a, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          tmem_st32(a, o);
        }
        tmem_wait_st();
      }
      if (close) {
        write_out(own, nullptr, open);
        store_lse(open);
        own_free();
      }
      // row l mod 64 of the item's P slab, K-major with the 128-byte swizzle
      if (q < n) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(own + lane * 128 + ((c ^ (lane & 7)) << 4)) =
              make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(leader(&sm.p_full));
      if (first) {
        open.tok = tok;
        open.slot = slot;
        open.whole = whole;
      }
    }
    if (i > 0) {  // the last piece
      sm.xl[i & 1][ch][l] = lsum;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.lbar);
      if (!warp_wait(&sm.lbar, 0, 60, p.wait_ns) || !warp_wait(&sm.pv_done, (i - 1) & 1, 65, p.wait_ns)) return false;
      tc_fence_after();
      open.sum = row_sum(sm.xl[i & 1]);
      open.m = m_used;
      store_lse(open);
      write_out(own, sm.ring[0] + (4 * ch + 2 * half + ((l >> 5) & 1)) * 3 * 4096, open);
    }
    if (one) bulk_wait_all();
    __syncwarp();
    return true;
  }
};

// ---------------------------------------------------------------- kernel
template <bool kSplit, typename Maps>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    chunk_pair_kernel(const __grid_constant__ Maps pool, const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ CUtensorMap qlomap, const __grid_constant__ CUtensorMap omap,
                      const __grid_constant__ CUtensorMap partmap, const __grid_constant__ Params p) {
  using G = Geo<kSplit>;
  extern __shared__ uint8_t smem_raw[];
  Smem<kSplit>& sm =
      *reinterpret_cast<Smem<kSplit>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = uni(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank(), worker = blockIdx.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < G::kSlots; ++s) {
      mbar_init(&sm.full[s], 2);
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.s_full[b], 1);
      mbar_init(&sm.xbar[b], kSoftmaxWarps);
    }
    mbar_init(&sm.p_full, 2 * kSoftmaxWarps);
    mbar_init(&sm.pv_done, 1);
    mbar_init(&sm.lbar, kSoftmaxWarps);
    for (int b = 0; b < kTiles; ++b) {
      mbar_init(&sm.tile_full[b], 1);
      mbar_init(&sm.tile_empty[b], kSoftmaxWarps + kLoadWarps + (rank == 0 ? 1 : 0));  // the MMA warp works in rank 0
    }
    mbar_init(&sm.fin, 1);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc_pair(&sm.tmem_base, kTmemCols);
    tmem_relinquish_pair();
  }
  if (warp == kPlanWarp && lane == 0) {
    prefetch_tensormap(&pool.end[sizeof(Maps) / sizeof(CUtensorMap) - 1]);
    prefetch_tensormap(&qmap);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are initialised
  tc_fence_after();
  const uint32_t tmem = uni(sm.tmem_base);
  pdl_wait();  // the queries, the tables and the appended rows come from the kernels before
  pdl_trigger();
  Cut cut{};
  if (p.q.batch > kWarpBatch) cut = sum_costs_of_block(p, reinterpret_cast<long long*>(sm.ring), sm.sums);

  if (warp < kSoftmaxWarps) {
    const int l = (warp & 3) * 32 + lane;
    Softmax<kSplit> so{sm, p, &omap, &partmap, tmem + ((uint32_t)((warp & 3) * 32) << 16), lane, l, l >> 6, warp >> 2,
                       kHalfH * rank + (l & 63), elect_one()};
    if (!so.run()) set_abort(sm);
  } else if (warp == kMmaWarp) {
    if (rank == 0) mma_role(sm, tmem, p);
  } else if (warp == kPlanWarp) {
    plan_role<kSplit, Maps>(sm, &qmap, p, cut, rank, worker, lane);
  } else {
    load_role<kSplit, Maps>(sm, pool, &qlomap, p, warp - kLoadWarp0, rank, lane);
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's MMAs and remote arrives are over before TMEM and shared memory go away
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- merge
// Joins the pieces of the tokens that several workers share:
//   o_lat = sum_i 2^(lse_i - M) O_i / sum_i 2^(lse_i - M).
// Grid (workers, 8); most calls' workers share few tokens or none, and a block
// without work costs its launch, so there are few.  join_of (chunk_plan.cuh) says
// which block joins what: of a token of few pieces four heads at a time, one to each
// 64 threads; of a token of many pieces (a long request) half a head at a time, the
// pieces dealt to the eight warps, over the blocks of up to 32 workers: 256 blocks
// that read 75 KB each of 74 pieces (28 us by 32 blocks of whole heads, 13 us by 128
// of one head).  A thread owns 8 latent columns; three loads are in flight, under no
// condition.  An idle worker's place counts as a piece without visible rows (lse
// -inf).  Sums run in a fixed order.
constexpr int kMergeThreads = 256;

__global__ void __launch_bounds__(kMergeThreads, 4) chunk_merge_kernel(const Shares* __restrict__ shares,
                                                                       const float* __restrict__ part_lse,
                                                                       const float* __restrict__ part_o,
                                                                       bf16* __restrict__ o_lat,
                                                                       float* __restrict__ lse_out) {
  pdl_wait();
  pdl_trigger();
  __shared__ float wt[kMaxWorkers + 4 * kMergeFew];  // weights: one list of many, or four of few
  __shared__ float4 sum[kMergeThreads / 32][2][32];
  const int w = blockIdx.x;
  const Join j = join_of(shares, w);
  const int tok = j.token, w0 = j.first, n = j.n, items = j.items(kH), step_item = j.step();
  if (tok < 0) return;
  const bool many = j.many();
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  float* list = many ? wt : wt + kMergeFew * (warp / 2);
  // piece i: the beginning with worker w0, the rest with the workers behind it
  const auto slot_of = [&](int i) { return 2 * (w0 + i) + (i == 0 ? 1 : 0); };
  for (int it = j.begin(w, blockIdx.y); it < items; it += step_item) {
    const int h = many ? it / 2 : 4 * it + warp / 2;
    const int d = many ? kDc / 2 * (it & 1) + 8 * lane : 8 * (threadIdx.x % 64);
    if (many ? warp == 0 : warp % 2 == 0) {
      float M = -INFINITY, Z = 0.f;
      for (int i = lane; i < n; i += 32) {
        const float x = part_lse[(long long)slot_of(i) * kH + h];
        list[i] = x;
        M = fmaxf(M, x);
        if (x != x) Z = x;  // the maximum passes over NaN, the sum must not
      }
      M = warp_max(M);
      for (int i = lane; i < n; i += 32) {
        const float x = M == -INFINITY ? 0.f : exp2f(list[i] - M);  // M = -inf: no piece has a visible row
        list[i] = x;
        Z += x;
      }
      Z = warp_sum(Z);
      const float inv = Z == 0.f ? 0.f : 1.f / Z;
      for (int i = lane; i < n; i += 32) list[i] *= inv;
      if (lse_out != nullptr && lane == 0 && d < kDc / 2)
        lse_out[(long long)tok * kH + h] = Z == 0.f ? -INFINITY : M + log2f(Z);
    }
    __syncthreads();
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const auto add = [&](int i, const float4& x, const float4& y) {
      const float f = i < n ? list[i] : 0.f;
      const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] = fmaf(f, f == 0.f ? 0.f : v[c], acc[c]);  // weight 0: nothing was written there
    };
    const auto at = [&](int i) {
      return reinterpret_cast<const float4*>(part_o + ((long long)slot_of(min(i, n - 1)) * kH + h) * kDc + d);
    };
    const int step = many ? kMergeThreads / 32 : 1;
    for (int i = many ? warp : 0; i < n; i += 3 * step) {
      const float4 x0 = __ldcs(at(i)), y0 = __ldcs(at(i) + 1);
      const float4 x1 = __ldcs(at(i + step)), y1 = __ldcs(at(i + step) + 1);
      if (n > 2) {
        const float4 x2 = __ldcs(at(i + 2 * step)), y2 = __ldcs(at(i + 2 * step) + 1);
        add(i, x0, y0);
        add(i + step, x1, y1);
        add(i + 2 * step, x2, y2);
      } else {
        add(i, x0, y0);
        add(i + 1, x1, y1);
      }
    }
    if (many) {
      sum[warp][0][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      sum[warp][1][lane] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int g = 1; g < kMergeThreads / 32; ++g) {
            const float4 v = sum[g][e][lane];
            acc[4 * e] += v.x;
            acc[4 * e + 1] += v.y;
            acc[4 * e + 2] += v.z;
            acc[4 * e + 3] += v.w;
          }
      }
    }
    if (!many || warp == 0)
      *reinterpret_cast<uint4*>(o_lat + ((long long)tok * kH + h) * kDc + d) =
          make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]), pack_bf16x2(acc[4], acc[5]),
                     pack_bf16x2(acc[6], acc[7]));
    __syncthreads();  // the lists are read before the next item's are made
  }
}

// ================================================================ host side
// The pool as pairdec::pool_map has it, ending at row `rows` of every page: the
// rows behind it read as zeros like those outside the page.
inline mla_status pool_map(const mla_cache* k, CUtensorMap* map, int rows) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) return MLA_ERR_CUDA;
  const cuuint64_t dims[3] = {(cuuint64_t)kRow, (cuuint64_t)rows, (cuuint64_t)k->num_blocks};
  const cuuint64_t strides[2] = {(cuuint64_t)kRow * 2, (cuuint64_t)kRow * 2 * kPage};
  const cuuint32_t box[3] = {64, (cuuint32_t)kPage, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, k->pool, dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MLA_OK : MLA_ERR_CUDA;
}

// Rows of 512 values, stored in boxes of 32 rows x 128 bytes: o_lat (bf16) or
// the workspace's pieces (fp32).
inline mla_status out_map(void* p, long long rows, CUtensorMapDataType type, int elem, CUtensorMap* map) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) return MLA_ERR_CUDA;
  const cuuint64_t dims[2] = {(cuuint64_t)kDc, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)kDc * elem};
  const cuuint32_t box[2] = {128u / elem, 32};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(map, type, 2, p, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace chunk
}  // namespace mla
