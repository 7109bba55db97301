// What the new tokens of a ragged batch see, and how that work is cut among
// the workers of the tensor-core kernel.
//
// Sequence b has the n_b = cu_q[b + 1] - cu_q[b] query rows (tokens)
// t = cu_q[b] + j and seq_lens[b] cached rows, its new ones included, so
// token t stands at position p = seq_lens[b] - n_b + j and sees
//   rows u <= p                                            (window = 0)
//   rows u <= p with u > p - window or u < n_sinks         (window > 0).
// The visible rows are walked page by page.  Item k of a token is a page and
// the range [a, b) of its rows that are visible: the sink pages first, then
// the pages of the window; while the window still touches the sinks the two
// are one run from row 0.  A page that holds both the end of the sinks and the
// start of the window is two items.  Page order does not matter to a softmax.
//
// The number of items of a token is a sum of floors of its position, so the
// cost of a whole run of tokens has a closed form, and the cut of all work
// into equal parts needs one prefix sum over the sequences, not over the
// tokens: a warp of every CTA makes it for itself (8 bytes read per sequence) and
// there is no planning launch ahead of the attention.
#pragma once

#include "common.cuh"

namespace mla {
namespace chunk {

constexpr int kPage = 64;
constexpr int kMaxBatch = 8192;   // sequences of a call: their prefix sums sit in shared memory
constexpr int kTilePages = 4;     // items of a tile of the tensor-core kernel
// Costs, in eighths of a full tile's time.  A tile takes its score MMAs whatever
// its items (half of a full tile's time, 4) and its value MMAs and loads by the
// item (1 each); a token on top of its tiles the change of queries and output.
constexpr int kTileCost = 4, kFullTile = kTileCost + kTilePages, kTokenCost = 4;
// What cutting tokens into pieces costs the call on top: pieces written to the
// workspace and joined by another kernel (about 10 us, a tile 2.5).
constexpr int kSplitCost = 4 * kFullTile;

struct Visible {
  int window, sinks;  // window = 0: all rows up to the token's own

  // first window row of a token at position p, 0 while the window touches the sinks
  __host__ __device__ int start(int p) const {
    if (window == 0) return 0;
    const int w0 = p - window + 1;  // p >= 0, window >= 1: no overflow
    return w0 <= sinks ? 0 : w0;
  }
  __host__ __device__ int sink_items() const { return sinks / kPage + (sinks % kPage != 0); }
  __host__ __device__ int items(int p) const {
    const int w0 = start(p);
    return (w0 > 0 ? sink_items() : 0) + p / kPage - w0 / kPage + 1;
  }
  __host__ __device__ int tiles(int p) const { return (items(p) + kTilePages - 1) / kTilePages; }
  __host__ __device__ int cost(int p) const { return kTileCost * tiles(p) + items(p); }
  // the most that a token may cost in sequences of up to `rows` rows
  __host__ __device__ long long most_cost(int rows) const {
    const long long all = rows / kPage + 1, some = (long long)sink_items() + window / kPage + 2;
    const long long n = window > 0 && some < all ? some : all;
    return kTokenCost + kTileCost * (n / kTilePages + 1) + n;
  }
  // sum over p < n of floor(p / step)
  __host__ __device__ static long long floors(long long n, int step) {
    const long long q = n / step, r = n % step;
    return step * (q * (q - 1) / 2) + q * r;
  }
  // Cost of the tokens at positions p0 .. p0 + n - 1.  Up to position sinks +
  // window - 1 a token sees one run from row 0: p / 64 + 1 items, p / 256 + 1
  // tiles.  Behind it the sink items and, with window - 1 = 64 a + c, a + 1 items
  // of the window, one more where p mod 64 < c.
  __host__ __device__ long long cost_of_run(long long p0, long long n) const {
    const long long end = p0 + n, apart = window == 0 ? end : (long long)sinks + window;
    const long long m = apart < p0 ? p0 : (apart < end ? apart : end);  // [p0, m): one run; [m, end): apart
    constexpr int kRun = kPage * kTilePages;
    long long s = (m - p0) * (kTileCost + 1) + kTileCost * (floors(m, kRun) - floors(p0, kRun)) + floors(m, kPage) -
                  floors(p0, kPage);
    if (m < end) {
      const int c = (window - 1) % kPage, few = sink_items() + (window - 1) / kPage + 1;
      const long long more = past(end, c) - past(m, c);  // tokens with one item more
      s += (end - m) * (kTileCost * ((few + kTilePages - 1) / kTilePages) + few) + more;
      if (few % kTilePages == 0) s += kTileCost * more;
    }
    return s;
  }
  // how many p < n have p mod 64 < c
  __host__ __device__ static long long past(long long n, int c) {
    const long long r = n % kPage;
    return n / kPage * c + (r < c ? r : c);
  }
};

// Item k of the token at position p: page, visible rows [a, b) of it.
struct Item {
  int page, a, b;
};
__host__ __device__ inline Item item_of(const Visible& vis, int p, int k) {
  const int w0 = vis.start(p);
  const int ns = w0 > 0 ? vis.sink_items() : 0;
  Item it;
  if (k < ns) {
    it.page = k;
    it.a = 0;
    it.b = vis.sinks - k * kPage < kPage ? vis.sinks - k * kPage : kPage;
  } else {
    it.page = w0 / kPage + (k - ns);
    it.a = w0 - it.page * kPage > 0 ? w0 - it.page * kPage : 0;
    it.b = p + 1 - it.page * kPage < kPage ? p + 1 - it.page * kPage : kPage;
  }
  return it;
}

// A ragged batch and what its tokens see.
struct Batch {
  const int32_t* cu_q;
  const int32_t* seq_lens;
  int batch, n_tok, max_rows;  // max_rows: what a block table row holds
  Visible vis;
};

// The query rows of one sequence: tokens [t0, t0 + n) at positions p0 + j.
// p0 < 0: its tokens see nothing.
struct Sequence {
  int t0, n, p0;
  enum { kFine, kBadRows, kBadLength } state;
};

// Sequence b, its lengths checked; a sequence whose entries do not fit has no
// tokens (cu_q out of order or past n_tok) or tokens that see nothing (no
// cached rows, or a length that does not hold them).
__host__ __device__ inline Sequence sequence_of(const Batch& q, int b) {
  Sequence s;
  const int lo = q.cu_q[b], hi = q.cu_q[b + 1], len = q.seq_lens[b];
  s.t0 = lo;
  s.n = hi - lo;
  s.p0 = len - s.n;
  s.state = Sequence::kFine;
  if (lo < 0 || hi < lo || hi > q.n_tok || (b == 0 && lo != 0)) {
    s.t0 = s.n = 0;
    s.p0 = -1;
    s.state = Sequence::kBadRows;
  } else if (s.n > 0 && (len < s.n || len > q.max_rows)) {
    s.p0 = -1;
    if (len != 0) s.state = Sequence::kBadLength;
  }
  return s;
}

__device__ __forceinline__ void report_sequence(const Batch& q, int b, const Sequence& s) {
  if (s.state == Sequence::kBadRows) report(MLA_ERR_BOUNDS, 20, b, q.cu_q[b + 1]);
  if (s.state == Sequence::kBadLength) report(MLA_ERR_BOUNDS, 21, b, q.seq_lens[b]);
}

// How the work is cut.  `single`: a token to a worker, none split, for calls of
// no more tokens than workers whose longest token is hardly longer than an equal
// part (a decode step of similar lengths); otherwise equal parts of cost.
struct Cut {
  long long total;  // cost of all tokens (their number, if single)
  int workers;
  float inv;        // 1 / workers
  int single;
  __host__ __device__ long long tokens(const Visible& vis, const Sequence& s, int n) const {
    return single ? n : (long long)kTokenCost * n + (s.p0 >= 0 ? vis.cost_of_run(s.p0, n) : 0);
  }
  // The cost where the range of worker w begins (w = workers: where the last
  // ends): growing in w, and the same for the worker that ends there.
  __host__ __device__ long long at(int w) const {
    if (w >= workers) return total;
    if (single) return w < total ? w : total;
    return (long long)((double)total * w * inv);
  }
};
__host__ __device__ inline bool one_token_each(long long tokens, long long total, long long longest, int workers) {
  return tokens <= workers && longest <= total / workers + kSplitCost;
}
// The longest cost that a token of the sequence may have.
__host__ __device__ inline long long longest_token(const Visible& vis, const Sequence& s) {
  return s.n > 0 && s.p0 >= 0 ? kTokenCost + vis.cost(s.p0 + s.n - 1) : 0;
}

// A place in the order of all items: sequence, token within it, item.
struct Place {
  int b, j, k;
};
__host__ __device__ inline bool before(const Place& x, const Place& y) {
  return x.b < y.b || (x.b == y.b && (x.j < y.j || (x.j == y.j && x.k < y.k)));
}

// The place at cost x, given the costs C[0 .. batch] of the sequences before
// each; its sequence and the cost ahead of that.  Inside a token it is moved back
// to a tile boundary.
struct Found {
  Place at;
  Sequence s;
  long long base;
};
__host__ __device__ inline Found place_at(const Batch& q, const Cut& cut, const long long* C, long long x) {
  Found f{{q.batch, 0, 0}, {0, 0, -1, Sequence::kFine}, cut.total};
  if (x >= cut.total) return f;
  int lo = 0, hi = q.batch - 1;  // the last sequence with C[b] <= x; it has tokens, as C[b + 1] > x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (C[mid] <= x) lo = mid; else hi = mid - 1;
  }
  f.s = sequence_of(q, lo);
  f.base = C[lo];
  const long long r = x - f.base;
  int a = 0, z = f.s.n - 1;
  while (a < z) {
    const int mid = (a + z + 1) >> 1;
    if (cut.tokens(q.vis, f.s, mid) <= r) a = mid; else z = mid - 1;
  }
  int k = 0;
  if (f.s.p0 >= 0 && !cut.single) {
    const long long i = r - cut.tokens(q.vis, f.s, a) - kTokenCost;  // below 0 in the token's fixed cost
    const int n = q.vis.tiles(f.s.p0 + a);
    k = i < 0 ? 0 : (int)(i / kFullTile < n ? i / kFullTile : n - 1) * kTilePages;
  }
  f.at = {lo, a, k};
  return f;
}

// A value that all lanes of a warp hold, in the warp-uniform datapath.
__host__ __device__ __forceinline__ int uni(int x) {
#ifdef __CUDA_ARCH__
  return __shfl_sync(0xffffffffu, x, 0);
#else
  return x;
#endif
}

// The pieces of a range in order: a piece is a run of items [at.k, k1) of one
// token (no items for a token that sees nothing).  Whole warps.
struct Walk {
  const Batch& q;
  Place at, to;
  Sequence s;
  int n_items, k1;  // items of the token; end of the piece
  // `seq`: the sequence of `from`
  __host__ __device__ Walk(const Batch& q_, Place from, Sequence seq, Place to_)
      : q(q_), at(from), to(to_), s(seq), n_items(0), k1(0) {
    settle();
  }
  __host__ __device__ bool valid() const { return before(at, to); }
  __host__ __device__ void load() {
    s = sequence_of(q, at.b);
    s.t0 = uni(s.t0);
    s.n = uni(s.n);
    s.p0 = uni(s.p0);
  }
  // the first sequence from b on that seems to have tokens (batch: none), 32 at a look
  __host__ __device__ int filled(int b) const {
#ifdef __CUDA_ARCH__
    for (; b < q.batch; b += 32) {
      const int i = b + (threadIdx.x & 31);
      const uint32_t some = __ballot_sync(0xffffffffu, i < q.batch && q.cu_q[i] < q.cu_q[i + 1]);
      if (some != 0) return b + __ffs(some) - 1;
    }
    return q.batch;
#else
    while (b < q.batch && q.cu_q[b] >= q.cu_q[b + 1]) ++b;
    return b;
#endif
  }
  // bring `at` to a token that exists, and measure its piece
  __host__ __device__ void settle() {
    while (valid() && at.j >= s.n) {
      at.j = 0;
      at.k = 0;
      if (++at.b >= q.batch) return;  // `to` is at most (batch, 0, 0): not valid any more
      load();
      if (s.n > 0) continue;
      at.b = filled(at.b + 1);
      if (at.b >= q.batch) return;
      load();
    }
    if (!valid()) return;
    n_items = s.p0 < 0 ? 0 : q.vis.items(s.p0 + at.j);
    k1 = at.b == to.b && at.j == to.j ? (to.k < n_items ? to.k : n_items) : n_items;
  }
  __host__ __device__ void next() {
    ++at.j;
    at.k = 0;
    settle();
  }
  __host__ __device__ int token() const { return s.t0 + at.j; }
  __host__ __device__ int position() const { return s.p0 + at.j; }
  __host__ __device__ bool whole() const { return at.k == 0 && k1 == n_items; }
  __host__ __device__ int tiles() const { return (k1 - at.k + kTilePages - 1) / kTilePages; }
};

// What worker w holds of tokens that it does not hold whole: the token that its
// range continues (-1: none), the token that its range begins and does not end
// (-1: none) and the last worker that holds a piece of that one; and, where its
// range begins inside a token, the worker that begins that one (-1 otherwise).
// Workers between the first and the last may be without work: they continue no
// token.
struct alignas(16) Shares {
  int continues, begins, last, first;
};
__host__ __device__ inline Shares shares_of(const Batch& q, const Cut& cut, const Found& from, const Found& to, int w) {
  const bool same = from.at.b == to.at.b && from.at.j == to.at.j, some = before(from.at, to.at);
  Shares e{-1, -1, w, -1};
  if (from.at.k > 0) {
    if (some) e.continues = from.s.t0 + from.at.j;
    // the last worker whose range begins at the token's first tile or ahead of it
    const long long inner = from.base + cut.tokens(q.vis, from.s, from.at.j) + kTokenCost + kFullTile;
    e.first = (int)((double)inner * cut.workers / cut.total);
    if (e.first > w) e.first = w;
    while (cut.at(e.first) >= inner) --e.first;
    while (cut.at(e.first + 1) < inner) ++e.first;
  }
  if (some && to.at.k > 0 && !(same && from.at.k > 0)) {
    e.begins = to.s.t0 + to.at.j;
    // a worker whose range begins at a cost below the token's end holds items of it
    const long long end = to.base + cut.tokens(q.vis, to.s, to.at.j + 1);
    e.last = (int)((double)end * cut.workers / cut.total);
    if (e.last >= cut.workers) e.last = cut.workers - 1;
    while (e.last + 1 < cut.workers && cut.at(e.last + 1) < end) ++e.last;
    while (cut.at(e.last) >= end) --e.last;
  }
  return e;
}

// What the merge's blocks of worker w join: the pieces of one token, which are with
// the workers first .. first + n - 1.  A token of up to kMergeFew pieces is joined by
// the blocks of the worker that begins it, in items of four heads; one of more by those
// of its first `helpers` workers, in items of half a head.  Block y takes the items
// begin(w, y), begin(w, y) + step(), ...
//
// A block has one token only, so the worker that ends a token is never among its
// helpers: its range goes on behind the token and may begin the next one, which it
// then joins.  The ranges of the workers between the first and the last lie inside
// the token whole, so those begin none.
constexpr int kMergeY = 8, kMergeFew = 8, kMergeMost = 32;
struct Join {
  int token, first, n, helpers;  // token -1: nothing
  __host__ __device__ bool many() const { return n > kMergeFew; }
  __host__ __device__ int items(int heads) const { return many() ? 2 * heads : heads / 4; }
  __host__ __device__ int begin(int w, int y) const { return y + kMergeY * (w - first); }
  __host__ __device__ int step() const { return kMergeY * helpers; }
};
__host__ __device__ inline Join join_of(const Shares* shares, int w) {
  Shares own = shares[w];
  int first = w;
  if (own.begins < 0 && own.first >= 0) {  // inside a token, or at its end
    first = own.first;
    own = shares[first];
  }
  const int n = own.last - first + 1;
  const int helpers = n <= kMergeFew ? 1 : n - 1 < kMergeMost ? n - 1 : kMergeMost;
  return {w - first < helpers ? own.begins : -1, first, n, helpers};
}

}  // namespace chunk
}  // namespace mla
