"""Ragged steps on a machine without a GPU: what a token sees and how the work
is cut (the kernels' own index arithmetic, compiled for the host, against
brute force), the reference's plan of a step, and the entry points' refusals."""

import ctypes
import random
import subprocess
from pathlib import Path

import pytest
import torch

from mla_latent_kv_39_b200 import Config, RaggedLayer, abi, build

ROOT = Path(__file__).resolve().parents[1]

# Reads cases "window sinks batch n_tok max_rows workers, cu_q.., seq_lens.."
# and prints for every worker its pieces: worker, sequence, token, position,
# first item, end item, items of the token; then its shares; then, per token
# with items, every item; and the closed-form item sums.
PROGRAM = r'''
#include <algorithm>
#include <cstdio>
#include <vector>
#include "chunk_plan.cuh"
using namespace mla::chunk;
int main() {
  int window, sinks, batch, n_tok, max_rows, workers;
  while (std::scanf("%d %d %d %d %d %d", &window, &sinks, &batch, &n_tok, &max_rows, &workers) == 6) {
    std::vector<int32_t> cu(batch + 1), len(batch);
    for (auto& x : cu) std::scanf("%d", &x);
    for (auto& x : len) std::scanf("%d", &x);
    const Batch q{cu.data(), len.data(), batch, n_tok, max_rows, Visible{window, sinks}};
    Cut cut{0, workers, 1.f / workers, 0};
    std::vector<long long> C(batch + 1, 0);
    long long tokens = 0, longest = 0;
    for (int b = 0; b < batch; ++b) {
      const Sequence s = sequence_of(q, b);
      cut.total += cut.tokens(q.vis, s, s.n);
      tokens += s.n;
      longest = std::max(longest, longest_token(q.vis, s));
    }
    std::printf("case %lld\n", cut.total);
    if (one_token_each(tokens, cut.total, longest, workers)) {
      cut.single = 1;
      cut.total = tokens;
    }
    for (int b = 0; b < batch; ++b) {
      const Sequence s = sequence_of(q, b);
      C[b + 1] = C[b] + cut.tokens(q.vis, s, s.n);
    }
    for (int w = 0; w < workers; ++w) {
      const Found from = place_at(q, cut, C.data(), cut.at(w)), to = place_at(q, cut, C.data(), cut.at(w + 1));
      for (Walk k(q, from.at, from.s, to.at); k.valid(); k.next())
        std::printf("piece %d %d %d %d %d %d %d %d\n", w, k.at.b, k.token(), k.position(), k.at.k, k.k1, k.n_items,
                    (int)k.whole());
      const Shares e = shares_of(q, cut, from, to, w);
      std::printf("shares %d %d %d %d %d\n", w, e.continues, e.begins, e.last, e.first);
    }
    for (int b = 0; b < batch; ++b) {
      const Sequence s = sequence_of(q, b);
      for (int j = 0; j < s.n && s.p0 >= 0; ++j) {
        const int n = q.vis.items(s.p0 + j);
        std::printf("token %d %d %d", b, s.t0 + j, n);
        for (int i = 0; i < n; ++i) {
          const Item it = item_of(q.vis, s.p0 + j, i);
          std::printf(" %d %d %d", it.page, it.a, it.b);
        }
        std::printf("\n");
      }
    }
  }
}
'''


def visible_rows(p, window, sinks):
    return [u for u in range(p + 1) if window == 0 or u > p - window or u < sinks]


def make_cases():
    r = random.Random(7)
    cases = []
    for _ in range(120):
        window = r.choice([0, 0, 1, 2, 17, 62, 63, 64, 65, 100, 128, 300])
        sinks = r.choice([0, 1, 4, 63, 64, 65, 130]) if window else 0
        new = [r.choice([0, 1, 1, 2, 5, 40]) for _ in range(r.choice([1, 1, 2, 3, 9]))]
        cached = [r.choice([0, 1, 63, 64, 65, 200, 700]) for _ in new]
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        lens = [c + n for c, n in zip(cached, new)]
        if r.random() < 0.2:
            lens[r.randrange(len(lens))] = 0                      # an empty sequence
        if r.random() < 0.1:
            lens[-1] = 5000                                       # more rows than the table holds
        n_tok = cu[-1] + r.choice([0, 3])
        cases.append((window, sinks, cu, lens, n_tok, r.choice([1, 2, 7, 74])))
    cases.append((0, 0, [0, 5, 3, 8], [5, 5, 5], 8, 4))           # prefix out of order
    cases.append((0, 0, [0, 5, 30], [5, 25], 20, 4))              # past the token rows
    cases.append((0, 0, [2, 5], [5], 5, 4))                       # not from 0
    return cases


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cu").write_text(PROGRAM)
    subprocess.run([build._nvcc(), *build.ARCH_FLAGS, "-std=c++17", f"-I{build.INCLUDE}", f"-I{build.CSRC}", "-o",
                    str(d / "plan"), str(d / "plan.cu")], check=True, capture_output=True)
    return d / "plan"


def test_pieces_cover_every_visible_row_once(plan):
    cases = make_cases()
    text = "".join(f"{w} {s} {len(lens)} {n} 1024 {k} " + " ".join(map(str, cu + lens)) + "\n"
                   for w, s, cu, lens, n, k in cases)
    out = subprocess.run([str(plan)], input=text, capture_output=True, text=True, check=True).stdout
    blocks = out.split("case ")[1:]
    assert len(blocks) == len(cases)
    for (window, sinks, cu, lens, n_tok, workers), block in zip(cases, blocks):
        lines = block.splitlines()
        total = int(lines[0])
        pieces, shares, items = [], {}, {}
        for ln in lines[1:]:
            f = ln.split()
            v = list(map(int, f[1:]))
            if f[0] == "piece":
                pieces.append(v)
            elif f[0] == "shares":
                shares[v[0]] = v[1:]
            else:
                items[v[0], v[1]] = [tuple(v[3 + 3 * i:6 + 3 * i]) for i in range(v[2])]
        # the tokens that are to be computed, and what they see
        want, cost = {}, 0
        for b in range(len(lens)):
            lo, hi, n = cu[b], cu[b + 1], cu[b + 1] - cu[b]
            if lo < 0 or hi < lo or hi > n_tok or (b == 0 and lo):
                continue
            for j in range(n):
                fine = n <= lens[b] <= 1024
                want[(b, lo + j)] = visible_rows(lens[b] - n + j, window, sinks) if fine else []
        for (b, t), rows in want.items():
            its = items[b, t] if rows else []
            got = [64 * page + u for page, a, e in its for u in range(a, e)]
            assert sorted(got) == rows, (window, sinks, t)
            assert all(0 <= a < e <= 64 for _, a, e in its)
            if window == 0 or window >= 64:        # a range cut on both sides needs a window shorter than a page
                assert all(a == 0 or e == 64 for _, a, e in its)
            cost += 4 + 4 * -(-len(its) // 4) + len(its)
        assert cost == total
        # every token's items exactly once, in order over the workers; cuts on tile boundaries
        seen = {}
        for w, b, t, p, k0, k1, n, whole in pieces:
            key = (b, t)
            assert key in want and n == (len(items[key]) if want[key] else 0)
            assert k0 == seen.get(key, (0, []))[0] and k0 % 4 == 0 and (k1 % 4 == 0 or k1 == n)
            assert k1 > k0 or n == 0
            assert bool(whole) == (k0 == 0 and k1 == n)
            seen[key] = (k1, seen.get(key, (0, []))[1] + [(w, k0, k1)])
        assert set(seen) == set(want)
        for key, (end, parts) in seen.items():
            assert end == (len(items[key]) if want[key] else 0)
            if len(parts) > 1:   # the merge finds them: begun by one, continued and ended by the others
                head, tail = parts[0][0], parts[-1][0]
                assert shares[head][1:3] == [key[1], tail]
                for w in range(head + 1, tail + 1):    # idle workers among them continue nothing
                    assert shares[w][0] == (key[1] if w in [q[0] for q in parts] else -1)
                    assert shares[w][3] == head
        begun = sum(1 for v in shares.values() if v[1] >= 0)
        assert begun == sum(1 for _, parts in seen.values() if len(parts) > 1)


# ---------------------------------------------------------------- refusals, before any launch

V3 = dict(hidden=7168, n_heads=128, d_c=512, d_r=64, qk_nope=128, v_head=128, q_lora=1536)
OK, ODD = 1 << 20, (1 << 20) + 8          # never dereferenced: every call below is refused


@pytest.fixture(scope="module")
def lib():
    build.build()
    return abi.load_library()


def _cfg(**kw):
    return abi.Config(**{**V3, "dtype": "bf16", **kw}).c()


def chunk(lib, cfg, window=None, **kw):
    a = dict(q=OK, q_rope=None, n_tok=4, cu_q=OK, batch=2, cache=abi.MLACache(OK, 8, OK, 2, 3), seq_lens=OK, workers=0,
             o_lat=OK, lse=OK, ws=OK, ws_bytes=1 << 40)
    a.update(kw)
    head = (ctypes.byref(cfg), a["q"], a["q_rope"], a["n_tok"], a["cu_q"], a["batch"], ctypes.byref(a["cache"]), a["seq_lens"])
    tail = (a["workers"], a["o_lat"], a["lse"], a["ws"], a["ws_bytes"], None)
    return lib.mla_chunk_attention(*head, *tail) if window is None else lib.mla_window_attention(*head, *window, *tail)


@pytest.mark.parametrize("window", [None, (64, 4)])
def test_attention_refuses_bad_arguments(lib, window):
    bf = _cfg()
    bad = abi.MLA_ERR_INVALID_ARG
    for kw in (dict(n_tok=-1), dict(batch=-1), dict(workers=-1), dict(q=None), dict(cu_q=None), dict(seq_lens=None),
               dict(o_lat=None), dict(ws=None), dict(q=ODD), dict(o_lat=ODD), dict(ws=ODD), dict(lse=OK + 2), dict(cu_q=OK + 1),
               dict(cache=abi.MLACache(ODD, 8, OK, 2, 3)), dict(cache=abi.MLACache(OK, 8, OK, 1, 3)),
               dict(cache=abi.MLACache(OK, 0, OK, 2, 3)), dict(q_rope=OK)):
        assert chunk(lib, bf, window, **kw) == bad, kw
    for kw in (dict(q_rope=None), dict(q_rope=OK, q=OK + 2), dict(q_rope=OK + 2)):     # fp32 storage takes two arrays
        assert chunk(lib, _cfg(dtype="f32"), window, **kw) == bad, kw
    assert chunk(lib, _cfg(fp8_cache=True), window, q_rope=OK) == bad                   # no row scales
    assert chunk(lib, bf, window, batch=9000, cache=abi.MLACache(OK, 8, OK, 9000, 3)) == abi.MLA_ERR_UNSUPPORTED
    assert chunk(lib, bf, window, n_tok=1 << 25) == abi.MLA_ERR_UNSUPPORTED
    assert chunk(lib, _cfg(d_c=1024), window) == abi.MLA_ERR_UNSUPPORTED                # rows past the CUDA-core kernel's
    need = lib.mla_chunk_workspace_size(ctypes.byref(bf), 4, 0)
    assert need > 0 and chunk(lib, bf, window, ws_bytes=need - 1) == abi.MLA_ERR_WORKSPACE
    assert need == lib.mla_chunk_workspace_size(ctypes.byref(bf), 1 << 20, 0)           # does not grow with the tokens
    assert lib.mla_chunk_workspace_size(ctypes.byref(bf), 4, 3) < need
    assert lib.mla_chunk_workspace_size(ctypes.byref(bf), -1, 0) == 0
    for kw in (dict(n_tok=0), dict(batch=0)):                                           # nothing to do
        assert chunk(lib, bf, window, **kw) == abi.MLA_OK


def test_window_and_sinks_are_checked(lib):
    for window in ((0, 0), (-1, 0), (5, -1)):
        assert chunk(lib, _cfg(), window) == abi.MLA_ERR_INVALID_ARG


def test_tables_refuse_bad_arguments(lib):
    c = _cfg()
    base = dict(batch=2, cached=OK, new=OK, free=OK, n_free=4, head=OK, num_blocks=8, table=OK, width=3, n_tok=5, cu=OK,
                lens=OK, idx=OK, pos=OK, slots=OK, out=OK)

    def call(**kw):
        a = {**base, **kw}
        return lib.mla_batch_tables(ctypes.byref(c), a["batch"], a["cached"], a["new"], a["free"], a["n_free"], a["head"],
                                    a["num_blocks"], a["table"], a["width"], a["n_tok"], a["cu"], a["lens"], a["idx"],
                                    a["pos"], a["slots"], a["out"], None)
    for kw in (dict(batch=-1), dict(n_free=-1), dict(num_blocks=0), dict(width=0), dict(n_tok=-1), dict(cached=None),
               dict(new=None), dict(free=None), dict(head=None), dict(table=None), dict(cu=None), dict(lens=None), dict(idx=None),
               dict(pos=None), dict(slots=None), dict(out=None), dict(slots=OK + 4), dict(pos=OK + 2), dict(batch=0)):
        assert call(**kw) == abi.MLA_ERR_INVALID_ARG, kw
    assert call(batch=20000) == abi.MLA_ERR_UNSUPPORTED
    assert call(width=1 << 26) == abi.MLA_ERR_UNSUPPORTED
    assert call(batch=0, n_tok=0) == abi.MLA_OK


def test_slots_and_stored_projection_refuse_bad_arguments(lib):
    c, P = _cfg(), ctypes.byref
    cache = abi.MLACache(OK, 8, OK, 2, 3)
    need = lib.mla_cache_append_workspace_size(P(c), 4)
    call = lambda pos=OK, slots=OK, ws=OK, n=need: lib.mla_cache_append_slots(P(c), OK, 4, OK, OK, pos, slots, P(cache), ws, n,
                                                                              None)
    for kw in (dict(pos=None), dict(slots=None), dict(ws=None), dict(slots=OK + 4), dict(pos=OK + 1)):
        assert call(**kw) == abi.MLA_ERR_INVALID_ARG
    assert call(n=need - 1) == abi.MLA_ERR_WORKSPACE
    need = lib.mla_out_proj_workspace_size(P(c), 4)
    assert lib.mla_out_proj_stored(P(c), ODD, 4, OK, OK, OK, OK, need, None) == abi.MLA_ERR_INVALID_ARG
    assert lib.mla_out_proj_stored(P(c), OK, 4, OK, OK, OK, OK, need - 1, None) == abi.MLA_ERR_WORKSPACE
    assert lib.mla_out_proj_stored(P(c), None, 4, OK, OK, OK, OK, need, None) == abi.MLA_ERR_INVALID_ARG
    assert lib.mla_out_proj_stored(P(c), None, 0, None, None, None, None, 0, None) == abi.MLA_OK


def test_a_ragged_layer_refuses_what_no_call_takes():
    from types import SimpleNamespace
    cache = SimpleNamespace(block_table=torch.zeros(abi.MAX_CHUNK_BATCH + 1, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="at most 8192 requests"):
        RaggedLayer(Config(**V3), {}, cache, 1)
    for bad in (dict(window=-1), dict(window=4, n_sinks=-1), dict(max_workers=-1)):
        with pytest.raises(ValueError, match="negative"):
            RaggedLayer(Config(**V3), {}, cache, 1, **bad)
