"""Ragged steps on the GPU: the attention of new tokens over the paged cache,
causal and windowed, against its definition in 64 bits; the request tables
against a plain count; slots, and the whole step of a ragged layer."""

import math

import pytest
import torch

from mla_latent_kv_39_b200 import Cache, Config, MLAError, abi, check_device_error, mla_get_device_error

from ragged_cases import TINY, V3, Ragged

pytestmark = pytest.mark.gpu

# (cached, new, padding): single rows, page and tile borders, ragged chunks with
# sequences that bring nothing, tokens cut over many workers, more tokens than workers
BATCHES = [
    ([0], [1], 0),
    ([1], [1], 3),
    ([62], [3], 0),
    ([255], [2], 1),
    ([256, 0, 64], [1, 5, 0], 2),
    ([0, 700, 63, 64, 1], [70, 1, 0, 33, 2], 5),
    ([9000], [1], 0),
    ([3000, 20], [2, 1], 0),
    ([200] * 40, [0, 1, 2, 3] * 10, 7),
]


@pytest.mark.parametrize("cached,new,pad", BATCHES)
def test_chunk_attention(cached, new, pad):
    r = Ragged(Config(**V3), cached, new, pad)
    r.run()
    check_device_error()
    r.check()


WINDOWS = [(1, 0), (1, 200), (17, 5), (62, 64), (63, 1), (64, 0), (65, 70), (300, 4), (256, 128), (10 ** 9, 3),
           (2 ** 31 - 1, 2 ** 31 - 1)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_window_attention(window, sinks):
    r = Ragged(Config(**V3), [0, 700, 63, 64, 1500], [70, 1, 0, 33, 3], 5)
    r.run(window, sinks)
    check_device_error()
    r.check(window, sinks)


@pytest.mark.parametrize("window,sinks", [(0, 0), (130, 70)])
def test_split_query(window, sinks):
    r = Ragged(Config(**V3, split_query=True), [300, 0, 1000], [2, 3, 40], 2, spread=2.0)
    r.run(window, sinks)
    check_device_error()
    r.check(window, sinks)


@pytest.mark.parametrize("cfg,kw", [
    (TINY, {}), (TINY, dict(block_size=16)), (TINY, dict(block_size=100, n_heads=3, d_c=40, d_r=6)),
    (V3, dict(n_heads=5)), (V3, dict(n_heads=2, d_c=96, d_r=32, block_size=48)), (V3, dict(n_heads=2, split_query=True)),
    (V3, dict(n_heads=4, fp8_cache=True)), (V3, dict(n_heads=1, d_c=960, d_r=64))], ids=lambda v: "-".join(
        f"{k}{x}" for k, x in v.items() if k in ("dtype", "block_size", "n_heads", "d_c", "fp8_cache", "split_query")))
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (33, 5), (64, 64), (500, 3)])
def test_other_shapes_run_on_cuda_cores(cfg, kw, window, sinks):
    r = Ragged(Config(**{**cfg, **kw}), [0, 300, 17, 63, 0], [1, 4, 0, 2, 70], 3)
    r.run(window, sinks)
    check_device_error()
    r.check(window, sinks)


def test_worker_count_does_not_change_what_is_computed():
    r = Ragged(Config(**V3), [3000, 70, 1500, 0], [3, 20, 1, 5], 2)
    for workers in (1, 2, 7, 31, 0):
        r.o_lat.fill_(7)
        r.lse.fill_(7)
        r.run(max_workers=workers)
        check_device_error()
        r.check()


@pytest.mark.parametrize("window,sinks", [(0, 0), (1000, 70)])
def test_results_do_not_depend_on_timing(window, sinks):
    r = Ragged(Config(**V3), [2500, 40, 0, 700], [90, 1, 130, 64], 0)
    r.run(window, sinks)
    a, b = r.o_lat.clone(), r.lse.clone()
    for _ in range(5):
        r.ws.fill_(0xFF)
        r.run(window, sinks)
        assert torch.equal(a, r.o_lat) and torch.equal(b, r.lse)
    check_device_error()


def test_many_short_tokens():
    """Tiles of one or two pages, several to a worker, again and again: the two
    CTAs of a pair must stay together although one of them loads nothing."""
    r = Ragged(Config(**V3), [0, 60, 100, 5] * 4, [100, 30, 20, 50] * 4)
    for _ in range(20):
        r.run()
    check_device_error()
    r.check()


def test_peaked_scores_rescale_the_running_sums():
    """Scores that grow along the rows: every tile raises the running maximum."""
    r = Ragged(Config(**V3), [1500, 200], [2, 1], spread=0.5)
    ramp = torch.linspace(0.1, 6.0, 1502, device="cuda")
    q = r.q64[:, :, :].mean(1, keepdim=True).expand_as(r.q64)
    r.q = q.bfloat16().contiguous()
    r.q64 = r.q.double()
    d = r.q64[0, 0] / r.q64[0, 0].norm()
    rows = (r.pool64[0] + ramp[:, None].double() * 20 * d).bfloat16()
    r.pool64[0] = rows.double()
    pages = (1502 + 63) // 64
    buf = torch.full((pages * 64, 576), math.nan, device="cuda")
    buf[:1502] = rows.float()
    r.pool[r.table[0, :pages].long()] = buf.view(pages, 64, 576).bfloat16()
    r.run()
    check_device_error()
    r.check()


@pytest.mark.parametrize("window,sinks", [(5, 0), (63, 3), (64, 64), (200, 1), (700, 130)])
def test_rows_that_no_token_sees_may_hold_anything(window, sinks):
    """One token a sequence: rows out of sight are NaN or infinite, and tables
    need no entry for pages out of sight."""
    r = Ragged(Config(**V3), [1200, 64, 700], [1, 1, 1], 2)
    for b, n in enumerate(r.lens):
        p = n - 1
        hidden = [u for u in range(n) if not (u > p - window or u < sinks)]
        for i, u in enumerate(hidden):
            page = int(r.table[b, u // 64])
            r.pool[page, u % 64] = math.nan if i % 2 else math.inf
        seen = {u // 64 for u in range(n)} - {u // 64 for u in hidden} | {u // 64 for u in range(n) if u not in set(hidden)}
        for k in range((n + 63) // 64):
            if k not in seen:
                r.table[b, k] = -7
    r.run(window, sinks)
    check_device_error()
    r.check(window, sinks)


def test_rows_of_later_tokens_may_hold_anything():
    """Token j of a chunk does not see the rows of the tokens behind it."""
    r = Ragged(Config(**V3), [100], [4])
    r.pool[int(r.table[0, 1]), 103 - 64] = math.nan      # the last token's own row
    r.run()
    check_device_error()
    o, lse, eo, el = r.expect()
    got = r.o_lat.double()
    assert ((got[:3] - o[:3]).abs() <= eo[:3]).all()
    assert got[3].isnan().all() and r.lse[3].isnan().all()


def test_nan_in_a_visible_row_reaches_its_tokens_only():
    r = Ragged(Config(**V3), [5000, 64, 0], [1, 1, 2])
    r.pool[int(r.table[0, 40]), 5] = math.nan            # seen by the first sequence, which is split over workers
    r.run()
    check_device_error()
    assert r.o_lat[0].isnan().all() and r.lse[0].isnan().all()
    r.pool64[0][40 * 64 + 5] = 0
    r.check(skip=[0])


def test_empty_sequences_and_bad_entries():
    r = Ragged(Config(**V3), [300, 200, 500, 64, 10], [2, 3, 2, 1, 1], 1)
    r.seq_lens[1] = 0                                    # an empty sequence
    r.run()
    check_device_error()
    assert (r.o_lat[2:5] == 0).all() and (r.lse[2:5] == -math.inf).all()
    r.check(skip=[1])
    r.seq_lens[2] = 1                                    # does not hold its two tokens
    r.run()
    status, detail = mla_get_device_error()
    assert status == abi.MLA_ERR_BOUNDS and detail[1] == 2
    assert (r.o_lat[5:7] == 0).all() and (r.lse[5:7] == -math.inf).all()
    r.check(skip=[1, 2])
    r.seq_lens[2] = 10 ** 6                              # more than a table row holds
    r.run()
    assert mla_get_device_error()[0] == abi.MLA_ERR_BOUNDS
    r.check(skip=[1, 2])


def test_a_block_id_outside_the_pool_is_not_visible():
    r = Ragged(Config(**V3), [300, 200], [2, 3], 1)
    keep = r.table.clone()
    for bad in (-1, r.pool.shape[0], 2 ** 31 - 1):
        r.table.copy_(keep)
        r.table[0, 1] = bad
        r.run()
        status, detail = mla_get_device_error()
        assert status == abi.MLA_ERR_BOUNDS and detail[1] == 0 and detail[2] == bad
        r.check(skip=[0])
        # the rest of the first sequence's rows is what its tokens see
        rows = r.pool64[0]
        save = rows.clone()
        u = torch.arange(302, device="cuda")
        for t in range(2):
            kv = rows[(u <= 300 + t) & ((u < 64) | (u >= 128))]
            w = torch.softmax(r.q64[t] @ kv.T / math.sqrt(192), -1)
            want = w @ kv[:, :512]
            assert ((r.o_lat[t].double() - want).abs() <= 2 ** -7 * (w @ kv[:, :512].abs() + want.abs())).all()
        assert torch.equal(save, rows)


def test_token_prefix_out_of_order_is_reported():
    r = Ragged(Config(**V3), [300, 200, 100], [2, 3, 4], 1)
    good = r.cu_q.clone()
    r.cu_q[2] = 100                                      # past the token rows, and the next one falls
    r.run()
    assert mla_get_device_error()[0] == abi.MLA_ERR_BOUNDS
    r.check(skip=[1, 2])
    r.cu_q.copy_(good)
    r.run()
    check_device_error()
    r.check()


def test_optional_lse_and_odd_alignment():
    r = Ragged(Config(**V3), [300, 5000], [20, 1], 2)
    flat = torch.full((r.o_lat.numel() + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    o = flat[8:].view_as(r.o_lat)                        # on a 16-byte boundary, not on a 32-byte one
    abi.mla_chunk_attention(r.cfg, r.q, r.cu_q, r.cache, r.seq_lens, o, r.ws)
    r.run()
    check_device_error()
    assert torch.equal(o, r.o_lat) and (flat[:8] == 7).all()
    r.check()


def test_streams_and_graphs():
    a = Ragged(Config(**V3), [2000, 10], [3, 60], 4, seed=1)
    b = Ragged(Config(**V3), [100, 900], [50, 1], 4, seed=2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):                                  # two calls at once, each with its workspace
        a.run(stream=s1)
        b.run(300, 4, stream=s2)
    torch.cuda.synchronize()
    check_device_error()
    a.check()
    b.check(300, 4)
    # captured once, replayed over other lengths
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run()
    for cached, new in (([1500, 0], [60, 3]), ([64, 2000], [1, 0]), ([7, 7], [0, 0])):
        c = Ragged(Config(**V3), cached, new, pad=a.n_tok - sum(new), seed=3)
        c_table = torch.full_like(a.table, -1)
        c_table[:, :c.table.shape[1]] = c.table[:, :a.table.shape[1]]
        n = min(c.pool.shape[0], a.pool.shape[0])
        ok = int(c.table.max()) < n
        assert ok
        a.pool[:n] = c.pool[:n]
        a.table.copy_(c_table)
        a.q.copy_(c.q)
        a.cu_q.copy_(c.cu_q)
        a.seq_lens.copy_(c.seq_lens)
        a.o_lat.fill_(7)
        a.lse.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        check_device_error()
        c.o_lat, c.lse = a.o_lat, a.lse
        c.check()


def test_arguments_are_checked():
    r = Ragged(Config(**V3), [10], [2])
    with pytest.raises(MLAError):
        r.run(-1, 0)
    with pytest.raises(MLAError):
        r.run(5, -1)
    with pytest.raises(MLAError):
        abi.mla_chunk_attention(r.cfg, r.q, r.cu_q, r.cache, r.seq_lens, r.o_lat, r.ws[:1024], r.lse)
    with pytest.raises(ValueError):
        abi.mla_chunk_attention(r.cfg, r.q.transpose(0, 1), r.cu_q, r.cache, r.seq_lens, r.o_lat, r.ws, r.lse)
    with pytest.raises(TypeError):
        abi.mla_chunk_attention(r.cfg, (r.q, r.q), r.cu_q, r.cache, r.seq_lens, r.o_lat, r.ws, r.lse)
    with pytest.raises(TypeError):
        abi.mla_chunk_attention(r.cfg, r.q, r.cu_q, r.cache, r.seq_lens, r.o_lat.float(), r.ws, r.lse)
    with pytest.raises(ValueError):
        abi.mla_chunk_attention(r.cfg, r.q, r.cu_q[:1], r.cache, r.seq_lens, r.o_lat, r.ws, r.lse)
    with pytest.raises(ValueError):
        abi.mla_chunk_attention(r.cfg, r.q.cpu(), r.cu_q, r.cache, r.seq_lens, r.o_lat, r.ws, r.lse)


# ---------------------------------------------------------------- request tables

class Tables:
    def __init__(self, cached, new, pad=0, bs=64, width=None, lead=3, spare=2, n_tok=None, seed=0, free=None):
        g = torch.Generator().manual_seed(seed)
        self.bs, self.cached, self.new = bs, list(cached), list(new)
        need = [-(-(c + n) // bs) for c, n in zip(cached, new)]
        have = [-(-c // bs) for c in cached]
        total = sum(need) + spare
        ids = torch.randperm(total, generator=g).int()
        self.width = width or max(need + [1]) + 1
        self.table = torch.full((len(new), self.width), -5, dtype=torch.int32)
        at = 0
        for b, h in enumerate(have):
            self.table[b, :h] = ids[at:at + h]
            at += h
        lead_ids = torch.full((lead,), 10 ** 6, dtype=torch.int32)
        self.free = torch.cat([lead_ids, ids[at:] if free is None else ids[at:at + free]])
        self.head, self.blocks = lead, total
        self.n_tok = sum(new) + pad if n_tok is None else n_tok

    def run(self, in_place=False):
        cfg = Config(**{**TINY, "block_size": self.bs})
        dev = lambda x, dt=torch.int32: torch.as_tensor(x, dtype=dt).cuda()
        B = len(self.new)
        t = dict(cached=dev(self.cached), new=dev(self.new), free=self.free.cuda(), head=dev([self.head]),
                 table=self.table.cuda(), cu_q=dev([9] * (B + 1)), seq_idx=dev([9] * self.n_tok), pos=dev([9] * self.n_tok),
                 slots=dev([9] * self.n_tok, torch.int64))
        t["seq_lens"] = t["cached"] if in_place else dev([9] * B)
        t["head_out"] = t["head"] if in_place else dev([9])
        abi.mla_batch_tables(cfg, t["cached"], t["new"], t["free"], t["head"], self.blocks, t["table"], t["cu_q"],
                             t["seq_lens"], t["seq_idx"], t["pos"], t["slots"], t["head_out"])
        torch.cuda.synchronize()
        return {k: t[k].cpu() for k in ("table", "cu_q", "seq_lens", "seq_idx", "pos", "slots", "head_out")}

    def expect(self):
        """One request and one token after the other."""
        bs, at, tok = self.bs, self.head, 0
        table, cu, lens = self.table.clone(), [0], []
        idx, pos, slots = [], [], []
        full = False
        for b, (c, n) in enumerate(zip(self.cached, self.new)):
            if c < 0 or n < 0 or c + n > self.width * bs:
                lens.append(0)
                cu.append(tok)
                continue
            want = -(-(c + n) // bs) - -(-c // bs)
            if full or tok + n > self.n_tok or at + want > len(self.free):
                full = True
                n = want = 0
            have = -(-c // bs)
            for k in range(want):
                table[b, have + k] = self.free[at + k]
            at += want
            for j in range(n):
                p = c + j
                idx.append(b)
                pos.append(p)
                slots.append(int(table[b, p // bs]) * bs + p % bs)
            tok += n
            cu.append(tok)
            lens.append(c + n)
        fill = self.n_tok - tok
        return dict(table=table, cu_q=torch.tensor(cu), seq_lens=torch.tensor(lens), seq_idx=torch.tensor(idx + [-1] * fill),
                    pos=torch.tensor(pos + [0] * fill), slots=torch.tensor(slots + [-1] * fill), head_out=torch.tensor([at]))

    def check(self, **kw):
        got, want = self.run(**kw), self.expect()
        for k in want:
            assert torch.equal(got[k].long(), want[k].long()), k


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("cached,new,pad,bs", [
    ([0], [1], 0, 64), ([64], [1], 3, 64), ([63], [1], 0, 64), ([5], [0], 4, 64), ([0, 100, 64, 7], [0, 1, 64, 200], 9, 64),
    ([10, 20, 30], [1, 2, 3], 0, 1), ([10, 0, 33], [90, 2, 1], 5, 16), ([1000] * 70, [1] * 70, 0, 64),
    ([3, 0, 70] * 500, [1, 0, 66] * 500, 11, 64), ([0, 5000], [9000, 1], 100, 64), (list(range(3000)), [1] * 3000, 0, 64)])
def test_batch_tables(cached, new, pad, bs, in_place):
    Tables(cached, new, pad, bs).check(in_place=in_place)
    check_device_error()


@pytest.mark.parametrize("kw", [dict(n_tok=20), dict(n_tok=0), dict(free=2), dict(free=0), dict(n_tok=67, free=3)])
def test_batch_tables_serves_what_fits(kw):
    t = Tables([0, 100, 64, 7, 0], [10, 1, 64, 200, 0], **kw)
    t.check()
    assert mla_get_device_error()[0] == abi.MLA_ERR_BOUNDS


def test_batch_tables_reports_bad_entries():
    t = Tables([0, 100, 64], [10, 1, 64])
    t.cached[1] = -3
    t.check()
    assert mla_get_device_error()[0] == abi.MLA_ERR_BOUNDS
    t = Tables([0, 100, 64], [10, 1, 64], width=3)
    t.new[1] = 500                                       # more rows than the table holds
    t.n_tok = 100
    t.check()
    assert mla_get_device_error()[0] == abi.MLA_ERR_BOUNDS
    t = Tables([0, 100, 64], [10, 1, 64])
    t.new = [2 ** 31 - 1, 1, 64]                         # a sum past 31 bits
    t.width = t.table.shape[1]
    t.check()
    assert mla_get_device_error()[0] == abi.MLA_ERR_BOUNDS
    t = Tables([0, 100, 64], [10, 1, 64])
    t.head = 10 ** 6                                     # a cursor past the list: nothing to hand out
    got = t.run()
    assert mla_get_device_error()[0] == abi.MLA_ERR_BOUNDS
    assert got["cu_q"].tolist() == [0, 0, 0, 0] and got["seq_lens"].tolist() == [0, 100, 64]
    t = Tables([0, 100, 64], [10, 1, 64])
    t.free[t.head] = t.blocks + 1                        # a free block outside the pool: no slot for its tokens
    got = t.run()
    assert mla_get_device_error()[0] == abi.MLA_ERR_BOUNDS
    assert (got["slots"][:10] == -1).all() and (got["slots"][10:] >= 0).all()


@pytest.mark.parametrize("bs", [1, 3, 100, 4096])
def test_tables_of_long_requests_at_odd_page_sizes(bs):
    Tables([2 ** 20, 2 ** 20 - 1, 5, 0], [3, 1, 0, 101], 2, bs).check()
    check_device_error()


def test_tables_at_the_largest_batch():
    n = 16384
    cached = [(7 * b) % 130 for b in range(n)]
    new = [(b * b) % 3 for b in range(n)]
    t = Tables(cached, new, pad=5)
    t.check()
    t.check(in_place=True)
    check_device_error()


@pytest.mark.parametrize("batch", [33, 1000, 8192])
def test_large_batches_with_few_tokens(batch):
    new = [1 if b % (batch // 20) == 7 else 0 for b in range(batch)]
    new[-1] = 40
    cached = [(3 * b) % 200 if new[b] else 5 for b in range(batch)]
    r = Ragged(Config(**V3), cached, new, 2)
    r.run()
    check_device_error()
    r.check()
    r.run(50, 3)
    check_device_error()
    r.check(50, 3)


@pytest.mark.parametrize("batch", [128, 129, 400])
def test_large_batches_whose_tokens_are_cut(batch):
    """More sequences than the plan warp sums up alone, a few of them long enough to be shared by workers."""
    new = [0 if b % 5 == 0 else 1 + (b * b) % 3 for b in range(batch)]
    cached = [(37 * b) % 150 for b in range(batch)]
    for b in (3, batch - 2):
        new[b], cached[b] = 2, 9000
    cached[6], new[6] = 0, 70
    r = Ragged(Config(**V3), cached, new, 3)
    for args in ((), (200, 5)):
        r.run(*args)
        check_device_error()
        r.check(*args)


@pytest.mark.parametrize("heads", [128, 2])
def test_caches_past_32_bits(heads):
    """Pages more than 4 GiB into the pool (and more than 2^31 values)."""
    r = Ragged(Config(**{**V3, "n_heads": heads}), [300, 64], [3, 1], 1)
    far = 65000
    pool = torch.zeros(far + r.pool.shape[0], 64, 576, dtype=torch.bfloat16, device="cuda")
    assert pool.numel() * 2 > 2 ** 32
    pool[far:] = r.pool
    r.table = torch.where(r.table >= 0, r.table + far, r.table)
    r.cache = Cache(pool, r.table)
    for window, sinks in ((0, 0), (100, 5)):
        r.run(window, sinks)
        check_device_error()
        r.check(window, sinks)


def test_one_workspace_under_two_graphs():
    a = Ragged(Config(**V3), [6000, 10], [1, 30], 4, seed=1)
    b = Ragged(Config(**V3), [100, 9000], [50, 1], 0, seed=2)
    b.ws = a.ws
    a.run()
    b.run(3000, 4)
    torch.cuda.synchronize()
    graphs = []
    for f in (lambda: a.run(), lambda: b.run(3000, 4)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for order in ((0, 1), (1, 0, 0, 1)):
        for x in (a, b):
            x.o_lat.fill_(7)
            x.lse.fill_(7)
        for k in order:
            graphs[k].replay()
        torch.cuda.synchronize()
        check_device_error()
        a.check()
        b.check(3000, 4)


def test_inputs_of_another_stream():
    """The call takes its stream as an argument: work queued there before it is waited for, the current stream's is not needed."""
    r = Ragged(Config(**V3), [700, 64], [5, 1], 1)
    good = r.q.clone()
    r.q.fill_(float("nan"))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        r.q.copy_(good)
    r.run(stream=s)
    s.synchronize()
    check_device_error()
    r.check()
