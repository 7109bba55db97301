"""Request tables for callers that have laid out their token rows by the requests'
lengths: a request that is refused must not move the rows of those behind it."""

import numpy as np
import pytest
import torch

import oracle
from mla_latent_kv_39_b200 import Config, abi, check_device_error, mla_get_device_error

from mla_gpu_cases import assert_close, tol_for
from ragged_cases import TINY
from test_gpu_ragged import Tables
from test_gpu_ragged_layer import Serving

pytestmark = pytest.mark.gpu


class Ordered(Tables):
    def run(self, in_place=False):
        cfg = Config(**{**TINY, "block_size": self.bs}, fixed_rows=True)
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
        """The requests ahead of the first bad one, then nothing new; a length that a table row holds is kept."""
        rows = self.width * self.bs
        new, cached = list(self.new), list(self.cached)
        ahead = True
        for b, (c, n) in enumerate(zip(cached, new)):
            ahead = ahead and c >= 0 and n >= 0 and c + n <= rows
            if not ahead:
                self.new[b] = 0
                self.cached[b] = c if 0 <= c <= rows else 0
        want = super().expect()
        self.new, self.cached = new, cached
        return want


BAD = [  # cached, new, table width: the first request that cannot be served is in the middle, first, last, one of several
    ([0, 100, 64, 7], [10, 500, 64, 3], 3), ([190, 1, 2], [3, 1, 1], 3), ([5, 6, 192], [1, 1, 1], 3),
    ([0, -3, 64], [10, 1, 64], 3), ([0, 40, 64], [10, -2, 64], 3), ([5, 300, 9], [70, 0, 4], 3),
    ([0, 100, 64], [2 ** 31 - 1, 1, 64], 3), ([1, 2, 190, 4, -1, 6], [1, 1, 9, 1, 1, 9], 3)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("cached,new,width", BAD)
def test_nothing_behind_a_refused_request_moves(cached, new, width, in_place):
    fine_c = [min(max(c, 0), width * 64) for c in cached]
    fine_n = [n if 0 <= n and c + n <= width * 64 else 0 for c, n in zip(fine_c, new)]
    t = Ordered(fine_c, fine_n, width=width, pad=80)
    t.cached, t.new = list(cached), list(new)
    t.check(in_place=in_place)
    assert mla_get_device_error()[0] == abi.MLA_ERR_BOUNDS


@pytest.mark.parametrize("batch,bad", [(3000, 1500), (16384, 9), (1025, 1024), (1024, 1023)])
def test_a_refused_request_of_a_large_batch(batch, bad):
    t = Ordered([(7 * b) % 130 for b in range(batch)], [(b * b) % 3 for b in range(batch)], width=4, pad=5)
    t.new[bad] = 1000
    t.check()
    status, detail = mla_get_device_error()
    assert status == abi.MLA_ERR_BOUNDS and detail[1] == bad


@pytest.mark.parametrize("kw", [dict(), dict(n_tok=20), dict(n_tok=0), dict(free=2), dict(n_tok=67, free=3)])
def test_fine_requests_are_served_as_ever(kw):
    a, b = Tables([0, 100, 64, 7, 0], [10, 1, 64, 200, 0], **kw), Ordered([0, 100, 64, 7, 0], [10, 1, 64, 200, 0], **kw)
    x, y = a.run(), b.run()
    assert all(torch.equal(x[k], y[k]) for k in x)
    if kw:
        assert mla_get_device_error()[0] == abi.MLA_ERR_BOUNDS
    else:
        check_device_error()


def test_a_layer_serves_what_lies_ahead_of_an_over_long_request():
    s = Serving("tiny_f32_b1_l128", 3, 160, width=2)
    s.check([60, 30, 20])
    new = [1, 100, 5]                                        # 130 rows: more than the second's two pages
    x = s.inputs(new)
    pool = s.layer.cache.pool.clone()
    s.layer.step(x.cuda(), s.cached, torch.tensor(new, dtype=torch.int32, device="cuda"), s.free, s.head)
    status, detail = mla_get_device_error()
    assert status == abi.MLA_ERR_BOUNDS and detail[1] == 1
    assert s.layer.seq_lens.tolist() == [61, 30, 20] and s.layer.cu_q.tolist() == [0, 1, 1, 1]
    want = s.expect(x, [1, 0, 0])
    assert_close(oracle.to64(s.layer.y[:1].cpu())[0], want[0], tol_for(s.shape), "y")
    changed = (pool.nan_to_num(7) != s.layer.cache.pool.nan_to_num(7)).any(-1).sum()
    assert changed == 1                                      # the first request's new row only
    s.cached.copy_(s.layer.seq_lens)
    s.check([1, 0, 5])                                       # the caller takes the second out; the third goes on
    assert np.array_equal(s.layer.seq_lens.cpu().numpy(), [62, 30, 25])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("cursor", [-1, 10 ** 6, -2 ** 31])
def test_a_cursor_outside_the_list_stays(cursor, in_place):
    """Only requests that need no page, ahead of the first that does, are served; the cursor is not replaced."""
    t = Tables([10, 100, 64, 7], [3, 1, 1, 2])
    t.head = cursor
    got = t.run(in_place=in_place)
    assert mla_get_device_error()[0] == abi.MLA_ERR_BOUNDS
    assert got["head_out"].tolist() == [cursor]
    assert got["cu_q"].tolist() == [0, 3, 4, 4, 4] and got["seq_lens"].tolist() == [13, 101, 64, 7]
    assert torch.equal(got["table"], t.table)


def test_a_cursor_at_the_end_of_the_list_is_fine():
    t = Tables([10, 100], [3, 1], spare=0, free=0)
    t.check()
    assert t.head == len(t.free)
    check_device_error()
