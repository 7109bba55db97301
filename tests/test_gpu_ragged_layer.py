"""The ragged operators together, as a serving loop uses them: request tables,
queries, rows stored through their slots, attention and projection, step after
step, against the fp64 oracle; and the step captured as one graph."""

import dataclasses

import numpy as np
import pytest
import torch

import oracle
from mla_synth import WORKLOADS, device_inputs, generate, reduced
from mla_latent_kv_39_b200 import (Cache, Config, DecodeLayer, MLAError, RaggedLayer, abi, check_device_error,
                                   mla_get_device_error)

from mla_gpu_cases import assert_close, tol_for

pytestmark = pytest.mark.gpu


class Serving:
    """Requests served step by step on the GPU, their cache rows kept by the oracle beside it."""

    def __init__(self, name, batch, n_tok, blocks=40, width=8, window=0, n_sinks=0, fp8=False, seed=3):
        wl = reduced(WORKLOADS[name], lengths=[1])
        self.shape, self.fp8 = wl.shape, fp8
        data = generate(dataclasses.replace(wl, seed=seed))
        self.W = data.weights
        dev = device_inputs(data, "cuda")
        self.cfg = Config.from_shape(wl.shape, fp8_cache=fp8)
        s = wl.shape
        row = s.d_c + s.d_r
        pool = torch.full((blocks, s.block_size, row), 0x7F if fp8 else float("nan"), device="cuda").to(self.cfg.cache_torch_dtype)
        scale = torch.ones(blocks, s.block_size, device="cuda") if fp8 else None
        table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
        self.layer = RaggedLayer(self.cfg, dev["weights"], Cache(pool, table, scale), n_tok, window, n_sinks)
        g = torch.Generator().manual_seed(seed)
        self.free = torch.randperm(blocks, generator=g).int().cuda()
        self.head = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cached = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.window, self.n_sinks, self.n_tok, self.g = window, n_sinks, n_tok, g
        self.rows = [np.zeros((0, row)) for _ in range(batch)]       # as the cache holds them

    def inputs(self, new):
        x = torch.randn(self.n_tok, self.shape.hidden, generator=self.g).to(self.cfg.torch_dtype)
        x[sum(new):] = float("nan")                                   # padding rows may hold anything
        return x

    def expect(self, x, new):
        """The oracle's y of the step's tokens; its cache rows move on."""
        s, W = self.shape, {k: oracle.to64(v) for k, v in self.W.items()}
        ys, at = [], 0
        for b, n in enumerate(new):
            if n == 0:
                continue
            xb = oracle.to64(x[at:at + n])
            pos = len(self.rows[b]) + np.arange(n)
            c, kr = oracle.latent_rows(xb, W["W_DKV"], W["W_KR"], pos, s.rope_theta, "fp8" if self.fp8 else s.dtype)
            q_nope, q_r = oracle.queries(xb, W, s.n_heads, s.qk_nope, s.d_r, pos, s.rope_theta)
            q_lat = oracle.absorb_query(q_nope, W["W_UK"], s.n_heads, s.qk_nope)
            self.rows[b] = np.concatenate([self.rows[b], np.concatenate([c, kr], 1)])
            scale = oracle.softmax_scale(s.qk_nope, s.d_r)
            for j in range(n):
                u = np.arange(len(self.rows[b]))
                see = u <= pos[j]
                if self.window:
                    see &= (u > pos[j] - self.window) | (u < self.n_sinks)
                kv = self.rows[b][see]
                o_lat, _, _ = oracle.attend_absorbed(q_lat[j], q_r[j], kv[:, :s.d_c], kv[:, s.d_c:], scale)
                ys.append(oracle.output_projection(oracle.heads_from_latent(o_lat, W["W_UV"], s.n_heads, s.v_head)[None],
                                                   W["W_O"])[0])
            at += n
        return np.stack(ys) if ys else np.zeros((0, s.hidden))

    def step(self, new):
        x = self.inputs(new)
        y = self.layer.step(x.cuda(), self.cached, torch.tensor(new, dtype=torch.int32, device="cuda"), self.free, self.head)
        torch.cuda.synchronize()
        check_device_error()
        self.cached.copy_(self.layer.seq_lens)
        return x, oracle.to64(y[:sum(new)].cpu())

    def check(self, new):
        x, y = self.step(new)
        want = self.expect(x, new)
        for t in range(len(want)):
            assert_close(y[t], want[t], tol_for(self.shape), f"y[{t}] of {new}")
        assert self.cached.tolist() == [len(r) for r in self.rows]


@pytest.mark.parametrize("window,n_sinks", [(0, 0), (50, 3)])
def test_steps_of_the_fp32_shape(window, n_sinks):
    s = Serving("tiny_f32_b1_l128", 4, 160, window=window, n_sinks=n_sinks)
    for new in ([70, 0, 5, 1], [1, 64, 0, 1], [0, 0, 0, 0], [1, 1, 1, 1], [60, 1, 64, 30]):
        s.check(new)


@pytest.mark.parametrize("fp8,window,n_sinks", [(False, 0, 0), (False, 100, 5), (True, 0, 0)])
def test_steps_of_the_bf16_shape(fp8, window, n_sinks):
    s = Serving("v3_b64_ragged1k_8k", 3, 140, window=window, n_sinks=n_sinks, fp8=fp8)
    for new in ([130, 0, 2], [1, 66, 0], [1, 1, 1]):
        s.check(new)


def test_one_token_each_equals_the_decode_layer():
    """The same batch through the uniform decode: the same rows in the cache, outputs within its roundings."""
    wl = reduced(WORKLOADS["v3_b64_ragged1k_8k"], lengths=[700, 64, 63])
    data = generate(wl)
    dev = device_inputs(data, "cuda")
    cfg = Config.from_shape(wl.shape)
    cache = Cache(dev["pool"], dev["block_table"])
    decode = DecodeLayer(cfg, dev["weights"], cache, 3, 1)
    y = decode.step(dev["x_new"], dev["seq_idx"], dev["pos"], dev["seq_lens"]).clone()
    rows = cache.pool.clone()
    table = dev["block_table"].clone()
    table[1, 1] = -1                                                   # the page of the second request's new token is not there yet
    pool = dev["pool"].clone()
    ragged = RaggedLayer(cfg, dev["weights"], Cache(pool, table), 3)
    free = dev["block_table"][1, 1:2].clone()
    y2 = ragged.step(dev["x_new"], dev["seq_lens"] - 1, torch.ones_like(dev["seq_lens"]), free,
                     torch.zeros(1, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    check_device_error()
    assert torch.equal(table, dev["block_table"])
    assert torch.equal(rows.nan_to_num(7), pool.nan_to_num(7))         # bit for bit
    # both round P, o_lat and the heads' outputs to bf16 (half a step 2^-8 each), on different cuts
    assert (y.double() - y2.double()).abs().max() <= 6 * 2.0 ** -8 * y.double().abs().max()


def test_the_captured_step_serves_other_steps():
    a = Serving("v3_b64_ragged1k_8k", 3, 140)
    b = Serving("v3_b64_ragged1k_8k", 3, 140)
    x = torch.zeros(140, a.shape.hidden, dtype=torch.bfloat16, device="cuda")
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    g = a.layer.capture_step(x, a.cached, new, a.free, a.head)
    eager = torch.zeros(1, a.shape.hidden, dtype=torch.bfloat16, device="cuda")   # an eager tensor of another step lives on
    for n in ([130, 0, 2], [1, 66, 0], [0, 0, 0], [1, 1, 1]):
        xb, yb = b.step(n)
        x.copy_(xb)
        new.copy_(torch.tensor(n))
        g.replay()
        torch.cuda.synchronize()
        check_device_error()
        a.cached.copy_(a.layer.seq_lens)
        assert torch.equal(a.cached, b.cached) and torch.equal(a.head, b.head)
        assert np.array_equal(oracle.to64(a.layer.y[:sum(n)].cpu()), yb)
    assert torch.equal(a.layer.cache.block_table, b.layer.cache.block_table)
    assert eager.abs().sum() == 0


def test_requests_that_do_not_fit_wait():
    s = Serving("tiny_f32_b1_l128", 3, 100, blocks=3)
    s.check([60, 30, 0])                                               # two pages
    new = torch.tensor([1, 0, 70], dtype=torch.int32, device="cuda")   # the third needs two pages, one is left
    xs = s.inputs([1, 0, 70])
    s.layer.step(xs.cuda(), s.cached, new, s.free, s.head)
    assert mla_get_device_error()[0] == abi.MLA_ERR_BOUNDS
    served = s.layer.seq_lens.tolist()
    assert served == [61, 30, 0] and s.head.tolist() == [2]
    want = s.expect(xs, [1, 0, 0])
    assert_close(oracle.to64(s.layer.y[:1].cpu())[0], want[0], tol_for(s.shape), "y")


@pytest.mark.parametrize("name,fp8", [("tiny_f32_b1_l128", False), ("v3_b64_ragged1k_8k", False), ("v3_b64_ragged1k_8k", True)])
def test_rows_stored_through_slots(name, fp8):
    wl = reduced(WORKLOADS[name], lengths=[70])
    data = generate(wl)
    dev = device_inputs(data, "cuda")
    cfg = Config.from_shape(wl.shape, fp8_cache=fp8)
    s, n = wl.shape, 9
    x = torch.randn(n, s.hidden, generator=torch.Generator().manual_seed(1)).to(cfg.torch_dtype).cuda()
    pos = torch.tensor([0, 1, 63, 64, 100, 5, 131072, 7, 8], dtype=torch.int32, device="cuda")
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
    make = lambda: (torch.zeros(4, 64, s.d_c + s.d_r, device="cuda").to(cfg.cache_torch_dtype),
                    torch.ones(4, 64, device="cuda") if fp8 else None)
    ws = torch.empty(abi.mla_cache_append_workspace_size(cfg, n), dtype=torch.uint8, device="cuda")
    W = dev["weights"]
    pa, sa = make()
    pb, sb = make()
    keep = torch.tensor([0, 1, 2, 3, 4, 5, 7], device="cuda")
    idx = torch.zeros(keep.numel(), dtype=torch.int32, device="cuda")
    abi.mla_cache_append(cfg, x[keep].contiguous(), W["W_DKV"], W["W_KR"], idx, pos[keep].contiguous(), Cache(pa, table, sa), ws)
    slots = torch.full((n,), -1, dtype=torch.int64, device="cuda")     # two tokens are padding
    p = pos[keep].long()
    slots[keep] = table[0, p // 64].long() * 64 + p % 64
    abi.mla_cache_append_slots(cfg, x, W["W_DKV"], W["W_KR"], pos, slots, Cache(pb, table, sb), ws)
    torch.cuda.synchronize()
    check_device_error()
    assert torch.equal(pa, pb) and (not fp8 or torch.equal(sa, sb))
    for bad in (4 * 64, -2, 2 ** 40):
        slots[6] = bad
        abi.mla_cache_append_slots(cfg, x, W["W_DKV"], W["W_KR"], pos, slots, Cache(pb, table, sb), ws)
        status, detail = mla_get_device_error()
        assert status == abi.MLA_ERR_BOUNDS and detail[1] == 6
        assert torch.equal(pa, pb)
    with pytest.raises(TypeError):
        abi.mla_cache_append_slots(cfg, x, W["W_DKV"], W["W_KR"], pos, slots.int(), Cache(pb, table, sb), ws)
    with pytest.raises(MLAError):
        abi.mla_cache_append_slots(cfg, x, W["W_DKV"], W["W_KR"], pos, slots, Cache(pb, table, sb), ws[:256])
