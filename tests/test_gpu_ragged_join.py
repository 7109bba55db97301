"""Ragged attention where workers hold parts of several long tokens: every head of
every token is joined from its pieces.  The outputs hold NaN before each call, so a row
that is never written is seen."""

import math

import pytest
import torch

from mla_latent_kv_39_b200 import Config, RaggedLayer, abi, check_device_error
from mla_synth import WORKLOADS, device_inputs, generate, reduced

from ragged_cases import V3, Ragged

pytestmark = pytest.mark.gpu


def run(r, *args, **kw):
    r.o_lat[:r.n] = math.nan
    r.lse[:r.n] = math.nan
    r.run(*args, **kw)
    check_device_error()


def unequal(n, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(2000, 60001, (n,), generator=g).tolist()


@pytest.mark.parametrize("cached,new", [
    (unequal(4, 1), [1] * 4), (unequal(6, 2), [1] * 6), (unequal(8, 3), [1] * 8), (unequal(12, 4), [1] * 12),
    (unequal(16, 5), [1] * 16), ([16383] * 4, [1] * 4), ([50000] * 5, [1] * 5), ([10000] * 6, [1] * 6),
    ([8000, 20000, 3000, 16000], [1] * 4), ([10000, 10000, 10000, 2000], [1] * 4), ([16000], [3]), ([16000], [10]),
    ([16384] * 2, [4] * 2), ([40000, 0, 30000], [1, 200, 1]), ([700, 30000, 0, 20000, 64], [90, 1, 130, 2, 1])],
    ids=lambda v: f"{len(v)}x{v[0]}")
def test_decodes_and_short_chunks_of_long_requests(cached, new):
    r = Ragged(Config(**V3), cached, new, 3)
    run(r)
    r.check()


@pytest.mark.parametrize("cached,window,sinks", [([16383] * 5, 8192, 4), ([30000, 12000, 9000, 50000, 20000, 7000], 6000, 130)])
def test_windowed_decodes_of_long_requests(cached, window, sinks):
    r = Ragged(Config(**V3), cached, [1] * len(cached), 2)
    run(r, window, sinks)
    r.check(window, sinks)


def test_split_query_decodes_of_long_requests():
    r = Ragged(Config(**V3, split_query=True), [16000, 9000, 24000, 30000], [1, 2, 1, 1], 2)
    run(r)
    r.check()


def test_other_worker_counts():
    r = Ragged(Config(**V3), [9000, 12000, 3000, 15000, 6000], [1, 1, 2, 1, 1], 2)
    for workers in (2, 9, 20, 33, 41, 73):
        run(r, max_workers=workers)
        r.check()


@pytest.mark.parametrize("window,sinks", [(0, 0), (9000, 70)])
def test_cut_tokens_repeat_bit_for_bit(window, sinks):
    r = Ragged(Config(**V3), [20000, 14000, 30000, 500], [1, 1, 2, 60], 0)
    run(r, window, sinks)
    a, b = r.o_lat.clone(), r.lse.clone()
    assert not a.isnan().any() and not b.isnan().any()
    for _ in range(5):
        r.ws.fill_(0xFF)
        run(r, window, sinks)
        assert torch.equal(a, r.o_lat) and torch.equal(b, r.lse)


def test_a_layer_leaves_nothing_of_the_step_before():
    """Six decodes of 10,000 rows through the layer, its buffers holding NaN as if from a step before."""
    wl = reduced(WORKLOADS["v3_b64_ragged1k_8k"], lengths=[1])
    dev = device_inputs(generate(wl), "cuda")
    cfg = Config.from_shape(wl.shape)
    r = Ragged(cfg, [10000] * 6, [1] * 6)
    layer = RaggedLayer(cfg, dev["weights"], r.cache, 6)
    layer.o_lat.fill_(math.nan)
    layer.lse.fill_(math.nan)
    x = torch.randn(6, cfg.hidden, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    free = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = layer.step(x, r.seq_lens - 1, torch.ones_like(r.seq_lens), free, torch.ones_like(free))
    torch.cuda.synchronize()
    check_device_error()
    assert not y.isnan().any() and not layer.o_lat.isnan().any() and not layer.lse.isnan().any()
    # the attention that the step ran, from its own queries and rows
    r.q64, r.o_lat, r.lse = layer.q.double(), layer.o_lat, layer.lse
    for b in range(6):
        pages = layer.cache.block_table[b, :157].long()
        r.pool64[b] = layer.cache.pool[pages].double().view(-1, 576)[:10001]
    r.check()
