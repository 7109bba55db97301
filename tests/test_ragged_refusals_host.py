"""What the ragged entry points refuse before anything is launched or changed, on a
machine without a GPU."""

from types import SimpleNamespace

import pytest
import torch

from mla_latent_kv_39_b200 import Config, RaggedLayer, abi, build

V3 = dict(hidden=7168, n_heads=128, d_c=512, d_r=64, qk_nope=128, v_head=128, q_lora=1536)


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


@pytest.mark.parametrize("kw", [
    dict(n_heads=64), dict(d_c=256), dict(d_r=32), dict(block_size=16), dict(hidden=7000), dict(v_head=64), dict(q_lora=1000),
    dict(n_heads=64, fp8_cache=True), dict(block_size=32, fp8_cache=True), dict(n_heads=16, split_query=True),
    dict(dtype="f32", d_c=1000)], ids=str)
def test_a_ragged_layer_refuses_shapes_that_no_step_computes(kw):
    """No kernel makes packed queries of these shapes (or takes rows so wide): the constructor says so, not the first step."""
    cache = SimpleNamespace(block_table=torch.zeros(2, 3, dtype=torch.int32), pool=torch.zeros(1))
    with pytest.raises(ValueError, match="RaggedLayer"):
        RaggedLayer(Config(**{**V3, **kw}), {}, cache, 4)


class Held(SimpleNamespace):
    """What the checks ask of a tensor, on a device of its own."""

    def __init__(self, shape, dtype=torch.int32, device=0):
        super().__init__(shape=torch.Size(shape), dtype=dtype, device=f"cuda:{device}", index=device)

    def get_device(self):
        return self.index

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def first_device(monkeypatch):
    def launched():
        raise AssertionError("a call with a tensor of another device went through")
    monkeypatch.setattr(abi, "_need", lambda *a, **k: None)
    monkeypatch.setattr(abi, "lib", launched)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


def test_slots_are_stored_on_the_current_device_only(first_device):
    cfg = Config(**V3, fp8_cache=True)
    names = ["x", "W_DKV", "W_KR", "pos", "slots", "pool", "table", "row_scale", "workspace"]
    for away in names + [None]:
        at = {n: int(n == away) for n in names}
        cache = SimpleNamespace(pool=Held((8, 64, 576), torch.uint8, at["pool"]), block_table=Held((2, 3), device=at["table"]),
                                row_scale=Held((8, 64), torch.float32, at["row_scale"]), c=abi.MLACache())
        args = (Held((4, 7168), torch.bfloat16, at["x"]), Held((7168, 512), torch.bfloat16, at["W_DKV"]),
                Held((7168, 64), torch.bfloat16, at["W_KR"]), Held((4,), device=at["pos"]), Held((4,), torch.int64, at["slots"]),
                cache, Held((1 << 20,), torch.uint8, at["workspace"]))
        with pytest.raises(AssertionError if away is None else ValueError):
            abi.mla_cache_append_slots(cfg, *args)


BIG = 2 ** 32 + 5          # its low 32 bits are 5: a number that would be taken


def test_numbers_past_32_bits_are_refused_not_cut(first_device):
    cfg = Config(**{**V3, "dtype": "f32"})
    n = 4
    cache = SimpleNamespace(pool=Held((8, 64, 576), torch.float32), block_table=Held((2, 3)), row_scale=None, c=abi.MLACache())
    q, cu, lens = Held((n, 128, 576), torch.float32), Held((3,)), Held((2,))
    o, ws = Held((n, 128, 512), torch.float32), Held((1 << 20,), torch.uint8)

    def window(window=64, n_sinks=4, max_workers=0):
        abi.mla_window_attention(cfg, (q, q), cu, cache, lens, window, n_sinks, o, ws, None, max_workers)

    def chunk(max_workers=0):
        abi.mla_chunk_attention(cfg, (q, q), cu, cache, lens, o, ws, None, max_workers)

    def tables(num_blocks=8):
        abi.mla_batch_tables(cfg, lens, lens, Held((5,)), Held((1,)), num_blocks, cache.block_table, cu, lens, Held((n,)),
                             Held((n,)), Held((n,), torch.int64))
    for call, names in ((window, ("window", "n_sinks", "max_workers")), (chunk, ("max_workers",)), (tables, ("num_blocks",))):
        with pytest.raises(AssertionError):          # goes through as it is
            call()
        for name in names:
            for bad in (BIG, 2 ** 31, -2 ** 31 - 1):
                with pytest.raises(ValueError, match=name):
                    call(**{name: bad})
    with pytest.raises(ValueError, match="n_tok"):
        abi.mla_chunk_workspace_size(cfg, BIG)
    with pytest.raises(ValueError, match="max_workers"):
        abi.mla_chunk_workspace_size(cfg, 4, BIG)


def test_a_ragged_layer_refuses_numbers_past_32_bits():
    cache = SimpleNamespace(block_table=torch.zeros(2, 3, dtype=torch.int32), pool=torch.zeros(1))
    for name in ("window", "n_sinks", "max_workers"):
        with pytest.raises(ValueError, match=name):
            RaggedLayer(Config(**V3), {}, cache, 4, **{"window": 64, name: BIG})


def test_a_config_keeps_its_numbers_when_a_caller_alters_the_struct():
    """c() is the caller's own; what later calls pass is not altered through it, and equal configurations stay equal."""
    cfg = Config(**V3)
    c = cfg.c()
    c.n_heads, c.flags = 7, 2
    assert cfg.c().n_heads == 128 and cfg.c().flags == 0
    assert abi.mla_chunk_workspace_size(cfg, 4) == abi.mla_chunk_workspace_size(Config(**V3), 4) > 256
    assert cfg == Config(**V3) and hash(cfg) == hash(Config(**V3))
    import copy
    import pickle
    for other in (copy.copy(cfg), copy.deepcopy(cfg), pickle.loads(pickle.dumps(cfg))):
        assert other == cfg and abi.mla_chunk_workspace_size(other, 4) == abi.mla_chunk_workspace_size(cfg, 4)
