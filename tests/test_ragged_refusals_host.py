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
