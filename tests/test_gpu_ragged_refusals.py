"""A refused step of a ragged layer changes nothing: the tables, the cursor and the
lengths are as they were, and the step can be made again."""

import pytest
import torch

from mla_latent_kv_39_b200 import check_device_error

from test_gpu_ragged_layer import Serving

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["tiny_f32_b1_l128", "v3_b64_ragged1k_8k"])
def test_a_refused_step_changes_nothing(name):
    s = Serving(name, 3, 20)
    s.check([7, 0, 3])
    layer, new = s.layer, torch.tensor([1, 0, 2], dtype=torch.int32, device="cuda")
    x = torch.zeros(20, s.shape.hidden, dtype=s.cfg.torch_dtype, device="cuda")
    held = lambda: [t.clone() for t in (layer.cache.block_table, layer.seq_lens, layer.cu_q, layer.slots, s.head, s.cached)]
    before = held()
    flat = torch.zeros(x.numel() + 8, dtype=x.dtype, device="cuda")
    wrong = [(x[:19], ValueError), (x[:, :-64].contiguous(), ValueError), (x.t().contiguous().t(), ValueError),
             (x.cpu(), ValueError), (x.double(), TypeError), (None, TypeError)]
    if x.dtype == torch.bfloat16:
        wrong.append((flat[1:1 + x.numel()].view_as(x), ValueError))     # off the tensor cores' 16 bytes
    for bad, error in wrong:
        with pytest.raises(error):
            layer.step(bad, s.cached, new, s.free, s.head)
    W = layer.W
    layer.W = {k: v for k, v in W.items() if k != "W_UV"}
    with pytest.raises(KeyError):
        layer.step(x, s.cached, new, s.free, s.head)
    layer.W = W
    torch.cuda.synchronize()
    check_device_error()
    assert all(torch.equal(a, b) for a, b in zip(before, held()))
    s.check([1, 0, 2])
