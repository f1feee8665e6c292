"""What the MX4 block runner refuses before it allocates or launches anything."""
import pytest

torch = pytest.importorskip("torch")

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402
from quantized_expert_ffn_sigmoid_gb300 import mx4_block  # noqa: E402


def block(**kw):
    d = dict(hidden=256, n_experts=8, n_groups=1, topk_group=1, top_k=2, inter=128, n_shared=1, shared_inter=128, weight_bits=4,
             routed_scaling_factor=1.0)
    d.update(kw)
    return mx4_block.Block(cm.Cfg(**d), *(None,) * 8)


@pytest.mark.parametrize("rank,size", [(0, 2), (1, 2), (3, 8)])
def test_shards_are_refused(rank, size):
    # a shard's layer leaves its part of y, which the norm behind it must not be given
    with pytest.raises(ValueError, match="shard"):
        mx4_block.Stack([block(), block(ep_rank=rank, ep_size=size)], torch.ones(256), 3, torch.float32)


@pytest.mark.parametrize("kw", [dict(hidden=128), dict(top_k=3), dict(weight_bits=8)])
def test_blocks_that_do_not_fit_are_refused(kw):
    with pytest.raises(ValueError, match="blocks"):
        mx4_block.Stack([block(), block(**kw)], torch.ones(256), 3, torch.float32)
