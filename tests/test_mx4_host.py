"""Host-side checks of the MX4 entry points that need no GPU."""
import types

import pytest

torch = pytest.importorskip("torch")

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402


def cfg(**kw):
    d = dict(hidden=256, n_experts=16, n_groups=1, topk_group=1, top_k=4, inter=128, n_shared=1, shared_inter=128,
             weight_bits=4, routed_scaling_factor=2.5)
    d.update(kw)
    return cm.Cfg.of(types.SimpleNamespace(**d))


def test_workspace_serves_the_router_too():
    for T in (0, 1, 7, 64, 300):
        n = cm.coli_mx4_workspace_size(cfg(), T)
        assert n >= cm.coli_moe_workspace_size(cfg(), T) > 0
    assert cm.coli_mx4_workspace_size(cfg(), 300) > cm.coli_mx4_workspace_size(cfg(), 64)


@pytest.mark.parametrize("bad", [dict(weight_bits=8), dict(weight_bits=2), dict(group_size=64), dict(hidden=200), dict(inter=100), dict(top_k=17),
                                 dict(n_experts=2000)])
def test_workspace_refuses_other_configs(bad):
    assert cm.coli_mx4_workspace_size(cfg(**bad), 4) == 0
    with pytest.raises(cm.ColiError):
        cm.new_mx4_workspace(cfg(**bad), 4)


def test_shards_without_shared_experts_need_less():
    whole = cm.coli_mx4_workspace_size(cfg(n_shared=2), 200)
    shard = cm.Cfg.of(types.SimpleNamespace(hidden=256, n_experts=16, n_groups=1, topk_group=1, top_k=4, inter=128, n_shared=2, shared_inter=128,
                                            weight_bits=4, routed_scaling_factor=2.5), 1, 2)
    assert 0 < cm.coli_mx4_workspace_size(shard, 200) < whole


def test_host_tensors_and_wrong_shapes_are_refused():
    x, q, s = torch.zeros(2, 64), torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        cm.coli_mx4_quantize(x, q, s)
    with pytest.raises(ValueError, match="GPU"):
        cm.coli_mx4_dequantize(q, s, x)
    with pytest.raises(ValueError, match="GPU"):
        cm.coli_moe_block_norm(x, n_out=x)
    with pytest.raises(ValueError):
        cm.coli_mx4_product(q, s, q, s, torch.zeros(2, 2), torch.zeros(8704, dtype=torch.uint8))
    with pytest.raises(ValueError):
        cm.coli_mx4_forward(cfg(), cm.Mx4Weights(), torch.zeros(2, 128), q, q, torch.zeros(2, 128), q)
    with pytest.raises(TypeError):
        cm.coli_mx4_quantize(x.double(), q, s)
    with pytest.raises(TypeError):
        cm.coli_moe_block_norm(x, x.half(), n_out=x)


def test_argument_errors_come_before_the_gpu():
    lib = cm.lib
    assert lib.coli_mx4_quantize(None, 0, 64, 0, 64, None, None, None) == cm.COLI_OK
    assert lib.coli_mx4_quantize(None, 0, 64, 1, 64, None, None, None) == cm.COLI_EINVAL
    assert lib.coli_mx4_quantize(16, 0, 64, 1, 65, 16, 16, None) == cm.COLI_EINVAL
    assert lib.coli_mx4_quantize(20, 0, 64, 1, 64, 16, 16, None) == cm.COLI_EALIGN
    assert lib.coli_mx4_product(16, 16, 1, 16, 16, 1, 8, 64, None, 16, 0, 8, 16, 100, None) == cm.COLI_EWORKSPACE
    assert lib.coli_mx4_product(16, 16, 1, 16, 16, 2, 8, 64, None, 16, 0, 8, 16, 8704, None) == cm.COLI_EINVAL
    a = cm.NormArgs(x=16, ldx=64, n_out=16, ld_n_out=64, type=0, n_type=0, eps=1e-6)
    assert lib.coli_moe_block_norm(a, 0, 64, None) == cm.COLI_OK
    assert lib.coli_moe_block_norm(a, 1, 65, None) == cm.COLI_EINVAL
    assert lib.coli_moe_block_norm(a, 1, 20000, None) == cm.COLI_EUNSUPPORTED
