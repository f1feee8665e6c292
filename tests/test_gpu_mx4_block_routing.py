"""The MX4 block runner with routers whose routing arrays are no multiple of
16 bytes (positions x slots not a multiple of 4)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402
from quantized_expert_ffn_sigmoid_gb300 import mx4_block  # noqa: E402

H = 256


@pytest.mark.parametrize("top_k", [1, 2, 3, 6])
def test_any_router_and_position_count(top_k):
    cfg = cm.Cfg(hidden=H, n_experts=8, n_groups=1, topk_group=1, top_k=top_k, inter=128, n_shared=1, shared_inter=128, weight_bits=4,
                 routed_scaling_factor=1.5)
    blocks = [mx4_block.random_block(cfg, i, torch.float32) for i in range(3)]
    pre = torch.ones(H, device="cuda")
    for T in (1, 2, 3, 5, 70):
        s = mx4_block.Stack(blocks, pre, T, torch.float32)
        x = torch.randn(T, H, generator=torch.Generator("cuda").manual_seed(T), device="cuda")
        s.x.copy_(x)
        s.step()
        ws = cm.new_mx4_workspace(cfg, T)
        n, y = torch.empty(T, H, device="cuda"), torch.empty(T, H, device="cuda")
        cm.coli_moe_block_norm(x, pre_w=pre, n_out=n)
        for i, b in enumerate(blocks):
            idx, w = torch.empty(T, top_k, dtype=torch.int32, device="cuda"), torch.empty(T, top_k, device="cuda")
            cm.coli_moe_route(cfg, n, b.router_w, b.corr_bias, idx, w, ws)
            cm.coli_mx4_forward(cfg, b.weights(), n, idx, w, y, ws)
            assert torch.equal(s.idx[i], idx) and torch.equal(s.w[i], w)
            cm.coli_moe_block_norm(x, y, post_w=b.post_w, gate=b.gate, res_scale=b.res_scale, pre_w=b.next_w, x_out=x, n_out=n)
        torch.cuda.synchronize()
        assert torch.equal(s.x, x) and torch.equal(s.norm, n)
        assert cm.coli_moe_status(s.ws) == 0 and cm.coli_moe_status(ws) == 0
        g = s.capture()
        g.replay()
        torch.cuda.synchronize()
        assert cm.coli_moe_status(s.ws) == 0 and torch.isfinite(s.x).all()
