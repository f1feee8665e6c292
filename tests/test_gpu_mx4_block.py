"""The MX4 block runner: a stack's step is exactly its library calls one after
the other (each of which is tested against the oracle on its own), and a graph
replay of it exactly the step."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402
from quantized_expert_ffn_sigmoid_gb300 import mx4_block  # noqa: E402


@pytest.fixture(scope="module", params=[1, 0])
def blocks(request):
    cfg = cm.Cfg(hidden=512, n_experts=32, n_groups=4, topk_group=2, top_k=4, inter=256, n_shared=request.param, shared_inter=256, weight_bits=4,
                 routed_scaling_factor=2.5)
    return [mx4_block.random_block(cfg, i, torch.bfloat16) for i in range(3)]


@pytest.mark.parametrize("T", [1, 9, 200])
def test_stack_is_its_calls(blocks, T):
    cfg = blocks[0].cfg
    H = cfg.hidden
    pre = torch.rand(H, device="cuda") + 0.5
    s = mx4_block.Stack(blocks, pre, T, torch.bfloat16)
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    s.x.copy_(x)
    s.step()
    ws = cm.new_mx4_workspace(cfg, T)
    n, y = torch.empty(T, H, device="cuda"), torch.empty_like(x)
    idx, w = torch.empty(T, 4, dtype=torch.int32, device="cuda"), torch.empty(T, 4, device="cuda")
    q, b = torch.empty(T, H // 2, dtype=torch.uint8, device="cuda"), torch.empty(T, H // 32, dtype=torch.uint8, device="cuda")
    cm.coli_moe_block_norm(x, pre_w=pre, n_out=n)
    for i, blk in enumerate(blocks):
        torch.cuda.synchronize()
        cm.coli_moe_route(cfg, n, blk.router_w, blk.corr_bias, idx, w, ws)
        cm.coli_mx4_quantize(n, q, b)   # the norm's own codes are those of its fp32 result
        cm.coli_mx4_forward(cfg, blk.weights(), q, idx, w, y, ws, x_scales=b)
        assert torch.equal(s.idx[i], idx) and torch.equal(s.w[i], w)
        x1 = torch.empty_like(x)
        cm.coli_moe_block_norm(x, y, post_w=blk.post_w, gate=blk.gate, res_scale=blk.res_scale, pre_w=blk.next_w, x_out=x1, n_out=n)
        x = x1
    torch.cuda.synchronize()
    assert torch.equal(s.x, x) and torch.equal(s.norm, n)
    assert torch.isfinite(x.float()).all() and cm.coli_moe_status(s.ws) == 0 and cm.coli_moe_status(ws) == 0


def test_graph_replay_is_the_step(blocks):
    T, H = 17, blocks[0].cfg.hidden
    s = mx4_block.Stack(blocks, torch.ones(H, device="cuda"), T, torch.bfloat16)
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    s.x.copy_(x)
    g = s.capture()
    assert torch.equal(s.x, x)
    s.step()
    want = s.x.clone(), s.norm.clone()
    for _ in range(3):
        s.x.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(s.x, want[0]) and torch.equal(s.norm, want[1])


def test_blocks_of_different_sizes_are_refused(blocks):
    other = mx4_block.random_block(cm.Cfg(hidden=256, n_experts=8, n_groups=1, topk_group=1, top_k=4, inter=128, n_shared=0, shared_inter=0,
                                          weight_bits=4, routed_scaling_factor=1.0), 9, torch.bfloat16)
    with pytest.raises(ValueError):
        mx4_block.Stack([blocks[0], other], torch.ones(512, device="cuda"), 4, torch.bfloat16)
