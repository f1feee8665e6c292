"""The int8 layer with shared experts of another inner size than the routed ones."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from quantized_expert_ffn_sigmoid_gb300 import i8_layer  # noqa: E402
from oracle import token8  # noqa: E402
from test_gpu_i8_layer import E, H, I, K, bits, check_codes, weights  # noqa: E402,F401


@pytest.mark.parametrize("T,ns,si", [(1, 1, 48), (7, 2, 512), (70, 1, 320)])
def test_shared_experts_of_their_own_size(weights, T, ns, si):  # noqa: F811
    (codes, scales), _, router = weights
    gen = torch.Generator(device="cuda").manual_seed(si)
    shared, shared_scales = i8_layer.random_records(ns, si, H, gen)
    both = i8_layer.Layer(codes, scales, router, I, T, torch.float32, K, shared=shared, shared_scales=shared_scales, shared_inter=si)
    routed = i8_layer.Layer(codes, scales, router, I, T, torch.float32, K)
    routed.x.copy_(torch.randn(T, H, generator=gen, device="cuda"))
    both.x.copy_(routed.x)
    y, r = both.step(), routed.step()
    assert both.status() == routed.status() == 0 and torch.equal(both.o, routed.o) and torch.equal(both.idx, routed.idx)
    q, sh, sc = both.xq.cpu().numpy(), shared.cpu().numpy(), shared_scales.cpu()
    off, rows, at = np.arange(ns + 1) * T, np.tile(np.arange(T), ns), np.repeat(np.arange(ns), T)
    gate_up, down = sh[:, :2 * si * H].reshape(ns, 2 * si, H), sh[:, 2 * si * H:].reshape(ns, H, si)
    assert torch.equal(both.s_gu.cpu(), bits(token8.sums(q, gate_up, off, rows), both.xs.cpu()[rows], sc[at, :2 * si], torch.float32))
    check_codes(both.s_gu, both.s_hq, both.s_hs)
    assert torch.equal(both.s_o.cpu(), bits(token8.sums(both.s_hq.cpu().numpy(), down, off, np.arange(ns * T)), both.s_hs.cpu(), sc[at, 2 * si:], torch.float32))
    ref = r.double() + both.s_o.double().view(ns, T, H).sum(0)
    # fp32 sums of ns + K terms, in another order than r's: half a unit a step on either side
    mag = both.s_o.abs().view(ns, T, H).sum(0).double() + (both.w[..., None] * both.o[both.slots.long()]).abs().sum(1).double()
    assert ((y.double() - ref).abs() <= 2 * (K + ns + 1) * 2.0 ** -24 * mag).all()
    g = both.capture()
    want = both.step().clone()
    both.y.zero_()
    g.replay()
    assert torch.equal(both.y, want)


def test_refusals(weights):  # noqa: F811
    (codes, scales), (shared, shared_scales), router = weights
    with pytest.raises(ValueError, match="int8 records"):
        i8_layer.Layer(codes, scales, router, I, 4, torch.float32, K, shared=shared, shared_scales=shared_scales, shared_inter=2 * I)
    with pytest.raises(ValueError, match="multiples of 16"):
        i8_layer.Layer(codes, scales, router, I, 4, torch.float32, K, shared=shared, shared_scales=shared_scales, shared_inter=I + 8)
