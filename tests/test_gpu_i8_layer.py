"""The int8 layer with activations quantised per token: every step from the
buffers of the step before it against the 64-bit forms, graph replays, shards."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402
from quantized_expert_ffn_sigmoid_gb300 import i8_layer  # noqa: E402
from oracle import token8  # noqa: E402

E, H, I, K = 16, 256, 128, 4


@pytest.fixture(scope="module")
def weights():
    gen = torch.Generator(device="cuda").manual_seed(5)
    return i8_layer.random_records(E, I, H, gen), i8_layer.random_records(2, I, H, gen), torch.randn(E, H, generator=gen, device="cuda") * H ** -0.5


def make(weights, T, dtype=torch.float32, ns=1, seed=0, **kw):
    (codes, scales), (shared, shared_scales), router = weights
    layer = i8_layer.Layer(codes, scales, router, I, T, dtype, K, shared=shared[:ns] if ns else None, shared_scales=shared_scales[:ns] if ns else None, **kw)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    layer.x.copy_(torch.randn(T, H, generator=gen, device="cuda"))
    return layer


def bits(S, sx, sw, dtype):
    return (torch.from_numpy(S).float() * sx[:, None] * sw).to(dtype)


def check_codes(gu, q, s):
    h = token8.swiglu(gu.double().cpu().numpy())
    s = s.double().cpu().numpy()
    assert (np.abs(q.double().cpu().numpy() * s[:, None] - h) <= s[:, None] * (0.5 + 127 * (2.0 ** -21 + 2.0 ** -22)) + 1e-37).all()


@pytest.mark.parametrize("T,ns,dtype", [(1, 1, torch.float32), (5, 0, torch.bfloat16), (40, 2, torch.bfloat16), (300, 1, torch.float16)])
def test_every_step(weights, T, ns, dtype):
    kw = dict(score=cm.SCORE_SIGMOID, bias=torch.linspace(-0.2, 0.2, E, device="cuda"), n_groups=4, topk_group=2, scaling=2.5) if T != 5 else {}
    s = make(weights, T, dtype, ns, T, **kw)
    y = s.step()
    assert s.status() == 0
    (codes, scales), (shared, shared_scales), router = weights
    w = codes.cpu().numpy()
    gate_up, down = w[:, :2 * I * H].reshape(E, 2 * I, H), w[:, 2 * I * H:].reshape(E, H, I)
    sc = scales.cpu()
    logits = s.x.double().cpu().numpy() @ router.double().cpu().numpy().T
    ids, wt, _ = token8.select(logits, K, bias=None if not kw else kw["bias"].cpu().numpy(), softmax=not kw, groups=4 if kw else 1, keep=2 if kw else 1,
                               scaling=2.5 if kw else 1.0)
    same = (s.idx.cpu().numpy() == ids).all(-1)        # (a near tie of random logits may fall either way)
    assert same.mean() > 0.97 and np.abs(s.w.cpu().numpy() - wt)[same].max() < 1e-5
    off, rows, slots = token8.group(s.idx.cpu().numpy(), E)
    assert np.array_equal(s.offsets.cpu().numpy(), off) and np.array_equal(s.rows.cpu().numpy(), rows) and np.array_equal(s.slots.cpu().numpy(), slots)
    q, _ = token8.quantize(s.x.double().cpu().numpy())
    assert np.array_equal(s.xq.cpu().numpy(), q)
    group = np.searchsorted(off, np.arange(T * K), side="right") - 1
    assert torch.equal(s.gu.cpu(), bits(token8.sums(q, gate_up, off, rows), s.xs.cpu()[rows], sc[group, :2 * I], dtype))
    check_codes(s.gu, s.hq, s.hs)
    assert torch.equal(s.o.cpu(), bits(token8.sums(s.hq.cpu().numpy(), down, off, np.arange(T * K)), s.hs.cpu(), sc[group, 2 * I:], dtype))
    add, mag0 = None, 0.0
    if ns:
        sh, ssc = shared[:ns].cpu().numpy(), shared_scales[:ns].cpu()
        soff, srows = np.arange(ns + 1) * T, np.tile(np.arange(T), ns)
        sg = np.repeat(np.arange(ns), T)
        assert torch.equal(s.s_gu.cpu(), bits(token8.sums(q, sh[:, :2 * I * H].reshape(ns, 2 * I, H), soff, srows), s.xs.cpu()[srows], ssc[sg, :2 * I], dtype))
        check_codes(s.s_gu, s.s_hq, s.s_hs)
        add = s.s_o.double().cpu().numpy().reshape(ns, T, H).sum(0)
        mag0 = np.abs(s.s_o.double().cpu().numpy()).reshape(ns, T, H).sum(0)
    ref, mag = token8.combine(s.o.double().cpu().numpy(), s.slots.cpu().numpy(), s.w.double().cpu().numpy(), add)
    eps = torch.finfo(dtype).eps / 2
    # the shared sum is rounded to y's type once before the routed one is added: half a unit of it more
    tol = (K + 2) * 2.0 ** -24 * (mag + mag0) * 1.01 + eps * (np.abs(ref) + (np.abs(add) if ns else 0.0)) * 1.02 + 2.0 ** -24 * (dtype == torch.float16) + 1e-37
    assert (np.abs(y.double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("T", [3, 70])
def test_graph_replay_is_the_step(weights, T):
    s = make(weights, T, torch.bfloat16)
    g = s.capture()
    for seed in (1, 2, 3):
        s.x.copy_(torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        want = s.step().clone()
        s.y.zero_()
        for _ in range(2):
            g.replay()
        assert torch.equal(s.y, want) and s.status() == 0


def test_two_layers_at_once(weights):
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    layers = [make(weights, T, torch.bfloat16, seed=T) for T in (9, 64)]
    want = [s.step().clone() for s in layers]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, s in zip((a, b), layers):
            with torch.cuda.stream(st):
                s.step()
    torch.cuda.synchronize()
    for s, y in zip(layers, want):
        assert torch.equal(s.y, y) and s.status() == 0


@pytest.mark.parametrize("T,P", [(1, 2), (33, 2), (20, 3)])
def test_shards_add_up(weights, T, P):
    (codes, scales), (shared, shared_scales), router = weights
    whole = make(weights, T).step().double()
    total = torch.zeros_like(whole)
    for r in range(P):
        s = i8_layer.Layer(codes[r::P].contiguous(), scales[r::P].contiguous(), router, I, T, torch.float32, K, shared=shared[:1],
                           shared_scales=shared_scales[:1], ep_rank=r, ep_size=P)
        s.x.copy_(make(weights, T).x)
        total += s.step().double()
        assert s.status() == 0
    # the same pairs' outputs bit for bit; the order of K + 1 terms differs
    assert (total - whole).abs().max() <= 2 * (K + P + 1) * 2.0 ** -24 * (K + 1) * whole.abs().max() * 4


def test_near_the_layer_without_quantisation(weights):
    (codes, scales), _, router = weights
    s = make(weights, 50, torch.float32, ns=0)
    y = s.step().double()
    w = codes.double()
    ref = torch.zeros_like(y)
    for t in range(50):
        for j in range(K):
            e = int(s.idx[t, j])
            gu = (w[e, :2 * I * H].view(2 * I, H) * scales[e, :2 * I, None]) @ s.x[t].double()
            h = gu[:I] * torch.sigmoid(gu[:I]) * gu[I:]
            ref[t] += s.w[t, j].double() * ((w[e, 2 * I * H:].view(H, I) * scales[e, 2 * I:, None]) @ h)
    # two roundings to steps of 1/127 of a row's largest value, a quarter of it typically: about 1 % each, and twice that through silu
    assert ((y - ref).norm(dim=1) / ref.norm(dim=1)).max() < 0.06


def test_refusals(weights):
    (codes, scales), _, router = weights
    with pytest.raises(ValueError, match="int8 records"):
        i8_layer.Layer(codes[:, :-1], scales, router, I, 4, torch.float32, K)
    with pytest.raises(ValueError, match="records of 8 experts"):
        i8_layer.Layer(codes, scales, router, I, 4, torch.float32, K, ep_size=2)
    with pytest.raises(ValueError, match="at least one position"):
        i8_layer.Layer(codes, scales, router, I, 0, torch.float32, K)
