"""The MX4 expert layer at sizes where its index arithmetic matters: records
beyond 32-bit offsets, tens of thousands of pairs, and the widest tiles.
Tolerances as in the tests of small layers (the oracle's bound)."""
import types

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402
from oracle import mx4  # noqa: E402


def layer_of(hidden, inter, experts, top_k, n_shared, filled, seed):
    """A layer whose experts `filled` hold random normal weights, the others zeros."""
    shape = types.SimpleNamespace(hidden=hidden, n_experts=experts, n_groups=1, topk_group=1, top_k=top_k, inter=inter, n_shared=n_shared,
                                  shared_inter=inter, weight_bits=4, routed_scaling_factor=1.0)
    g = torch.Generator("cuda").manual_seed(seed)
    tensors = []
    for n, which in ((experts, filled), (n_shared, range(n_shared))):
        codes = torch.zeros(n, 3 * inter * hidden // 2, dtype=torch.uint8, device="cuda")
        scales = torch.zeros(n, 3 * inter * hidden // 32, dtype=torch.uint8, device="cuda")
        for e in which:
            for at, rows, k in ((0, 2 * inter, hidden), (2 * inter * hidden, hidden, inter)):
                m = torch.randn(rows, k, generator=g, device="cuda") * k ** -0.5
                cm.coli_mx4_quantize(m, codes[e, at // 2:(at + m.numel()) // 2].view(rows, k // 2),
                                     scales[e, at // 32:(at + m.numel()) // 32].view(rows, k // 32))
        tensors += [codes, scales]

    def values(codes, scales):
        c, s = codes.cpu().numpy(), scales.cpu().numpy()
        out = []
        for at, rows, k in ((0, inter, hidden), (inter * hidden, inter, hidden), (2 * inter * hidden, hidden, inter)):
            n = rows * k
            out.append(mx4.values(c[at // 2:(at + n) // 2].reshape(rows, -1), s[at // 32:(at + n) // 32].reshape(rows, -1)))
        return out

    routed = lambda e: values(tensors[0][e], tensors[1][e])   # noqa: E731
    shared = lambda s: values(tensors[2][s], tensors[3][s])   # noqa: E731
    return shape, tensors, routed, shared


def run(shape, tensors, x, idx, w):
    cfg = cm.Cfg.of(shape)
    weights = cm.make_mx4_weights(*tensors)
    ws = cm.new_mx4_workspace(cfg, len(x))
    y = torch.full((len(x), shape.hidden), 777.0, device="cuda")
    cm.coli_mx4_forward(cfg, weights, x, idx, w, y, ws)
    assert cm.coli_moe_status(ws) == 0
    return y


def check(y, ref, bound):
    err = np.abs(y.double().cpu().numpy() - ref)
    bound = bound + 2.0 ** -24 * (np.abs(ref) + bound)
    assert (err <= bound).all(), np.max(err / bound)
    assert np.linalg.norm(err) <= 0.02 * np.linalg.norm(ref)


def test_records_beyond_32_bit_offsets():
    # 240 records of 18 MB of codes: the last begin past 2^32 bytes
    E, last = 240, [0, 7, 238, 239]
    shape, tensors, routed, shared = layer_of(6144, 2048, E, 4, 0, last, 1)
    assert tensors[0][238].data_ptr() - tensors[0].data_ptr() > 2 ** 32
    x = torch.randn(3, 6144, generator=torch.Generator("cuda").manual_seed(2), device="cuda")
    idx = torch.tensor([[0, 239, 5, 238], [238, 7, 239, 100], [239, -1, -1, 238]], dtype=torch.int32, device="cuda")
    w = torch.rand(3, 4, generator=torch.Generator("cuda").manual_seed(3), device="cuda")
    y = run(shape, tensors, x, idx, w)
    keep = torch.where(torch.isin(idx, torch.tensor(last, device="cuda")), idx, -1).cpu().numpy()   # the others hold zeros
    check(y, *mx4.layer(shape, routed, shared, x.cpu().numpy(), keep, w.cpu().numpy()))


@pytest.mark.parametrize("T,experts,top_k,n_shared", [(9000, 40, 6, 1), (5000, 1000, 8, 0)])
def test_many_pairs(T, experts, top_k, n_shared):
    shape, tensors, routed, shared = layer_of(256, 128, experts, top_k, n_shared, range(experts), 4)
    g = torch.Generator("cuda").manual_seed(T)
    x = torch.randn(T, 256, generator=g, device="cuda")
    score = torch.rand(T, experts, generator=g, device="cuda")
    score[:, 3] += 0.5                                        # one expert far more often than the others
    idx = score.topk(top_k, -1)[1].int()
    idx[torch.rand(T, top_k, generator=g, device="cuda") < 0.1] = -1
    w = torch.rand(T, top_k, generator=g, device="cuda")
    y = run(shape, tensors, x, idx, w)
    check(y, *mx4.layer(shape, routed, shared, x.cpu().numpy(), idx.cpu().numpy(), w.cpu().numpy()))
    # the order of an expert's rows may differ from call to call, the result may not
    for _ in range(5):
        assert torch.equal(y, run(shape, tensors, x, idx, w))


def test_wide_layer_of_many_positions():
    shape, tensors, routed, shared = layer_of(2048, 1024, 8, 2, 1, range(8), 5)
    g = torch.Generator("cuda").manual_seed(6)
    T = 900
    x = torch.randn(T, 2048, generator=g, device="cuda")
    idx = torch.rand(T, 8, generator=g, device="cuda").topk(2, -1)[1].int()
    w = torch.rand(T, 2, generator=g, device="cuda")
    y = run(shape, tensors, x, idx, w)
    check(y, *mx4.layer(shape, routed, shared, x.cpu().numpy(), idx.cpu().numpy(), w.cpu().numpy()))
