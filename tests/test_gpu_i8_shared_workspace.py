"""A workspace shared, in stream order, by the products of codes and the older operators: the header that
coli_moe_workspace_init clears belongs to its owners (status, counters, the router's tagged words)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import synth  # noqa: E402
import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402
from gpu_harness import DeviceLayer  # noqa: E402

HEADER = 8704


def product(P, N, K, G=1, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-127, 128, (P, K), generator=gen, device="cuda").to(torch.int8)
    w = torch.randint(-127, 128, (G, N, K), generator=gen, device="cuda").to(torch.int8)
    xs, sc = torch.rand(P, generator=gen, device="cuda"), torch.rand(G, N, generator=gen, device="cuda")
    off = torch.linspace(0, P, G + 1, device="cuda").to(torch.int32)
    y = torch.empty(P, N, device="cuda")
    return lambda ws: (cm.coli_i8_product(x, xs, w, sc, y, ws, offsets=off), y)[1]


# few rows, sums in parts, whole sums, tiles of two CTAs
@pytest.mark.parametrize("P,N,K,G", [(3, 300, 512, 1), (16, 4096, 6144, 1), (60, 200, 4096, 3), (500, 300, 1008, 1), (700, 2500, 6144, 3)])
def test_products_leave_the_header(P, N, K, G):
    f, ws = product(P, N, K, G), cm.new_i8_product_workspace(P, K)
    want = f(ws).clone()
    torch.cuda.synchronize()
    assert not ws[:HEADER].any()
    ws[4:HEADER] = 0xa5                      # (the first word is the status)
    assert torch.equal(f(ws), want)
    torch.cuda.synchronize()
    assert (ws[4:HEADER] == 0xa5).all() and not ws[:4].any()


def test_selection_and_grouping_leave_the_header():
    T, H, E, k = 12, 256, 64, 4
    ws = torch.zeros(max(cm.coli_moe_select_workspace_size(T, H, E), cm.coli_moe_group_workspace_size(T, k, E)), dtype=torch.uint8, device="cuda")
    ws[4:HEADER] = 0xa5
    x, wr = torch.randn(T, H, device="cuda"), torch.randn(E, H, device="cuda")
    for n in (T, 1):
        idx, w = torch.empty(n, k, dtype=torch.int32, device="cuda"), torch.empty(n, k, device="cuda")
        cm.coli_moe_select(x[:n], idx, w, router_w=wr, ws=ws)
        cm.coli_moe_group(idx, torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(n * k, dtype=torch.int32, device="cuda"), torch.empty_like(idx), ws)
    torch.cuda.synchronize()
    assert (ws[4:HEADER] == 0xa5).all() and not ws[:4].any()


def test_layers_between_products():
    # one position through the fused layer, whose router exchanges logits by tagged words, and split products
    # (four parts and more) in turn on one workspace: as on workspaces of their own, whatever number a call has
    layer = DeviceLayer(synth.TINY, synth.WORKLOADS["tiny_t8"][1])
    s = layer.shape
    jobs = [product(16, 4096, 6144), product(16, 130, 4096, seed=1), product(60, 200, 4096, 3, seed=2)]
    n = max(cm.coli_moe_workspace_size(layer.cfg, 1), cm.coli_i8_product_workspace_size(60, 6144))
    one, own = torch.empty(n, dtype=torch.uint8, device="cuda"), cm.new_workspace(layer.cfg, 1)
    cm.coli_moe_workspace_init(one)
    spaces = [cm.new_i8_product_workspace(60, 6144) for _ in jobs]
    want = [f(ws).clone() for f, ws in zip(jobs, spaces)]
    xs = torch.from_numpy(synth.token_batch(s, layer.seed, "between", range(64))).cuda()

    def run(x, ws):
        idx, w, y = torch.empty(1, s.top_k, dtype=torch.int32, device="cuda"), torch.empty(1, s.top_k, device="cuda"), torch.empty(1, s.hidden, device="cuda")
        cm.coli_moe_layer(layer.cfg, layer.W, x, layer.wr_d, layer.bias_d, idx, w, y, ws)
        return idx, w, y

    for i in range(64):
        a = run(xs[i:i + 1], own)
        y = jobs[i % 3](one)
        b = run(xs[i:i + 1], one)
        assert all(torch.equal(p, q) for p, q in zip(a, b)), i
        assert torch.equal(y, want[i % 3]), i
    assert cm.coli_moe_status(one) == 0 and cm.coli_moe_status(own) == 0
