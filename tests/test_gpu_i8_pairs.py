"""Products whose tiles two CTAs take together, where offsets, rows and strides are out of the ordinary: by the
tile sizes' expected times these shapes are a sixth or more away from the smaller tiles."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402
from test_gpu_i8 import check, make, want  # noqa: E402

P, N, K = 1500, 6200, 2100
OFFSETS = [
    [0, 0, 700, 700, 1500, 1500],               # empty groups
    [64, 700, 700, 1400],                       # rows of no group at both ends
    [0, 900, 300, 2000, 1500, 1200],            # not ascending, beyond P
    [-7, 5, 99999],
    [0, 0, 0, 0],                               # no rows at all
    [1500, 1500, 1500],
    [0, 1, 17, 48, 81, 208, 336, 465, 1500],    # tiles of 1, 16, 31, 33, 127, 128 and 129 rows
    [0, 1499, 1500],
]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("offsets", OFFSETS)
def test_offsets(offsets, gather):
    check(P, len(offsets) - 1, N, K, "bf16", seed=len(offsets), X=P if not gather else 500, gather=gather, offsets=offsets)


def test_rows_out_of_range():
    x, xs, w, ws = make(200, 4, N, K, 3)
    rows = torch.randint(0, 200, (P,), device="cuda").to(torch.int32)
    bad = [0, 1, 127, 128, 700, P - 2, P - 1]
    rows[bad] = torch.tensor([-1, 200, 2 ** 31 - 1, -2 ** 31, 201, -5, 10 ** 9], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 130, 130, 701, P - 1], dtype=torch.int32, device="cuda")      # the last row is of no group
    y, space = torch.full((P, N), 3.0, device="cuda"), cm.new_i8_product_workspace(P, K)
    cm.coli_i8_product(x, xs, w, ws, y, space, offsets=off, rows=rows)
    ref, live = want(x, xs, w, ws, off.tolist(), rows, torch.float32)
    assert cm.coli_moe_status(space) == cm.STATUS_BADIDX
    assert torch.equal(torch.nan_to_num(y[live], nan=-7.0), torch.nan_to_num(ref[live], nan=-7.0))
    assert torch.isnan(y[bad[:-1]]).all() and (y[-1] == 3.0).all()
    rows[bad[:-1]] = 0
    cm.coli_i8_product(x, xs, w, ws, y, space, offsets=off, rows=rows)                  # (the row of no group is not looked at)
    assert cm.coli_moe_status(space) == 0


def test_weights_at_any_stride():
    G = 5
    x, xs, w, ws = make(P, G, N, K, 21)
    cuts = [0, 190, 190, 760, P - 1, P]
    off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    mixed = torch.zeros(N, G, 2112, dtype=torch.int8, device="cuda").permute(1, 0, 2)[:, :, :K]      # rows between one another
    mixed.copy_(w)
    for weights, scales in ((w[:1].expand(G, N, K), ws), (w[:1].expand(G, N, K), ws[:1].expand(G, N)), (mixed, ws)):
        y, space = torch.empty(P, N, device="cuda"), cm.new_i8_product_workspace(P, K)
        cm.coli_i8_product(x, xs, weights, scales, y, space, offsets=off)
        ref, live = want(x, xs, weights, scales, cuts, torch.arange(P, device="cuda"), torch.float32)
        assert live.all() and torch.equal(y, ref)


def test_scales_without_value():
    x, xs, w, ws = make(P, 2, N, K, 1)
    xs[1], xs[2], ws[1, 5] = float("nan"), 0.0, float("inf")
    y, space = torch.empty(P, N, device="cuda"), cm.new_i8_product_workspace(P, K)
    cm.coli_i8_product(x, xs, w, ws, y, space, offsets=torch.tensor([0, 700, P], dtype=torch.int32, device="cuda"))
    assert torch.isnan(y[1]).all() and (y[2] == 0).all() and torch.isfinite(y[3:700]).all() and not torch.isfinite(y[700:, 5]).any()
    assert torch.isfinite(y[700:, :5]).all() and torch.isfinite(y[700:, 6:]).all()


def test_same_bits_in_every_call_size():
    n, k = 2000, 3300
    x, xs, w, ws = make(3000, 1, n, k, 4)
    space = cm.new_i8_product_workspace(3000, k)
    y = torch.empty(3000, n, device="cuda")
    cm.coli_i8_product(x, xs, w, ws, y, space)
    for p in (1, 4, 9, 33, 65, 129, 1000, 2999):
        z = torch.empty(p, n, device="cuda")
        cm.coli_i8_product(x[:p], xs[:p].clone(), w, ws, z, space)
        assert torch.equal(z, y[:p])


@pytest.mark.parametrize("small", [False, True])
def test_the_longest_rows(small):
    # the largest sums in runs of 512, and one run over the whole row
    p, n, k = 300, 5000, 131071
    x, xs, w, ws = make(p, 1, n, k, 6, extreme=not small)
    if small:
        x.copy_((torch.rand(x.shape, device="cuda") < 0.3).to(torch.int8))
    y, space = torch.empty(p, n, device="cuda"), cm.new_i8_product_workspace(p, k)
    cm.coli_i8_product(x, xs, w, ws, y, space)
    ref, _ = want(x, xs, w, ws, [0, p], torch.arange(p, device="cuda"), torch.float32)
    assert torch.equal(y, ref) and cm.coli_moe_status(space) == 0
