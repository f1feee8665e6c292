"""SwiGLU of the MX4 expert layer to the last fp32 bits, seen through 4-bit
codes: gate and up sums are exact by construction (16 terms, one per block,
digits of one 24-bit number), and up is chosen so that h lands just beside a
border between two codes.

fp32 silu(g) * u = g / (1 + exp(-g)) * u takes an exponential, an addition, a
division and a product: within 8 units of 2**-24 (oracle.mx4.expert's bound for
h), so an h that is more than 8 units from its border has to get the code of
its exact value.  Those here are 9 to 15 units away.  The down matrix hands
every h code to y unchanged."""
import types

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402
from oracle import mx4  # noqa: E402

H, I, E = 512, 128, 8
DIGITS = 12                      # base 4
UNIT = 2.0 ** -24
BORDERS = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])


def on_grid(v, top):
    """v rounded towards 0 to DIGITS base-4 digits of which the first counts 4**top."""
    step = np.exp2(2.0 * (top - DIGITS + 1))
    return np.trunc(v / step) * step


def digit_rows(v, top):
    """Codes and scales of rows of H values that sum to v [n] (on that grid): digit j at element 32 j."""
    n = len(v)
    top = np.broadcast_to(np.asarray(top), (n,))
    step = np.exp2(2.0 * (top - DIGITS + 1))
    left = np.rint(np.abs(v) / step).astype(np.int64)
    assert (left * step == np.abs(v)).all() and (left < 1 << 2 * DIGITS).all()
    vals = np.zeros((n, H))
    scales = np.full((n, H // 32), 127, np.uint8)
    codes = np.zeros((n, H // 2), np.uint8)
    for j in range(DIGITS):
        digit = left >> 2 * (DIGITS - 1 - j) & 3
        codes[:, 16 * j] = np.array([0, 2, 4, 5], np.uint8)[digit] | np.where(v < 0, 8, 0).astype(np.uint8)
        scales[:, j] = 127 + np.rint(2.0 * (top - j)).astype(np.int64)
        vals[:, 32 * j] = digit * np.exp2(2.0 * (top - j)) * np.sign(v)
    assert (mx4.values(codes, scales) == vals).all() and (vals.sum(-1) == v).all()
    return codes, scales


def layer_of(g, u, u_top, g_top):
    """Weights of E experts with gate sums g and up sums u [E, I] for the row of ones at elements 32 j."""
    codes, scales = [], []
    down = np.zeros((H, I // 2), np.uint8)
    for n in range(I):
        down[n, n // 2] = 2 << 4 * (n % 2)
    for e in range(E):
        parts = [digit_rows(g[e], g_top), digit_rows(u[e], u_top[e]), (down, np.full((H, I // 32), 127, np.uint8))]
        codes.append(np.concatenate([p[0].ravel() for p in parts]))
        scales.append(np.concatenate([p[1].ravel() for p in parts]))
    return np.stack(codes), np.stack(scales)


def run(codes, scales):
    cfg = cm.Cfg.of(types.SimpleNamespace(hidden=H, n_experts=E, n_groups=1, topk_group=1, top_k=1, inter=I, n_shared=0, shared_inter=0,
                                          weight_bits=4, routed_scaling_factor=1.0))
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    x = torch.zeros(E, H, device="cuda")
    x[:, ::32] = 1.0
    x[:, 32 * DIGITS:] = 0.0
    ec, es = dev(codes), dev(scales)
    # the gate and up sums are what they are meant to be, exactly
    xc, xs = torch.empty(E, H // 2, dtype=torch.uint8, device="cuda"), torch.empty(E, H // 32, dtype=torch.uint8, device="cuda")
    cm.coli_mx4_quantize(x, xc, xs)
    sums = torch.empty(1, 2 * I, device="cuda")
    got = []
    for e in range(E):
        cm.coli_mx4_product(xc[:1], xs[:1], ec[e, :I * H].view(2 * I, H // 2).clone(), es[e, :2 * I * H // 32].view(2 * I, H // 32).clone(), sums,
                            cm.new_mx4_product_workspace())
        got.append(sums.double().cpu().numpy().reshape(2, I))
    ws = cm.new_mx4_workspace(cfg, E)
    y = torch.full((E, H), 777.0, device="cuda")
    idx = torch.arange(E, dtype=torch.int32, device="cuda")[:, None].contiguous()
    cm.coli_mx4_forward(cfg, cm.make_mx4_weights(ec, es), x, idx, torch.ones(E, 1, device="cuda"), y, ws)
    assert cm.coli_moe_status(ws) == 0
    return np.stack(got), y.double().cpu().numpy()


@pytest.mark.parametrize("lo,hi,g_top", [(-5.0, -0.25, 2), (-60.0, -5.0, 2), (-87.3, -60.0, 3), (-88.7, -87.35, 3), (0.25, 6.0, 2), (6.0, 60.0, 2)])
def test_codes_beside_their_borders(lo, hi, g_top):
    rng = np.random.default_rng(int(1000 + lo))
    S = 2.0 ** -10                                               # the scale of every block of h
    g = on_grid(rng.uniform(lo, hi, (E, I)), g_top)
    border = BORDERS[rng.integers(0, len(BORDERS), (E, I))]
    side = rng.choice([-1.0, 1.0], (E, I))
    target = border * (1.0 + side * 12.0 * UNIT) * S
    target[:, ::32] = 4.6 * S                                    # sets the block's scale, far from a border
    silu = g / (1.0 + np.exp(-g))
    want_u = target / np.abs(silu)
    # the top digit is 1 to 3 and the number at least 2 of it: 23 or 24 significant bits
    u_top = np.floor(np.log2(want_u) / 2.0)
    u_top = np.where(want_u < 2.0 * 4.0 ** u_top, u_top - 0.5, u_top)
    u = on_grid(want_u, u_top)
    h = silu * u
    off = (np.abs(h) / (border * S) - 1.0) / UNIT * side
    aimed = np.ones((E, I), bool)
    aimed[:, ::32] = False
    assert (off[aimed] >= 9.0).all() and (off[aimed] <= 15.0).all()
    hq = mx4.values(*mx4.quantize(h))
    got, y = run(*layer_of(g, u, u_top, g_top))
    assert (got[:, 0] == g).all() and (got[:, 1] == u).all()
    wrong = y[:, :I] != hq
    assert not wrong.any(), f"{wrong.sum()} of {wrong.size} codes on the wrong side"
    assert not y[:, I:].any()


def test_far_negative_gates_vanish():
    rng = np.random.default_rng(3)
    g = on_grid(rng.uniform(-1000.0, -110.0, (E, I)), 4)
    g[:, ::32] = 4.0
    u = on_grid(rng.uniform(2.0, 3.9, (E, I)), np.zeros((E, I)))
    hq = mx4.values(*mx4.quantize(np.where(np.arange(I) % 32 == 0, 4.0 / (1.0 + np.exp(-4.0)) * u, 0.0)))
    got, y = run(*layer_of(g, u, np.zeros((E, I)), 4))
    assert (got[:, 0] == g).all() and (got[:, 1] == u).all()
    assert (y[:, :I] == hq).all() and not y[:, I:].any()
