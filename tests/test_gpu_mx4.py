"""The MX4 operators on the GPU against the numpy oracle (fp64).

Tolerances.  Quantisation and its inverse are exact in fp32, so codes, scales
and values are compared bit for bit.  A product of K terms summed in fp32 in
any order, each addition rounded or truncated, is within K * 2**-23 * sum|x w|
of the exact sum; storing y adds half a unit of y's type.  The expert layer
adds the effect of every code of h that these sums can move across a rounding
boundary (oracle.mx4.layer).  A norm of H terms: H * 2**-24 relative for the
sum of squares (halved by the square root) plus a few roundings."""
import types

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402
from oracle import mx4  # noqa: E402

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_UNIT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # 24, 8 and 11 significant bits
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}
ACC = 2.0 ** -23


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.double().cpu().numpy()


def strided(a, dtype, pad):
    """`a` on the GPU as rows of a buffer `pad` values wider, poisoned with NaN."""
    buf = torch.full((a.shape[0], a.shape[1] + pad), float("nan"), device="cuda").to(DTYPES[dtype])
    buf[:, :a.shape[1]] = dev(a).to(DTYPES[dtype])
    return buf[:, :a.shape[1]]


def empty_mx4(*lead, K):
    return (torch.full((*lead, K // 2), 0xAB, dtype=torch.uint8, device="cuda"),
            torch.full((*lead, K // 32), 0xAB, dtype=torch.uint8, device="cuda"))


# --------------------------------------------------------------- quantisation
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,K,pad", [(1, 32, 0), (1, 6144, 0), (3, 64, 8), (5, 1024, 5), (7, 1056, 1), (33, 96, 2048), (130, 2080, 0)])
def test_quantize_and_back(dtype, T, K, pad):
    rng = np.random.default_rng(T * K)
    x = rng.standard_normal((T, K)) * np.exp2(rng.integers(-12, 8, (T, K // 32)).repeat(32, 1))
    xs = strided(x, dtype, pad)
    codes, scales = empty_mx4(T, K=K)
    cm.coli_mx4_quantize(xs, codes, scales)
    c, b = mx4.quantize(host(xs))
    assert np.array_equal(scales.cpu().numpy(), b)
    assert np.array_equal(codes.cpu().numpy(), c)
    for out_type in DTYPES:
        buf = torch.full((T, K + pad), 777.0, dtype=DTYPES[out_type], device="cuda")
        cm.coli_mx4_dequantize(codes, scales, buf[:, :K])
        assert torch.equal(buf[:, :K].cpu(), torch.from_numpy(mx4.values(c, b)).to(DTYPES[out_type]))
        assert (buf[:, K:] == 777.0).all()


def test_quantize_special_blocks():
    # every magnitude class: zero, smallest subnormals, around powers of two, ties, largest, infinities, NaN
    rows = [np.zeros(32)]
    for s in (2.0 ** -149, 2.0 ** -140, 2.0 ** -127, 2.0 ** -126, 2.0 ** -125, 2.0 ** -3, 1.0, 2.0 ** 60, 2.0 ** 125):
        rows.append(s * np.resize([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 5.5, 6, 7, 7.75], 32)
                    * np.resize([1, -1, 1], 32))
    rows.append(np.full(32, np.finfo(np.float32).max))
    for bad in (np.inf, -np.inf, np.nan):
        r = np.arange(32.0)
        r[17] = bad
        rows.append(r)
    r = np.full(32, np.nan)
    rows += [r, np.arange(32.0)]
    with np.errstate(over="ignore"):
        x = np.stack(rows).astype(np.float32)
    codes, scales = empty_mx4(len(x), K=32)
    cm.coli_mx4_quantize(dev(x), codes, scales)
    c, b = mx4.quantize(x)
    assert np.array_equal(scales.cpu().numpy(), b)
    assert np.array_equal(codes.cpu().numpy(), c)
    out = torch.empty(len(x), 32, device="cuda")
    cm.coli_mx4_dequantize(codes, scales, out)
    assert np.array_equal(out.cpu().numpy(), mx4.values(c, b).astype(np.float32), equal_nan=True)


def test_dequantize_every_code_and_scale():
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (256, 1))
    scales = np.repeat(np.arange(256, dtype=np.uint8), 16).reshape(-1, 1)
    out = torch.empty(len(codes), 32, device="cuda")
    cm.coli_mx4_dequantize(dev(codes), dev(scales), out)
    with np.errstate(over="ignore"):
        ref = mx4.values(codes, scales).astype(np.float32)
    assert np.array_equal(out.cpu().numpy(), ref, equal_nan=True)


# -------------------------------------------------------------------- product
def random_mx4(rng, *lead, K, spread=3):
    c = rng.integers(0, 256, (*lead, K // 2), dtype=np.uint8)
    b = rng.integers(127 - spread, 128 + spread, (*lead, K // 32)).astype(np.uint8)
    return c, b


def check_product(P, G, N, K, y_type="f32", pad=0, offsets=None, seed=0, spread=3):
    rng = np.random.default_rng(seed + P + 31 * N + 7 * K + G)
    xc, xb = random_mx4(rng, P, K=K, spread=spread)
    wc, wb = random_mx4(rng, G, N, K=K, spread=spread)
    if offsets is None:
        offsets = [0] + sorted(rng.integers(0, P + 1, G - 1).tolist()) + [P]
    buf = torch.full((P, N + pad), 777.0, dtype=DTYPES[y_type], device="cuda")
    ws = cm.new_mx4_product_workspace()
    off = None if G == 1 and seed % 2 else dev(np.array(offsets, np.int32))
    cm.coli_mx4_product(dev(xc), dev(xb), dev(wc), dev(wb), buf[:, :N], ws, offsets=off)
    ref, mag = mx4.product(mx4.values(xc, xb), mx4.values(wc, wb), offsets)
    y = host(buf[:, :N])
    bound = K * ACC * mag + HALF_UNIT[y_type] * (np.abs(ref) + K * ACC * mag) + TINY[y_type]
    assert (np.abs(y - ref) <= bound).all(), np.max(np.abs(y - ref) / bound)
    assert (buf[:, N:] == 777.0).all()
    assert cm.coli_moe_status(ws) == 0
    return buf, (xc, xb, wc, wb, offsets)


@pytest.mark.parametrize("P", [1, 2, 7, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 255, 257, 300, 515])
def test_product_rows(P):
    check_product(P, 1, 200, 544)


@pytest.mark.parametrize("N", [1, 3, 31, 32, 64, 65, 127, 128, 129, 250, 384, 1000])
def test_product_columns(N):
    check_product(33, 1, N, 288, pad=3)


@pytest.mark.parametrize("K", [32, 64, 96, 128, 224, 256, 288, 480, 512, 544, 992, 1024, 1056, 1536, 2048, 6144])
def test_product_reduction(K):
    check_product(20, 1, 130, K, seed=1)
    check_product(140, 1, 130, K)


@pytest.mark.parametrize("y_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_product_types_and_strides(y_type, pad):
    check_product(50, 3, 136, 320, y_type, pad)


@pytest.mark.parametrize("P,G,N,K", [(1, 4, 64, 64), (5, 9, 128, 96), (64, 8, 129, 512), (333, 7, 100, 544), (700, 33, 256, 256),
                                     (1000, 1000, 40, 64), (3, 1024, 33, 32)])
def test_product_groups(P, G, N, K):
    check_product(P, G, N, K)


@pytest.mark.parametrize("offsets", [[0, 0, 0, 40], [0, 40, 40, 40], [0, 13, 13, 40], [0, 1, 39, 40]])
def test_product_empty_groups(offsets):
    check_product(40, 3, 96, 160, offsets=offsets)


def test_product_rows_of_no_group_are_not_written():
    buf, (xc, xb, wc, wb, _) = check_product(40, 2, 64, 64, offsets=[0, 10, 40])
    y = torch.full((40, 64), 777.0, device="cuda")
    ws = cm.new_mx4_product_workspace()
    cm.coli_mx4_product(dev(xc), dev(xb), dev(wc), dev(wb), y, ws, offsets=dev(np.array([3, 10, 31], np.int32)))
    assert (y[:3] == 777.0).all() and (y[31:] == 777.0).all() and torch.equal(y[3:31], buf[3:31])


def test_product_offsets_are_clamped():
    # out of range and descending: the clamped ranges are [0, 5), [5, 40), [40, 40)
    buf, (xc, xb, wc, wb, _) = check_product(40, 3, 64, 64, offsets=[0, 5, 40, 40])
    y = torch.full((40, 64), 777.0, device="cuda")
    ws = cm.new_mx4_product_workspace()
    cm.coli_mx4_product(dev(xc), dev(xb), dev(wc), dev(wb), y, ws, offsets=dev(np.array([-7, 5, 1 << 30, -9], np.int32)))
    assert torch.equal(y, buf)


def test_product_wide_scales_and_lost_blocks():
    rng = np.random.default_rng(11)
    P, N, K = 24, 70, 128
    xc, xb = random_mx4(rng, P, K=K)
    wc, wb = random_mx4(rng, 1, N, K=K)
    xb[:, 0], wb[..., 0] = 127 + 60, 127 - 60       # large times small
    xb[5, 2] = 255                                  # a block without a value: its row of y has none
    wb[0, 9, 3] = 255                               # and its column
    y = torch.empty(P, N, device="cuda")
    cm.coli_mx4_product(dev(xc), dev(xb), dev(wc), dev(wb), y, cm.new_mx4_product_workspace())
    ref, mag = mx4.product(mx4.values(xc, xb), mx4.values(wc, wb))
    yh = host(y)
    assert np.isnan(yh[5]).all() and np.isnan(yh[:, 9]).all()
    ok = ~np.isnan(ref)
    assert ok.sum() == (P - 1) * (N - 1) and (np.abs(yh - ref)[ok] <= K * ACC * mag[ok]).all()


def test_product_repeats_bit_for_bit_and_runs_on_other_streams():
    buf, (xc, xb, wc, wb, off) = check_product(300, 5, 384, 1024, y_type="bf16")
    d = [dev(v) for v in (xc, xb, wc, wb)]
    offs, ws = dev(np.array(off, np.int32)), cm.new_mx4_product_workspace()
    ys = [torch.empty_like(buf) for _ in range(3)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    cm.coli_mx4_product(*d, ys[0], ws, offsets=offs, stream=s)
    with torch.cuda.stream(s):
        cm.coli_mx4_product(*d, ys[1], ws, offsets=offs)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="thread_local"):
        cm.coli_mx4_product(*d, ys[2], ws, offsets=offs)
    g.replay()
    torch.cuda.synchronize()
    for y in ys:
        assert torch.equal(y, buf)


def test_product_weights_beyond_32_bit_offsets():
    # 36 groups of 128 MiB of codes; only the last group has rows
    G, N, K = 36, 32768, 8192
    wc = torch.zeros(G, N, K // 2, dtype=torch.uint8, device="cuda")
    wb = torch.full((G, N, K // 32), 127, dtype=torch.uint8, device="cuda")
    assert wc.numel() > 2 ** 32
    rng = np.random.default_rng(2)
    P = 5
    xc, xb = random_mx4(rng, P, K=K)
    rows = [0, 1, 777, N - 2, N - 1]
    c, b = random_mx4(rng, len(rows), K=K)
    for i, r in enumerate(rows):
        wc[G - 1, r], wb[G - 1, r] = dev(c[i]), dev(b[i])
    y = torch.full((P, N), 777.0, device="cuda")
    off = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    off[G] = P
    ws = cm.new_mx4_product_workspace()
    cm.coli_mx4_product(dev(xc), dev(xb), wc, wb, y, ws, offsets=off)
    ref, mag = mx4.product(mx4.values(xc, xb), mx4.values(c, b)[None])
    assert (np.abs(host(y[:, rows]) - ref) <= K * ACC * mag).all()
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert (y[:, rest] == 0).all() and cm.coli_moe_status(ws) == 0


def test_product_outputs_beyond_32_bit_offsets():
    P, N, K = 33000, 33000, 32     # 1.09e9 values of y in rows 2 * N apart: the last at element 2.2e9
    rng = np.random.default_rng(4)
    xc, xb = random_mx4(rng, P, K=K)
    wc, wb = random_mx4(rng, N, K=K)
    buf = torch.zeros(P, 2 * N, dtype=torch.bfloat16, device="cuda")
    cm.coli_mx4_product(dev(xc), dev(xb), dev(wc), dev(wb), buf[:, :N], cm.new_mx4_product_workspace())
    for rows in (slice(0, 3), slice(P - 200, P)):
        ref, mag = mx4.product(mx4.values(xc[rows], xb[rows]), mx4.values(wc, wb)[None])
        bound = (K * ACC) * mag * 1.01 + HALF_UNIT["bf16"] * np.abs(ref) + TINY["bf16"]
        assert (np.abs(host(buf[rows, :N]) - ref) <= bound).all()
    assert not buf[:, N:].any()


# ---------------------------------------------------------------- expert layer
def shape_of(**kw):
    d = dict(hidden=256, n_experts=16, n_groups=1, topk_group=1, top_k=4, inter=128, n_shared=1, shared_inter=128,
             weight_bits=4, routed_scaling_factor=2.5)
    d.update(kw)
    return types.SimpleNamespace(**d)


class Layer:
    def __init__(self, seed=0, ep_rank=0, ep_size=0, **kw):
        self.shape = s = shape_of(**kw)
        self.cfg = cm.Cfg.of(s, ep_rank, ep_size)
        rng = np.random.default_rng(seed)

        def records(n, inter):
            out = [[mx4.quantize(rng.standard_normal(d) * d[1] ** -0.5) for d in ((inter, s.hidden), (inter, s.hidden), (s.hidden, inter))]
                   for _ in range(n)]
            codes = np.stack([np.concatenate([m[0].ravel() for m in r]) for r in out]) if n else np.zeros((0, 1), np.uint8)
            scales = np.stack([np.concatenate([m[1].ravel() for m in r]) for r in out]) if n else np.zeros((0, 1), np.uint8)
            return [[mx4.values(*m) for m in r] for r in out], codes, scales

        self.routed, ec, es = records(s.n_experts, s.inter)
        self.shared, sc, ss = records(s.n_shared, s.shared_inter)
        if ep_size > 1:
            ec, es = ec[ep_rank::ep_size], es[ep_rank::ep_size]
        self.dev = [dev(v) for v in (ec, es, sc, ss)]
        self.weights = cm.make_mx4_weights(*self.dev)

    def routing(self, rng, T, skip=0.0):
        s = self.shape
        idx = np.stack([rng.permutation(s.n_experts)[:s.top_k] for _ in range(T)]).astype(np.int32)
        idx[rng.random(idx.shape) < skip] = -1
        return idx, rng.random((T, s.top_k)).astype(np.float32)

    def run(self, x, idx, w, y_type="f32", ws=None, stream=None, x_scales=None):
        T = idx.shape[0]
        self.ws = cm.new_mx4_workspace(self.cfg, T) if ws is None else ws
        y = torch.full((T, self.shape.hidden), 777.0, dtype=DTYPES[y_type], device="cuda")
        torch.cuda.synchronize()
        cm.coli_mx4_forward(self.cfg, self.weights, x, dev(idx), dev(w), y, self.ws, x_scales=x_scales, stream=stream)
        torch.cuda.synchronize()
        return y

    def check(self, x, idx, w, y, y_type="f32"):
        ref, bound = mx4.layer(self.shape, self.routed.__getitem__, self.shared.__getitem__, x, idx, w)
        bound = bound + HALF_UNIT[y_type] * (np.abs(ref) + bound) + TINY[y_type]
        err = np.abs(host(y) - ref)
        assert (err <= bound).all(), np.max(err / bound)
        # the bound is an estimate of the worst case: on the whole the result is much nearer
        assert np.linalg.norm(err) <= 0.02 * np.linalg.norm(ref) + 1e-30


@pytest.fixture(scope="module")
def tiny():
    return Layer(seed=1)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 16, 17, 33, 64, 70, 130, 257])
def test_layer_positions(tiny, T):
    rng = np.random.default_rng(T)
    x = rng.standard_normal((T, 256)).astype(np.float32)
    idx, w = tiny.routing(rng, T)
    tiny.check(x, idx, w, tiny.run(dev(x), idx, w))
    assert cm.coli_moe_status(tiny.ws) == 0


@pytest.mark.parametrize("kw", [dict(n_shared=0), dict(n_shared=2, shared_inter=384), dict(inter=384, shared_inter=128), dict(top_k=1, n_shared=0),
                                dict(n_experts=5, top_k=5), dict(hidden=1152, inter=640), dict(hidden=128, inter=128),
                                dict(n_experts=200, top_k=8, n_shared=1)])
@pytest.mark.parametrize("T", [1, 6, 90])
def test_layer_shapes(kw, T):
    layer = Layer(seed=2, **kw)
    rng = np.random.default_rng(T)
    x = rng.standard_normal((T, layer.shape.hidden)).astype(np.float32)
    idx, w = layer.routing(rng, T)
    layer.check(x, idx, w, layer.run(dev(x), idx, w))


@pytest.mark.parametrize("x_type", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("y_type", ["f32", "bf16", "f16"])
def test_layer_types(tiny, x_type, y_type):
    rng = np.random.default_rng(9)
    x = dev(rng.standard_normal((11, 256))).to(DTYPES[x_type])
    idx, w = tiny.routing(rng, 11)
    tiny.check(host(x), idx, w, tiny.run(x, idx, w, y_type), y_type)


def test_layer_takes_codes(tiny):
    rng = np.random.default_rng(10)
    for T in (1, 7, 80):
        x = rng.standard_normal((T, 256)).astype(np.float32)
        idx, w = tiny.routing(rng, T)
        codes, scales = empty_mx4(T, K=256)
        cm.coli_mx4_quantize(dev(x), codes, scales)
        assert torch.equal(tiny.run(codes, idx, w, x_scales=scales), tiny.run(dev(x), idx, w))


@pytest.mark.parametrize("T", [1, 5, 70])
def test_layer_skipped_and_repeated_slots(tiny, T):
    rng = np.random.default_rng(20 + T)
    x = rng.standard_normal((T, 256)).astype(np.float32)
    idx, w = tiny.routing(rng, T, skip=0.4)
    idx[0] = -1                                     # a position with no routed expert at all
    idx[T // 2, :2] = 3                             # one expert twice
    w[-1, 0] = 0.0
    tiny.check(x, idx, w, tiny.run(dev(x), idx, w))
    none = Layer(seed=3, n_shared=0)
    y = none.run(dev(x), np.full_like(idx, -1), w)
    assert (y == 0).all() and cm.coli_moe_status(none.ws) == 0


def test_layer_one_expert_takes_all(tiny):
    T = 300
    rng = np.random.default_rng(30)
    x = rng.standard_normal((T, 256)).astype(np.float32)
    idx = np.full((T, 4), -1, np.int32)
    idx[:, 2] = 7
    idx[5, 0] = 15
    w = rng.random((T, 4)).astype(np.float32)
    tiny.check(x, idx, w, tiny.run(dev(x), idx, w))


def test_layer_bad_ids_and_lost_values(tiny):
    rng = np.random.default_rng(31)
    x = rng.standard_normal((9, 256)).astype(np.float32)
    idx, w = tiny.routing(rng, 9)
    good = tiny.run(dev(x), idx, w)
    bad = idx.copy()
    bad[2, 1], bad[4, 0] = 16, -5
    skipped = np.where((bad < -1) | (bad >= 16), -1, bad)
    y = tiny.run(dev(x), bad, w)
    assert cm.coli_moe_status(tiny.ws) == cm.STATUS_BADIDX
    assert cm.coli_moe_status(tiny.ws) == 0
    assert torch.equal(y, tiny.run(dev(x), skipped.astype(np.int32), w))
    xn = x.copy()
    xn[3, 100] = np.inf
    y = tiny.run(dev(xn), idx, w)
    assert cm.coli_moe_status(tiny.ws) & cm.STATUS_NONFINITE
    keep = np.arange(9) != 3
    assert torch.isnan(y[3]).all() and torch.equal(y[keep], good[keep])


def test_layer_workspace_reuse_streams_and_graph(tiny):
    rng = np.random.default_rng(32)
    ws = cm.new_mx4_workspace(tiny.cfg, 100)
    s = torch.cuda.Stream()
    for T in (100, 1, 33, 2, 64):
        x = rng.standard_normal((T, 256)).astype(np.float32)
        idx, w = tiny.routing(rng, T)
        a = tiny.run(dev(x), idx, w, ws=ws)
        for _ in range(3):
            assert torch.equal(a, tiny.run(dev(x), idx, w, ws=ws, stream=s))
        xd, idxd, wd, y = dev(x), dev(idx), dev(w), torch.empty_like(a)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="thread_local"):
            cm.coli_mx4_forward(tiny.cfg, tiny.weights, xd, idxd, wd, y, ws)
            cm.coli_mx4_forward(tiny.cfg, tiny.weights, xd, idxd, wd, y, ws)
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, y)


def test_layer_and_products_on_several_streams_at_once(tiny):
    # calls on different streams share the SMs: each claims its work as it gets them
    rng = np.random.default_rng(33)
    streams = [torch.cuda.Stream() for _ in range(4)]
    jobs = []
    for i, T in enumerate((70, 1, 33, 130)):
        x = dev(rng.standard_normal((T, 256)).astype(np.float32))
        idx, w = tiny.routing(rng, T)
        want = tiny.run(x, idx, w)
        jobs.append((x, dev(idx), dev(w), torch.empty_like(want), cm.new_mx4_workspace(tiny.cfg, T), want, T))
    xc, xb = random_mx4(rng, 500, K=512)
    wc, wb = random_mx4(rng, 6, 700, K=512)
    p = [dev(v) for v in (xc, xb, wc, wb)]
    off = dev(np.array([0, 50, 50, 200, 210, 499, 500], np.int32))
    pw = [cm.new_mx4_product_workspace() for _ in streams]
    py = [torch.empty(500, 700, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (x, idx, w, y, ws, _, _), pws, y2 in zip(streams, jobs, pw, py):
            cm.coli_mx4_forward(tiny.cfg, tiny.weights, x, idx, w, y, ws, stream=s)
            cm.coli_mx4_product(*p, y2, pws, offsets=off, stream=s)
    torch.cuda.synchronize()
    for (_, _, _, y, ws, want, _), pws, y2 in zip(jobs, pw, py):
        assert torch.equal(y, want) and torch.equal(y2, py[0])
        assert cm.coli_moe_status(ws) == 0 and cm.coli_moe_status(pws) == 0


@pytest.mark.parametrize("T", [1, 40])
def test_layer_shards_sum_to_the_layer(T):
    rng = np.random.default_rng(40)
    whole = Layer(seed=4, n_experts=10)
    x = rng.standard_normal((T, 256)).astype(np.float32)
    idx, w = whole.routing(rng, T)
    total = 0.0
    for r in range(3):
        shard = Layer(seed=4, n_experts=10, ep_rank=r, ep_size=3)
        part = shard.run(dev(x), idx, w)
        total = total + part.double()
        assert cm.coli_moe_status(shard.ws) == 0
    whole.check(x, idx, w, total)


def test_layer_route_shares_the_workspace():
    layer = Layer(seed=5, n_groups=4, topk_group=2)
    rng = np.random.default_rng(50)
    T = 12
    x = rng.standard_normal((T, 256)).astype(np.float32)
    ws = cm.new_mx4_workspace(layer.cfg, T)
    idx = torch.empty(T, 4, dtype=torch.int32, device="cuda")
    w = torch.empty(T, 4, device="cuda")
    wr, bias = dev(rng.standard_normal((16, 256)).astype(np.float32) * 0.1), torch.zeros(16, device="cuda")
    y = torch.empty(T, 256, device="cuda")
    cm.coli_moe_route(layer.cfg, dev(x), wr, bias, idx, w, ws)
    cm.coli_mx4_forward(layer.cfg, layer.weights, dev(x), idx, w, y, ws)
    assert cm.coli_moe_status(ws) == 0
    layer.check(x, idx.cpu().numpy(), w.cpu().numpy(), y)


# ----------------------------------------------------------------------- norms
def norm_case(T, H, dtype, post=True, gate="token", pre=True, with_y=True, pad=0, n_type=None, codes=False, inplace=False, seed=0):
    rng = np.random.default_rng(seed + T * 7 + H)
    n_type = n_type or dtype
    x, y = strided(rng.standard_normal((T, H)), dtype, pad), strided(rng.standard_normal((T, H)) * 3, dtype, pad)
    pw = dev((1 + 0.2 * rng.standard_normal(H)).astype(np.float32)) if post else None
    nw = dev((1 + 0.2 * rng.standard_normal(H)).astype(np.float32)) if pre else None
    g = {"none": None, "channel": dev(rng.random(H)).to(DTYPES[dtype]), "token": strided(rng.random((T, H)), dtype, pad)}[gate]
    xo, no = mx4.block_norm(host(x), host(y) if with_y else None, host(pw) if post else None, None if g is None else host(g), 0.7,
                            host(nw) if pre else None, 1e-5)
    x_in = host(x)
    xbuf = torch.full((T, H + pad), 777.0, dtype=DTYPES[dtype], device="cuda")
    nbuf = torch.full((T, H + pad), 777.0, dtype=DTYPES[n_type], device="cuda")
    x_out = x if inplace else xbuf[:, :H]
    q = empty_mx4(T, K=H) if codes else (None, None)
    cm.coli_moe_block_norm(x, y if with_y else None, post_w=pw, gate=g, res_scale=0.7, pre_w=nw, eps=1e-5, x_out=x_out, n_out=nbuf[:, :H],
                           codes=q[0], scales=q[1])
    rel = (H + 32) * 2.0 ** -24
    ex = rel * (np.abs(x_in) + np.abs(xo - x_in))
    assert (np.abs(host(x_out) - xo) <= ex + HALF_UNIT[dtype] * (np.abs(xo) + ex) + TINY[dtype]).all()
    # n = x' * c * w: x' off by ex, c by its own sum and the relative size of ex in the row
    c = (np.abs(host(nw)) if pre else 1.0) / np.sqrt((xo * xo).mean(-1, keepdims=True) + 1e-5)
    en = ex * c + np.abs(no) * (rel + np.linalg.norm(ex, axis=-1, keepdims=True) / np.linalg.norm(xo, axis=-1, keepdims=True))
    assert (np.abs(host(nbuf[:, :H]) - no) <= en + HALF_UNIT[n_type] * (np.abs(no) + en) + TINY[n_type]).all()
    assert (nbuf[:, H:] == 777.0).all() and (inplace or (xbuf[:, H:] == 777.0).all())
    if codes:
        v0, reach = mx4._quant_reach(no, en)
        v = mx4.values(q[0].cpu().numpy(), q[1].cpu().numpy())
        assert (np.abs(v - v0) <= reach).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,H", [(1, 1), (2, 7), (5, 33), (9, 64), (3, 255), (17, 256), (4, 257), (1, 512), (3, 520), (2, 1000), (170, 2049), (1, 6144),
                                 (200, 6144), (160, 8192), (2, 8200), (155, 16384), (1, 16384)])
def test_norm_sizes(dtype, T, H):
    norm_case(T, H, dtype)


@pytest.mark.parametrize("kw", [dict(post=False), dict(gate="none"), dict(gate="channel"), dict(pre=False), dict(with_y=False, post=False, gate="none"),
                                dict(post=False, gate="none", pre=False), dict(pad=8), dict(pad=3), dict(n_type="f32"), dict(inplace=True)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H", [320, 1024])
def test_norm_options(kw, dtype, H):
    norm_case(37, H, dtype, **kw)


@pytest.mark.parametrize("T,H", [(1, 32), (40, 96), (3, 512), (1, 544), (7, 1056), (1, 6144), (300, 6144), (2, 16384)])
@pytest.mark.parametrize("pad", [0, 5])
def test_norm_codes(T, H, pad):
    norm_case(T, H, "bf16", pad=pad, codes=True, n_type="f32")
    norm_case(T, H, "f32", pad=pad, codes=True)


def test_norm_codes_alone_and_lost_rows():
    x = torch.randn(6, 128, device="cuda")
    x[2, 5] = float("nan")
    x[4] = 0.0
    codes, scales = empty_mx4(6, K=128)
    cm.coli_moe_block_norm(x, codes=codes, scales=scales, eps=1e-6)
    b = scales.cpu().numpy()
    assert (b[2] == 255).all() and not (np.delete(b, 2, 0) == 255).any()
    assert (b[4] == 0).all() and not codes[4].any()


# -------------------------------------------------------------------- refusals
def code_of(fn, *a, **k):
    with pytest.raises(cm.ColiError) as e:
        fn(*a, **k)
    return e.value.code


def test_refusals():
    lib, f = cm.lib, torch.zeros(1 << 16, device="cuda")
    p, s = f.data_ptr(), 0
    q = lambda *a: lib.coli_mx4_quantize(*a, s)  # noqa: E731
    assert q(p, 0, 64, 4, 48, p, p) == cm.COLI_EINVAL            # K not a multiple of 32
    assert q(p, 0, 32, 4, 64, p, p) == cm.COLI_EINVAL            # rows overlap
    assert q(p, 3, 64, 4, 64, p, p) == cm.COLI_EINVAL            # not a value type
    assert q(p, 0, 64, -1, 64, p, p) == cm.COLI_EINVAL
    assert q(None, 0, 64, 1, 64, p, p) == cm.COLI_EINVAL
    assert q(p + 4, 0, 64, 1, 64, p, p) == cm.COLI_EALIGN
    assert q(p, 0, 64, 1, 64, p, p + 8) == cm.COLI_EALIGN
    assert q(None, 0, 64, 0, 64, None, None) == cm.COLI_OK       # nothing to do
    d = lambda *a: lib.coli_mx4_dequantize(*a, s)  # noqa: E731
    assert d(p, p, 4, 64, p, 9, 64) == cm.COLI_EINVAL
    assert d(p, p, 4, 64, p + 2, 1, 64) == cm.COLI_EALIGN
    assert d(None, None, 0, 64, None, 0, 64) == cm.COLI_OK

    ws = cm.new_mx4_product_workspace()
    w, n = ws.data_ptr(), ws.numel()

    def prod(xc=p, xs=p, P=4, wc=p, wsc=p, G=1, N=8, K=64, off=None, y=p, yt=0, ldy=8, wp=w, wn=n):
        return lib.coli_mx4_product(xc, xs, P, wc, wsc, G, N, K, off, y, yt, ldy, wp, wn, s)
    assert prod(K=40) == cm.COLI_EINVAL and prod(K=0) == cm.COLI_EINVAL
    assert prod(G=0) == cm.COLI_EINVAL and prod(N=0) == cm.COLI_EINVAL and prod(P=-1) == cm.COLI_EINVAL
    assert prod(G=2) == cm.COLI_EINVAL                           # several groups need offsets
    assert prod(G=1025, off=p) == cm.COLI_EUNSUPPORTED
    assert prod(ldy=7) == cm.COLI_EINVAL and prod(yt=3) == cm.COLI_EINVAL
    assert prod(wc=None) == cm.COLI_EINVAL and prod(wp=None) == cm.COLI_EINVAL
    assert prod(xc=p + 8) == cm.COLI_EALIGN and prod(off=p + 2) == cm.COLI_EALIGN
    assert prod(wn=n - 1) == cm.COLI_EWORKSPACE
    assert prod(P=0, xc=None) == cm.COLI_OK
    assert prod(P=1 << 30) == cm.COLI_EUNSUPPORTED

    layer = Layer(seed=6)
    for bad in (dict(weight_bits=8), dict(weight_bits=2), dict(weight_bits=4, group_size=64), dict(hidden=200), dict(top_k=17)):
        cfg = cm.Cfg.of(types.SimpleNamespace(**{**vars(layer.shape), **bad}))
        assert cm.coli_mx4_workspace_size(cfg, 4) == 0
        with pytest.raises(cm.ColiError):
            cm.new_mx4_workspace(cfg, 4)
    ws = cm.new_mx4_workspace(layer.cfg, 4)
    rng = np.random.default_rng(0)
    idx, wt = layer.routing(rng, 8)
    x, y = torch.zeros(8, 256, device="cuda"), torch.zeros(8, 256, device="cuda")
    assert code_of(cm.coli_mx4_forward, layer.cfg, layer.weights, x, dev(idx), dev(wt), y,
                   torch.empty(cm.coli_mx4_workspace_size(layer.cfg, 8) // 2, dtype=torch.uint8, device="cuda")) == cm.COLI_EWORKSPACE
    none = cm.Mx4Weights(layer.dev[0].data_ptr(), layer.dev[1].data_ptr(), None, None)
    assert code_of(cm.coli_mx4_forward, layer.cfg, none, x[:4], dev(idx[:4]), dev(wt[:4]), y[:4], ws) == cm.COLI_EINVAL
    with pytest.raises(ValueError):
        cm.coli_mx4_forward(layer.cfg, layer.weights, x, dev(idx[:4]), dev(wt[:4]), y, ws)
    with pytest.raises(TypeError):
        cm.coli_mx4_forward(layer.cfg, layer.weights, x.double(), dev(idx), dev(wt), y, ws)
    e = torch.zeros(0, 256, device="cuda")
    cm.coli_mx4_forward(layer.cfg, layer.weights, e, torch.zeros(0, 4, dtype=torch.int32, device="cuda"), torch.zeros(0, 4, device="cuda"), e, ws)

    xn = torch.zeros(4, 64, device="cuda")
    out = torch.empty_like(xn)
    q4, q1 = empty_mx4(4, K=64)
    assert code_of(cm.coli_moe_block_norm, xn) == cm.COLI_EINVAL                       # nothing to write
    assert code_of(cm.coli_moe_block_norm, xn, n_out=out, codes=q4) == cm.COLI_EINVAL   # codes without scales
    assert code_of(cm.coli_moe_block_norm, xn, gate=xn, n_out=out) == cm.COLI_EINVAL    # a gate for nothing
    assert code_of(cm.coli_moe_block_norm, xn, n_out=out, eps=-1.0) == cm.COLI_EINVAL
    assert code_of(cm.coli_moe_block_norm, torch.zeros(1, 16385, device="cuda"), n_out=torch.zeros(1, 16385, device="cuda")) == cm.COLI_EUNSUPPORTED
    assert code_of(cm.coli_moe_block_norm, xn, n_out=out.half()) == cm.COLI_EINVAL
    odd = torch.zeros(4, 40, device="cuda")
    assert code_of(cm.coli_moe_block_norm, odd, codes=torch.zeros(4, 20, dtype=torch.uint8, device="cuda"),
                   scales=torch.zeros(4, 1, dtype=torch.uint8, device="cuda")) == cm.COLI_EINVAL
    with pytest.raises(ValueError):
        cm.coli_moe_block_norm(xn, xn[:2], n_out=out)
    with pytest.raises(TypeError):
        cm.coli_moe_block_norm(xn, xn.half(), n_out=out)
    with pytest.raises(ValueError):
        cm.coli_moe_block_norm(xn.t(), n_out=out.t())
    cm.coli_moe_block_norm(xn[:0], n_out=out[:0])
