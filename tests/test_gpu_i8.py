"""Codes of activations and products of codes with a scale for each token and
channel, against plain 64-bit forms.

Codes without SwiGLU and integer sums have one right value, and every rounding of
a product's value is fixed (the sum to fp32, times the token's scale, times the
channel's, to the type of y): both are compared bit for bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402
from oracle import token8  # noqa: E402

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def rows_of(t, k, pitch, dtype, fill=None):
    """A [t, k] view of rows `pitch` apart, and the buffer."""
    buf = torch.zeros(t, pitch, dtype=dtype, device="cuda") if fill is None else torch.full((t, pitch), fill, dtype=dtype, device="cuda")
    return buf[:, :k], buf


# ------------------------------------------------------------------------ codes
@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("T,K,pad", [(1, 1, 0), (3, 7, 0), (5, 32, 8), (2, 1000, 0), (9, 1024, 3), (4, 1032, 8), (3, 6144, 0), (2, 8192, 5), (2, 8200, 0),
                                     (1, 20001, 0), (70, 96, 0)])
def test_codes(T, K, pad, name):
    gen = torch.Generator(device="cuda").manual_seed(T * K)
    x = (torch.randn(T, K + pad, generator=gen, device="cuda") * torch.exp(4 * torch.randn(T, 1, generator=gen, device="cuda"))).to(TYPES[name])
    x[0, 0] = x[0].abs().max()           # a largest value and half of it: the middle of 63 and 64
    if K > 1:
        x[0, 1] = -x[0, 0] / 2
    x = x[:, :K]
    codes, buf = rows_of(T, K, K + 3 * (pad > 0), torch.int8, 77)
    scales = torch.empty(T, device="cuda")
    cm.coli_i8_quantize(x, codes, scales)
    q, s = token8.quantize(x.double().cpu().numpy())
    top = x.float().abs().amax(-1).cpu()
    assert np.array_equal(codes.cpu().numpy(), q)
    assert np.array_equal(scales.cpu().numpy(), top.numpy() / np.float32(127.0))
    assert (buf[:, K:] == 77).all()
    out, obuf = rows_of(T, K, K + pad, TYPES[name], 5.0)
    cm.coli_i8_dequantize(codes, scales, out)
    assert torch.equal(out, (codes.float() * scales[:, None]).to(TYPES[name])) and (obuf[:, K:] == 5.0).all()


def test_codes_next_to_the_middle():
    # every neighbourhood of a middle between two codes, for several maxima that are no powers of two
    for top in (1.0, 3.1415927, 0.73, 1e-20, 2.3e30):
        mid = (np.arange(-127, 127) + 0.5) * np.float64(np.float32(top)) / 127.0
        near = mid.astype(np.float32)
        x = np.concatenate([np.nextafter(near, np.float32(-np.inf)), near, np.nextafter(near, np.float32(np.inf)), [np.float32(top)]])[None].astype(np.float32)
        codes, scales = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
        cm.coli_i8_quantize(torch.from_numpy(x).cuda(), codes, scales)
        assert np.array_equal(codes.cpu().numpy(), token8.quantize(x)[0])


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("T,K,pad", [(1, 1, 0), (3, 7, 1), (5, 32, 8), (2, 1000, 0), (3, 2048, 0), (2, 2052, 0), (2, 9000, 0)])
def test_swiglu_codes(T, K, pad, name):
    gen = torch.Generator(device="cuda").manual_seed(T * K + 1)
    x = (torch.randn(T, 2 * K + pad, generator=gen, device="cuda") * 4).to(TYPES[name])[:, :2 * K]
    if K > 2:
        x[0, :3] = torch.tensor([-60.0, 60.0, 0.0])
    codes, scales = torch.empty(T, K, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    cm.coli_i8_quantize(x, codes, scales, swiglu=True)
    h = token8.swiglu(x.double().cpu().numpy())
    s = scales.double().cpu().numpy()
    # fp32 silu * u: exp 1 ulp (2^-23), sum, fast division 2 ulp (2^-22), three products: below 2^-21 of the value
    rel = 2.0 ** -21
    top = np.abs(h).max(-1)
    assert (np.abs(s - top / 127) <= top / 127 * (rel + 2.0 ** -23)).all()
    assert (np.abs(codes.double().cpu().numpy() * s[:, None] - h) <= s[:, None] * (0.5 + 127 * (rel + 2.0 ** -22)) + 1e-37).all()


@pytest.mark.parametrize("K", [16, 1500, 9001])
def test_rows_without_values(K):
    x = torch.randn(6, K, device="cuda")
    x[0, K // 2], x[1, 0], x[2, K - 1] = float("nan"), float("inf"), float("-inf")
    x[3] = 0.0
    x[4] = 1e-42                                        # below 2^-100
    codes, scales = torch.full((6, K), 9, dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
    cm.coli_i8_quantize(x, codes, scales)
    assert torch.isnan(scales[:3]).all() and (scales[3:5] == 0).all() and scales[5] > 0
    assert (codes[:5] == 0).all() and (codes[5].abs().max() == 127)


def test_no_rows():
    codes, scales = torch.empty(0, 8, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda")
    cm.coli_i8_quantize(torch.empty(0, 8, device="cuda"), codes, scales)
    cm.coli_i8_dequantize(codes, scales, torch.empty(0, 8, device="cuda"))
    cm.coli_i8_product(codes, scales, torch.zeros(4, 16, dtype=torch.int8, device="cuda")[:, :8], torch.ones(4, device="cuda"),
                       torch.empty(0, 4, device="cuda"), cm.new_i8_product_workspace(0, 8))
    torch.cuda.synchronize()


# ------------------------------------------------------------------------ products
def make(X, G, N, K, seed, extreme=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pitch = (K + 15) // 16 * 16
    x = torch.randint(-127, 128, (X, pitch), generator=gen, device="cuda").to(torch.int8)[:, :K]
    w = torch.randint(-128, 128, (G, N, pitch), generator=gen, device="cuda").to(torch.int8)[:, :, :K]
    if extreme:  # the largest sums
        x.fill_(-128)
        w.fill_(-128)
        w[:, ::2] = 127
    xs = torch.rand(X, generator=gen, device="cuda") * 0.01 + 1e-4
    ws = torch.rand(G, N, generator=gen, device="cuda") * 0.01 + 1e-4
    return x, xs, w, ws


def want(x, xs, w, ws, offsets, rows, dtype):
    """Every row's right bits, NaN for rows without activations, and which rows belong to a group."""
    P = len(rows)
    S = torch.zeros(P, w.shape[1], dtype=torch.float64, device="cuda")
    sx, sw, live = torch.zeros(P, device="cuda"), torch.zeros(P, w.shape[1], device="cuda"), torch.zeros(P, dtype=torch.bool, device="cuda")
    top = 0
    for g in range(w.shape[0]):
        a = top = max(top, min(max(int(offsets[g]), 0), P))
        b = max(a, min(max(int(offsets[g + 1]), 0), P))
        if b > a:
            r = rows[a:b].long()
            ok = (r >= 0) & (r < len(x))
            S[a:b] = x[r.clamp(0, len(x) - 1)].double() @ w[g].double().T   # whole numbers below 2^31: exact in 64 bits
            sx[a:b] = torch.where(ok, xs[r.clamp(0, len(x) - 1)], float("nan"))
            sw[a:b] = ws[g]
            live[a:b] = True
    return (S.float() * sx[:, None] * sw).to(dtype), live


def check(P, G, N, K, name, seed=0, X=None, gather=False, offsets=None, extreme=False, ldy=0):
    X = X or P
    x, xs, w, ws = make(X, G, N, K, seed, extreme)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    rows = torch.randint(0, X, (P,), generator=gen, device="cuda").to(torch.int32) if gather else torch.arange(P, device="cuda", dtype=torch.int32)
    y, buf = rows_of(P, N, max(N, ldy), TYPES[name], 3.0)
    space = cm.new_i8_product_workspace(P, K)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    cm.coli_i8_product(x, xs, w, ws, y, space, offsets=off, rows=rows if gather else None)
    ref, live = want(x, xs, w, ws, [0, P] if offsets is None else offsets, rows, TYPES[name])
    assert cm.coli_moe_status(space) == 0
    assert torch.equal(y[live], ref[live]), (y[live].float() - ref[live].float()).abs().max()
    assert (y[~live] == 3.0).all() and (buf[:, N:] == 3.0).all()
    return y


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("P,N,K", [(1, 1, 1), (1, 48, 40), (2, 300, 1000), (3, 17, 129), (4, 64, 6144), (5, 128, 64), (8, 1000, 6400), (1, 6144, 2048), (7, 33, 20000)])
def test_few_rows(P, N, K, name):
    check(P, 1, N, K, name, seed=P + N)


@pytest.mark.parametrize("name", list(TYPES))
@pytest.mark.parametrize("P,N,K", [(9, 1, 1), (9, 128, 64), (16, 130, 65), (17, 48, 128), (32, 300, 1000), (33, 128, 1024), (64, 129, 1040), (65, 1000, 544),
                                   (100, 256, 2048), (128, 128, 3001), (191, 200, 4096)])
def test_many_rows(P, N, K, name):
    check(P, 1, N, K, name, seed=P + N)


@pytest.mark.parametrize("P,N,K", [(192, 128, 64), (256, 130, 1024), (257, 128, 1025), (300, 300, 512), (384, 128, 513), (385, 256, 1537), (1000, 1100, 2500), (700, 64, 8200)])
def test_rows_of_wide_tiles(P, N, K):
    check(P, 1, N, K, "bf16", seed=P + N)
    check(P, 1, N, K, "f32", seed=P + N, ldy=N + 5)


@pytest.mark.parametrize("P,N,K", [(9, 130, 700), (40, 300, 5000), (100, 1000, 3001), (1000, 4000, 6100), (300, 256, 20000)])
def test_one_run_over_all_of_K(P, N, K):
    # activations whose magnitudes add up to less than 2^24 / 255: other runs than those of the largest sums
    x, xs, w, ws = make(P, 1, N, K, P)
    x.copy_((torch.randn(x.shape, device="cuda") * (60000.0 / K)).clamp(-127, 127).round().to(torch.int8))
    x[0] = 0
    x[1 % P, :min(K, 517)] = 127                     # just below, and (two more rows) just above
    for grow in (0, 3):
        if grow:
            x[2 % P, :min(K, 517 + grow)] = 127
        y, space = torch.empty(P, N, device="cuda"), cm.new_i8_product_workspace(P, K)
        cm.coli_i8_product(x, xs, w, ws, y, space)
        ref, _ = want(x, xs, w, ws, [0, P], torch.arange(P, device="cuda"), torch.float32)
        assert torch.equal(y, ref) and cm.coli_moe_status(space) == 0


@pytest.mark.parametrize("P", [3, 40, 300])
@pytest.mark.parametrize("K", [1023, 16384, 131071])
def test_largest_sums(P, K):
    check(P, 1, 40, K, "f32", extreme=True)


GROUPS = [
    (6, [0, 1, 1, 4, 6]),                       # an empty group
    (8, [0, 8, 8, 8]),
    (8, [2, 3, 3, 5]),                          # rows of no group at both ends
    (5, [0, 5, 3, 9]),                          # not ascending, beyond P
    (7, [-4, 2, 99]),
    (12, [0, 1, 12, 12, 12]),
    (100, [0, 0, 33, 34, 100]),
    (100, [10, 60, 20, 90]),
    (130, [0, 129, 130]),
    (600, [0, 5, 5, 300, 590]),                 # tiles of 256 rows
    (600, [0, 0, 0, 0]),                        # no rows at all
]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("P,offsets", GROUPS)
def test_groups(P, offsets, gather):
    check(P, len(offsets) - 1, 200, 300, "bf16", seed=P, X=P if not gather else max(1, P // 3), gather=gather, offsets=offsets)


def test_many_groups():
    rng = np.random.default_rng(5)
    for G, P in ((1024, 2000), (300, 8), (257, 31), (40, 9000)):
        off = [0] + sorted(rng.integers(0, P + 1, G - 1).tolist()) + [P]
        check(P, G, 130, 200, "f32", seed=G, X=50, gather=True, offsets=off)


@pytest.mark.parametrize("P", [4, 50, 400])
def test_rows_out_of_range(P):
    x, xs, w, ws = make(20, 2, 70, 96, 3)
    rows = torch.randint(0, 20, (P,), device="cuda").to(torch.int32)
    rows[1], rows[P - 2], rows[P - 1] = -1, 20, 2 ** 31 - 1
    off = torch.tensor([0, P // 2, P - 1], dtype=torch.int32, device="cuda")     # the last row is of no group
    y, space = torch.full((P, 70), 3.0, device="cuda"), cm.new_i8_product_workspace(P, 96)
    cm.coli_i8_product(x, xs, w, ws, y, space, offsets=off, rows=rows)
    ref, live = want(x, xs, w, ws, off.tolist(), rows, torch.float32)
    assert cm.coli_moe_status(space) == cm.STATUS_BADIDX
    assert torch.equal(torch.nan_to_num(y[:-1], nan=-7.0), torch.nan_to_num(ref[:-1], nan=-7.0)) and torch.isnan(y[1]).all() and (y[-1] == 3.0).all()
    # rows behind the last group are not looked at
    off = torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda")
    rows[0] = 3
    cm.coli_i8_product(x, xs, w, ws, y, space, offsets=off, rows=rows)
    assert cm.coli_moe_status(space) == 0


def test_expert_records_as_weights():
    # the matrices of int8 records [gate, up, down] and their scales, in place
    E, H, I, P = 5, 256, 128, 40
    rec = torch.randint(-127, 128, (E, 3 * I * H), device="cuda").to(torch.int8)
    sc = torch.rand(E, 2 * I + H, device="cuda") + 0.1
    off = torch.tensor([0, 3, 3, 20, 39, 40], dtype=torch.int32, device="cuda")
    for rows_, K, w, s in ((2 * I, H, rec[:, :2 * I * H].view(E, 2 * I, H), sc[:, :2 * I]), (H, I, rec[:, 2 * I * H:].view(E, H, I), sc[:, 2 * I:])):
        for n in (P, 6):
            x, xs, _, _ = make(n, 1, 1, K, 9)
            y, space = torch.empty(n, rows_, device="cuda"), cm.new_i8_product_workspace(n, K)
            cm.coli_i8_product(x, xs, w, s, y, space, offsets=off.clamp(max=n))
            ref, live = want(x, xs, w, s, off.clamp(max=n).tolist(), torch.arange(n, device="cuda"), torch.float32)
            assert live.all() and torch.equal(y, ref)


@pytest.mark.parametrize("P", [6, 40, 700])
def test_weights_at_any_stride(P):
    # one matrix for all groups (stride 0), and matrices whose rows stand between one another
    G, N, K = 5, 140, 200
    x, xs, w, ws = make(P, G, N, K, 21)
    cuts = [0, P // 8, P // 8, P // 2, P - 1, P]
    off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    mixed = torch.zeros(N, G, 208, dtype=torch.int8, device="cuda").permute(1, 0, 2)[:, :, :K]
    mixed.copy_(w)
    for weights, scales in ((w[:1].expand(G, N, K), ws), (w[:1].expand(G, N, K), ws[:1].expand(G, N)), (mixed, ws)):
        y, space = torch.empty(P, N, device="cuda"), cm.new_i8_product_workspace(P, K)
        cm.coli_i8_product(x, xs, weights, scales, y, space, offsets=off)
        ref, live = want(x, xs, weights, scales, cuts, torch.arange(P, device="cuda"), torch.float32)
        assert live.all() and torch.equal(y, ref)


def test_scales_without_value():
    for P in (4, 64):
        x, xs, w, ws = make(P, 1, 130, 200, 1)
        xs[1] = float("nan")
        xs[2] = 0.0
        y, space = torch.empty(P, 130, device="cuda"), cm.new_i8_product_workspace(P, 200)
        cm.coli_i8_product(x, xs, w[0], ws[0], y, space)
        assert torch.isnan(y[1]).all() and (y[2] == 0).all() and torch.isfinite(y[3:]).all()


def test_same_bits_in_every_call_size():
    # a row's result does not depend on the rows beside it
    x, xs, w, ws = make(700, 1, 150, 2100, 4)
    space = cm.new_i8_product_workspace(700, 2100)
    y = torch.empty(700, 150, device="cuda")
    cm.coli_i8_product(x, xs, w, ws, y, space)
    for n in (1, 2, 4, 8, 9, 33, 64, 128, 192, 300):
        z = torch.empty(n, 150, device="cuda")
        cm.coli_i8_product(x[:n], xs[:n].clone(), w, ws, z, space)
        assert torch.equal(z, y[:n])


@pytest.mark.parametrize("P", [2, 60, 500])
def test_graph_replays(P):
    x, xs, w, ws = make(P, 3, 256, 700, 8)
    off = torch.tensor([0, P // 2, P // 2, P], dtype=torch.int32, device="cuda")
    y, space = torch.empty(P, 256, dtype=torch.bfloat16, device="cuda"), cm.new_i8_product_workspace(P, 700)
    cm.coli_i8_product(x, xs, w, ws, y, space, offsets=off)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="thread_local"):
        cm.coli_i8_product(x, xs, w, ws, y, space, offsets=off)
    for seed in (1, 2):
        x.copy_(make(P, 1, 1, 700, seed)[0])
        off.copy_(torch.tensor([0, P // 3, P - 1, P], dtype=torch.int32))
        g.replay()
        ref, _ = want(x, xs, w, ws, off.tolist(), torch.arange(P, device="cuda"), torch.bfloat16)
        assert torch.equal(y, ref)


def test_two_streams_at_once():
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    jobs = []
    for i, (st, P) in enumerate(((a, 300), (b, 40), (a, 5), (b, 260))):
        x, xs, w, ws = make(P, 1, 500, 1200, i)
        jobs.append((st, x, xs, w, ws, torch.empty(P, 500, device="cuda"), cm.new_i8_product_workspace(P, 1200)))
    torch.cuda.synchronize()
    for _ in range(3):
        for st, x, xs, w, ws, y, space in jobs:
            cm.coli_i8_product(x, xs, w, ws, y, space, stream=st)
    torch.cuda.synchronize()
    for st, x, xs, w, ws, y, space in jobs:
        assert torch.equal(y, want(x, xs, w, ws, [0, len(x)], torch.arange(len(x), device="cuda"), torch.float32)[0]) and cm.coli_moe_status(space) == 0


@pytest.mark.parametrize("P,G,N,K", [(7152, 23, 700, 5573), (1500, 9, 384, 2048), (500, 5, 300, 1000), (60, 5, 256, 1500)])
def test_many_calls_one_behind_the_other(P, G, N, K):
    # the pipeline of one call starts while the call before ends, and its copies land in any order
    gen = torch.Generator(device="cuda").manual_seed(P)
    x, xs, w, ws = make(P, G, N, K, P)
    x.copy_((x.float() * 0.1).round().to(torch.int8))      # sums small enough for one run over all of K
    off = [0] + sorted(torch.randint(0, P + 1, (G - 1,), generator=gen, device="cuda").tolist()) + [P]
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    space = cm.new_i8_product_workspace(P, K)
    ref, _ = want(x, xs, w, ws, off, torch.arange(P, device="cuda"), torch.bfloat16)
    ys = [torch.zeros(P, N, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    for _ in range(100):
        for y in ys:
            cm.coli_i8_product(x, xs, w, ws, y, space, offsets=offsets)
    for y in ys:
        assert torch.equal(y, ref)
    assert cm.coli_moe_status(space) == 0


def test_weights_beyond_32_bit_offsets():
    G, N, K = 180, 4096, 6144                      # 4.5 GB of codes
    for P in (6, 400):
        gen = torch.Generator(device="cuda").manual_seed(P)
        w = torch.zeros(G, N, K, dtype=torch.int8, device="cuda")
        for g in (0, 88, G - 1):
            w[g] = torch.randint(-128, 128, (N, K), generator=gen, device="cuda").to(torch.int8)
        ws = torch.rand(G, N, generator=gen, device="cuda")
        x, xs, _, _ = make(P, 1, 1, K, P)
        cuts = torch.full((G + 1,), P // 2, dtype=torch.int32, device="cuda")
        cuts[0], cuts[1:89], cuts[G] = 0, P // 3, P
        y, space = torch.empty(P, N, device="cuda"), cm.new_i8_product_workspace(P, K)
        cm.coli_i8_product(x, xs, w, ws, y, space, offsets=cuts)
        for g, a, b in ((0, 0, P // 3), (88, P // 3, P // 2), (G - 1, P // 2, P)):
            ref, _ = want(x[a:b], xs[a:b], w[g:g + 1], ws[g:g + 1], [0, b - a], torch.arange(b - a, device="cuda"), torch.float32)
            assert torch.equal(y[a:b], ref)
        del w


def test_rows_beyond_32_bit_offsets():
    # codes, their activations and the results of products, each beyond 2^31 bytes or values
    T, K = 40000, 60000
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    some = torch.tensor([0, 17895, 35791, 35792, T - 1], device="cuda")
    x[some] = torch.randn(5, K, device="cuda").bfloat16()
    codes, scales = torch.empty(T, K, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    cm.coli_i8_quantize(x, codes, scales)
    q, _ = token8.quantize(x[some].double().cpu().numpy())
    assert np.array_equal(codes[some].cpu().numpy(), q) and int((scales != 0).sum()) == 5
    cm.coli_i8_dequantize(codes, scales, x)
    assert torch.equal(x[some], (codes[some].float() * scales[some][:, None]).bfloat16())
    del x
    w, ws = torch.randint(-128, 128, (64, K), device="cuda").to(torch.int8), torch.rand(64, device="cuda")
    y, space = torch.empty(T, 64, device="cuda"), cm.new_i8_product_workspace(T, K)
    cm.coli_i8_product(codes, scales, w, ws, y, space)
    ref, _ = want(codes[some], scales[some], w[None], ws[None], [0, 5], torch.arange(5, device="cuda"), torch.float32)
    assert cm.coli_moe_status(space) == 0 and torch.equal(y[some], ref)
    del space, codes
    x, xs, w, ws = make(T, 1, K, 64, 3)
    y, space = torch.empty(T, K, dtype=torch.bfloat16, device="cuda"), cm.new_i8_product_workspace(T, 64)
    cm.coli_i8_product(x, xs, w[0], ws[0], y, space)
    ref, _ = want(x[some], xs[some], w, ws, [0, 5], torch.arange(5, device="cuda"), torch.bfloat16)
    assert torch.equal(y[some], ref)


# calls whose tiles two CTAs take together: more rows than 64 and enough tiles
PAIRS = [(333, 1, 6100, 6144), (5000, 1, 2100, 3001), (2000, 40, 2100, 3001), (700, 3, 2500, 6144), (9000, 150, 4200, 1500)]


@pytest.mark.parametrize("P,G,N,K", PAIRS)
def test_tiles_of_two_ctas(P, G, N, K):
    gen = torch.Generator(device="cuda").manual_seed(P + G)
    cuts = None if G == 1 else [0] + sorted(torch.randint(0, P + 1, (G - 1,), generator=gen, device="cuda").tolist()) + [P]
    check(P, G, N, K, "bf16", seed=P + N, offsets=cuts, gather=G > 1, X=P // 2 + 7 if G > 1 else None)   # runs of 512 codes
    check(P, G, N, K, "f32", seed=P + N, offsets=cuts, extreme=True, ldy=N + 3)


@pytest.mark.parametrize("P,G,N,K", PAIRS)
def test_tiles_of_two_ctas_in_many_calls(P, G, N, K):
    x, xs, w, ws = make(P, G, N, K, P)
    x.copy_((x.float() * 0.1).round().to(torch.int8))      # one run over all of K
    gen = torch.Generator(device="cuda").manual_seed(P)
    off = [0] + sorted(torch.randint(0, P + 1, (G - 1,), generator=gen, device="cuda").tolist()) + [P]
    offsets, space = torch.tensor(off, dtype=torch.int32, device="cuda"), cm.new_i8_product_workspace(P, K)
    ref, _ = want(x, xs, w, ws, off, torch.arange(P, device="cuda"), torch.float16)
    y, few = torch.zeros(P, N, dtype=torch.float16, device="cuda"), torch.zeros(40, N, dtype=torch.float16, device="cuda")
    for _ in range(60):
        cm.coli_i8_product(x, xs, w, ws, y, space, offsets=offsets)
        cm.coli_i8_product(x, xs, w[0], ws[0], few, space, rows=torch.arange(40, dtype=torch.int32, device="cuda"))   # another kernel between
    assert cm.coli_moe_status(space) == 0 and torch.equal(y, ref)


@pytest.mark.parametrize("P,G,N,K", [(333, 1, 6100, 6144), (2000, 40, 2100, 3001)])
def test_tiles_of_two_ctas_on_two_streams_and_in_a_graph(P, G, N, K):
    x, xs, w, ws = make(P, G, N, K, P)
    off = torch.linspace(0, P, G + 1, device="cuda").to(torch.int32)
    ref, _ = want(x, xs, w, ws, off.tolist(), torch.arange(P, device="cuda"), torch.float32)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [cm.new_i8_product_workspace(P, K) for _ in range(2)]
    ys = [torch.zeros(P, N, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for st, space, y in zip(streams, spaces, ys):
            with torch.cuda.stream(st):
                cm.coli_i8_product(x, xs, w, ws, y, space, offsets=off)
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref) for y in ys)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cm.coli_i8_product(x, xs, w, ws, ys[0], spaces[0], offsets=off)
    ys[0].zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ref) and all(cm.coli_moe_status(space) == 0 for space in spaces)
