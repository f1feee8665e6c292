"""Selection of experts, grouping of the pairs and the weighted sum, against
plain 64-bit forms."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402
from oracle import token8  # noqa: E402

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------ selection
def spread(rng, T, E):
    """Logits whose scores lie apart, so that a selection has one answer in 32 and in 64 bits: a grid of distinct
    values, the gaps of whose sigmoids and softmaxes are far above fp32's error, in random order."""
    base = np.linspace(-3.0, 3.0, E)
    return np.stack([rng.permutation(base) for _ in range(T)])


def run_select(l, k, dtype=torch.float32, pad=0, **kw):
    T, E = l.shape
    x = torch.full((T, E + pad), 9e9 if dtype != torch.float16 else 6e4, dtype=dtype, device="cuda")
    x[:, :E] = torch.from_numpy(l).to(dtype)
    idx, w = torch.full((T, k), 7, dtype=torch.int32, device="cuda"), torch.full((T, k), 7.0, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = dict(kw)
    if args.get("bias") is not None:
        args["bias"] = torch.from_numpy(np.asarray(args["bias"], np.float32)).cuda()
    cm.coli_moe_select(x[:, :E], idx, w, ws=ws, **args)
    b = None if kw.get("bias") is None else np.asarray(kw["bias"], np.float32)
    ids, wt, bad = token8.select(x[:, :E].double().cpu().numpy(), k, bias=b, softmax=kw.get("score", cm.SCORE_SOFTMAX) == cm.SCORE_SOFTMAX,
                                 groups=kw.get("n_groups", 1), keep=kw.get("topk_group", 1), top2=kw.get("group_score", 0) == cm.GROUP_TOP2,
                                 renorm=kw.get("renorm", True), scaling=kw.get("scaling", 1.0))
    assert np.array_equal(idx.cpu().numpy(), ids)
    # exp of a rounded difference (|l - m| 2^-24), 1 ulp exp, fast division 2 ulp, a sum of E <= 1024 in 5 + 32 steps, the quotient of two such, the scaling
    span = np.ptp(np.where(np.isfinite(l), l, 0.0)) + 1
    assert np.abs(w.cpu().numpy() - wt).max() <= 2 * (span + 50) * 2.0 ** -24 * np.abs(wt).max(initial=1e-30)
    assert cm.coli_moe_status(ws) == (cm.STATUS_NONFINITE if bad.any() else 0)
    return idx, w


SHAPES = [(1, 1, 1, 1, 1), (1, 8, 1, 1, 8), (3, 16, 4, 2, 4), (7, 60, 1, 1, 4), (5, 64, 8, 3, 6), (4, 160, 8, 3, 6), (33, 256, 8, 4, 8), (2, 256, 1, 1, 8),
          (3, 384, 12, 5, 12), (9, 512, 16, 4, 32), (2, 1024, 32, 7, 32), (2, 1000, 10, 3, 20), (1, 96, 3, 2, 32), (700, 128, 4, 4, 2), (3, 32, 32, 9, 9)]


@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("T,E,G,keep,k", SHAPES)
def test_select(T, E, G, keep, k, softmax):
    rng = np.random.default_rng(E + T)
    l = spread(rng, T, E)
    for renorm, top2, scaling in ((True, True, 1.0), (False, False, 2.5)):
        run_select(l, k, n_groups=G, topk_group=keep, score=cm.SCORE_SOFTMAX if softmax else cm.SCORE_SIGMOID, renorm=renorm,
                   group_score=cm.GROUP_TOP2 if top2 else cm.GROUP_MAX, scaling=scaling)


@pytest.mark.parametrize("T,E,G,keep,k", SHAPES)
def test_select_with_a_bias(T, E, G, keep, k):
    rng = np.random.default_rng(E)
    # biased scores on a grid of 2^-10: sigmoids of logits 0, biases distinct multiples
    l = np.zeros((T, E))
    bias = rng.permutation(E) * 2.0 ** -10
    run_select(l, k, n_groups=G, topk_group=keep, score=cm.SCORE_SIGMOID, bias=bias)
    run_select(l, k, n_groups=G, topk_group=keep, score=cm.SCORE_SIGMOID, bias=bias - 3.0, group_score=cm.GROUP_MAX)
    # logits that differ, biases far apart: the bias decides, the weights are the scores'
    run_select(spread(rng, T, E), k, n_groups=G, topk_group=keep, score=cm.SCORE_SOFTMAX, bias=rng.permutation(E) * 4.0, renorm=False)


@pytest.mark.parametrize("name", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_types_strides_and_ties(name, pad):
    rng = np.random.default_rng(pad)
    l = rng.integers(-3, 4, (40, 128)).astype(np.float64)      # many equal logits: the lower id
    run_select(l, 8, dtype=TYPES[name], pad=pad)
    run_select(l, 8, dtype=TYPES[name], pad=pad, score=cm.SCORE_SIGMOID, n_groups=4, topk_group=4)
    run_select(np.zeros((2, 128)), 8, dtype=TYPES[name], pad=pad, n_groups=4, topk_group=2, group_score=cm.GROUP_MAX)
    z = np.zeros((1, 64))
    z[0, 1::2] = -0.0                                            # equal to 0
    run_select(z, 4, dtype=TYPES[name], pad=pad)


def test_scores_that_underflow_still_rank():
    l = np.array([[-200.0, -150.0, -300.0, -120.0], [100.0, 101.0, 99.0, 102.0]])
    idx, w = run_select(l, 3, score=cm.SCORE_SIGMOID, renorm=False)
    assert idx.tolist() == [[3, 1, 0], [3, 1, 0]]
    run_select(l, 3)
    idx, w = run_select(np.full((1, 8), -1000.0), 2, score=cm.SCORE_SIGMOID)
    assert idx.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]     # a sum of 0 stays 0


def test_masked_and_non_finite():
    inf, nan = np.inf, np.nan
    rng = np.random.default_rng(1)
    l = spread(rng, 9, 32)
    l[1, 3:] = -inf                      # three experts take part
    l[2, :] = -inf                       # none
    l[3, 5] = nan
    l[4, 6] = inf
    l[5, 8:16] = -inf                    # a whole group
    l[6, 1:] = -inf
    for kw in (dict(), dict(score=cm.SCORE_SIGMOID), dict(n_groups=4, topk_group=2), dict(n_groups=4, topk_group=2, score=cm.SCORE_SIGMOID, group_score=cm.GROUP_MAX),
               dict(n_groups=4, topk_group=4)):
        idx, w = run_select(l, 4, **kw)
        assert (idx[2] == -1).all() and (w[2] == 0).all() and (idx[3:5] == -1).all()
    bias = np.zeros(32)
    bias[::2] = -inf                     # excluded everywhere
    idx, _ = run_select(l, 4, bias=bias, score=cm.SCORE_SIGMOID)
    assert (idx[0] % 2 == 1).all()
    bias[1] = nan
    idx, _ = run_select(l, 4, bias=bias, score=cm.SCORE_SIGMOID)
    assert (idx == -1).all()


@pytest.mark.parametrize("T", [1, 2, 8, 9, 70])
@pytest.mark.parametrize("E,H", [(32, 16), (60, 272), (256, 6144), (8, 128)])
def test_select_from_the_hidden_state(T, E, H):
    # hidden states and weights of small whole numbers: logits are exact in fp32 in any order
    rng = np.random.default_rng(T + E)
    x, wr = rng.integers(-3, 4, (T, H)), rng.integers(-2, 3, (E, H))
    l = x.astype(np.float64) @ wr.T.astype(np.float64)
    xd, wd = torch.from_numpy(x).float().cuda(), torch.from_numpy(wr).float().cuda()
    idx, w = torch.empty(T, 4, dtype=torch.int32, device="cuda"), torch.empty(T, 4, device="cuda")
    ws = cm.new_select_workspace(T, H, E)
    for _ in range(2):
        cm.coli_moe_select(xd, idx, w, router_w=wd, ws=ws, renorm=True, scaling=2.0)
        ids, wt, _ = token8.select(l, 4, scaling=2.0)
        assert np.array_equal(idx.cpu().numpy(), ids) and cm.coli_moe_status(ws) == 0
        assert np.abs(w.cpu().numpy() - wt).max() <= 2 * (np.ptp(l) + 50) * 2.0 ** -24 * 2.0
    # the library's own router is the case of sigmoid scores, a bias and the sum of two per group
    if E % 4 == 0 and H % 128 == 0:
        cfg = cm.Cfg(hidden=H, n_experts=E, n_groups=4, topk_group=2, top_k=4, inter=128, n_shared=0, shared_inter=0, weight_bits=8, routed_scaling_factor=2.5)
        bias = torch.arange(E, device="cuda").float() * 0.25
        xd = xd * 0.01
        i2, w2 = torch.empty_like(idx), torch.empty_like(w)
        cm.coli_moe_route(cfg, xd, wd, bias, i2, w2, cm.new_workspace(cfg, T))
        cm.coli_moe_select(xd, idx, w, router_w=wd, bias=bias, ws=ws, score=cm.SCORE_SIGMOID, n_groups=4, topk_group=2, scaling=2.5)
        assert torch.equal(idx, i2) and (w - w2).abs().max() < 2e-5


def test_hidden_state_without_value():
    # no logit of a hidden state masks an expert, not even -inf everywhere
    x, wr = torch.randn(12, 64, device="cuda"), -torch.rand(20, 64, device="cuda") - 0.1
    x[1, 3], x[4, 0], x[5, 7] = float("inf"), float("nan"), float("-inf")
    for T in (12, 6):
        idx, w, ws = torch.empty(T, 4, dtype=torch.int32, device="cuda"), torch.empty(T, 4, device="cuda"), cm.new_select_workspace(T, 64, 20)
        cm.coli_moe_select(x[:T].contiguous(), idx, w, router_w=wr, ws=ws)
        bad = torch.tensor([t in (1, 4, 5) for t in range(T)], device="cuda")
        assert cm.coli_moe_status(ws) == cm.STATUS_NONFINITE
        assert (idx[bad] == -1).all() and (w[bad] == 0).all() and (idx[~bad] >= 0).all() and torch.allclose(w[~bad].sum(-1), torch.ones((), device="cuda"))


def test_no_positions():
    e, f = torch.empty(0, 4, dtype=torch.int32, device="cuda"), torch.empty(0, 4, device="cuda")
    cm.coli_moe_select(torch.empty(0, 16, device="cuda"), e, f)
    off = torch.full((17,), 5, dtype=torch.int32, device="cuda")
    cm.coli_moe_group(e, off, torch.empty(0, dtype=torch.int32, device="cuda"), e, cm.new_group_workspace(0, 4, 16))
    assert (off == 0).all()
    cm.coli_moe_combine(torch.empty(0, 8, device="cuda"), e, f, torch.empty(0, 8, device="cuda"))


@pytest.mark.parametrize("T", [1, 3000])
def test_bias_of_the_kernel_before(T):
    # a bias that the step before on the stream updates
    E, k = 64, 4
    gen = torch.Generator(device="cuda").manual_seed(T)
    l = torch.linspace(-1.0, 1.0, E, device="cuda").expand(T, E).contiguous()
    biases = 4 * torch.stack([torch.randperm(E, generator=gen, device="cuda") for _ in range(40)]).float()  # (whole numbers: v lie apart)
    bias = torch.zeros(E, device="cuda")
    idx = torch.empty(40, T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(40, T, k, device="cuda")
    torch.cuda.synchronize()
    for i in range(40):
        bias.copy_(biases[i])
        cm.coli_moe_select(l, idx[i], w[i], bias=bias, score=cm.SCORE_SIGMOID)
    assert torch.equal(idx, biases.topk(k, -1).indices.int()[:, None].expand(40, T, k))


# ------------------------------------------------------------------------ grouping
def run_group(idx, E, rank=0, size=0):
    T, k = idx.shape
    P = max(size, 1)
    mine = len(range(rank, E, P))
    d = torch.from_numpy(idx.astype(np.int32)).cuda()
    off, rows, slots = (torch.full((n,), 77, dtype=torch.int32, device="cuda") for n in (mine + 1, T * k, T * k))
    ws = cm.new_group_workspace(T, k, E)
    cm.coli_moe_group(d, off, rows, slots.view(T, k), ws, n_experts=E, ep_rank=rank, ep_size=size)
    o, r, s = token8.group(idx, E, rank, P)
    assert np.array_equal(off.cpu().numpy(), o) and np.array_equal(slots.view(T, k).cpu().numpy(), s)
    assert np.array_equal(rows[:len(r)].cpu().numpy(), r) and (rows[len(r):] == 77).all()
    return cm.coli_moe_status(ws)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (5, 3, 7), (32, 8, 256), (256, 8, 256), (257, 8, 64), (300, 7, 1024), (2049, 1, 3), (4096, 4, 100), (700, 32, 128)])
def test_group(T, k, E):
    rng = np.random.default_rng(T)
    idx = rng.integers(-1, E, (T, k))
    assert run_group(idx, E) == 0
    if E >= 4:
        for rank in (0, 3):
            assert run_group(idx, E, rank, 4) == 0
    assert run_group(np.full((T, k), -1), E) == 0
    assert run_group(np.full((T, k), E - 1), E) == 0      # one expert, the same one in every slot


def test_group_bad_ids():
    idx = np.array([[0, 5], [-2, 1], [4, 2 ** 31 - 1], [3, -2 ** 31]])
    assert run_group(idx, 4) == cm.STATUS_BADIDX
    big = np.random.default_rng(0).integers(0, 9, (3000, 2))
    assert run_group(big, 8) == cm.STATUS_BADIDX


def test_group_of_many_pairs():
    T, k, E = 150000, 8, 384
    idx = torch.randint(-1, E, (T, k), device="cuda", dtype=torch.int32)
    off, rows, slots = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(T * k, dtype=torch.int32, device="cuda"), torch.empty_like(idx)
    cm.coli_moe_group(idx, off, rows, slots, cm.new_group_workspace(T, k, E))
    flat = idx.flatten().long()
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices
    n = int((flat >= 0).sum())
    assert torch.equal(rows[:n].long(), order[:n] // k) and int(off[-1]) == n
    place = torch.full_like(flat, -1)
    place[order[:n]] = torch.arange(n, device="cuda")
    assert torch.equal(slots.flatten().long(), place)
    assert torch.equal(off[1:].long(), torch.bincount(flat[flat >= 0], minlength=E).cumsum(0))


# ------------------------------------------------------------------------ weighted sum
@pytest.mark.parametrize("ot,yt", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("bf16", "f32"), ("f16", "bf16")])
@pytest.mark.parametrize("T,H,k,P,pad,add", [(1, 1, 1, 1, 0, False), (3, 7, 2, 5, 1, True), (5, 264, 8, 40, 8, True), (2, 1000, 3, 6, 0, False), (4, 6144, 8, 32, 0, True),
                                           (33, 129, 5, 100, 0, True), (2, 40, 40, 9, 0, True), (6, 24, 9, 0, 0, True)])
def test_combine(T, H, k, P, pad, add, ot, yt):
    gen = torch.Generator(device="cuda").manual_seed(T * H)
    o = torch.randn(P, H + pad, generator=gen, device="cuda").to(TYPES[ot])[:, :H]
    slots = torch.randint(-1, P + 2, (T, k), generator=gen, device="cuda").to(torch.int32)     # some skipped, some behind the end
    w = torch.randn(T, k, generator=gen, device="cuda")
    w[(slots < 0) | (slots >= P)] = float("nan")
    a = torch.randn(T, H + pad, generator=gen, device="cuda").to(TYPES[yt])[:, :H] if add else None
    ybuf = torch.full((T, H + pad), 3.0, dtype=TYPES[yt], device="cuda")
    y = ybuf[:, :H]
    cm.coli_moe_combine(o, slots, w, y, add=a)
    ref, mag = token8.combine(o.double().cpu().numpy(), slots.cpu().numpy(), w.double().cpu().numpy(), None if a is None else a.double().cpu().numpy())
    # k fused steps of half a unit of fp32 each, then one rounding to y's type
    tol = k * 2.0 ** -24 * mag * 1.01 + torch.finfo(TYPES[yt]).eps / 2 * np.abs(ref) * 1.01 + 2.0 ** -25 * (yt == "f16") + 1e-38
    assert (np.abs(y.double().cpu().numpy() - ref) <= tol).all() and (ybuf[:, H:] == 3.0).all()
    if add:  # into the added rows themselves
        cm.coli_moe_combine(o, slots, w, a, add=a)
        assert torch.equal(a, y)


def test_combine_rows_beyond_32_bit_offsets():
    H, P = 8192, 300000
    o = torch.zeros(P, H, dtype=torch.bfloat16, device="cuda")
    o[P - 1] = 2.0
    o[P // 2] = 1.0
    slots = torch.tensor([[P - 1, P // 2], [P // 2, -1]], dtype=torch.int32, device="cuda")
    y = torch.empty(2, H, device="cuda")
    cm.coli_moe_combine(o, slots, torch.tensor([[1.0, 0.5], [3.0, 1.0]], device="cuda"), y)
    assert (y[0] == 2.5).all() and (y[1] == 3.0).all()
