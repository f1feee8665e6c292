"""Groups of experts whose scores saturate or underflow in 32 bits: without a bias their logits still tell them
apart, as they do for the experts."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402

INF = np.inf


def group_order(l, softmax, top2):
    """Groups of l [G, per] best first, from the logits in 64 bits, in a form that neither saturates nor underflows.

    log of s1 + s2 up to what all groups share: log(e^l1 + e^l2) for softmax; for the sigmoid by the distance
    from 0, 1 or 2 (s = 1 - c with c the sigmoid of -l): s1 + s2 = 2 - c1 - c2 = 1 + s2 - c1."""
    best = -np.sort(-l, axis=1)
    l1, l2 = best[:, 0], best[:, 1] if l.shape[1] > 1 else np.full(len(l), -INF)
    if not top2:
        return sorted(range(len(l)), key=lambda g: (-l1[g], g))

    def logs(z):            # log of the sigmoid
        return np.minimum(z, 0) - np.log1p(np.exp(-np.abs(z)))

    def rank(g):
        a, b = l1[g], l2[g]
        if softmax:
            return (0, np.logaddexp(a, b))
        s = np.exp(logs(a)) + np.exp(logs(b))
        if s < 0.5:
            return (0, np.logaddexp(logs(a), logs(b)))
        if s < 1.5:
            return (1, np.exp(logs(b)) - np.exp(logs(-a)))
        return (2, -np.logaddexp(logs(-a), logs(-b)))
    # (equal in 64 bits with the same l1: the larger l2 is the larger sum)
    return sorted(range(len(l)), key=lambda g: (-rank(g)[0], -rank(g)[1], -l1[g], -l2[g], g))


def check(groups, keep, k, softmax, top2, dtype=torch.float32):
    """groups [T, G, per] logits."""
    l = np.asarray(groups, np.float64)
    T, G, per = l.shape
    x = torch.from_numpy(l.reshape(T, G * per)).to(dtype).cuda()
    l = x.double().cpu().numpy().reshape(T, G, per)
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    cm.coli_moe_select(x, idx, w, score=cm.SCORE_SOFTMAX if softmax else cm.SCORE_SIGMOID, n_groups=G, topk_group=keep,
                       group_score=cm.GROUP_TOP2 if top2 else cm.GROUP_MAX)
    for t in range(T):
        kept = group_order(l[t], softmax, top2)[:keep]
        cand = sorted(((-l[t, g, j], g * per + j) for g in kept for j in range(per) if l[t, g, j] > -INF))[:k]
        want = [e for _, e in cand] + [-1] * (k - len(cand))
        assert idx[t].tolist() == want, (t, kept, l[t].max(1), idx[t].tolist(), want)
    assert torch.isfinite(w).all()


def rows(G, per, bests, rest):
    """One position: group g's two best logits bests[g] at its end, all others `rest`."""
    l = np.full((1, G, per), float(rest))
    for g, b in enumerate(bests):
        l[0, g, per - len(b):] = b
    return l


# groups of fewer than 32 experts, of 32 with a group a register, and of 32 and 64 otherwise
SHAPES = [(2, 4), (4, 16), (2, 32), (4, 32), (3, 32), (2, 64)]


@pytest.mark.parametrize("top2", [False, True])
@pytest.mark.parametrize("G,per", SHAPES)
def test_sigmoids_that_saturate(G, per, top2):
    up = [(18.0 + 4 * g, 17.5 + 4 * g) for g in range(G)]              # the last group is the best
    check(rows(G, per, up, 0.0), 1, 2, False, top2)
    check(rows(G, per, [(a + 100, b + 100) for a, b in up], 90.0), 1, 2, False, top2)
    # the best logit alone does not decide a sum of two: the second is farther from 1
    check(rows(G, per, [(40.0, 18.0)] + [(22.0 + g, 21.0) for g in range(1, G)], 0.0), 1, 2, False, top2)
    # one saturated, the other negligible
    check(rows(G, per, [(30.0, -30.0 + g) for g in range(G)], -60.0), 1, 2, False, top2)


@pytest.mark.parametrize("top2", [False, True])
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("G,per", SHAPES)
def test_scores_that_underflow(G, per, softmax, top2):
    low = [(-200.0 + 3 * g, -203.0 + 2 * g) for g in range(G)]
    check(rows(G, per, low, -400.0), 1, 2, softmax, top2)
    # two equal ones, whose sum is the largest, against one that is a little larger than either
    check(rows(G, per, [(-200.0, -200.0)] + [(-198.5 - g, -300.0) for g in range(1, G)], -400.0), 1, 2, softmax, top2)
    if softmax and G > 2:   # one group far above the others, of which one more is kept
        check(rows(G, per, low[:-1] + [(10.0, 9.0)], -400.0), 2, per + 1 if per < 8 else 9, True, top2)


@pytest.mark.parametrize("top2", [False, True])
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wide_logits_and_ties(softmax, top2, dtype):
    rng = np.random.default_rng(7)
    # whole multiples of 8: scores of different groups are equal only with the same logits (then: the lower group), or
    # differ by a factor that no rounding hides
    for G, per in SHAPES:
        l = 8.0 * rng.integers(-8, 9, (50, G, per))
        if top2 and not softmax:
            l = np.where(l > 0, -l, l)      # (sums that are near 1 or 2: above)
        check(l, max(1, G // 2), 3, softmax, top2, dtype)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("G,per", SHAPES)
def test_masked_groups(G, per, softmax):
    for top2 in (False, True):
        l = rows(G, per, [(20.0 + 2 * g, -INF) for g in range(G)], -INF)          # one expert a group
        check(l, 1, 1, softmax, top2)
        l[0, G - 1] = -INF
        check(l, 1, 2, softmax, top2)
        check(np.full((1, G, per), -INF), 1, 2, softmax, top2)
