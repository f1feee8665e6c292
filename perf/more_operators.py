"""Timed cases of the operators around an expert layer with 8-bit codes that
have one scale for each token and one for each channel: the selection of
experts from scores, the grouping of the routed pairs by expert, the codes of
activations (with SwiGLU before them, where they are the experts' hidden
values), the products of codes grouped by expert, and the weighted sum that
brings the pairs back to their positions.

``run`` computes a case in one of two ways: with ``own`` false in plain form
(elementary torch operations in 32 bits, rounded once at the end), with ``own``
true through this repository's package.  ``exact`` computes the same values in
64 bits from the definitions.

The codes of a row are whole numbers in [-127, 127] with one 32-bit scale: the
row's largest magnitude over 127.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TINY = 2.0 ** -100  # rows of no larger values are zeros
_held = {}  # the package and the workspaces that a user's program keeps


# ------------------------------------------------------------------------ cases
def listed():
    return [
        # the router of one decoded token, from its hidden state: latency alone
        dict(name="select_token", op="select", rows=1, experts=256, hidden=6144, score="softmax", bias=False, groups=1, keep=1, group_score="top2",
             top_k=8, renorm=True, type="f32", pad=0, masked=0.0),
        # the logits of a batch of long prompts: sigmoid scores, a bias for balance, half of the groups kept
        dict(name="select_prompt", op="select", rows=16384, experts=256, hidden=0, score="sigmoid", bias=True, groups=8, keep=4,
             group_score="top2", top_k=8, renorm=True, type="f32", pad=0, masked=0.0),
        # the pairs of a batch of decoding streams
        dict(name="group_batch", op="group", rows=32, experts=256, top_k=8, skip=0.0),
        # the pairs of a batch of long prompts, some slots skipped
        dict(name="group_prompt", op="group", rows=16384, experts=256, top_k=8, skip=0.1),
        # the experts' outputs of a batch of decoding streams back to its positions
        dict(name="combine_batch", op="combine", rows=32, hidden=6144, top_k=8, skip=0.0, add=True, type="bf16"),
        # the same for a prompt
        dict(name="combine_prompt", op="combine", rows=2048, hidden=6144, top_k=8, skip=0.1, add=True, type="bf16"),
        # the activations of a long prompt before their products
        dict(name="quantize_prompt", op="quantize", rows=8192, cols=6144, swiglu=False, pad=0, type="bf16"),
        # the hidden values of a prompt's routed pairs before the down product
        dict(name="quantize_hidden", op="quantize", rows=16384, cols=2048, swiglu=True, pad=0, type="bf16"),
        # one decoded token through one projection: latency, 25 MB of weights
        dict(name="product_token", op="product", rows=1, experts=1, top_k=1, n=4096, k=6144, type="bf16"),
        # the gate and up products of a batch of decoding streams: streams nearly every expert for a row or two
        dict(name="product_batch", op="product", rows=32, experts=256, top_k=8, n=4096, k=6144, type="bf16"),
        # the same for a prompt, about 64 rows an expert
        dict(name="product_experts", op="product", rows=2048, experts=256, top_k=8, n=4096, k=6144, type="bf16"),
        # a dense projection of a long prompt: bound by arithmetic
        dict(name="product_prompt", op="product", rows=8192, experts=1, top_k=1, n=4096, k=6144, type="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "group", "combine", "quantize", "product", "product"])
    if op == "select":
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * rng.choice([8, 16, 20, 32])
        keep = rng.randint(1, groups)
        hidden = 128 * _log_int(rng, 1, 48) if rng.random() < 0.3 else 0
        return dict(op=op, rows=_log_int(rng, 1, 64 if hidden else 16384), experts=experts, hidden=hidden, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, keep=keep, group_score=rng.choice(["top2", "max"]),
                    top_k=rng.randint(1, min(8, keep * (experts // groups))), renorm=rng.random() < 0.7,
                    type="f32" if hidden else rng.choice(["f32", "f32", "bf16", "f16"]), pad=0 if hidden else rng.choice([0, 0, 3, 8]),
                    masked=0.0 if hidden else rng.choice([0.0, 0.0, 0.2]))
    if op == "group":
        experts = _log_int(rng, 16, 512)
        return dict(op=op, rows=_log_int(rng, 8, 16384), experts=experts, top_k=rng.randint(1, 8), skip=rng.choice([0.0, 0.0, 0.25]))
    if op == "combine":
        hidden, top_k = _log_int(rng, 33, 8192), rng.randint(1, 8)
        return dict(op=op, rows=min(_log_int(rng, 1, 8192), (1 << 26) // (hidden * top_k)), hidden=hidden, top_k=top_k,
                    skip=rng.choice([0.0, 0.25]), add=rng.random() < 0.5, type=rng.choice(["f32", "bf16", "f16"]))
    if op == "quantize":
        cols = _log_int(rng, 17, 8192)
        return dict(op=op, rows=min(_log_int(rng, 1, 16384), (1 << 25) // cols), cols=cols, swiglu=rng.random() < 0.4, pad=rng.choice([0, 0, 8, 5]),
                    type=rng.choice(["f32", "bf16", "f16"]))
    experts = rng.choice([1, 1, _log_int(rng, 2, 128)])
    n, k = _log_int(rng, 48, 6144), _log_int(rng, 40, 6144)
    experts = max(1, min(experts, (1 << 29) // (n * k)))
    top_k = rng.randint(1, min(8, experts))
    rows = max(1, min(_log_int(rng, 1, 8192), (1 << 37) // (n * k * top_k)))
    return dict(op=op, rows=rows, experts=experts, top_k=top_k, n=n, k=k, type=rng.choice(["f32", "bf16", "bf16", "f16"]))


def work(case):
    c, size = case, lambda name: torch.empty(0, dtype=DTYPES[name]).element_size()
    t = c["rows"]
    if c["op"] == "select":
        scores, out = t * c["experts"], 8 * t * c["top_k"]
        if c["hidden"]:
            return {"bytes": 4 * (t + c["experts"]) * c["hidden"] + out, "flops": 2 * scores * c["hidden"]}
        return {"bytes": scores * size(c["type"]) + out, "flops": 10 * scores}
    if c["op"] == "group":  # the ids in; the pairs' slots and rows and the experts' offsets out
        return {"bytes": 12 * t * c["top_k"] + 4 * c["experts"], "flops": 4 * t * c["top_k"]}
    if c["op"] == "combine":
        pairs = t * c["top_k"] * (1.0 - c["skip"])
        return {"bytes": (pairs + t * (1 + c["add"])) * c["hidden"] * size(c["type"]) + 8 * t * c["top_k"], "flops": 2 * pairs * c["hidden"]}
    if c["op"] == "quantize":  # values in, codes and scales out, codes and scales in, their values out
        n = t * c["cols"]
        return {"bytes": n * ((1 + c["swiglu"]) * size(c["type"]) + 2 + 2) + 8 * t, "flops": 4 * n + 6 * n * c["swiglu"]}
    pairs, e = t * c["top_k"], c["experts"]
    hit = e * (1.0 - (1.0 - c["top_k"] / e) ** t) if e > 1 else 1
    return {"bytes": hit * c["n"] * (c["k"] + 4) + t * (c["k"] + 4) + pairs * (c["n"] * size(c["type"]) + 4), "flops": 2 * pairs * c["n"] * c["k"]}


# ------------------------------------------------------------------------ inputs
def _group_scores(v, c):
    """Scores of the groups from scores v [T, E] of the experts, -inf for the excluded: the sum of a group's two best, or its best."""
    top = v.unflatten(-1, (c["groups"], -1)).sort(-1, descending=True).values[..., :2]
    if c["group_score"] == "max":
        return top[..., 0]
    return torch.where(top[..., 0] == -math.inf, -math.inf, torch.where(top == -math.inf, 0.0, top).sum(-1))


def _near(c, logits, bias):
    """Rows whose selection hangs on a difference that 32 bits may turn: a selection has one right answer in 32 and in 64 bits."""
    margin = 5e-5 if c["hidden"] else 2e-6
    l = logits.double()
    s = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, -1)
    s = torch.where(l == -math.inf, -math.inf, s if bias is None else s + bias.double())
    bad = torch.zeros(len(l), dtype=torch.bool, device=l.device)
    rank = s if bias is not None else l
    if c["keep"] < c["groups"]:
        g, order = _group_scores(s, c).sort(-1, descending=True)
        last, next_ = g[:, c["keep"] - 1], g[:, c["keep"]]
        bad |= last - next_ < margin * (next_.abs() if bias is None else 1.0)
        kept = (order[:, :c["keep"], None] == torch.arange(c["groups"], device="cuda")).any(1)
        rank = torch.where(kept.repeat_interleave(c["experts"] // c["groups"], -1), rank, -math.inf)
    if bias is not None or c["hidden"]:  # otherwise the logits themselves decide, and their ties go to the lower id
        v = rank.sort(-1, descending=True).values[:, :c["top_k"] + 1]
        bad |= (v[:, :-1] - v[:, 1:] < margin).any(-1)
    return bad


def _select_inputs(c, gen):
    t, e = c["rows"], c["experts"]
    s = {"bias": None, "x": None, "router_w": None}
    if c["bias"]:
        s["bias"] = (torch.rand(e, generator=gen, device="cuda") - 0.5) * 0.2
    if c["hidden"]:
        s["router_w"] = torch.randn(e, c["hidden"], generator=gen, device="cuda") * c["hidden"] ** -0.5
    favour = torch.randn(e, generator=gen, device="cuda") * 0.5

    def rows(n):
        if c["hidden"]:
            return torch.randn(n, c["hidden"], generator=gen, device="cuda")
        v = torch.randn(n, e + c["pad"], generator=gen, device="cuda") * 1.5
        v[:, :e] += favour
        if c["masked"]:
            v[:, :e] = torch.where(torch.rand(n, e, generator=gen, device="cuda") < c["masked"], -math.inf, v[:, :e])
        return v.to(DTYPES[c["type"]])

    def logits(v):
        return (v.double() @ s["router_w"].double().T) if c["hidden"] else v[:, :e]

    v = rows(t)
    for _ in range(40):
        bad = _near(c, logits(v), s["bias"])
        n = int(bad.sum())
        if n == 0:
            break
        v[bad] = rows(n)
    if c["hidden"]:
        s["x"] = v
    else:
        s["logits"] = v[:, :e]
    return s


def _routing(c, gen):
    """Distinct experts for every position, some sought more than others; and the pairs in expert order."""
    t, e, k = c["rows"], c["experts"], c["top_k"]
    score = torch.rand(t, e, generator=gen, device="cuda") + 0.3 * torch.rand(e, generator=gen, device="cuda")
    weight, idx = score.topk(k, dim=-1)
    if c.get("skip"):
        idx = torch.where(torch.rand(t, k, generator=gen, device="cuda") < c["skip"], -1, idx)
    return idx.to(torch.int32), weight / weight.sum(-1, keepdim=True) * 2.5


def _group(idx, experts):
    """Offsets of the experts' pairs, each pair's position (-1 behind the last pair), each slot's pair (-1: none)."""
    flat = idx.long().flatten()
    key = torch.where(flat >= 0, flat, experts)  # skipped slots behind all others
    order = key.argsort(dim=0, stable=True)
    offsets = (key[:, None] < torch.arange(experts + 1, device="cuda")).sum(0) if len(key) * experts < 1 << 20 else \
        torch.searchsorted(key[order], torch.arange(experts + 1, device="cuda"))
    place = torch.arange(len(key), device="cuda")
    live = place < offsets[-1]
    rows = torch.where(live, order // idx.shape[1], -1)
    slots = torch.empty_like(place)
    slots[order] = torch.where(live, place, -1)
    return offsets.int(), rows.int(), slots.int().view(idx.shape)


def _activations(gen, rows, cols, dtype, pad=0):
    """Normal values, with a few channels that are larger; rows of a buffer `pad` wider."""
    x = torch.randn(rows, cols + pad, generator=gen, device="cuda")
    big = torch.rand(cols + pad, generator=gen, device="cuda") < 0.01
    return torch.where(big, x * 6.0, x).to(DTYPES[dtype])[:, :cols]


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": c}
    t = c["rows"]
    if c["op"] == "select":
        s.update(_select_inputs(c, gen))
        s["idx"] = torch.empty(t, c["top_k"], dtype=torch.int32, device="cuda")
        s["weight"] = torch.empty(t, c["top_k"], device="cuda")
    elif c["op"] == "group":
        s["idx"], _ = _routing(c, gen)
        s["offsets"] = torch.empty(c["experts"] + 1, dtype=torch.int32, device="cuda")
        s["rows"] = torch.full((t * c["top_k"],), -1, dtype=torch.int32, device="cuda")  # behind the last pair it stays as it is
        s["slots"] = torch.empty(t, c["top_k"], dtype=torch.int32, device="cuda")
    elif c["op"] == "combine":
        pairs, h, dtype = t * c["top_k"], c["hidden"], DTYPES[c["type"]]
        s["o"] = torch.randn(pairs, h, generator=gen, device="cuda").to(dtype)
        drop = torch.rand(t, c["top_k"], generator=gen, device="cuda") < c["skip"]
        slots = torch.randperm(pairs, generator=gen, device="cuda").view(t, c["top_k"])
        s["slots"] = torch.where(drop, -1, slots).to(torch.int32)
        weight = torch.rand(t, c["top_k"], generator=gen, device="cuda")
        s["weight"] = weight / weight.sum(-1, keepdim=True) * 2.5
        s["add"] = torch.randn(t, h, generator=gen, device="cuda").to(dtype) if c["add"] else None
        s["out"] = torch.empty(t, h, dtype=dtype, device="cuda")
    elif c["op"] == "quantize":
        k = c["cols"]
        s["x"] = _activations(gen, t, k * (1 + c["swiglu"]), c["type"], c["pad"])
        s["codes"] = torch.empty(t, k, dtype=torch.int8, device="cuda")
        s["scales"] = torch.empty(t, device="cuda")
        s["out"] = torch.empty(t, k, dtype=torch.bfloat16, device="cuda")
    else:
        e, n, k, pitch = c["experts"], c["n"], c["k"], -(-c["k"] // 16) * 16  # rows begin on 16-byte boundaries
        x = _activations(gen, t, k, "f32")
        top = x.abs().amax(-1)
        s["x"] = torch.zeros(t, pitch, dtype=torch.int8, device="cuda")[:, :k]
        s["x"].copy_(torch.round(x / top[:, None] * 127.0))
        s["x_scales"] = top / 127.0
        s["w"] = torch.empty(e, n, pitch, dtype=torch.int8, device="cuda")[:, :, :k]
        step = max(1, (1 << 28) // (n * k))
        for i in range(0, e, step):
            m = min(step, e - i)
            s["w"][i:i + m] = torch.randn(m, n, k, generator=gen, device="cuda").mul_(30.0).round_().clamp_(-127, 127)
        s["w_scales"] = (0.5 + torch.rand(e, n, generator=gen, device="cuda")) * (k ** -0.5 / 30.0)
        if e > 1:
            idx, _ = _routing(c, gen)
            s["offsets"], s["rows"], _ = _group(idx, e)
            s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        s["out"] = torch.empty(t * c["top_k"], n, dtype=DTYPES[c["type"]], device="cuda")
    return s


# ------------------------------------------------------------------------ plain form
def _plain_select(s):
    c, e = s["case"], s["case"]["experts"]
    l = s["x"] @ s["router_w"].T if c["hidden"] else s["logits"].float()
    masked = l == -math.inf
    if c["score"] == "softmax":
        p = torch.exp(l - l.amax(-1, keepdim=True).clamp(min=-3e38))
        p = p / p.sum(-1, keepdim=True).clamp(min=1e-38)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    b = p if s["bias"] is None else p + s["bias"]
    b = torch.where(masked, -math.inf, b)
    rank = l if s["bias"] is None else b  # without a bias the logits have the order of the scores
    if c["groups"] > 1:
        kept = _group_scores(b, c).argsort(dim=-1, descending=True, stable=True)[:, :c["keep"]]
        ok = (kept[:, :, None] == torch.arange(c["groups"], device="cuda")).any(1)
        rank = torch.where(ok.repeat_interleave(e // c["groups"], -1), rank, -math.inf)
    order = rank.argsort(dim=-1, descending=True, stable=True)[:, :c["top_k"]]
    live = rank.gather(-1, order) > -math.inf
    w = torch.where(live, p.gather(-1, order), 0.0)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-38)
    return {"idx": torch.where(live, order, -1).int(), "weight": w * 2.5}


def _plain_group(s):
    offsets, rows, slots = _group(s["idx"], s["case"]["experts"])
    return {"offsets": offsets, "rows": rows, "slots": slots}


def _plain_combine(s):
    slots = s["slots"].long()
    o = s["o"][slots.clamp(min=0)].float()
    y = torch.where(slots >= 0, s["weight"], 0.0)[..., None] * o
    y = y.sum(1)
    if s["add"] is not None:
        y = y + s["add"].float()
    return {"y": y.to(s["out"].dtype)}


def _plain_quantize(s):
    x = s["x"].float()
    if s["case"]["swiglu"]:
        g, u = x.chunk(2, -1)
        x = g / (1.0 + torch.exp(-g)) * u
    top = x.abs().amax(-1, keepdim=True)
    some = top >= TINY
    codes = torch.where(some, torch.round(x.double() * 127.0 / top.clamp(min=TINY).double()).float(), 0.0)  # next to a border 32 bits may turn a code
    return {"values": (codes * torch.where(some, top / 127.0, 0.0)).to(s["out"].dtype)}


def _plain_product(s):
    c = s["case"]
    x, n, e = s["x"].float(), c["n"], c["experts"]
    if e == 1:
        return {"y": (x @ s["w"][0].float().T * s["x_scales"][:, None] * s["w_scales"][0]).to(s["out"].dtype)}
    # every expert's rows, filled up to the longest
    off, rows = s["offsets"].long(), s["rows"].long()
    at = (off[:-1, None] + torch.arange(s["most"], device="cuda")).clamp(max=len(rows) - 1)
    row = torch.arange(len(rows), device="cuda")
    group = (row[:, None] >= off[1:]).sum(-1)
    y = torch.empty(e, s["most"], n, device="cuda")
    step = max(1, (1 << 32) // (n * c["k"]))
    for i in range(0, e, step):
        y[i:i + step] = torch.bmm(x[rows[at[i:i + step]]], s["w"][i:i + step].float().transpose(1, 2))
    y = y[group, row - off[group]] * s["x_scales"][rows][:, None] * s["w_scales"][group]
    return {"y": y.to(s["out"].dtype)}


# ------------------------------------------------------------------------ the package
def _package():
    if "package" not in _held:
        import quantized_expert_ffn_sigmoid_gb300 as cm
        _held["package"] = cm
    return _held["package"]


def _workspace(key, make):
    if key not in _held:
        _held[key] = make()
    return _held[key]


def _own_select(s):
    cm, c = _package(), s["case"]
    ws = None
    if c["hidden"]:
        ws = _workspace(("select", c["rows"], c["hidden"], c["experts"]), lambda: cm.new_select_workspace(c["rows"], c["hidden"], c["experts"]))
    cm.coli_moe_select(s["x"] if c["hidden"] else s["logits"], s["idx"], s["weight"], router_w=s["router_w"], bias=s["bias"],
                       score=cm.SCORE_SOFTMAX if c["score"] == "softmax" else cm.SCORE_SIGMOID, n_groups=c["groups"], topk_group=c["keep"],
                       group_score=cm.GROUP_TOP2 if c["group_score"] == "top2" else cm.GROUP_MAX, renorm=c["renorm"], scaling=2.5, ws=ws)
    return {"idx": s["idx"], "weight": s["weight"]}


def _own_group(s):
    cm, c = _package(), s["case"]
    ws = _workspace(("group", c["rows"], c["top_k"], c["experts"]), lambda: cm.new_group_workspace(c["rows"], c["top_k"], c["experts"]))
    cm.coli_moe_group(s["idx"], s["offsets"], s["rows"], s["slots"], ws)
    return {"offsets": s["offsets"], "rows": s["rows"], "slots": s["slots"]}


def _own_combine(s):
    _package().coli_moe_combine(s["o"], s["slots"], s["weight"], s["out"], add=s["add"])
    return {"y": s["out"]}


def _own_quantize(s):
    cm = _package()
    cm.coli_i8_quantize(s["x"], s["codes"], s["scales"], swiglu=s["case"]["swiglu"])
    cm.coli_i8_dequantize(s["codes"], s["scales"], s["out"])
    return {"values": s["out"]}


def _own_product(s):
    cm, c = _package(), s["case"]
    ws = _workspace(("product", s["out"].shape[0], c["k"]), lambda: cm.new_i8_product_workspace(s["out"].shape[0], c["k"]))
    cm.coli_i8_product(s["x"], s["x_scales"], s["w"], s["w_scales"], s["out"], ws, offsets=s.get("offsets"), rows=s.get("rows"))
    return {"y": s["out"]}


_RUN = {("select", False): _plain_select, ("group", False): _plain_group, ("combine", False): _plain_combine, ("quantize", False): _plain_quantize,
        ("product", False): _plain_product, ("select", True): _own_select, ("group", True): _own_group, ("combine", True): _own_combine,
        ("quantize", True): _own_quantize, ("product", True): _own_product}


def run(state):
    return _RUN[state["case"]["op"], bool(own)](state)


# ------------------------------------------------------------------------ 64 bits
def _select64(s):
    c = s["case"]
    t, e, k, per = c["rows"], c["experts"], c["top_k"], c["experts"] // c["groups"]
    l = s["x"].double() @ s["router_w"].double().T if c["hidden"] else s["logits"].double()
    p = torch.softmax(l, -1).nan_to_num(0.0) if c["score"] == "softmax" else torch.sigmoid(l)
    v = p + (0.0 if s["bias"] is None else s["bias"].double())
    order = l if s["bias"] is None else v  # the same order, and one that no score's underflow blurs
    order = torch.where(torch.isneginf(l), -math.inf, order)
    if c["groups"] > 1:
        v = torch.where(torch.isneginf(l), -math.inf, v).view(t, c["groups"], per)
        best = v.max(-1).values
        if c["group_score"] == "top2" and per > 1:
            second = v.topk(2, -1).values[..., 1]
            best = best + torch.where(second == -math.inf, 0.0, second)
        # a group is kept if fewer than `keep` come before it
        before = (best[:, None, :] > best[:, :, None]) | ((best[:, None, :] == best[:, :, None]) & torch.ones(
            c["groups"], c["groups"], dtype=torch.bool, device="cuda").tril(-1))
        kept = before.sum(-1) < c["keep"]
        order = torch.where(kept.repeat_interleave(per, 1), order, -math.inf)
    idx = torch.full((t, k), -1, dtype=torch.int64, device="cuda")
    for j in range(k):
        best = order.amax(-1, keepdim=True)
        first = torch.where(order == best, torch.arange(e, device="cuda"), e).amin(-1)
        live = best[:, 0] > -math.inf
        idx[:, j] = torch.where(live, first, -1)
        order = order.scatter(1, first[:, None], -math.inf)
    w = torch.where(idx >= 0, p.gather(1, idx.clamp(min=0)), 0.0)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    return {"idx": idx.int(), "weight": w * 2.5}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "select":
        return _select64(s)
    if c["op"] == "group":
        flat = s["idx"].long().flatten()
        hit = (flat[:, None] == torch.arange(c["experts"], device="cuda")).int()
        offsets = torch.cat((hit.new_zeros(1), hit.sum(0))).cumsum(0)
        place = ((hit.cumsum(0, dtype=torch.int32) - 1) * hit).sum(1)  # among the pairs of the same expert
        slots = torch.where(flat >= 0, offsets[flat.clamp(min=0)] + place, -1)
        rows = torch.full((len(flat) + 1,), -1, dtype=torch.int64, device="cuda")
        rows[torch.where(flat >= 0, slots, len(flat))] = torch.arange(len(flat), device="cuda") // c["top_k"]
        return {"offsets": offsets.int(), "rows": rows[:-1].int(), "slots": slots.int().view(s["idx"].shape)}
    if c["op"] == "combine":
        y = torch.zeros(c["rows"], c["hidden"], dtype=torch.float64, device="cuda") if s["add"] is None else s["add"].double()
        for j in range(c["top_k"]):
            at = s["slots"][:, j].long()
            y += torch.where(at[:, None] >= 0, s["weight"][:, j, None].double() * s["o"][at.clamp(min=0)].double(), 0.0)
        return {"y": y}
    if c["op"] == "quantize":
        x = s["x"].double()
        if c["swiglu"]:
            x = x[:, :c["cols"]] * torch.sigmoid(x[:, :c["cols"]]) * x[:, c["cols"]:]
        unit = x.abs().amax(-1, keepdim=True) / 127.0
        return {"values": torch.where(unit * 127.0 >= TINY, torch.round(x / unit.clamp(min=1e-300)) * unit, 0.0)}
    y = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    off = s["offsets"].tolist() if c["experts"] > 1 else [0, c["rows"]]
    for g in range(c["experts"]):
        if off[g + 1] > off[g]:
            at = s["rows"][off[g]:off[g + 1]].long() if c["experts"] > 1 else slice(None)
            x = s["x"][at].double() * s["x_scales"][at].double()[:, None]
            y[off[g]:off[g + 1]] = x @ (s["w"][g].double() * s["w_scales"][g].double()[:, None]).T
    return {"y": y}
