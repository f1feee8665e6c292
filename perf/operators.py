"""Timed cases of the 4-bit microscaled (MX4) operators: quantisation of
activations, matrix products grouped by expert, the routed expert layer on
them, and the norms around a block.

``run`` computes a case in one of two ways: with ``own`` false in plain form
(elementary torch operations in 32 bits, rounded once at the end), with ``own``
true through this repository's package.  ``exact`` computes the same values in
64 bits from the definitions.

An MX4 row is a run of 4-bit codes (sign, two exponent bits, one mantissa bit:
0, 0.5, 1, 1.5, 2, 3, 4, 6) with one power-of-two scale byte per 32 of them
(exponent + 127; 255 marks a block with no value).  Element 2j is the low half
of byte j.
"""
import math
import random

import torch

own = False

BLOCK = 32
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
_held = {}  # the package and the workspaces that a user's program keeps


# ------------------------------------------------------------------------ cases
def listed():
    glm = dict(op="experts", hidden=6144, experts=256, inter=2048, top_k=8, shared=1, skip=0.0, x="bf16", y="bf16")
    return [
        # the hidden state of one decoded token, quantised before its products: latency alone
        dict(name="quantize_token", op="quantize", rows=1, cols=6144, pad=0, x="f32"),
        # the activations of a long prompt, rows of a wider buffer
        dict(name="quantize_prompt", op="quantize", rows=8192, cols=6144, pad=2048, x="bf16"),
        # one token through one down projection that stays in the L2 cache
        dict(name="product_token", op="product", rows=1, groups=1, n=6144, k=2048, split=0, y="bf16"),
        # ragged groups, some empty, no size a multiple of a tile
        dict(name="product_odd", op="product", rows=333, groups=7, n=1000, k=544, split=3, y="f16"),
        # the gate and up products of one expert-parallel shard (32 of 256 experts) for a prompt
        dict(name="product_shard", op="product", rows=4096, groups=32, n=4096, k=6144, split=1, y="bf16"),
        # a dense projection of a long prompt: bound by arithmetic
        dict(name="product_prompt", op="product", rows=8192, groups=1, n=4096, k=6144, split=0, y="bf16"),
        # the routed layer for one decoded token: streams 8 routed experts and the shared one
        dict(glm, name="experts_token", rows=1),
        # the verification of a few drafted tokens
        dict(glm, name="experts_verify", rows=4),
        # a batch of decoding streams
        dict(glm, name="experts_batch", rows=32),
        # a prompt: every expert is read, about 64 tokens each
        dict(glm, name="experts_prompt", rows=2048),
        # the norms around a block for one decoded token
        dict(name="norm_token", op="norm", rows=1, hidden=6144, post=True, gate="channel", mx4=True, x="f32"),
        # the same for a prompt, with a gate of its own for every token
        dict(name="norm_prompt", op="norm", rows=4096, hidden=6144, post=True, gate="token", mx4=True, x="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "experts", "experts", "norm"])
    if op == "quantize":
        cols = BLOCK * _log_int(rng, 1, 192)
        return dict(op=op, rows=min(_log_int(rng, 1, 8192), (1 << 25) // cols), cols=cols, pad=rng.choice([0, 0, 8, 2048, 5]),
                    x=rng.choice(["f32", "bf16", "f16"]))
    if op == "product":
        groups, n, k = rng.choice([1, 1, _log_int(rng, 2, 64)]), _log_int(rng, 48, 6144), BLOCK * _log_int(rng, 1, 192)
        groups = max(1, min(groups, (1 << 29) // (n * k)))
        rows = max(1, min(_log_int(rng, 1, 8192), (1 << 37) // (n * k)))
        return dict(op=op, rows=rows, groups=groups, n=n, k=k, split=rng.randrange(1, 1 << 20), y=rng.choice(["bf16", "bf16", "f16"]))
    if op == "experts":
        experts = rng.choice([8, 16, 60, 64, 128, 256])
        hidden, inter = 128 * _log_int(rng, 2, 48), 128 * _log_int(rng, 1, 16)
        return dict(op=op, rows=_log_int(rng, 1, 1792), hidden=hidden, experts=experts, inter=inter, top_k=rng.choice([1, 2, 4, 6, 8]),
                    shared=rng.choice([0, 1, 1, 2]), skip=rng.choice([0.0, 0.0, 0.25]), x=rng.choice(["f32", "bf16", "f16"]),
                    y=rng.choice(["bf16", "f16"]))
    mx4 = rng.random() < 0.5
    hidden = BLOCK * _log_int(rng, 1, 256) if mx4 else _log_int(rng, 33, 8192)
    return dict(op=op, rows=min(_log_int(rng, 1, 8192), (1 << 24) // hidden), hidden=hidden, post=rng.random() < 0.7,
                gate=rng.choice(["none", "channel", "token"]), mx4=mx4, x=rng.choice(["f32", "bf16", "f16"]))


def _offsets(c):
    """The first row of each group and the end: cuts at random places, so that some groups are large and some empty."""
    rng = random.Random(c["split"])
    return [0] + sorted(rng.randint(0, c["rows"]) for _ in range(c["groups"] - 1)) + [c["rows"]]


def _row_bytes(k):
    return k // 2 + k // BLOCK


def work(case):
    c, size = case, lambda name: torch.empty(0, dtype=DTYPES[name]).element_size()
    if c["op"] == "quantize":  # values in, codes out, codes in, values out
        n = c["rows"] * c["cols"]
        return {"bytes": n * 2 * size(c["x"]) + 2 * c["rows"] * _row_bytes(c["cols"]), "flops": 4 * n}
    if c["op"] == "product":
        off = _offsets(c)
        used = sum(b > a for a, b in zip(off, off[1:]))
        return {"bytes": (used * c["n"] + c["rows"]) * _row_bytes(c["k"]) + c["rows"] * c["n"] * size(c["y"]),
                "flops": 2 * c["rows"] * c["n"] * c["k"]}
    if c["op"] == "experts":  # each expert that is hit is read once
        h, i = c["hidden"], c["inter"]
        k, keep = min(c["top_k"], c["experts"]), 1.0 - c["skip"]
        hit = c["experts"] * (1.0 - (1.0 - keep * k / c["experts"]) ** c["rows"]) + c["shared"]
        pairs = c["rows"] * (k * keep + c["shared"])
        return {"bytes": hit * (2 * i * _row_bytes(h) + h * _row_bytes(i)) + c["rows"] * h * (size(c["x"]) + size(c["y"])) + 8 * c["rows"] * k,
                "flops": pairs * 6 * h * i}
    n, e = c["rows"] * c["hidden"], size(c["x"])
    streams = 3 + 1 + (c["gate"] == "token")  # the stream, the block's output, the gate; the new stream and its norm
    codes = 2 * c["rows"] * _row_bytes(c["hidden"]) + 2 * n if c["mx4"] else 0  # codes out, codes in, values out
    return {"bytes": n * e * streams + codes + 4 * c["hidden"] * (1 + c["post"] + (c["gate"] == "channel")), "flops": 12 * n}


# ------------------------------------------------------------------ MX4, plain form
def _scale_of(byte):
    """2 ** (byte - 127), and no value for 255."""
    s = (byte.int() << 23).view(torch.float32)
    s = torch.where(byte == 0, torch.full_like(s, 2.0 ** -127), s)
    return torch.where(byte == 255, torch.full_like(s, float("nan")), s)


def _quantize(x):
    """x [..., K] -> codes [..., K/2], scales [..., K/32] (bytes)."""
    v = x.float().unflatten(-1, (-1, BLOCK))
    top = v.abs().amax(-1, keepdim=True)
    exponent = top.view(torch.int32) >> 23
    lost = exponent == 255  # a block with an infinity or NaN
    byte = torch.where(lost, exponent, (exponent - 2).clamp(min=0))
    v = torch.where(lost, torch.zeros_like(v), v * ((254 - byte.clamp(max=253)) << 23).view(torch.float32))
    a = v.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte.squeeze(-1).to(torch.uint8)


def _values(codes, scales):
    """The values that codes [..., K/2] and scales [..., K/32] stand for, in 32 bits."""
    b = codes.int()
    halves = torch.stack((b & 15, b >> 4), -1).flatten(-2)
    del b
    # the three low bits are a float's exponent and mantissa of their own, 2 ** 126 too small
    v = (((halves & 7) << 22) | ((halves & 8) << 28)).view(torch.float32)
    del halves
    v *= 2.0 ** 126
    v = v.unflatten(-1, (-1, BLOCK))
    v *= _scale_of(scales).unsqueeze(-1)
    return v.flatten(-2)


# ------------------------------------------------------------------------ inputs
def _random_weights(gen, count, rows, k, std):
    """Normal weights of `count` matrices [rows, k] as codes and scales."""
    codes = torch.empty(count, rows, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(count, rows, k // BLOCK, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (rows * k))
    for i in range(0, count, step):
        n = min(step, count - i)
        w = torch.randn(n, rows, k, generator=gen, device="cuda").mul_(std)
        codes[i:i + n], scales[i:i + n] = _quantize(w)
    return codes, scales


def _hidden(gen, rows, cols, dtype, pad=0):
    """Activations: normal, with a few channels that are much larger; rows of a buffer `pad` wider."""
    x = torch.randn(rows, cols + pad, generator=gen, device="cuda")
    big = torch.rand(cols + pad, generator=gen, device="cuda") < 0.01
    return torch.where(big, x * 12.0, x).to(DTYPES[dtype])[:, :cols]


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "quantize":
        s["x"] = _hidden(gen, c["rows"], c["cols"], c["x"], c["pad"])
        s["codes"] = torch.empty(c["rows"], c["cols"] // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(c["rows"], c["cols"] // BLOCK, dtype=torch.uint8, device="cuda")
        s["out"] = torch.empty(c["rows"], c["cols"], dtype=s["x"].dtype, device="cuda")
    elif c["op"] == "product":
        off = _offsets(c)
        s["most"] = max(b - a for a, b in zip(off, off[1:]))
        s["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda")
        s["x"], s["x_scales"] = _quantize(_hidden(gen, c["rows"], c["k"], "f32"))
        s["w"], s["w_scales"] = _random_weights(gen, c["groups"], c["n"], c["k"], c["k"] ** -0.5)
        s["out"] = torch.empty(c["rows"], c["n"], dtype=DTYPES[c["y"]], device="cuda")
    elif c["op"] == "experts":
        t, h, e, i, n = c["rows"], c["hidden"], c["experts"], c["inter"], c["shared"]
        k = min(c["top_k"], e)
        s["x"] = _hidden(gen, t, h, c["x"])
        # one record an expert: gate [i][h], up [i][h], down [h][i], codes and scales alike
        for name, count in (("experts", e), ("shared", n)):
            s[name] = torch.empty(count, 3 * i * h // 2, dtype=torch.uint8, device="cuda")
            s[name + "_scales"] = torch.empty(count, 3 * i * h // BLOCK, dtype=torch.uint8, device="cuda")
            for j in range(count):
                for at, r, kk in ((0, 2 * i, h), (2 * i * h, h, i)):
                    q, b = _random_weights(gen, 1, r, kk, kk ** -0.5)
                    s[name][j, at // 2:at // 2 + q.numel()] = q.view(-1)
                    s[name + "_scales"][j, at // BLOCK:at // BLOCK + b.numel()] = b.view(-1)
        score = torch.rand(t, e, generator=gen, device="cuda")
        weight, idx = score.topk(k, dim=-1)
        drop = torch.rand(t, k, generator=gen, device="cuda") < c["skip"]
        s["idx"] = torch.where(drop, torch.full_like(idx, -1), idx).to(torch.int32)
        s["weight"] = weight / weight.sum(-1, keepdim=True) * 2.5
        s["most"] = int(torch.bincount(idx.flatten()).max())
        s["out"] = torch.empty(t, h, dtype=DTYPES[c["y"]], device="cuda")
    else:
        t, h = c["rows"], c["hidden"]
        s["x"], s["y"] = _hidden(gen, t, h, c["x"]), _hidden(gen, t, h, c["x"])
        s["pre"] = 1.0 + 0.1 * torch.randn(h, generator=gen, device="cuda")
        s["post"] = 1.0 + 0.1 * torch.randn(h, generator=gen, device="cuda") if c["post"] else None
        s["gate"] = None
        if c["gate"] != "none":
            g = torch.rand(t if c["gate"] == "token" else 1, h, generator=gen, device="cuda").to(s["x"].dtype)
            s["gate"] = g if c["gate"] == "token" else g[0]
        s["stream"], s["norm"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        if c["mx4"]:
            s["codes"] = torch.empty(t, h // 2, dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty(t, h // BLOCK, dtype=torch.uint8, device="cuda")
            s["out"] = torch.empty(t, h, dtype=torch.bfloat16, device="cuda")
    return s


RES_SCALE = 0.7  # the scale of the residual branch


# ------------------------------------------------------------------------ plain form
def _plain_quantize(s):
    codes, scales = _quantize(s["x"])
    return {"values": _values(codes, scales).to(s["x"].dtype)}


def _plain_product(s):
    c, off = s["case"], s["offsets"].long()
    x, w = _values(s["x"], s["x_scales"]), _values(s["w"], s["w_scales"])
    if c["groups"] == 1:
        return {"y": (x @ w[0].T).to(DTYPES[c["y"]])}
    # every group's rows, filled up to the longest group
    at = off[:-1, None] + torch.arange(s["most"], device="cuda")
    y = torch.bmm(x[at.clamp(max=c["rows"] - 1)], w.transpose(1, 2))
    row = torch.arange(c["rows"], device="cuda")
    group = (row[:, None] >= off[1:]).sum(-1)
    return {"y": y[group, row - off[group]].to(DTYPES[c["y"]])}


def _ffn(x, codes, scales, h, i):
    """x [B, M, h] through the experts of records codes [B, ...], scales [B, ...]."""
    b, cut, cut_s = codes.shape[0], i * h, 2 * i * h // BLOCK
    gu = torch.bmm(x, _values(codes[:, :cut].reshape(b, 2 * i, h // 2), scales[:, :cut_s].reshape(b, 2 * i, h // BLOCK)).transpose(1, 2))
    gate, up = gu[..., :i], gu[..., i:]
    hid = _values(*_quantize(gate / (1.0 + torch.exp(-gate)) * up))
    return torch.bmm(hid, _values(codes[:, cut:].reshape(b, h, i // 2), scales[:, cut_s:].reshape(b, h, i // BLOCK)).transpose(1, 2))


def _plain_experts(s):
    c, idx = s["case"], s["idx"].long()
    t, h, e, i = c["rows"], c["hidden"], c["experts"], c["inter"]
    k = idx.shape[1]
    x = _values(*_quantize(s["x"]))
    w = torch.where(idx >= 0, s["weight"], torch.zeros_like(s["weight"]))
    idx = idx.clamp(min=0)
    if t * k < e:  # few pairs: each with its own expert's weights
        o = _ffn(x.repeat_interleave(k, 0)[:, None], s["experts"][idx.flatten()], s["experts_scales"][idx.flatten()], h, i)
        y = (o.view(t, k, h) * w[..., None]).sum(1)
    else:  # every expert over its pairs, filled up to the longest
        flat = s["idx"].long().flatten()
        hit = (flat[:, None] == torch.arange(e, device="cuda")).int()
        place = (hit.cumsum(0) * hit).sum(1) - 1  # among the pairs of the same expert; -1 where there is none
        token = torch.arange(t * k, device="cuda") // k
        rows = torch.full((e, s["most"] + 1), t, device="cuda")
        rows[flat.clamp(min=0), torch.where(flat >= 0, place, torch.full_like(place, s["most"]))] = token
        o = _ffn(torch.cat((x, x.new_zeros(1, h)))[rows[:, :-1]], s["experts"], s["experts_scales"], h, i)
        y = (o[idx.flatten(), place.clamp(min=0)].view(t, k, h) * w[..., None]).sum(1)
    if c["shared"]:
        y = y + _ffn(x.expand(c["shared"], t, h), s["shared"], s["shared_scales"], h, i).sum(0)
    return {"y": y.to(DTYPES[c["y"]])}


def _rms(v, weight):
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * weight


def _plain_norm(s):
    y = s["y"].float()
    if s["post"] is not None:
        y = _rms(y, s["post"])
    if s["gate"] is not None:
        y = y * s["gate"].float()
    stream = s["x"].float() + RES_SCALE * y
    norm = _rms(stream, s["pre"])
    out = {"stream": stream.to(s["x"].dtype), "norm": norm.to(s["x"].dtype)}
    if s["case"]["mx4"]:
        out["values"] = _values(*_quantize(norm)).to(torch.bfloat16)
    return out


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


def _own_quantize(s):
    cm = _package()
    cm.coli_mx4_quantize(s["x"], s["codes"], s["scales"])
    cm.coli_mx4_dequantize(s["codes"], s["scales"], s["out"])
    return {"values": s["out"]}


def _own_product(s):
    cm = _package()
    ws = _workspace("product", cm.new_mx4_product_workspace)
    cm.coli_mx4_product(s["x"], s["x_scales"], s["w"], s["w_scales"], s["out"], ws, offsets=s["offsets"])
    return {"y": s["out"]}


def _own_experts(s):
    cm, c = _package(), s["case"]
    if "layer" not in s:
        cfg = cm.Cfg(hidden=c["hidden"], n_experts=c["experts"], n_groups=1, topk_group=1, top_k=s["idx"].shape[1], inter=c["inter"],
                     n_shared=c["shared"], shared_inter=c["inter"], weight_bits=4, routed_scaling_factor=2.5)
        s["layer"] = cfg, cm.make_mx4_weights(s["experts"], s["experts_scales"], s["shared"], s["shared_scales"])
    cfg, weights = s["layer"]
    ws = _workspace(tuple(sorted(c.items())), lambda: cm.new_mx4_workspace(cfg, c["rows"]))
    cm.coli_mx4_forward(cfg, weights, s["x"], s["idx"], s["weight"], s["out"], ws)
    return {"y": s["out"]}


def _own_norm(s):
    cm, mx4 = _package(), s["case"]["mx4"]
    cm.coli_moe_block_norm(s["x"], s["y"], post_w=s["post"], gate=s["gate"], res_scale=RES_SCALE, pre_w=s["pre"], eps=EPS,
                           x_out=s["stream"], n_out=s["norm"], codes=s["codes"] if mx4 else None, scales=s["scales"] if mx4 else None)
    out = {"stream": s["stream"], "norm": s["norm"]}
    if mx4:
        cm.coli_mx4_dequantize(s["codes"], s["scales"], s["out"])
        out["values"] = s["out"]
    return out


_RUN = {("quantize", False): _plain_quantize, ("product", False): _plain_product, ("experts", False): _plain_experts, ("norm", False): _plain_norm,
        ("quantize", True): _own_quantize, ("product", True): _own_product, ("experts", True): _own_experts, ("norm", True): _own_norm}


def run(state):
    return _RUN[state["case"]["op"], bool(own)](state)


# ------------------------------------------------------------------------ 64 bits
_GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _decode64(codes, scales):
    table = torch.tensor(_GRID + [-g for g in _GRID], dtype=torch.float64, device=codes.device)
    v = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=codes.device)
    v[..., 0::2] = table[(codes % 16).long()]
    v[..., 1::2] = table[(codes // 16).long()]
    p = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=codes.device), scales.double() - 127.0)
    p[scales == 255] = float("nan")
    return v * p.repeat_interleave(BLOCK, -1)


def _to_grid64(x):
    """x [..., K] in 64 bits -> the nearest MX4 values, half to even."""
    v = x.double().reshape(*x.shape[:-1], -1, BLOCK)
    top = v.abs().amax(-1, keepdim=True)
    _, ex = torch.frexp(torch.where(top > 0, top, torch.ones_like(top)))
    p = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=x.device), (ex - 3).clamp(min=-127).double())
    a = v.abs() / p
    r = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2)).clamp(max=6.0)
    r = torch.copysign(r * p, v)
    return torch.where(torch.isfinite(top), r, torch.full_like(r, float("nan"))).reshape(x.shape)


def _norm64(v, weight):
    return v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS) * weight.double()


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "quantize":
        return {"values": _to_grid64(s["x"])}
    if c["op"] == "product":
        x, off = _decode64(s["x"], s["x_scales"]), _offsets(c)
        y = torch.zeros(c["rows"], c["n"], dtype=torch.float64, device="cuda")
        for g in range(c["groups"]):
            if off[g + 1] > off[g]:
                y[off[g]:off[g + 1]] = x[off[g]:off[g + 1]] @ _decode64(s["w"][g], s["w_scales"][g]).T
        return {"y": y}
    if c["op"] == "experts":
        h, i = c["hidden"], c["inter"]
        x, y = _to_grid64(s["x"]), torch.zeros(c["rows"], h, dtype=torch.float64, device="cuda")

        def expert(name, j, rows):
            q, b = s[name][j], s[name + "_scales"][j]
            m = [_decode64(q[a // 2:(a + i * h) // 2].view(r, -1), b[a // BLOCK:(a + i * h) // BLOCK].view(r, -1))
                 for a, r in ((0, i), (i * h, i), (2 * i * h, h))]
            g = rows @ m[0].T
            return _to_grid64(g * torch.sigmoid(g) * (rows @ m[1].T)) @ m[2].T

        for j in torch.unique(s["idx"]).tolist():
            if j >= 0:
                t, slot = torch.nonzero(s["idx"] == j, as_tuple=True)
                y[t] += s["weight"][t, slot].double()[:, None] * expert("experts", j, x[t])
        for j in range(c["shared"]):
            y += expert("shared", j, x)
        return {"y": y}
    y = s["y"].double()
    if s["post"] is not None:
        y = _norm64(y, s["post"])
    if s["gate"] is not None:
        y = y * s["gate"].double()
    stream = s["x"].double() + RES_SCALE * y
    norm = _norm64(stream, s["pre"])
    out = {"stream": stream, "norm": norm}
    if c["mx4"]:
        out["values"] = _to_grid64(norm)
    return out
