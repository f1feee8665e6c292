"""The MX4 operators in plain numpy, fp64: the format, products grouped by
expert, the routed expert layer and the norms around a block.

A row of K values (K % 32 == 0) is K/2 bytes of codes (element 2j in the low
half of byte j; sign, two exponent bits, one mantissa bit) and K/32 scale
bytes (b stands for 2**(b - 127), 255 for a block without a value).
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
_SIGNED = np.concatenate([MAGNITUDES, -MAGNITUDES])


def scale_bytes(amax):
    """Scale byte of blocks from their largest magnitudes: floor(log2) - 2, at least 2**-127."""
    amax = np.asarray(amax, np.float64)
    _, ex = np.frexp(np.where(np.isfinite(amax) & (amax > 0), amax, 1.0))
    b = np.where(amax > 0, np.maximum(ex - 1 - 2 + 127, 0), 0)
    return np.where(np.isfinite(amax), b, 255).astype(np.uint8)


def round_codes(a):
    """Code (0..7) of magnitudes already divided by their scale: nearest, ties to the even code, 6 at most."""
    a = np.asarray(a, np.float64)
    mid = (MAGNITUDES[:-1] + MAGNITUDES[1:]) / 2
    code = np.searchsorted(mid, a, side="left")          # a tie stays with the lower code ...
    tie = (code < 7) & (a == mid[np.minimum(code, 6)])
    return np.where(tie & (code % 2 == 1), code + 1, code).astype(np.uint8)   # ... unless that is odd


def quantize(x):
    """x [..., K] -> codes [..., K/2], scales [..., K/32]."""
    x = np.asarray(x, np.float64)
    v = x.reshape(*x.shape[:-1], -1, BLOCK)
    with np.errstate(invalid="ignore"):
        amax = np.abs(v).max(-1)
        b = scale_bytes(np.where(np.isnan(v).any(-1), np.nan, amax))
        ok = (b != 255)[..., None]
        c = round_codes(np.where(ok, np.abs(v), 0.0) * np.exp2(127.0 - np.where(b == 255, 127, b).astype(np.float64))[..., None])
    c = np.where(ok, c | (np.signbit(v).astype(np.uint8) << 3), 0).astype(np.uint8).reshape(x.shape)
    return c[..., 0::2] | (c[..., 1::2] << 4), b


def values(codes, scales):
    """The values that codes [..., K/2] and scales [..., K/32] stand for."""
    codes = np.asarray(codes, np.uint8)
    v = np.empty((*codes.shape[:-1], codes.shape[-1] * 2))
    v[..., 0::2] = _SIGNED[codes & 15]
    v[..., 1::2] = _SIGNED[codes >> 4]
    s = np.exp2(np.asarray(scales, np.float64) - 127.0)
    s = np.where(np.asarray(scales) == 255, np.nan, s)
    return v * np.repeat(s, BLOCK, axis=-1)


def product(xv, wv, offsets=None):
    """Rows of xv [P, K] times the matrix of their group, wv [G, N, K]; also sum |x||w|, for error bounds."""
    if offsets is None:
        offsets = [0, xv.shape[0]]
    y = np.zeros((xv.shape[0], wv.shape[1]))
    mag = np.zeros_like(y)
    for g in range(wv.shape[0]):
        a, b = offsets[g], offsets[g + 1]
        y[a:b] = xv[a:b] @ wv[g].T
        mag[a:b] = np.abs(xv[a:b]) @ np.abs(wv[g]).T
    return y, mag


def silu_mul(g, u):
    return g / (1.0 + np.exp(-g)) * u


def _quant_reach(h, err):
    """MX4 values of h [T, I], and how far they can move when h moves by up to err (elementwise)."""
    v0 = values(*quantize(h))
    reach = np.zeros_like(v0)
    hb, eb = h.reshape(len(h), -1, BLOCK), err.reshape(len(h), -1, BLOCK)
    amax = np.abs(hb)
    lo, hi = scale_bytes((amax - eb).clip(min=0).max(-1)), scale_bytes((amax + eb).max(-1))
    for b in (lo, hi):
        s = np.exp2(b.astype(np.float64) - 127.0)[..., None]
        for m in (hb - eb, hb + eb):
            q = np.copysign(MAGNITUDES[round_codes(np.abs(m) / s)], m) * s
            reach = np.maximum(reach, np.abs(q.reshape(h.shape) - v0))
    return v0, reach


def expert(xv, gate, up, down, acc_eps):
    """One expert's output rows and an elementwise bound on what fp32 sums (relative error acc_eps per
    reduction element, against sum |x||w|) and the code changes of h they allow can move it."""
    g, gm = product(xv, gate[None])
    u, um = product(xv, up[None])
    h = silu_mul(g, u)
    eg, eu = acc_eps * xv.shape[1] * gm, acc_eps * xv.shape[1] * um
    # |d silu| <= 1.1; a few fp32 roundings of silu and the product
    eh = 1.1 * eg * np.abs(u) + (np.abs(silu_mul(g, 1.0)) + 1.1 * eg) * eu + 8 * 2.0 ** -24 * np.abs(h)
    hv, reach = _quant_reach(h, eh)
    o, om = product(hv, down[None])
    bound = acc_eps * h.shape[1] * om + product(reach, np.abs(down)[None])[0] * (1 + 1e-3)
    return o, bound


def layer(shape, routed, shared, x, idx, w, acc_eps=2.0 ** -23):
    """The MX4 expert layer: routed(e) / shared(s) give (gate, up, down) values; returns y and its bound."""
    xv = values(*quantize(x))
    y = np.zeros((len(x), shape.hidden))
    bound = np.zeros_like(y)
    for e in sorted(set(int(i) for i in np.ravel(idx) if 0 <= i < shape.n_experts)):
        t, j = np.nonzero(idx == e)
        o, b = expert(xv[t], *routed(e), acc_eps)
        np.add.at(y, t, w[t, j][:, None].astype(np.float64) * o)
        np.add.at(bound, t, np.abs(w[t, j])[:, None] * (b + 2.0 ** -22 * np.abs(o)))
    for s in range(shape.n_shared):
        o, b = expert(xv, *shared(s), acc_eps)
        y += o
        bound += b + 2.0 ** -22 * np.abs(o)
    return y, bound


def block_norm(x, y=None, post_w=None, gate=None, res_scale=1.0, pre_w=None, eps=1e-6):
    """(x', n) of the norms around a block, fp64."""
    def rms(v, w):
        return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps) * (1.0 if w is None else w)

    x = np.asarray(x, np.float64)
    if y is not None:
        r = np.asarray(y, np.float64)
        if post_w is not None:
            r = rms(r, np.asarray(post_w, np.float64))
        if gate is not None:
            r = r * np.asarray(gate, np.float64)
        x = x + res_scale * r
    return x, rms(x, None if pre_w is None else np.asarray(pre_w, np.float64))
