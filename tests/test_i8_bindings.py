"""The bindings of the 8-bit token and channel operators look at every tensor
before the library is called, and the library at every size and address before
it launches.  No GPU: stand-ins answer what the bindings ask of a tensor, a
recorder takes the library's place; the library's own refusals come before any
CUDA call."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402
from test_mx4_bindings import Stand, calls  # noqa: E402,F401

F, I, B, H = torch.float32, torch.int32, torch.int8, torch.bfloat16


def select_logits():
    return cm.coli_moe_select, dict(x=Stand(3, 16, dtype=H), topk_idx=Stand(3, 4, dtype=I), topk_w=Stand(3, 4, dtype=F), bias=Stand(16, dtype=F), ws=Stand(256))


def select_hidden():
    return cm.coli_moe_select, dict(x=Stand(3, 32, dtype=F), topk_idx=Stand(3, 4, dtype=I), topk_w=Stand(3, 4, dtype=F), router_w=Stand(16, 32, dtype=F),
                                    bias=Stand(16, dtype=F), ws=Stand(1 << 20))


def group():
    return cm.coli_moe_group, dict(topk_idx=Stand(3, 4, dtype=I), offsets=Stand(17, dtype=I), rows=Stand(12, dtype=I), slots=Stand(3, 4, dtype=I), ws=Stand(1 << 20))


def combine():
    return cm.coli_moe_combine, dict(o=Stand(12, 32, dtype=H), slots=Stand(3, 4, dtype=I), topk_w=Stand(3, 4, dtype=F), y=Stand(3, 32, dtype=F), add=Stand(3, 32, dtype=F))


def quantize():
    return cm.coli_i8_quantize, dict(x=Stand(3, 32, dtype=H), codes=Stand(3, 32, dtype=B), scales=Stand(3, dtype=F))


def swiglu():
    f, a = quantize()
    return (lambda **kw: f(**kw, swiglu=True)), dict(a, x=Stand(3, 64, dtype=H))


def dequantize():
    return cm.coli_i8_dequantize, dict(codes=Stand(3, 32, dtype=B), scales=Stand(3, dtype=F), out=Stand(3, 32, dtype=H))


def product():
    return cm.coli_i8_product, dict(x_codes=Stand(5, 32, dtype=B), x_scales=Stand(5, dtype=F), w_codes=Stand(2, 8, 32, dtype=B), w_scales=Stand(2, 8, dtype=F),
                                    y=Stand(9, 8, dtype=H), ws=Stand(1 << 20), offsets=Stand(3, dtype=I), rows=Stand(9, dtype=I))


ALL = [select_logits, select_hidden, group, combine, quantize, swiglu, dequantize, product]


def with_(t, **kw):
    d = dict(dtype=t.dtype, index=t.index, strides=None if t.dense else t.strides)
    shape = kw.pop("shape", t.shape)
    d.update(kw)
    return Stand(*shape, **d)


@pytest.mark.parametrize("make", ALL, ids=lambda f: f.__name__)
def test_a_valid_call_is_made(calls, make):  # noqa: F811
    f, args = make()
    f(**args)
    assert len(calls) == 1


@pytest.mark.parametrize("make", ALL, ids=lambda f: f.__name__)
def test_every_tensor_is_looked_at(calls, make):  # noqa: F811
    f, args = make()
    for name, t in args.items():
        bad = [with_(t, index=1), with_(t, index=-1)]
        if name != "ws":
            bad.append(with_(t, dtype=torch.int64))
            if name != "o" and not (name == "offsets" and make is group):     # (which choose a size of the call)
                bad.append(with_(t, shape=(*t.shape[:-1], t.shape[-1] + 1)))
            if len(t.shape) > 1:
                bad.append(with_(t, shape=(*t.shape[:-1], t.shape[-1] + 3) if name == "o" else t.shape, strides=None if name == "o" else
                                 (*[s * 2 for s in t.strides[:-1]], 2)))
        else:
            bad.append(Stand(2, 128, strides=(256, 1)))
        for b in bad:
            with pytest.raises((ValueError, TypeError)):
                f(**dict(args, **{name: b}))
    everywhere = {n: with_(t, index=-1) for n, t in args.items()}
    with pytest.raises(ValueError):
        f(**everywhere)
    other = {n: with_(t, index=1) for n, t in args.items()}
    with pytest.raises(ValueError, match="current device"):
        f(**other)
    assert not calls


def test_strides_that_are_taken(calls):  # noqa: F811
    f, a = product()
    f(**dict(a, x_codes=Stand(5, 32, dtype=B, strides=(48, 1)), w_codes=Stand(2, 8, 32, dtype=B, strides=(4096, 64, 1)),
             w_scales=Stand(2, 8, dtype=F, strides=(100, 1)), y=Stand(9, 8, dtype=H, strides=(11, 1))))
    f(**dict(a, w_codes=Stand(8, 32, dtype=B), w_scales=Stand(8, dtype=F), offsets=None, x_codes=Stand(9, 32, dtype=B), x_scales=Stand(9, dtype=F), rows=None))
    f, a = quantize()
    f(**dict(a, x=Stand(3, 32, dtype=H, strides=(37, 1)), codes=Stand(3, 32, dtype=B, strides=(33, 1))))
    f, a = combine()
    f(**dict(a, o=Stand(12, 32, dtype=H, strides=(40, 1)), add=a["y"]))
    f, a = select_logits()
    f(**dict(a, x=Stand(3, 16, dtype=H, strides=(19, 1)), bias=None, ws=None))
    assert len(calls) == 5


def test_other_refusals(calls):  # noqa: F811
    f, a = group()
    with pytest.raises(ValueError, match="17"):
        f(**dict(a, n_experts=16, offsets=Stand(9, dtype=I)))
    f(**dict(a, n_experts=16, offsets=Stand(6, dtype=I), ep_rank=1, ep_size=3))
    with pytest.raises(ValueError, match="6 values"):
        f(**dict(a, n_experts=16, ep_rank=1, ep_size=3))
    f, a = combine()
    with pytest.raises(TypeError, match="add must have y's type"):
        f(**dict(a, add=Stand(3, 32, dtype=H)))
    f, a = select_hidden()
    with pytest.raises(TypeError, match="x must be"):
        f(**dict(a, x=Stand(3, 32, dtype=H)))
    f, a = dequantize()
    with pytest.raises(ValueError, match="32 bits"):
        f(codes=Stand(1 << 31, 1, dtype=B), scales=Stand(1 << 31, dtype=F), out=Stand(1 << 31, 1, dtype=H))
    f, a = product()
    with pytest.raises(ValueError, match="32 bits"):
        f(**dict(a, y=Stand(1 << 31, 8, dtype=H), rows=Stand(1 << 31, dtype=I)))
    assert len(calls) == 1


# ------------------------------------------------------------------- the library
P = ctypes.c_void_p(4096)


def c_select(**kw):
    d = dict(x=4096, ldx=64, router_w=None, bias=None, topk_idx=4096, topk_w=4096, ws=4096, ws_bytes=1 << 30, type=cm.COLI_F32, hidden=0, n_experts=64,
             n_groups=8, topk_group=4, top_k=8, score=0, group_score=0, renorm=1, scaling=1.0, T=5)
    d.update(kw)
    return cm.lib.coli_moe_select(cm.SelectArgs(*(d[f] for f, _ in cm.SelectArgs._fields_)), d["T"], None)


@pytest.mark.parametrize("code,kw", [
    (cm.COLI_EINVAL, dict(T=-1)), (cm.COLI_EINVAL, dict(n_experts=0)), (cm.COLI_EINVAL, dict(n_experts=60)), (cm.COLI_EINVAL, dict(topk_group=9)),
    (cm.COLI_EINVAL, dict(topk_group=0)), (cm.COLI_EINVAL, dict(top_k=0)), (cm.COLI_EINVAL, dict(topk_group=1, top_k=9)), (cm.COLI_EINVAL, dict(score=2)),
    (cm.COLI_EINVAL, dict(group_score=-1)), (cm.COLI_EINVAL, dict(scaling=float("nan"))), (cm.COLI_EINVAL, dict(type=cm.COLI_MX4)), (cm.COLI_EINVAL, dict(ldx=63)),
    (cm.COLI_EINVAL, dict(x=None)), (cm.COLI_EINVAL, dict(topk_idx=None)), (cm.COLI_EINVAL, dict(topk_w=None)),
    (cm.COLI_EUNSUPPORTED, dict(n_experts=2048, ldx=2048)), (cm.COLI_EUNSUPPORTED, dict(n_groups=64)), (cm.COLI_EUNSUPPORTED, dict(top_k=33, topk_group=8)),
    (cm.COLI_EALIGN, dict(x=4100)), (cm.COLI_EALIGN, dict(bias=4100)), (cm.COLI_EALIGN, dict(topk_w=4104)), (cm.COLI_EALIGN, dict(ws=4104)),
    (cm.COLI_EWORKSPACE, dict(ws_bytes=128)),
    (cm.COLI_EINVAL, dict(router_w=4096, hidden=64, type=cm.COLI_BF16)), (cm.COLI_EINVAL, dict(router_w=4096, hidden=40, ldx=40)),
    (cm.COLI_EINVAL, dict(router_w=4096, hidden=64, ldx=80)), (cm.COLI_EINVAL, dict(router_w=4096, hidden=64, ws=None, ws_bytes=0)),
    (cm.COLI_EWORKSPACE, dict(router_w=4096, hidden=64, ws_bytes=9000)), (cm.COLI_OK, dict(T=0, x=None)),
])
def test_select_refuses(code, kw):
    assert c_select(**kw) == code


def c_group(**kw):
    d = dict(idx=P, T=5, k=4, E=16, rank=0, size=0, offsets=P, rows=P, slots=P, ws=P, n=1 << 30)
    d.update(kw)
    return cm.lib.coli_moe_group(*(d[n] for n in ("idx", "T", "k", "E", "rank", "size", "offsets", "rows", "slots", "ws", "n")), None)


@pytest.mark.parametrize("code,kw", [
    (cm.COLI_EINVAL, dict(T=-1)), (cm.COLI_EINVAL, dict(k=0)), (cm.COLI_EINVAL, dict(E=0)), (cm.COLI_EINVAL, dict(size=17)), (cm.COLI_EINVAL, dict(rank=1)),
    (cm.COLI_EINVAL, dict(rank=2, size=2)), (cm.COLI_EINVAL, dict(rank=-1, size=2)), (cm.COLI_EINVAL, dict(size=-1)), (cm.COLI_EINVAL, dict(idx=None)),
    (cm.COLI_EINVAL, dict(offsets=None)), (cm.COLI_EINVAL, dict(ws=None)), (cm.COLI_EUNSUPPORTED, dict(k=33)), (cm.COLI_EUNSUPPORTED, dict(E=1025)),
    (cm.COLI_EUNSUPPORTED, dict(T=1 << 30)), (cm.COLI_EALIGN, dict(rows=ctypes.c_void_p(4100))), (cm.COLI_EWORKSPACE, dict(n=9000)),
])
def test_group_refuses(code, kw):
    assert c_group(**kw) == code


def c_combine(**kw):
    d = dict(o=P, ot=0, ldo=32, P=12, slots=P, w=P, T=3, k=4, H=32, add=None, lda=0, y=P, yt=0, ldy=32)
    d.update(kw)
    return cm.lib.coli_moe_combine(*(d[n] for n in ("o", "ot", "ldo", "P", "slots", "w", "T", "k", "H", "add", "lda", "y", "yt", "ldy")), None)


@pytest.mark.parametrize("code,kw", [
    (cm.COLI_EINVAL, dict(T=-1)), (cm.COLI_EINVAL, dict(P=-1)), (cm.COLI_EINVAL, dict(k=0)), (cm.COLI_EINVAL, dict(H=0)), (cm.COLI_EINVAL, dict(ot=3)),
    (cm.COLI_EINVAL, dict(yt=3)), (cm.COLI_EINVAL, dict(ldo=31)), (cm.COLI_EINVAL, dict(ldy=31)), (cm.COLI_EINVAL, dict(add=P, lda=31)),
    (cm.COLI_EINVAL, dict(o=None)), (cm.COLI_EINVAL, dict(slots=None)), (cm.COLI_EINVAL, dict(y=None)), (cm.COLI_EALIGN, dict(y=ctypes.c_void_p(4104))),
    (cm.COLI_OK, dict(T=0)),
])
def test_combine_refuses(code, kw):
    assert c_combine(**kw) == code


@pytest.mark.parametrize("code,kw", [
    (cm.COLI_EINVAL, dict(T=-1)), (cm.COLI_EINVAL, dict(K=0)), (cm.COLI_EINVAL, dict(ty=3)), (cm.COLI_EINVAL, dict(act=2)), (cm.COLI_EINVAL, dict(ldx=31)),
    (cm.COLI_EINVAL, dict(ldc=31)), (cm.COLI_EINVAL, dict(act=1, ldx=63)), (cm.COLI_EINVAL, dict(x=None)), (cm.COLI_EINVAL, dict(s=None)),
    (cm.COLI_EUNSUPPORTED, dict(K=131072, ldx=131072, ldc=131072)), (cm.COLI_EALIGN, dict(c=ctypes.c_void_p(4097))), (cm.COLI_OK, dict(T=0)),
])
def test_quantize_refuses(code, kw):
    d = dict(x=P, ty=0, ldx=32, T=3, K=32, act=0, c=P, ldc=32, s=P)
    d.update(kw)
    assert cm.lib.coli_i8_quantize(*(d[n] for n in ("x", "ty", "ldx", "T", "K", "act", "c", "ldc", "s")), None) == code
    if "act" not in kw:
        assert cm.lib.coli_i8_dequantize(d["c"], d["ldc"], d["s"], d["T"], d["K"], d["x"], d["ty"], d["ldx"], None) == code


def c_product(**kw):
    d = dict(x_codes=4096, ldx=64, x_scales=4096, rows=None, w_codes=4096, ldw=64, w_group=512 * 64, w_scales=4096, w_scale_group=512, offsets=4096, y=4096,
             ldy=512, ws=4096, ws_bytes=1 << 34, x_rows=20, P=20, G=3, N=512, K=60, y_type=0)
    d.update(kw)
    return cm.lib.coli_i8_product(cm.I8ProductArgs(*(d[f] for f, _ in cm.I8ProductArgs._fields_)), None)


@pytest.mark.parametrize("code,kw", [
    (cm.COLI_EINVAL, dict(P=-1)), (cm.COLI_EINVAL, dict(x_rows=-1)), (cm.COLI_EINVAL, dict(G=0)), (cm.COLI_EINVAL, dict(N=0)), (cm.COLI_EINVAL, dict(K=0)),
    (cm.COLI_EINVAL, dict(y_type=3)), (cm.COLI_EINVAL, dict(ldx=48)), (cm.COLI_EINVAL, dict(ldw=48)), (cm.COLI_EINVAL, dict(ldy=511)),
    (cm.COLI_EINVAL, dict(w_group=-16)), (cm.COLI_EINVAL, dict(w_scale_group=-1)), (cm.COLI_EINVAL, dict(offsets=None)), (cm.COLI_EINVAL, dict(x_rows=19)),
    (cm.COLI_EINVAL, dict(x_codes=None)), (cm.COLI_EINVAL, dict(w_scales=None)), (cm.COLI_EINVAL, dict(y=None)), (cm.COLI_EINVAL, dict(ws=None)),
    (cm.COLI_EUNSUPPORTED, dict(K=131072, ldx=131072, ldw=131072)), (cm.COLI_EUNSUPPORTED, dict(G=1025)), (cm.COLI_EUNSUPPORTED, dict(P=1 << 26, x_rows=1 << 26)),
    (cm.COLI_EUNSUPPORTED, dict(N=1 << 26, ldy=1 << 26)), (cm.COLI_EALIGN, dict(x_codes=4104)), (cm.COLI_EALIGN, dict(w_codes=4104)),
    (cm.COLI_EALIGN, dict(ldx=72)), (cm.COLI_EALIGN, dict(ldw=72)), (cm.COLI_EALIGN, dict(w_group=512 * 64 + 8)), (cm.COLI_EALIGN, dict(offsets=4100)),
    (cm.COLI_EWORKSPACE, dict(ws_bytes=10000)), (cm.COLI_EWORKSPACE, dict(P=3, ws_bytes=8000)), (cm.COLI_OK, dict(P=0, x_codes=None)),
])
def test_product_refuses(code, kw):
    assert c_product(**kw) == code


def test_workspace_sizes():
    for f, bad in ((lambda T: cm.coli_moe_select_workspace_size(T, 6144, 256), (cm.coli_moe_select_workspace_size(4, 100, 8), cm.coli_moe_select_workspace_size(4, 64, 1025))),
                   (lambda T: cm.coli_moe_group_workspace_size(T, 8, 256), (cm.coli_moe_group_workspace_size(4, 33, 8), cm.coli_moe_group_workspace_size(1 << 30, 4, 8))),
                   (lambda T: cm.coli_i8_product_workspace_size(T, 6144), (cm.coli_i8_product_workspace_size(4, 131072), cm.coli_i8_product_workspace_size(4, 0)))):
        sizes = [f(T) for T in (0, 1, 7, 8, 9, 32, 33, 64, 65, 100, 128, 700, 5000, 70000)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])) and sizes[0] >= 8704      # serves every smaller call
        assert not any(bad) and f(-1) == 0
    for new in (lambda: cm.new_select_workspace(4, 100, 8, "cpu"), lambda: cm.new_group_workspace(4, 33, 8, "cpu"), lambda: cm.new_i8_product_workspace(4, 0, "cpu")):
        with pytest.raises(cm.ColiError):
            new()
