"""The MX4 bindings look at every tensor before the library is called.  No GPU:
stand-ins answer what the bindings ask of a tensor, and a recorder takes the
library's place, so nothing is launched whatever passes."""
import gc
import types
import weakref

import pytest

torch = pytest.importorskip("torch")

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402


class Stand:
    """What a GPU tensor of this shape and type would answer."""

    def __init__(self, *shape, dtype=torch.uint8, index=0, strides=None):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, index
        dense, n = [], 1
        for s in reversed(shape):
            dense.insert(0, n)
            n *= s
        self.strides = tuple(dense) if strides is None else strides
        self.dense = self.strides == tuple(dense)
        self.count = n

    @property
    def device(self):
        return f"cuda:{self.index}" if self.index >= 0 else "cpu"

    @property
    def is_cuda(self):
        return self.index >= 0

    @property
    def nbytes(self):
        return self.count * self.element_size()

    def get_device(self):
        return self.index

    def stride(self):
        return self.strides

    def is_contiguous(self):
        return self.dense

    def numel(self):
        return self.count

    def dim(self):
        return len(self.shape)

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def data_ptr(self):
        return 256 if self.count else 0


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(cm, "lib", rec)
    cm._torch_names()
    monkeypatch.setattr(cm, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(cm, "_raw_device", lambda: 0, raising=False)
    return rec.calls


def cfg(ep_rank=0, ep_size=0, **kw):
    d = dict(hidden=256, n_experts=16, n_groups=1, topk_group=1, top_k=4, inter=128, n_shared=1, shared_inter=384,
             weight_bits=4, routed_scaling_factor=2.5)
    d.update(kw)
    return cm.Cfg.of(types.SimpleNamespace(**d), ep_rank, ep_size)


def records(n, hidden=256, inter=128):
    return Stand(n, 3 * inter * hidden // 2), Stand(n, 3 * inter * hidden // 32)


def layer_args(T=3, hidden=256, k=4):
    f = torch.float32
    return [Stand(T, hidden, dtype=torch.bfloat16), Stand(T, k, dtype=torch.int32), Stand(T, k, dtype=f), Stand(T, hidden, dtype=f),
            Stand(1 << 20)]


# ------------------------------------------------------------------- the records
@pytest.mark.parametrize("c,n", [(cfg(), 16), (cfg(n_shared=0), 16), (cfg(0, 3), 6), (cfg(1, 3), 5), (cfg(2, 3), 5), (cfg(0, 16), 1)])
def test_records_of_the_configuration_are_taken(calls, c, n):
    w = cm.make_mx4_weights(*records(n), *records(c.n_shared, inter=384))
    cm.coli_mx4_forward(c, w, *layer_args())
    assert calls == ["coli_mx4_forward"]


def test_shared_records_are_looked_at_where_they_are_used(calls):
    w = cm.make_mx4_weights(*records(16))                      # no shared experts at all: the library's own answer
    cm.coli_mx4_forward(cfg(n_shared=0), w, *layer_args())
    w = cm.make_mx4_weights(*records(5), *records(7))          # a shard that owns no shared experts ignores them
    cm.coli_mx4_forward(cfg(1, 3), w, *layer_args())
    assert len(calls) == 2


@pytest.mark.parametrize("c,routed,shared", [
    (cfg(), records(15), records(1, inter=384)),                                       # an expert short
    (cfg(), records(6), records(1, inter=384)),                                        # a shard's records, the whole layer's configuration
    (cfg(1, 3), records(16), ()),                                                      # the whole layer's, a shard's configuration
    (cfg(), records(16, inter=64), records(1, inter=384)),                             # another layer's inter
    (cfg(), records(16, hidden=128), records(1, inter=384)),
    (cfg(), (records(16)[0], records(15)[1]), records(1, inter=384)),                  # scales of another count
    (cfg(), records(16), records(1, inter=128)),                                       # shared_inter
    (cfg(n_shared=2), records(16), records(1, inter=384)),
    (cfg(), records(16), (records(1, inter=384)[0], records(1, inter=128)[1])),
])
def test_other_records_are_refused(calls, c, routed, shared):
    w = cm.make_mx4_weights(*routed, *shared)
    with pytest.raises(ValueError, match="record"):
        cm.coli_mx4_forward(c, w, *layer_args())
    assert not calls


def test_weights_are_dense_bytes_on_the_gpu():
    e, s = records(16)
    for bad in (Stand(16, 3 * 128 * 256 // 2, index=-1), Stand(16, 3 * 128 * 256 // 2, strides=(1 << 20, 1)),
                Stand(16, 3 * 128 * 256 // 2, dtype=torch.int32)):
        with pytest.raises(ValueError, match="experts"):
            cm.make_mx4_weights(bad, s)
        with pytest.raises(ValueError, match="expert_scales"):
            cm.make_mx4_weights(e, bad)
        with pytest.raises(ValueError, match="shared"):
            cm.make_mx4_weights(e, s, bad, s)
        with pytest.raises(ValueError, match="shared_scales"):
            cm.make_mx4_weights(e, s, e, bad)


def test_the_struct_keeps_its_tensors_alive():
    e, s = records(16)
    seen = [weakref.ref(t) for t in (e, s)]
    w = cm.make_mx4_weights(e, s)
    del e, s
    gc.collect()
    assert all(r() is not None for r in seen)
    del w
    gc.collect()
    assert all(r() is None for r in seen)


# --------------------------------------------------------------------- the types
def test_ids_weights_and_offsets_have_their_types(calls):
    f, i = torch.float32, torch.int32
    w = cm.make_mx4_weights(*records(16), *records(1, inter=384))
    x, idx, tw, y, ws = layer_args()
    for bad_idx, bad_w in ((tw, idx), (tw, tw), (idx, idx), (Stand(3, 4, dtype=torch.uint32), tw)):
        with pytest.raises(TypeError, match="topk_"):
            cm.coli_mx4_forward(cfg(), w, x, bad_idx, bad_w, y, ws)
    with pytest.raises(TypeError, match="offsets"):
        cm.coli_mx4_product(Stand(5, 32), Stand(5, 2), Stand(2, 8, 32), Stand(2, 8, 2), Stand(5, 8, dtype=f), Stand(8704), offsets=Stand(3, dtype=f))
    h = Stand(3, 64, dtype=f)
    for kw in (dict(post_w=Stand(64, dtype=i), y=h), dict(pre_w=Stand(64, dtype=i))):
        with pytest.raises(TypeError, match=next(iter(kw))):
            cm.coli_moe_block_norm(h, n_out=h, **kw)
    assert not calls
    cm.coli_mx4_product(Stand(5, 32), Stand(5, 2), Stand(2, 8, 32), Stand(2, 8, 2), Stand(5, 8, dtype=f), Stand(8704), offsets=Stand(3, dtype=i))
    cm.coli_moe_block_norm(h, y=h, n_out=h, post_w=Stand(64, dtype=f), pre_w=Stand(64, dtype=f))
    assert len(calls) == 2


# ------------------------------------------------------------------- the devices
def every_call(index=0, other=None, at=None):
    """One valid call of each entry point on GPU `index`; argument `other` of it on GPU `at`."""
    f = torch.float32

    def place(name, *shape, dtype=torch.uint8):
        return Stand(*shape, dtype=dtype, index=at if name == other else index)

    def layer(codes):
        rec = [place(n, *t.shape) for n, t in zip(("experts", "expert_scales", "shared", "shared_scales"), (*records(16), *records(1, inter=384)))]
        w = cm.make_mx4_weights(*rec)
        x = place("x", 3, 128) if codes else place("x", 3, 256, dtype=f)
        cm.coli_mx4_forward(cfg(), w, x, place("topk_idx", 3, 4, dtype=torch.int32), place("topk_w", 3, 4, dtype=f), place("y", 3, 256, dtype=f),
                            place("ws", 1 << 20), x_scales=place("x_scales", 3, 8) if codes else None)

    def norm():
        h = lambda n: place(n, 3, 64, dtype=f)  # noqa: E731
        cm.coli_moe_block_norm(h("x"), y=h("y"), gate=h("gate"), x_out=h("x_out"), n_out=h("n_out"), post_w=place("post_w", 64, dtype=f),
                               pre_w=place("pre_w", 64, dtype=f), codes=place("codes", 3, 32), scales=place("scales", 3, 2))

    def channel_gate():
        cm.coli_moe_block_norm(place("x", 3, 64, dtype=f), y=place("y", 3, 64, dtype=f), gate=place("gate", 64, dtype=f),
                               n_out=place("n_out", 3, 64, dtype=f))

    return {
        "quantize": (("x", "codes", "scales"),
                     lambda: cm.coli_mx4_quantize(place("x", 3, 64, dtype=f), place("codes", 3, 32), place("scales", 3, 2))),
        "dequantize": (("codes", "scales", "out"),
                       lambda: cm.coli_mx4_dequantize(place("codes", 3, 32), place("scales", 3, 2), place("out", 3, 64, dtype=f))),
        "product": (("x_codes", "x_scales", "w_codes", "w_scales", "y", "ws", "offsets"),
                    lambda: cm.coli_mx4_product(place("x_codes", 5, 32), place("x_scales", 5, 2), place("w_codes", 2, 8, 32),
                                                place("w_scales", 2, 8, 2), place("y", 5, 8, dtype=f), place("ws", 8704),
                                                offsets=place("offsets", 3, dtype=torch.int32))),
        "layer": (("experts", "expert_scales", "shared", "shared_scales", "x", "topk_idx", "topk_w", "y", "ws"), lambda: layer(False)),
        "layer of codes": (("x", "x_scales"), lambda: layer(True)),
        "norm": (("x", "y", "gate", "x_out", "n_out", "post_w", "pre_w", "codes", "scales"), norm),
        "norm, channel gate": (("gate",), channel_gate),
    }


ARGUMENTS = [(call, name) for call, (names, _) in every_call().items() for name in names]


@pytest.mark.parametrize("at", [1, -1])
@pytest.mark.parametrize("call,name", ARGUMENTS)
def test_every_argument_is_on_the_same_gpu(calls, monkeypatch, call, name, at):
    monkeypatch.setattr(cm, "_raw_device", lambda: 0, raising=False)
    every_call()[call][1]()
    assert len(calls) == 1
    with pytest.raises(ValueError, match="GPU"):
        every_call(other=name, at=at)[call][1]()
    assert len(calls) == 1


@pytest.mark.parametrize("call", list(every_call()))
def test_the_tensors_gpu_is_the_current_one(calls, monkeypatch, call):
    monkeypatch.setattr(cm, "_raw_device", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="current"):
        every_call(index=1)[call][1]()
    assert not calls
    monkeypatch.setattr(cm, "_raw_device", lambda: 1, raising=False)
    every_call(index=1)[call][1]()
    assert len(calls) == 1


def test_a_given_stream_is_of_the_same_gpu(calls, monkeypatch):
    monkeypatch.setattr(cm, "_raw_device", lambda: 0, raising=False)
    args = Stand(3, 64, dtype=torch.float32), Stand(3, 32), Stand(3, 2)
    with pytest.raises(ValueError, match="stream"):
        cm.coli_mx4_quantize(*args, stream=types.SimpleNamespace(cuda_stream=7, device_index=1))
    assert not calls
    cm.coli_mx4_quantize(*args, stream=types.SimpleNamespace(cuda_stream=7, device_index=0))
    cm.coli_mx4_quantize(*args, stream=types.SimpleNamespace(cuda_stream=7))
    assert len(calls) == 2


def test_workspaces_are_dense(calls, monkeypatch):
    monkeypatch.setattr(cm, "_raw_device", lambda: 0, raising=False)
    sparse = Stand(8704, strides=(2,))
    with pytest.raises(ValueError, match="ws"):
        cm.coli_mx4_product(Stand(5, 32), Stand(5, 2), Stand(8, 32), Stand(8, 2), Stand(5, 8, dtype=torch.float32), sparse)
    w = cm.make_mx4_weights(*records(16), *records(1, inter=384))
    with pytest.raises(ValueError, match="ws"):
        cm.coli_mx4_forward(cfg(), w, *layer_args()[:4], sparse)
    assert not calls


# --------------------------------------------------------------------- the sizes
@pytest.mark.parametrize("n", [1 << 31, (1 << 32) + 64])
def test_sizes_beyond_32_bits_are_refused(calls, n):
    # the library counts rows and values in int32: a larger size must not arrive there as its low half
    f, u = torch.float32, lambda *s: Stand(*s)
    w = cm.make_mx4_weights(*records(16), *records(1, inter=384))
    x, idx, tw, y, ws = layer_args(T=n)
    for call in (lambda: cm.coli_mx4_quantize(Stand(1, n, dtype=f), u(1, n // 2), u(1, n // 32)),
                 lambda: cm.coli_mx4_quantize(Stand(n, 32, dtype=f), u(n, 16), u(n, 1)),
                 lambda: cm.coli_mx4_dequantize(u(1, n // 2), u(1, n // 32), Stand(1, n, dtype=f)),
                 lambda: cm.coli_mx4_dequantize(u(n, 16), u(n, 1), Stand(n, 32, dtype=f)),
                 lambda: cm.coli_mx4_product(u(n, 16), u(n, 1), u(8, 16), u(8, 1), Stand(n, 8, dtype=f), u(8704)),
                 lambda: cm.coli_mx4_product(u(1, 16), u(1, 1), u(n, 16), u(n, 1), Stand(1, n, dtype=f), u(8704)),
                 lambda: cm.coli_mx4_product(u(1, n // 2), u(1, n // 32), u(8, n // 2), u(8, n // 32), Stand(1, 8, dtype=f), u(8704)),
                 lambda: cm.coli_mx4_product(u(1, 16), u(1, 1), u(n, 1, 16), u(n, 1, 1), Stand(1, 1, dtype=f), u(8704),
                                             offsets=Stand(n + 1, dtype=torch.int32)),
                 lambda: cm.coli_mx4_forward(cfg(), w, x, idx, tw, y, ws),
                 lambda: cm.coli_moe_block_norm(Stand(n, 1, dtype=f), n_out=Stand(n, 1, dtype=f)),
                 lambda: cm.coli_moe_block_norm(Stand(1, n, dtype=f), n_out=Stand(1, n, dtype=f))):
        with pytest.raises(ValueError, match="32 bits"):
            call()
    with pytest.raises(ValueError, match="32 bits"):
        cm.coli_mx4_workspace_size(cfg(), n)
    assert not calls
