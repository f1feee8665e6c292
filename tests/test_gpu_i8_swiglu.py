"""Codes after SwiGLU are the exact rounding of the fp32 values silu(gate) * up.

From a gate of 18 on, exp(-gate) < 2^-25, so 1 + exp(-gate) is 1 in fp32 and silu(gate) is the gate itself: the
value is the fp32 product gate * up, known here bit for bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402
from oracle import token8  # noqa: E402


def check(gate, up, pad=0):
    """gate, up [T, K] of one torch type, all gates of at least 18."""
    T, K = gate.shape
    x = torch.zeros(T, 2 * K + pad, dtype=gate.dtype, device="cuda")[:, :2 * K]
    x[:, :K], x[:, K:] = gate.cuda(), up.cuda()
    codes, scales = torch.empty(T, K, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    cm.coli_i8_quantize(x, codes, scales, swiglu=True)
    v = gate.float() * up.float()                            # one fp32 rounding, as in the kernel
    q, _ = token8.quantize(v.double().numpy())
    assert np.array_equal(codes.cpu().numpy(), q), int((codes.cpu().numpy() != q).sum())
    assert np.array_equal(scales.cpu().numpy(), v.abs().amax(-1).numpy() / np.float32(127.0))


@pytest.mark.parametrize("top", [1.0, 3.1415927, 0.73, 1e-20, 2.3e30])
@pytest.mark.parametrize("gate", [18.0, 64.0, 128.0])
def test_next_to_the_middle(top, gate):
    # every neighbourhood of a middle between two codes, for several maxima that are no powers of two
    mid = ((np.arange(-127, 127) + 0.5) * np.float64(np.float32(top)) / 127.0 / gate).astype(np.float32)
    u = np.concatenate([np.nextafter(mid, np.float32(-np.inf)), mid, np.nextafter(mid, np.float32(np.inf)), [np.float32(top / gate)]])[None]
    u = torch.from_numpy(u.astype(np.float32))
    check(torch.full_like(u, gate), u)


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,K,pad", [(40, 1, 0), (30, 7, 1), (64, 1000, 0), (50, 2048, 8), (5, 9000, 0)])
def test_random_rows(T, K, pad, name):
    gen = torch.Generator().manual_seed(T * K)
    dtype = dict(f32=torch.float32, bf16=torch.bfloat16, f16=torch.float16)[name]
    gate = (18 + 40 * torch.rand(T, K, generator=gen)).to(dtype).clamp(min=18)
    up = torch.randn(T, K, generator=gen).to(dtype)
    if K > 2:
        # the row's largest value and, of the same gate, its half: the middle of 63 and 64
        gate[:, :2], up[:, 0] = 64.0, 8.0
        up[:, 1] = -up[:, 0] / 2
    check(gate, up, pad)
