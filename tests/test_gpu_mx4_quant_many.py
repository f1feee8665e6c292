"""MX4 quantisation and its inverse in calls of many rows, on both sides of the
rule that gives a warp a longer run of a row: rows that fill such runs and rows
that do not, with and without 16-byte aligned strides.  Exact, on a sample of
rows against the oracle and on all rows against the values themselves."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402
from oracle import mx4  # noqa: E402

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T,K,pad", [(1600, 6144, 0), (1700, 6144, 0), (1700, 6144, 3), (6000, 2048, 8), (6000, 1568, 0), (6000, 1504, 0),
                                     (6000, 1568, 1), (20000, 512, 0), (3000, 4128, 0), (700, 16384, 0)])
def test_many_rows(dtype, T, K, pad):
    g = torch.Generator("cuda").manual_seed(T + K)
    buf = torch.full((T, K + pad), float("nan"), device="cuda").to(DTYPES[dtype])
    x = buf[:, :K]
    x.copy_(torch.randn(T, K, generator=g, device="cuda") * torch.exp2(torch.randint(-6, 5, (T, K // 32), generator=g, device="cuda").float())
            .repeat_interleave(32, 1))
    codes = torch.full((T, K // 2), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((T, K // 32), 0xAB, dtype=torch.uint8, device="cuda")
    cm.coli_mx4_quantize(x, codes, scales)
    rows = sorted({0, 1, T // 3, T - 2, T - 1, *np.random.default_rng(T).integers(0, T, 40).tolist()})
    c, b = mx4.quantize(x[rows].double().cpu().numpy())
    assert np.array_equal(codes[rows].cpu().numpy(), c) and np.array_equal(scales[rows].cpu().numpy(), b)
    out = torch.full((T, K + pad), 777.0, device="cuda").to(DTYPES[dtype])
    cm.coli_mx4_dequantize(codes, scales, out[:, :K])
    assert (out[:, K:] == 777.0).all()
    # the values of the codes are their own nearest codes: a second pass finds the same
    again, scales2 = torch.zeros_like(codes), torch.zeros_like(scales)
    cm.coli_mx4_quantize(out[:, :K], again, scales2)
    assert torch.equal(again, codes) and torch.equal(scales2, scales)
    assert torch.equal(out[rows, :K].cpu(), torch.from_numpy(mx4.values(c, b)).to(DTYPES[dtype]))
