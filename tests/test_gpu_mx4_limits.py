"""MX4 rows of the longest length the entry points take (2**30 values): the
last stages, the last blocks and one block in the middle carry values, chosen
so that every sum is exact in fp32 whatever its order."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402

K = 1 << 30
PLACES = [0, 33, (1 << 29) + 7, K - 512, K - 31, K - 1]


def test_longest_row_there_and_back():
    x = torch.zeros(1, K, dtype=torch.bfloat16, device="cuda")
    x[0, PLACES] = torch.tensor([1.0, -2.0, 3.0, 0.5, 6.0, -1.5], dtype=torch.bfloat16, device="cuda")
    codes = torch.full((1, K // 2), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((1, K // 32), 0xAB, dtype=torch.uint8, device="cuda")
    cm.coli_mx4_quantize(x, codes, scales)
    out = torch.full_like(x, 777.0)
    cm.coli_mx4_dequantize(codes, scales, out)
    assert torch.equal(out, x)


def test_longest_product():
    x = torch.zeros(1, K // 2, dtype=torch.uint8, device="cuda")
    w = torch.zeros(2, K // 2, dtype=torch.uint8, device="cuda")
    xs = torch.full((1, K // 32), 127, dtype=torch.uint8, device="cuda")
    ws = torch.full((2, K // 32), 127, dtype=torch.uint8, device="cuda")
    for i, k in enumerate(PLACES):          # x: 1 at the places; w: 1, 2, 3, ... and all 0.5
        x[0, k // 2] |= 2 << 4 * (k % 2)
        w[0, k // 2] |= (i + 1) << 4 * (k % 2)
        w[1, k // 2] |= 1 << 4 * (k % 2)
    y = torch.full((1, 2), 777.0, device="cuda")
    ws_ = cm.new_mx4_product_workspace()
    cm.coli_mx4_product(x, xs, w, ws, y, ws_)
    assert cm.coli_moe_status(ws_) == 0
    assert y.tolist() == [[0.5 + 1.0 + 1.5 + 2.0 + 3.0 + 4.0, 3.0]]
