"""Products without activation rows: every row of y of a group is out of range."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402
from test_gpu_i8 import make  # noqa: E402


@pytest.mark.parametrize("P,N,K", [(4, 70, 96), (50, 70, 96), (1500, 6200, 2100)])
def test_no_activation_rows(P, N, K):
    _, _, w, ws = make(1, 3, N, K, 1)
    x, xs = torch.empty(0, K, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda")
    rows, space = torch.arange(P, dtype=torch.int32, device="cuda"), cm.new_i8_product_workspace(P, K)
    for cuts, live in (([1, 2, 2, P - 1], slice(1, P - 1)), ([0, 0, 0, 0], slice(0, 0))):
        y = torch.full((P, N), 3.0, device="cuda")
        cm.coli_i8_product(x, xs, w, ws, y, space, offsets=torch.tensor(cuts, dtype=torch.int32, device="cuda"), rows=rows)
        want = torch.full_like(y, 3.0)
        want[live] = float("nan")
        assert torch.equal(torch.nan_to_num(y, nan=-7.0), torch.nan_to_num(want, nan=-7.0))
        assert cm.coli_moe_status(space) == (cm.STATUS_BADIDX if live.stop else 0)
