"""Sizes at the ends of what the 8-bit token and channel operators take.  No GPU: the library looks at sizes and
addresses before any CUDA call, and answers COLI_ECUDA where it would have launched."""
import pytest

pytest.importorskip("torch")

import torch  # noqa: E402

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402
from test_i8_bindings import c_product, c_select  # noqa: E402

if torch.cuda.is_available():
    pytest.skip("addresses that are none: only where nothing can be launched", allow_module_level=True)


def test_no_activation_rows():
    # every row of y is out of range then, which is no reason to refuse the call
    for P in (3, 20):
        assert c_product(P=P, x_rows=0, x_codes=None, x_scales=None, rows=4096) == cm.COLI_ECUDA
        assert c_product(P=P, x_rows=1, x_codes=None, rows=4096) == cm.COLI_EINVAL
        assert c_product(P=P, x_rows=0, x_codes=None, x_scales=None, rows=None) == cm.COLI_EINVAL     # (P > x_rows)


def test_positions_of_a_selection_from_the_hidden_state():
    most = 65535 * 64
    kw = dict(router_w=4096, hidden=64, ws_bytes=1 << 50)
    assert c_select(T=most, **kw) == cm.COLI_ECUDA and c_select(T=most + 1, **kw) == cm.COLI_EUNSUPPORTED
    assert c_select(T=most + 1) == cm.COLI_ECUDA                       # from logits: any number
    assert cm.coli_moe_select_workspace_size(most, 64, 64) > 0 == cm.coli_moe_select_workspace_size(most + 1, 64, 64)
