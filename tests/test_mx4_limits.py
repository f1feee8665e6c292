"""Limits of the MX4 entry points that are answered on the host, before any
launch (the addresses here are never read)."""
import pytest

pytest.importorskip("torch")

import quantized_expert_ffn_sigmoid_gb300 as cm  # noqa: E402

MAX_K = 1 << 30
LONGEST = (1 << 31) - 32   # the longest multiple of 32 an int32 holds


@pytest.mark.parametrize("K", [MAX_K + 32, (1 << 31) - 2048, (1 << 31) - 512, LONGEST])
def test_rows_beyond_the_longest_are_refused(K):
    lib = cm.lib
    assert lib.coli_mx4_quantize(16, 0, K, 1, K, 16, 16, None) == cm.COLI_EUNSUPPORTED
    assert lib.coli_mx4_dequantize(16, 16, 1, K, 16, 0, K, None) == cm.COLI_EUNSUPPORTED
    assert lib.coli_mx4_product(16, 16, 1, 16, 16, 1, 8, K, None, 16, 0, 8, 16, 8704, None) == cm.COLI_EUNSUPPORTED


@pytest.mark.parametrize("K", [32, MAX_K])
def test_rows_up_to_the_longest_pass_the_checks(K):
    lib = cm.lib
    assert lib.coli_mx4_quantize(None, 0, K, 0, K, None, None, None) == cm.COLI_OK
    assert lib.coli_mx4_dequantize(None, None, 0, K, None, 0, K, None) == cm.COLI_OK
    assert lib.coli_mx4_product(None, None, 0, None, None, 1, 8, K, None, None, 0, 8, None, 0, None) == cm.COLI_OK
