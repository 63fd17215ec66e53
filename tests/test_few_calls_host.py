"""More host-side checks of the calls for a few tokens (no GPU needed)."""
import pytest

from mxfp8_precision_gemms_fp8bw_gb300 import binding as B
from mxfp8_precision_gemms_fp8bw_gb300 import build
from mxfp8_precision_gemms_fp8bw_gb300 import few_binding as FB

P = 1 << 20  # a fake, 16-byte aligned "device" address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return FB.lib()


def test_self_tests_take_the_calls_arguments_and_a_limit(lib):
    n = lib.mx_few_linear_workspace_bytes(5, 64, 2048)
    linear = [P, 2 * P, 3 * P, 4, 5, 64, 2048, 4 * P, 5 * P, n]
    assert lib.fp8bw_selftest_few_linear(*linear, 2_000_000_001, None) == B.ERR_ARG
    assert "wait_ns" in B.last_error()
    assert lib.fp8bw_selftest_few_linear(*linear[:6], 40, *linear[7:], 0, None) == B.ERR_SHAPE
    n = lib.mx_few_moe_workspace_bytes(3, 8, 2, 64, 96)
    layer = [P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, 7 * P, 4, 3, 8, 2, 64, 96, 1, 1, 1, 0, 1, 1.0, 8 * P, 9 * P, n]
    assert lib.fp8bw_selftest_few_moe(*layer, 2_000_000_001, None) == B.ERR_ARG
    assert lib.fp8bw_selftest_few_moe(*layer[:7], 5, *layer[8:], 0, None) == B.ERR_ARG
