"""Where the product's launches would pass 2^32 threads the call is refused, and not before (no GPU:
the size call checks what the launches do)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    from clebsch_gordan_tensor_cgtp_amd import _lib
    _lib.lib()
    return _lib


def test_rows_of_the_longest_calls(L):
    b = ctypes.c_size_t()
    size = lambda *a: L.lib().cgtp_linear_act_workspace_size(*a, ctypes.byref(b))  # noqa: E731
    most = (1 << 30) - 1
    # 256 threads to 64 rows of 65 to 128 fp32 inputs: 2^24 blocks are too many
    for K in (65, 128):
        assert size(L.CGTP_F32, most, K, 8, 0) == L.CGTP_ERR_UNSUPPORTED
        assert size(L.CGTP_F32, most - 62, K, 8, 0) == L.CGTP_ERR_UNSUPPORTED
        assert size(L.CGTP_F32, most - 63, K, 8, 0) == L.CGTP_OK
    # 128 rows to a block elsewhere
    assert size(L.CGTP_F32, most, 64, 8, 0) == L.CGTP_OK and size(L.CGTP_BF16, most, 128, 8, 0) == L.CGTP_OK
