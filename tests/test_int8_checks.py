"""What the 8-bit integer entry points and their test support refuse on the
host (no GPU needed)."""
import pytest

from bit_codebook_quantized_router_b200 import _lib


@pytest.fixture(scope="module")
def L():
    from bit_codebook_quantized_router_b200 import build
    build.build()
    return _lib.lib()


def test_selftest_hold_rejects_bad_times(L):
    for us in (0, 3000001):
        assert L.moe_q4_selftest_hold(us, None) == _lib.EINVAL
