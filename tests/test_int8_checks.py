"""What the 8-bit integer entry points and their test support refuse on the
host (no GPU needed)."""
import bit_codebook_quantized_router_b200 as q4
from bit_codebook_quantized_router_b200 import _lib


def test_selftest_hold_rejects_bad_times():
    for us in (0, 3000001):
        assert q4.lib().moe_q4_selftest_hold(us, None) == _lib.EINVAL
