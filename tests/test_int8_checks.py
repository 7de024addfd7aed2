"""What the 8-bit integer entry points and their test support refuse on the
host (no GPU needed)."""
import numpy as np
import pytest
import torch

import bit_codebook_quantized_router_b200 as q4
from bit_codebook_quantized_router_b200 import _lib


@pytest.fixture(scope="module")
def L():
    from bit_codebook_quantized_router_b200 import build
    build.build()
    return _lib.lib()


def test_selftest_hold_rejects_bad_times(L):
    for us in (0, 3000001):
        assert L.moe_q4_selftest_hold(us, None) == _lib.EINVAL


class OnDevice:
    """What the binding asks of a tensor on CUDA device `dev`, without one (its memory is never used)."""

    def __init__(self, shape, dtype, dev, strides=None):
        self.shape, self.dtype, self.dev = torch.Size(shape), dtype, dev
        self.strides = strides or tuple(int(np.prod(shape[i + 1:])) for i in range(len(shape)))
        self.device, self.is_cuda = torch.device("cuda", dev), True

    def get_device(self):
        return self.dev

    def dim(self):
        return len(self.shape)

    def numel(self):
        return int(np.prod(self.shape))

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]

    def is_contiguous(self):
        return self.strides == tuple(int(np.prod(self.shape[i + 1:])) for i in range(len(self.shape)))

    def data_ptr(self):
        return 1 << 20


def layer_on(dev, E=2, H=64, I=32):
    u = lambda *s: OnDevice(s, torch.uint8, dev)  # noqa: E731
    return q4.Layer(u(E, I, H // 2), u(E, I, H // 32), u(E, I, H // 2), u(E, I, H // 32), u(E, H, I // 2), u(E, H, I // 32),
                    np.linspace(0.1, 2, 8, dtype=np.float32), np.zeros(E, np.uint8))


def mlp_on(dev, H=64, I=32):
    f = lambda n: OnDevice((n,), torch.float32, dev)  # noqa: E731
    return q4.MlpI8(OnDevice((2 * I, H), torch.int8, dev), f(2 * I), OnDevice((H, I), torch.int8, dev), f(H))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("layer_dev,mlp_dev,row_dev,scale_dev", [(0, 1, None, None), (1, 0, None, None), (1, 1, None, None),
                                                                 (0, 0, 1, 1), (0, 0, 0, 1), (0, 0, 1, 0)])
def test_a_forward_refuses_parts_on_different_devices(gated, layer_dev, mlp_dev, row_dev, scale_dev):
    T, H, E = 4, 64, 2
    x = OnDevice((T, H), torch.bfloat16, 0)
    rows = {} if row_dev is None else dict(xq=OnDevice((T, H), torch.int8, row_dev), x_scale=OnDevice((T,), torch.float32, scale_dev))
    with pytest.raises(ValueError, match="cuda:|device"):
        if gated:
            q4.forward_gated(layer_on(layer_dev), mlp_on(mlp_dev), OnDevice((E, H), torch.bfloat16, 0), x, 2, **rows)
        else:
            q4.forward_ex(layer_on(layer_dev), mlp_on(mlp_dev), x, OnDevice((T, E), torch.float32, 0), 2, **rows)


def test_parts_on_one_device_pass():
    x, xq, s = OnDevice((4, 64), torch.bfloat16, 1), OnDevice((4, 64), torch.int8, 1), OnDevice((4,), torch.float32, 1)
    assert _lib._shared_rows(layer_on(1), mlp_on(1), x, xq, s) == 64
    assert _lib._shared_rows(layer_on(1), mlp_on(1), x, None, None) == 0


def test_mlp_refuses_a_workspace_that_repeats_its_bytes():
    x, s, out = OnDevice((4, 64), torch.int8, 0), OnDevice((4,), torch.float32, 0), OnDevice((4, 64), torch.bfloat16, 0)
    m = mlp_on(0)
    ws = OnDevice((q4.mlp_i8_workspace(m, 4),), torch.uint8, 0, strides=(0,))
    with pytest.raises(ValueError, match="contiguous"):
        q4.mlp_i8(m, x, s, out=out, ws=ws)
