"""Bounded waits of the int8 products that run out: in the debug build one block
never asks for its first tokens, or sends its partial sums late.  The call
returns, its status word says MOE_Q4_ETIMEOUT, nothing is written out of bounds
and the next call is right."""
import ctypes

import pytest
import torch

import bit_codebook_quantized_router_b200 as q4
from bit_codebook_quantized_router_b200 import _lib, build
from tests.gpu_support import Guarded
from tests.test_gpu_int8 import F, mlp_weights, rows

pytestmark = pytest.mark.gpu

LIMIT_US, RELEASE_US = 5000, 2000000


@pytest.fixture(scope="module")
def L():
    lib = ctypes.CDLL(build.LIB_DEBUG)
    for name in ("moe_q4_linear_i8", "moe_q4_mlp_i8"):
        getattr(lib, name).argtypes = getattr(q4.lib(), name).argtypes
        getattr(lib, name).restype = ctypes.c_int
    lib.moe_q4_debug_withhold.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_uint]
    lib.moe_q4_debug_withhold.restype = ctypes.c_int
    lib.moe_q4_i8_status.argtypes, lib.moe_q4_i8_status.restype = [ctypes.c_void_p], ctypes.c_int
    return lib


@pytest.fixture
def withhold(L):
    def f(block, late=0):
        assert L.moe_q4_debug_withhold(block, late, LIMIT_US if block >= 0 else RELEASE_US) == _lib.OK

    yield f
    f(-1)


def stream():
    return torch.cuda.current_stream().cuda_stream


def linear(L, x, xs, w, ws, out, status):
    T, K = x.shape
    assert L.moe_q4_linear_i8(x.data_ptr(), x.stride(0), xs.data_ptr(), w.data_ptr(), w.stride(0), ws.data_ptr(), None, T,
                              w.shape[0], K, out.data_ptr(), 1, out.stride(0), _lib._ptr(status), stream()) == _lib.OK
    torch.cuda.synchronize()


# clusters of one to eight blocks, pairs alone, and two and four pairs a cluster
@pytest.mark.parametrize("T,N,K,blocks", [(64, 400, 2176, (0, 5, 31)), (100, 300, 1600, (1, 4)), (20, 30000, 1024, (7,)),
                                          (300, 400, 512, (0, 1, 3)), (200, 400, 2600, (0, 3)), (200, 100, 5200, (1, 6))])
def test_tokens_that_never_come(L, withhold, T, N, K, blocks):
    x, xs = q4.quant_rows(rows(T, K, 1, spread=False).cuda())
    w, ws = q4.quant_rows(rows(N, K, 2, spread=False).cuda())
    want = q4.linear_i8(x, xs, w, ws, dtype=F)
    out, status = Guarded((T, N), F), torch.zeros(1, dtype=torch.int32, device="cuda")
    for block in blocks:
        withhold(block)
        linear(L, x, xs, w, ws, out.view, status.zero_())
        assert status.item() == _lib.ETIMEOUT
        out.check("out")
        withhold(-1)
        linear(L, x, xs, w, ws, out.view, status.zero_())
        assert status.item() == _lib.OK and torch.equal(out.view, want)


@pytest.mark.parametrize("T,N,K,block", [(64, 400, 2176, 0), (64, 400, 2176, 13), (100, 300, 1600, 2)])
def test_partial_sums_that_come_late(L, withhold, T, N, K, block):
    # the other blocks of the cluster give up before the sums come, and stay
    # until they have come
    x, xs = q4.quant_rows(rows(T, K, 3, spread=False).cuda())
    w, ws = q4.quant_rows(rows(N, K, 4, spread=False).cuda())
    want = q4.linear_i8(x, xs, w, ws, dtype=F)
    out, status = Guarded((T, N), F), torch.zeros(1, dtype=torch.int32, device="cuda")
    withhold(block, late=1)
    linear(L, x, xs, w, ws, out.view, status)
    assert status.item() == _lib.ETIMEOUT
    out.check("out")
    withhold(-1)
    linear(L, x, xs, w, ws, out.view, status.zero_())
    assert status.item() == _lib.OK and torch.equal(out.view, want)


@pytest.mark.parametrize("T,H,I", [(64, 2560, 2176), (300, 512, 256)])
def test_mlp_whose_products_give_up(L, withhold, T, H, I):
    m = mlp_weights(H, I, 5)
    x, xs = q4.quant_rows(rows(T, H, 6, spread=False).cuda())
    want = q4.mlp_i8(m, x, xs, dtype=F)
    out, status = Guarded((T, H), F), torch.zeros(1, dtype=torch.int32, device="cuda")
    work = Guarded((q4.mlp_i8_workspace(m, T),), torch.uint8)
    for block, code in ((1, _lib.ETIMEOUT), (-1, _lib.OK)):
        withhold(block)
        status.zero_()
        assert L.moe_q4_mlp_i8(m.ref, x.data_ptr(), x.stride(0), xs.data_ptr(), T, out.view.data_ptr(), 1, H,
                               status.data_ptr(), work.view.data_ptr(), work.view.numel(), stream()) == _lib.OK
        torch.cuda.synchronize()
        assert status.item() == code
        out.check("out")
        work.check("workspace")
    assert torch.equal(out.view, want)


@pytest.mark.parametrize("T", [64, 300])
def test_calls_without_a_status_word(L, withhold, T):
    x, xs = q4.quant_rows(rows(T, 2176, 7, spread=False).cuda())
    w, ws = q4.quant_rows(rows(200, 2176, 8, spread=False).cuda())
    out = torch.empty((T, 200), device="cuda")
    assert L.moe_q4_i8_status(stream()) == _lib.OK
    withhold(0)
    linear(L, x, xs, w, ws, out, None)
    withhold(-1)
    linear(L, x, xs, w, ws, out, None)
    # a right call behind it does not hide it; returned once
    assert L.moe_q4_i8_status(stream()) == _lib.ETIMEOUT
    assert L.moe_q4_i8_status(stream()) == _lib.OK
    # a call with a word of its own reports there alone
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    withhold(0)
    linear(L, x, xs, w, ws, out, status)
    assert status.item() == _lib.ETIMEOUT and L.moe_q4_i8_status(stream()) == _lib.OK
    assert torch.equal(q4.linear_i8(x, xs, w, ws, dtype=F), q4.linear_i8(x, xs, w, ws, out=out))
    assert q4.i8_status() == _lib.OK and q4.i8_status(device=0, stream=torch.cuda.Stream()) == _lib.OK
