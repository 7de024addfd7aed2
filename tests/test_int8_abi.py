"""The 8-bit integer entry points refuse bad arguments on the host, before any
launch (no GPU needed)."""
import ctypes

import pytest
import torch

import bit_codebook_quantized_router_b200 as q4
from bit_codebook_quantized_router_b200 import _lib
from tests import int8_plain
from tests.test_abi import _layer

P, Q = 1 << 20, 1 << 21  # addresses that are never dereferenced: validation fails first
BF16, F32 = 0, 1


@pytest.fixture(scope="module")
def L():
    from bit_codebook_quantized_router_b200 import build
    build.build()
    return _lib.lib()


def test_quant_rows_refusals(L):
    ok = dict(x=P, xt=BF16, ldx=64, T=4, K=64, q=Q, ldq=64, scale=P, stream=None)
    f = lambda **k: L.moe_q4_quant_rows(*{**ok, **k}.values())  # noqa: E731
    for bad in (dict(x=None), dict(q=None), dict(scale=None), dict(xt=2), dict(xt=-1), dict(T=-1), dict(K=0),
                dict(ldx=63), dict(ldq=63), dict(x=P + 1), dict(x=P + 2, xt=F32), dict(scale=P + 2)):
        assert f(**bad) == _lib.EINVAL, bad
    assert f(T=0, x=None, q=None, scale=None) == _lib.OK
    assert f(K=(1 << 30) + 1, ldx=1 << 31, ldq=1 << 31) == _lib.ENOTSUP


def test_add_norm_refusals(L):
    ok = dict(x=P, xt=BF16, ldx=64, res=P, rt=F32, ldr=64, ro=Q, ldro=64, w=P, wt=BF16, eps=1e-6, T=4, H=64, out=P,
              ldo=64, q=Q, ldq=64, scale=P, stream=None)
    f = lambda **k: L.moe_q4_add_norm(*{**ok, **k}.values())  # noqa: E731
    for bad in (dict(x=None), dict(xt=3), dict(rt=3), dict(wt=3), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(T=-1), dict(H=0), dict(ldx=63), dict(ldr=63), dict(ldro=63),
                dict(ldo=63), dict(ldq=63), dict(ro=None), dict(res=None), dict(q=None), dict(scale=None),
                dict(out=None, q=None, scale=None), dict(out=Q, ro=Q), dict(x=P + 1), dict(res=P + 2),
                dict(ro=Q + 2), dict(w=P + 1), dict(out=P + 1), dict(scale=P + 1)):
        assert f(**bad) == _lib.EINVAL, bad
    assert f(T=0, x=None) == _lib.OK
    # in place only where a row's results go where that row was read
    for bad in (dict(ro=P, res=P, ldr=64, ldro=72), dict(x=P, ro=P, res=Q, rt=F32), dict(xt=F32, ro=P, res=Q, ldro=72),
                dict(x=P, out=P, xt=F32), dict(x=P, out=P, ldo=72)):
        assert f(**bad) == _lib.EINVAL, bad
    assert f(H=(1 << 30) + 1, **{k: 1 << 31 for k in ("ldx", "ldr", "ldro", "ldo", "ldq")}) == _lib.ENOTSUP


def test_linear_refusals(L):
    ok = dict(x=P, ldx=64, xs=P, w=Q, ldw=64, ws=P, bias=None, T=4, N=8, K=64, out=P, ot=BF16, ldo=8, status=None, stream=None)
    f = lambda **k: L.moe_q4_linear_i8(*{**ok, **k}.values())  # noqa: E731
    for bad in (dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(out=None), dict(T=-1), dict(N=0),
                dict(K=0), dict(ldx=48), dict(ldx=72), dict(ldw=48), dict(ldw=72), dict(ldo=7), dict(ot=2),
                dict(x=P + 8), dict(w=Q + 8), dict(xs=P + 2), dict(ws=P + 2), dict(bias=P + 2), dict(out=P + 1),
                dict(out=P + 2, ot=F32), dict(status=P + 2)):
        assert f(**bad) == _lib.EINVAL, bad
    # int32 sums of any codes: K to 131071
    assert f(K=131072, ldx=131072, ldw=131072) == _lib.ENOTSUP
    assert f(T=(1 << 30) + 1) == f(N=(1 << 30) + 1, ldo=1 << 31) == _lib.ENOTSUP
    assert f(T=0, x=None, out=None) == _lib.OK


def _mlp(H=64, I=32, gu=P, ldg=64, gus=P, dn=Q, ldd=32, ds=P):
    return _lib._MlpStruct(H, I, gu, ldg, gus, dn, ldd, ds)


def test_mlp_refusals(L):
    n = L.moe_q4_mlp_i8_workspace(ctypes.byref(_mlp()), 4)
    assert n > 0 and L.moe_q4_mlp_i8_workspace(ctypes.byref(_mlp()), 0) == 0
    assert L.moe_q4_mlp_i8_workspace(None, 4) == 0
    ok = dict(x=P, ldx=64, xs=P, T=4, out=P, ot=BF16, ldo=64, status=None, ws=P, n=n, stream=None)
    f = lambda m=_mlp(), **k: L.moe_q4_mlp_i8(ctypes.byref(m), *{**ok, **k}.values())  # noqa: E731
    for m in (_mlp(H=0), _mlp(I=0), _mlp(gu=None), _mlp(dn=None), _mlp(gus=None), _mlp(ds=None), _mlp(ldg=48),
              _mlp(ldg=72), _mlp(ldd=16), _mlp(ldd=40), _mlp(gu=P + 8), _mlp(ds=P + 1)):
        assert L.moe_q4_mlp_i8_workspace(ctypes.byref(m), 4) == 0
        assert f(m) == _lib.EINVAL
    assert f(_mlp(I=131072, ldd=131072)) == _lib.ENOTSUP
    for bad in (dict(x=None), dict(xs=None), dict(out=None), dict(T=-1), dict(ldx=48), dict(ldx=72), dict(ldo=63),
                dict(ot=5), dict(x=P + 8), dict(out=P + 1), dict(xs=P + 1), dict(status=P + 1)):
        assert f(**bad) == _lib.EINVAL, bad
    for bad in (dict(ws=None), dict(ws=P + 128), dict(n=n - 1)):
        assert f(**bad) == _lib.EWORKSPACE, bad
    assert f(T=0, x=None, ws=None, n=0) == _lib.OK


def test_forward_with_int8_shared_expert_refusals(L):
    st, keep = _layer()
    lay = ctypes.byref(st)
    good = _mlp(H=256, ldg=256)
    m = ctypes.byref(good)
    base = L.moe_q4_forward_workspace(lay, 4, 2)
    n = L.moe_q4_forward_ex_i8_workspace(lay, m, 4, 2)
    ng = L.moe_q4_forward_gated_i8_workspace(lay, m, 4, 2)
    assert base < n < ng
    wrong = ctypes.byref(_mlp(H=128, ldg=128))  # not the layer's H
    for bad in (wrong, None):
        assert L.moe_q4_forward_ex_i8_workspace(lay, bad, 4, 2) == 0
        assert L.moe_q4_forward_gated_i8_workspace(lay, bad, 4, 2) == 0
    ok = dict(x=P, xq=None, ldxq=0, xs=None, logits=P, T=4, k=2, out=P, o32=None, ids=None, w=None, c=None, ws=P, n=n,
              s=None)
    f = lambda mm=m, **k: L.moe_q4_forward_ex_i8(lay, mm, *{**ok, **k}.values())  # noqa: E731
    assert f(wrong) == f(None) == _lib.EINVAL
    for bad in (dict(x=None), dict(logits=None), dict(out=None), dict(xq=P), dict(xs=P), dict(xq=P, xs=P, ldxq=128),
                dict(xq=P, xs=P, ldxq=264), dict(xq=P + 8, xs=P, ldxq=256), dict(k=9)):
        assert f(**bad) == _lib.EINVAL, bad
    assert f(n=n - 1) == f(ws=None) == _lib.EWORKSPACE
    okg = dict(rw=P, x=P, xq=None, ldxq=0, xs=None, T=4, k=2, out=P, o32=None, lg=None, ids=None, w=None, c=None,
               ws=P, n=ng, s=None)
    g = lambda mm=m, **k: L.moe_q4_forward_gated_i8(lay, mm, *{**okg, **k}.values())  # noqa: E731
    assert g(wrong) == g(None) == _lib.EINVAL
    for bad in (dict(rw=None), dict(x=None), dict(out=None), dict(xq=P), dict(rw=P + 2)):
        assert g(**bad) == _lib.EINVAL, bad
    assert g(n=n) == _lib.EWORKSPACE


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((2, 32))
    s = torch.zeros(2)
    q = torch.zeros((2, 32), dtype=torch.int8)
    with pytest.raises(ValueError):
        q4.quant_rows(x)
    with pytest.raises(ValueError):
        q4.add_norm(x, None)
    with pytest.raises(ValueError):
        q4.linear_i8(q, s, q, s)
    with pytest.raises(ValueError):
        q4.MlpI8(q, s, q, s)


def test_plain_form_against_arithmetic_by_hand():
    # m = 254: quotients 127 v / 254 = v / 2, so odd values are ties
    codes, m = int8_plain.quant(torch.tensor([[254.0, 1, 3, -1, -3, 5, 0]], dtype=torch.float64))
    assert m.item() == 254 and codes.tolist() == [[127, 0, 2, 0, -2, 2, 0]]
    # the norm of a constant row c is weight (up to eps), its codes the weight's
    r, p, codes, s = int8_plain.add_norm(torch.full((1, 4), 2.0), torch.tensor([1.0, 0.5, -1.0, 0.25]), 1e-12)
    assert torch.allclose(p, torch.tensor([[1.0, 0.5, -1.0, 0.25]], dtype=torch.float64), atol=1e-12)
    assert codes.tolist() == [[127, 64, -127, 32]]
