"""GPU parity of the 8-bit integer operators against their plain 64-bit forms:
codes and integer sums exact, the rest within the roundings counted at each
test."""
import threading

import pytest
import torch

import bit_codebook_quantized_router_b200 as q4
from tests import int8_plain as plain
from tests.gpu_support import Guarded

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(T, K, seed, dtype=BF, spread=True):
    """Rows with outlier channels, a row of zeros and rows of very different size."""
    x = torch.randn((T, K), generator=gen(seed))
    x[:, 5::37] *= 9
    if spread and T > 3:
        x[1] = 0
        x[2] *= 1e-4
        x[3] *= 1e4
    return x.to(dtype)


def strided(t, ld, offset=0, fill=float("nan")):
    """t on the GPU with row stride ld, `offset` elements into its memory, in
    the midst of `fill`."""
    T, K = t.shape
    big = torch.full((offset + T * ld + 64,), fill if t.dtype.is_floating_point else 77, dtype=t.dtype, device="cuda")
    v = big[offset:offset + T * ld].view(T, ld)[:, :K]
    v.copy_(t)
    return v


def check_codes(q, codes):
    same = q.cpu().double() == codes
    assert bool(same.all()), (~same).nonzero()[:4].tolist()


# ---- rows to codes ------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,K", [(1, 1), (1, 6144), (3, 7), (5, 8), (9, 129), (4, 256), (4, 257), (300, 523),
                                 (7, 2048), (400, 2048), (2, 8200), (2, 40001), (1, 65536), (301, 6144)])
def test_quant_rows(T, K, dtype):
    x = rows(T, K, T + K, dtype)
    q, s = q4.quant_rows(x.cuda())
    codes, m = plain.quant(x.double())
    check_codes(q, codes)
    # the scale is one correctly rounded fp32 division
    assert torch.equal(s.cpu(), m.float() / 127)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("ldx,offset,ldq", [(72, 0, 80), (72, 8, 72), (65, 0, 64), (72, 1, 64), (71, 3, 67), (80, 4, 66)])
def test_quant_rows_strides_and_bounds(ldx, offset, ldq, dtype):
    x = rows(50, 64, 11, dtype)
    q, s = Guarded((50, ldq), torch.int8), Guarded((50,), F)
    q.view.fill_(99)
    q4.quant_rows(strided(x, ldx, offset), q=q.view[:, :64], scale=s.view)
    q.check("codes")
    s.check("scales")
    check_codes(q.view[:, :64], plain.quant(x.double())[0])
    assert bool((q.view[:, 64:] == 99).all())  # what lies between the rows stays


def test_quant_rows_ties_and_borders():
    # m = 254 and 2 m: every odd value is a tie; and values one bf16 / fp32 step beside a tie
    v = torch.arange(-254, 255, dtype=F)
    x = torch.stack([v, v * 2.0 ** -60, v * 2.0 ** 100])
    for dtype in (F, BF):
        d = x.to(dtype)
        q, _ = q4.quant_rows(d.cuda())
        check_codes(q, plain.quant(d.double())[0])
    near = torch.nextafter(v, torch.full_like(v, 1e9)), torch.nextafter(v, torch.full_like(v, -1e9))
    x = torch.stack([torch.cat([torch.full((1,), 254.0), n.clamp(-254, 254)]) for n in near])
    q, _ = q4.quant_rows(x.cuda())
    check_codes(q, plain.quant(x.double())[0])
    # fp32 quotients at random with a maximum of many bits: borders from both sides
    x = torch.rand((64, 4096), generator=gen(5)) * 1.7
    q, _ = q4.quant_rows(x.cuda())
    check_codes(q, plain.quant(x.double())[0])


@pytest.mark.parametrize("m", [1e-30, 1e-36, 1e-38, 1e-44, 1e38, 3.4e38])
def test_quant_rows_smallest_and_largest(m):
    # (the fp32 steps of linspace overflow at the largest: a row that is not finite)
    for x in (torch.linspace(-m, m, 65), torch.linspace(-m, m, 65, dtype=torch.float64).float()):
        x = x.repeat(3, 1).contiguous()
        q, s = q4.quant_rows(x.cuda())
        codes, top = plain.quant(x.double())
        check_codes(q, codes)
        assert torch.allclose(s.cpu(), top.float() / 127, rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("K", [40, 41, 3000, 40001])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_rows_that_are_not_finite(bad, K):
    x = rows(6, K, 3, F)
    x[2, K // 2] = bad
    x[4, :] = bad
    q, s = q4.quant_rows(x.cuda())
    assert torch.isnan(s.cpu()).tolist() == [False, False, True, False, True, False]
    fine = [0, 1, 3, 5]
    check_codes(q[fine], plain.quant(x[fine].double())[0])
    assert not q[[2, 4]].any()
    r, out, q, s = q4.add_norm(x.cuda(), None, residual=torch.zeros_like(x).cuda())
    assert torch.isnan(s.cpu()).tolist() == [False, False, True, False, True, False]
    assert torch.isnan(out[[2, 4]]).all() and not q[[2, 4]].any() and torch.isfinite(out[fine]).all()
    # every product with such a row is NaN, the others are not touched
    w, ws = q4.quant_rows(rows(9, K, 4, spread=False).cuda())
    y = q4.linear_i8(q, s, w, ws)
    assert torch.isnan(y[[2, 4]]).all() and torch.isfinite(y[fine]).all()


# ---- residual, norm, codes ----------------------------------------------------

def check_add_norm(x, w, eps, res, got, H):
    r, out, q, s = got
    er, ep, codes, es = plain.add_norm(x, w, eps, res)
    if res is not None:
        assert torch.equal(r.cpu(), er)
    if q is not None:
        check_codes(q, codes)
    # The factor: squares and their sum, at most H / 1024 + 48 additions deep,
    # halved by the root; the mean, eps and the root are 2^-24 to 2^-22 each.
    f = (H / 1024 + 48) * 2.0 ** -25 + 5 * 2.0 ** -24
    if s is not None:
        assert bool(((s.cpu().double() - es).abs() <= (f + 2.0 ** -23) * es).all())
    if out is not None:
        d = (out.cpu().double() - ep).abs()
        assert bool((d <= (plain.HALF_STEP[BF] + f + 2.0 ** -23) * ep.abs() * 1.01 + 1e-38).all())


@pytest.mark.parametrize("xt,rt,wt", [(BF, BF, BF), (F, BF, BF), (BF, F, BF), (F, F, F), (BF, None, BF), (F, None, None),
                                      (BF, BF, F), (BF, BF, None)])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 6144), (5, 8), (6, 100), (9, 1021), (310, 1021), (400, 256), (2, 33000),
                                 (2, 40001)])
def test_add_norm(T, H, xt, rt, wt):
    x = rows(T, H, H, xt)
    res = None if rt is None else rows(T, H, H + 1, rt)
    w = None if wt is None else (1 + 0.3 * torch.randn(H, generator=gen(H + 2))).to(wt)
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = q4.add_norm(c(x), c(w), 1e-5, residual=c(res))
    check_add_norm(x, w, 1e-5, res, got, H)


@pytest.mark.parametrize("H", [64, 61, 40001])
def test_add_norm_in_place_and_parts(H):
    x, res, w = rows(7, H, 1), rows(7, H, 2), (1 + 0.3 * torch.randn(H, generator=gen(3))).to(BF)
    a = q4.add_norm(x.cuda(), w.cuda(), residual=res.cuda())
    # the residual and the input in place
    xd, rd = x.cuda(), res.cuda()
    b = q4.add_norm(xd, w.cuda(), residual=rd, residual_out=rd, out=xd)
    assert b[0] is rd and b[1] is xd
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    xd = x.cuda()
    assert torch.equal(q4.add_norm(xd, w.cuda(), residual=res.cuda(), residual_out=xd)[0], a[0])
    # one output alone
    r, out, q, s = q4.add_norm(x.cuda(), w.cuda(), residual=res.cuda(), quant=False)
    assert q is None and s is None and torch.equal(out, a[1]) and torch.equal(r, a[0])
    r, out, q, s = q4.add_norm(x.cuda(), w.cuda(), residual=res.cuda(), bf16=False)
    assert out is None and torch.equal(q, a[2]) and torch.equal(s, a[3])
    # without a residual x itself is normed
    z = a[0]
    c = q4.add_norm(z, w.cuda())
    assert c[0] is None and torch.equal(c[1], a[1]) and torch.equal(c[2], a[2]) and torch.equal(c[3], a[3])


@pytest.mark.parametrize("ld,offset", [(72, 0), (65, 0), (72, 1), (80, 8)])
def test_add_norm_strides_and_bounds(ld, offset):
    x, res, w = rows(40, 64, 21), rows(40, 64, 22, F), torch.ones(64, dtype=BF)
    ro, out, q, s = (Guarded((40, ld), F), Guarded((40, ld), BF), Guarded((40, ld), torch.int8), Guarded((40,), F))
    for g in (ro, out, q):
        g.view.fill_(55)
    got = q4.add_norm(strided(x, ld, offset), w.cuda(), 1e-6, residual=strided(res, ld, offset),
                      residual_out=ro.view[:, :64], out=out.view[:, :64], q=q.view[:, :64], scale=s.view)
    check_add_norm(x, w, 1e-6, res, got, 64)
    for g in (ro, out, q, s):
        g.check()
    for g in (ro, out, q):
        assert bool((g.view[:, 64:] == 55).all())


def test_add_norm_zero_rows_and_overflowing_squares():
    x = torch.zeros((4, 512))
    x[1] = 1e20  # finite, but the squares' sum is not: the row is marked
    x[2] = 1e-30
    r, out, q, s = q4.add_norm(x.cuda(), None, 1e-6)
    assert not out[0].any() and not q[0].any() and s[0] == 0
    assert torch.isnan(out[1]).all() and torch.isnan(s[1]) and not q[1].any()
    assert bool((q[2] == 127).all())


# ---- products -----------------------------------------------------------------

def int8_rows(T, K, seed, extreme=False):
    q = torch.randint(-128 if extreme else -127, 128, (T, K), generator=gen(seed), dtype=torch.int8)
    s = torch.rand(T, generator=gen(seed + 1)) * 0.01
    return q, s


def on_gpu(q, ld=None):
    return strided(q, ld or -(-q.shape[1] // 16) * 16)


def check_linear(got, x, xs, w, ws, bias):
    d = (got.cpu().double() - plain.linear(x, xs, w, ws, bias)).abs()
    bound = plain.linear_bound(x, xs, w, ws, bias, got.dtype)
    assert bool((d <= bound).all()), float((d / bound).max())


LINEAR_SIZES = [(1, 1, 1), (1, 16, 64), (1, 17, 15), (1, 600, 1000), (2, 33, 16), (7, 100, 129), (8, 128, 256),
                (9, 65, 527), (16, 256, 512), (17, 257, 1031), (31, 64, 2048), (33, 129, 100), (45, 1003, 1990),
                (64, 384, 640), (100, 130, 130), (128, 256, 128), (129, 255, 257), (200, 1000, 523), (256, 512, 1024),
                (257, 300, 384), (300, 700, 77), (511, 129, 1000), (513, 513, 513), (1000, 1000, 1000), (1030, 2050, 260)]


@pytest.mark.parametrize("T,N,K", LINEAR_SIZES)
@pytest.mark.parametrize("dtype,bias", [(BF, False), (F, True)])
def test_linear(T, N, K, dtype, bias):
    x, xs = int8_rows(T, K, K, extreme=True)
    w, ws = int8_rows(N, K, K + 7, extreme=True)
    b = torch.randn(N, generator=gen(N)) if bias else None
    out = Guarded((T, N), dtype)
    got = q4.linear_i8(on_gpu(x), xs.cuda(), on_gpu(w), ws.cuda(), bias=None if b is None else b.cuda(), out=out.view)
    out.check("out")
    check_linear(got, x, xs, w, ws, b)


@pytest.mark.parametrize("T,N,K", [(129, 100, 2560), (129, 100, 2559), (256, 515, 2700), (200, 77, 5120),
                                   (257, 300, 5121), (300, 1800, 5200),
                                   (256, 2049, 5120), (256, 4000, 2561), (256, 4200, 4096), (400, 2100, 4500), (256, 8192, 4097),
                                   (256, 8200, 4097), (1000, 1000, 2600), (900, 100, 131071)])
@pytest.mark.parametrize("dtype,bias", [(BF, False), (F, True)])
def test_linear_long_rows_of_many_tokens(T, N, K, dtype, bias):
    # K over a cluster's pairs, and both sides of the limits: exact sums against
    # a split of the same product into calls of few tokens, and the plain form
    x, xs = int8_rows(T, K, K, extreme=True)
    w, ws = int8_rows(N, K, K + 7, extreme=True)
    b = torch.randn(N, generator=gen(N)).cuda() if bias else None
    xg, xsg, wg, wsg = on_gpu(x), xs.cuda(), on_gpu(w), ws.cuda()
    out, status = Guarded((T, N), dtype), torch.zeros(1, dtype=torch.int32, device="cuda")
    got = q4.linear_i8(xg, xsg, wg, wsg, bias=b, out=out.view, status=status)
    out.check("out")
    assert status.item() == 0
    for lo in (0, T // 2, T - 16):
        few = q4.linear_i8(xg[lo:lo + 16], xsg[lo:lo + 16], wg, wsg, bias=b, dtype=dtype)
        assert torch.equal(few, got[lo:lo + 16])
    some = slice(T - 5, T)
    check_linear(got[some], x[some], xs[some], w, ws, None if b is None else b.cpu())


@pytest.mark.parametrize("T,H,I", [(129, 2560, 65), (256, 5200, 130), (256, 4100, 2050), (256, 5120, 1030), (513, 2600, 400)])
def test_mlp_long_rows_of_many_tokens(T, H, I):
    m = mlp_weights(H, I, H + I)
    q, s = q4.quant_rows(rows(T, H, T, spread=False).cuda())
    got = q4.mlp_i8(m, q, s, dtype=F)
    for lo in (0, T // 2, T - 9):
        assert torch.equal(q4.mlp_i8(m, q[lo:lo + 9], s[lo:lo + 9], dtype=F), got[lo:lo + 9])
    check_mlp(got[-5:], m, q[-5:].cpu(), s[-5:].cpu())


@pytest.mark.parametrize("T", [1, 20, 130, 600])
@pytest.mark.parametrize("ldx,ldw,ldo", [(64, 80, 101), (128, 64, 104), (80, 192, 112)])
def test_linear_strides(T, ldx, ldw, ldo):
    x, xs = int8_rows(T, 63, 1)
    w, ws = int8_rows(99, 63, 2)
    for dtype in (BF, F):
        out = Guarded((T, ldo), dtype)
        out.view.fill_(7)
        got = q4.linear_i8(on_gpu(x, ldx), xs.cuda(), on_gpu(w, ldw), ws.cuda(), out=out.view[:, :99])
        out.check("out")
        check_linear(got, x, xs, w, ws, None)
        assert bool((out.view[:, 99:] == 7).all())
    # an output that starts anywhere
    flat = torch.zeros(T * 99 + 1, dtype=BF, device="cuda")
    got = q4.linear_i8(on_gpu(x), xs.cuda(), on_gpu(w), ws.cuda(), out=flat[1:].view(T, 99))
    check_linear(got, x, xs, w, ws, None)


@pytest.mark.parametrize("T", [1, 12, 64, 300])
def test_linear_largest_sums(T):
    # 131071 products of 2^14: the largest sum is 2^31 - 16384
    K = 131071
    x = torch.full((T, K), -128, dtype=torch.int8)
    w = torch.full((40, K), -128, dtype=torch.int8)
    w[1] = 127
    w[2] = 0
    got = q4.linear_i8(on_gpu(x), torch.ones(T).cuda(), on_gpu(w), torch.ones(40).cuda(), dtype=F).cpu()
    want = torch.full((40,), K * 16384, dtype=torch.int64)
    want[1] = -128 * 127 * K
    want[2] = 0
    assert torch.equal(got, want.float().expand(T, 40))


def test_linear_rows_are_independent_and_repeat():
    x, xs = int8_rows(700, 1000, 1)
    w, ws = int8_rows(515, 1000, 2)
    xg, xsg, wg, wsg = on_gpu(x), xs.cuda(), on_gpu(w), ws.cuda()
    full = q4.linear_i8(xg, xsg, wg, wsg, dtype=F)
    assert torch.equal(full, q4.linear_i8(xg, xsg, wg, wsg, dtype=F))
    for lo, hi in ((0, 1), (3, 10), (100, 113), (200, 233), (300, 400), (0, 250), (90, 600)):
        assert torch.equal(q4.linear_i8(xg[lo:hi], xsg[lo:hi], wg, wsg, dtype=F), full[lo:hi])


@pytest.mark.parametrize("N,K", [(515, 1000), (515, 2000), (130, 100)])
def test_linear_rows_with_bias_are_independent(N, K):
    x, xs = int8_rows(700, K, 1)
    w, ws = int8_rows(N, K, 2)
    b = torch.randn(N, generator=gen(3)).cuda()
    xg, xsg, wg, wsg = on_gpu(x), xs.cuda(), on_gpu(w), ws.cuda()
    full = q4.linear_i8(xg, xsg, wg, wsg, bias=b, dtype=F)
    for lo, hi in ((0, 1), (3, 10), (100, 113), (200, 233), (300, 400), (0, 250), (90, 600)):
        assert torch.equal(q4.linear_i8(xg[lo:hi], xsg[lo:hi], wg, wsg, bias=b, dtype=F), full[lo:hi])


def test_linear_empty_and_refusals():
    w, ws = q4.quant_rows(rows(8, 32, 1, spread=False).cuda())
    x = torch.empty((0, 32), dtype=torch.int8, device="cuda")
    assert q4.linear_i8(x, torch.empty(0, device="cuda"), w, ws).shape == (0, 8)
    assert q4.quant_rows(torch.empty((0, 32), device="cuda"))[0].shape == (0, 32)
    assert q4.add_norm(torch.empty((0, 32), device="cuda"), None)[1].shape == (0, 32)
    m = q4.MlpI8(*q4.quant_rows(rows(8, 32, 1).cuda()), *q4.quant_rows(rows(32, 4, 2).cuda()))
    assert q4.mlp_i8(m, x, torch.empty(0, device="cuda")).shape == (0, 32)
    q, s = q4.quant_rows(rows(4, 32, 2).cuda())
    with pytest.raises(ValueError):
        q4.linear_i8(q, s, w[:, :16], ws)  # K differs
    with pytest.raises(ValueError):
        q4.linear_i8(q, s[:3], w, ws)
    with pytest.raises(ValueError):
        q4.linear_i8(q.t(), s, w, ws)
    with pytest.raises(ValueError):
        q4.linear_i8(q, s, w, ws, bias=torch.zeros(8, device="cuda", dtype=BF))
    with pytest.raises(ValueError):
        q4.linear_i8(q, s, w, ws.cpu())
    with pytest.raises(q4.MoeQ4Error):
        q4.linear_i8(torch.zeros((4, 33), dtype=torch.int8, device="cuda")[:, 1:], s, w, ws)  # not on 16 bytes
    with pytest.raises(q4.MoeQ4Error):
        q4.linear_i8(torch.zeros((1, 32), dtype=torch.int8, device="cuda").expand(4, 32), s, w, ws)


def test_offsets_past_32_bits():
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB")
    # 2^31 elements and more in each matrix; rows from the far end are checked
    T, K = 70001, 32768
    x = torch.zeros((T, K), dtype=BF, device="cuda")
    far = torch.tensor([0, 65535, 65536, T - 1])
    src = rows(4, K, 9, spread=False)
    x[far.cuda()] = src.cuda()
    q, s = q4.quant_rows(x)
    check_codes(q[far.cuda()], plain.quant(src.double())[0])
    r, out, q2, s2 = q4.add_norm(x, None, 1e-6, residual=x, residual_out=x)
    check_add_norm(src, None, 1e-6, src, (r[far.cuda()], out[far.cuda()], q2[far.cuda()], s2[far.cuda()]), K)
    del x, r, out, q2, s2
    w, ws = int8_rows(16, K, 5)
    y = q4.linear_i8(q, s, on_gpu(w), ws.cuda(), dtype=F)  # x past 2^31
    check_linear(y[far.cuda()], q[far.cuda()].cpu(), s[far.cuda()].cpu(), w, ws, None)
    del y
    few = q[far.cuda()].contiguous()
    y = q4.linear_i8(few, s[far.cuda()], q, s, dtype=F)  # w past 2^31
    check_linear(y[:, far.cuda()], few.cpu(), s[far.cuda()].cpu(), q[far.cuda()].cpu(), s[far.cuda()].cpu(), None)
    a, sa = int8_rows(T, 32, 6)
    b, sb = int8_rows(K, 32, 7)
    y = q4.linear_i8(on_gpu(a), sa.cuda(), on_gpu(b), sb.cuda())  # the output past 2^31
    check_linear(y[far.cuda()], a[far], sa[far], b, sb, None)


# ---- the MLP ------------------------------------------------------------------

def mlp_weights(H, I, seed):
    gu = (0.05 * torch.randn((2 * I, H), generator=gen(seed))).to(BF)
    dn = (0.05 * torch.randn((H, I), generator=gen(seed + 1))).to(BF)
    return q4.MlpI8(*q4.quant_rows(gu.cuda()), *q4.quant_rows(dn.cuda()))


def check_mlp(got, m, x, xs):
    gu, gus, dn, ds = (t.cpu() for t in m.tensors)
    want, h = plain.mlp(x, xs, gu, gus, dn, ds)
    # h in fp32 is within 2^-20 of its value, so at most 2 * 2^-20 / 2^-8 of the
    # h round to the neighbouring bf16, which moves a code by one step at most
    # (2^-7 |h| < max|h| / 127).  One step is max|h| / 127, below 0.1 of the
    # rows' rms for maxima to 12 rms: 0.1 * sqrt(2^-11) = 2.2e-3 of the result.
    d = got.cpu().double() - want
    own = plain.HALF_STEP[got.dtype]
    assert d.norm() <= (2.0 ** -8 + own) * want.norm()
    # and no element may be further off than all of its h by one step
    wd = dn.double().abs() * ds.double()[:, None]
    step = h.abs().amax(1) * (1 + 2.0 ** -7) / 127
    bound = step[:, None] * wd.sum(1)[None] * 1.01 + own * want.abs() * 1.01
    assert bool((d.abs() <= bound + 1e-30).all())


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T,H,I", [(1, 16, 1), (1, 1000, 523), (1, 2048, 768), (3, 64, 33), (8, 512, 256), (9, 256, 128),
                                   (33, 1000, 523), (64, 512, 384), (130, 300, 200), (257, 640, 300), (600, 512, 260)])
def test_mlp(T, H, I, dtype):
    m = mlp_weights(H, I, H + I)
    x = rows(T, H, T, spread=False)
    q, s = q4.quant_rows(x.cuda())
    out, ws = Guarded((T, H), dtype), Guarded((q4.mlp_i8_workspace(m, T),), torch.uint8)
    got = q4.mlp_i8(m, q, s, out=out.view, ws=ws.view)
    out.check("out")
    ws.check("workspace")
    check_mlp(got, m, q.cpu(), s.cpu())
    # the same bits again, in a workspace that holds other bytes
    ws.view.fill_(255)
    assert torch.equal(got.clone(), q4.mlp_i8(m, q, s, dtype=dtype, ws=ws.view))


@pytest.mark.parametrize("T,I", [(1, 5400), (1, 5600), (1, 8192), (1, 8193), (2, 4096), (2, 4097), (3, 2730), (4, 2048),
                                 (5, 1638), (7, 1170), (8, 1024), (8, 1025)])
def test_mlp_few_tokens_of_long_rows(T, I):
    # rows of h to 8192 values and past them, for few tokens
    m = mlp_weights(40, I, I)
    q, s = q4.quant_rows(rows(T, 40, T, spread=False).cuda())
    got = q4.mlp_i8(m, q, s, dtype=F)
    check_mlp(got, m, q.cpu(), s.cpu())
    for t in range(T):
        assert torch.equal(q4.mlp_i8(m, q[t:t + 1], s[t:t + 1], dtype=F), got[t:t + 1])


def test_mlp_rows_are_independent():
    m = mlp_weights(512, 272, 5)
    q, s = q4.quant_rows(rows(400, 512, 6).cuda())
    full = q4.mlp_i8(m, q, s, dtype=F)
    assert not full[1].any()  # a row of zeros
    for lo, hi in ((0, 1), (5, 12), (20, 45), (40, 140), (0, 300)):
        assert torch.equal(q4.mlp_i8(m, q[lo:hi], s[lo:hi], dtype=F), full[lo:hi])
    # a row that is not finite is NaN, and only that
    s2 = s.clone()
    s2[7] = float("nan")
    bad = q4.mlp_i8(m, q, s2, dtype=F)
    keep = [i for i in range(400) if i != 7]
    assert torch.isnan(bad[7]).all() and torch.equal(bad[keep], full[keep])


# ---- streams, graphs, threads ---------------------------------------------------

def chain(m, x, res, w, stream=None):
    r, h, q, s = q4.add_norm(x, w, residual=res, stream=stream)
    return r, h, q4.mlp_i8(m, q, s, stream=stream)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_another_stream(T):
    m = mlp_weights(512, 256, 1)
    x, res, w = rows(T, 512, 2).cuda(), rows(T, 512, 3).cuda(), torch.ones(512, dtype=BF, device="cuda")
    want = chain(m, x, res, w)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = chain(m, x, res, w, stream=st)
    with torch.cuda.stream(st):
        again = chain(m, x, res, w)
    st.synchronize()
    for a, b, c in zip(want, got, again):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_captured_and_replayed(T):
    m = mlp_weights(512, 256, 1)
    w = torch.ones(512, dtype=BF, device="cuda")
    xs = [(rows(T, 512, 10 + i).cuda(), rows(T, 512, 20 + i).cuda()) for i in range(3)]
    want = [chain(m, x, r, w) for x, r in xs]
    x, r = (t.clone() for t in xs[0])
    ws = q4.alloc_workspace(q4.mlp_i8_workspace(m, T))
    graphs = []
    for _ in range(2):  # two graphs that share a workspace
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            ro, h, q, s = q4.add_norm(x, w, residual=r)
            y = q4.mlp_i8(m, q, s, ws=ws)
        graphs.append((g, (ro, h, y)))
    for i, (xi, ri) in enumerate(xs):
        x.copy_(xi)
        r.copy_(ri)
        for g, out in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, out in graphs:
            for a, b in zip(want[i], out):
                assert torch.equal(a, b)


def test_two_threads_on_two_streams():
    m = mlp_weights(512, 256, 1)
    w = torch.ones(512, dtype=BF, device="cuda")
    xs = [(rows(T, 512, T).cuda(), rows(T, 512, T + 1).cuda()) for T in (5, 300)]
    want = [chain(m, x, r, w) for x, r in xs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(50):
                got = chain(m, *xs[i], w)
                st.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(want[i], got)):
                    bad.append(i)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad


@pytest.mark.parametrize("T", [1, 6, 40, 300])
def test_operands_written_just_before(T):
    # every operand of the calls is rewritten by the kernels right in front of
    # them, with no wait between: launches overlap, results may not
    H, I = 2048, 1024
    gus = [(0.05 * torch.randn((2 * I, H), generator=gen(i))).to(BF).cuda() for i in range(3)]
    dns = [(0.05 * torch.randn((H, I), generator=gen(9 + i))).to(BF).cuda() for i in range(3)]
    xs = [rows(T, H, 20 + i).cuda() for i in range(3)]
    gu, dn = q4.quant_rows(gus[0]), q4.quant_rows(dns[0])
    m = q4.MlpI8(*gu, *dn)
    q, s = q4.quant_rows(xs[0])
    ws = q4.alloc_workspace(q4.mlp_i8_workspace(m, T))

    def step(i):
        q4.quant_rows(xs[i], q=q, scale=s)
        q4.quant_rows(gus[i], q=gu[0], scale=gu[1])
        y = q4.linear_i8(q, s, gu[0], gu[1])
        r, h, _, _ = q4.add_norm(y[:, :H].contiguous(), None, residual=xs[i], q=q, scale=s)
        q4.quant_rows(dns[i], q=dn[0], scale=dn[1])
        return y, h, q4.mlp_i8(m, q, s, ws=ws)

    want = []
    for i in range(3):
        want.append([t.clone() for t in step(i)])
        torch.cuda.synchronize()
    got = [step(i % 3) for i in range(30)]
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        for a, b in zip(want[i % 3], out):
            assert torch.equal(a, b)
