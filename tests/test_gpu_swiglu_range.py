"""The SwiGLU at the ends of fp32's range: silu(g) u is 0 for g far below 0,
however large u is."""
import pytest
import torch

import bit_codebook_quantized_router_b200 as q4
from bit_codebook_quantized_router_b200 import inputs
from tests.test_gpu_int8 import BF, F, check_mlp, gen, mlp_weights, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [4, 40, 300])
def test_routed_experts(T):
    # g = -256 and u = 2^124 or so: silu(g) u is 0 in fp32, g u is out of range
    sh = inputs.TINY
    tables, tid = inputs.layer_tables(inputs.WORKLOADS["tiny"])
    gate = torch.full((sh.E, sh.I, sh.H), -1.0, dtype=BF, device="cuda")
    up = torch.full((sh.E, sh.I, sh.H), 2.0 ** 116, dtype=BF, device="cuda")
    down = torch.ones((sh.E, sh.H, sh.I), dtype=BF, device="cuda")
    layer = q4.Layer(*q4.pack(gate, tables, tid), *q4.pack(up, tables, tid), *q4.pack(down, tables, tid), tables, tid)
    x = torch.ones((T, sh.H), dtype=BF, device="cuda")
    logits = torch.randn((T, sh.E), generator=gen(T)).cuda()
    out32 = torch.empty((T, sh.H), device="cuda")
    out = q4.forward(layer, x, logits, 2, out_f32=out32)
    assert not out32.any() and not out.any()  # (a NaN counts as not zero)


def extreme_mlp(H, I, g, u):
    """Weights, and the codes of one row, that make channel 3's gate g and up u, both exact, beside normal channels."""
    q = torch.randint(-127, 128, (2 * I, H), generator=gen(H), dtype=torch.int8)
    s = torch.rand(2 * I, generator=gen(I)) * 1e-5
    for row, v in ((3, g), (I + 3, u)):
        q[row] = 0
        q[row, :2] = 64 if v > 0 else -64  # sum 2^13 with the codes of x below
        s[row] = abs(v) / 2.0 ** 13
    x = torch.randint(-127, 128, (1, H), generator=gen(7), dtype=torch.int8)
    x[0, :2] = 64
    down, ds = torch.randint(-127, 128, (H, I), generator=gen(8), dtype=torch.int8), torch.rand(H, generator=gen(9)) * 1e-3
    pad = lambda t: torch.nn.functional.pad(t, (0, -t.shape[1] % 16)).cuda()[:, :t.shape[1]]  # noqa: E731
    return q4.MlpI8(pad(q), s.cuda(), pad(down), ds.cuda()), pad(x)


@pytest.mark.parametrize("T,H,I", [(1, 300, 40), (9, 1000, 64), (40, 6144, 100), (70, 1600, 300), (200, 640, 90), (200, 2600, 90)])
@pytest.mark.parametrize("g,u", [(-200.0, 2.0 ** 123), (-100.0, -2.0 ** 125), (-2.0 ** 100, 2.0 ** 100), (-1000.0, 2.0 ** 126)])
def test_int8_mlp(T, H, I, g, u):
    m, x = extreme_mlp(H, I, g, u)
    x, xs = x.expand(T, H).contiguous(), torch.ones(T, device="cuda")
    x = torch.nn.functional.pad(x, (0, -H % 16))[:, :H]
    got = q4.mlp_i8(m, x, xs, dtype=F)
    check_mlp(got, m, x.cpu(), xs.cpu())


@pytest.mark.parametrize("T,H,I", [(1, 300, 40), (9, 1000, 64), (40, 6144, 100), (70, 1600, 300), (200, 640, 90), (200, 2600, 90)])
@pytest.mark.parametrize("g,u", [(-87.5, 2.0 ** 124), (-88.5, 2.0 ** 126), (-20.0, 2.0 ** 30), (-60.0, -2.0 ** 86)])
def test_int8_mlp_small_sigmoids(T, H, I, g, u):
    # silu(g) is small and u makes up for it: the channel is the row's largest,
    # so its code is 127 in size and the row's scale is |h| / 127
    m, x = extreme_mlp(H, I, g, u)
    x = torch.nn.functional.pad(x.expand(T, H).contiguous(), (0, -H % 16))[:, :H]
    xs = torch.ones(T, device="cuda")
    check_mlp(q4.mlp_i8(m, x, xs, dtype=F), m, x.cpu(), xs.cpu())


def fp32_formula(m, x, xs):
    """The MLP's definition step by step in fp32, sums exact."""
    gu, gus, dn, ds = m.tensors
    product = lambda a, sa, b, sb: (a.double() @ b.double().T).float() * sa[:, None] * sb  # noqa: E731
    g, u = product(x, xs, gu, gus).chunk(2, 1)
    q, s = q4.quant_rows((g / (1 + torch.exp(-g)) * u).to(BF))
    return product(q, s, dn, ds)


@pytest.mark.parametrize("T", [1, 40, 300])
@pytest.mark.parametrize("g,u", [(6 * 2.0 ** -149, 2.0 ** 127), (1.7 * 2.0 ** -130, 2.0 ** 126), (torch.finfo(F).max, 2.0 ** -126), (1e30, 1e-20),
                                 (-88.6, 2.0 ** 126), (-88.9, 2.0 ** 126), (0.0, 2.0 ** 127), (-2.0 ** -149, 2.0 ** 127)])
def test_h_of_the_smallest_and_largest_gates(T, g, u):
    # one channel alone, its sums 1, so that the scales are g and u
    H, I = 2304, 64
    q = torch.zeros((2 * I, H), dtype=torch.int8)
    q[3, 0], q[I + 3, 0] = (-1 if g < 0 else 1), 1
    s = torch.ones(2 * I)
    s[3], s[I + 3] = abs(g), u
    down = torch.randint(-127, 128, (H, I), generator=gen(1), dtype=torch.int8)
    m = q4.MlpI8(q.cuda(), s.cuda(), down.cuda(), torch.ones(H, device="cuda"))
    x = torch.ones((T, H), dtype=torch.int8, device="cuda")
    xs = torch.ones(T, device="cuda")
    got, want = q4.mlp_i8(m, x, xs, dtype=F), fp32_formula(m, x, xs)
    assert torch.equal(got, want) and torch.isfinite(got).all()


@pytest.mark.parametrize("T,H,I,size", [(3, 640, 300, 1.0), (40, 2304, 256, 30.0), (100, 1600, 300, 8.0), (700, 512, 1000, 1.0),
                                        (700, 512, 1000, 40.0), (300, 2600, 200, 8.0)])
def test_h_is_the_fp32_formula_rounded_to_bf16(T, H, I, size):
    # every step of the definition in fp32 (sums exact), on gates of about `size`:
    # the MLP's result has the same bits
    m = mlp_weights(H, I, T)
    gu, gus, dn, ds = m.tensors
    gus = gus * size
    m = q4.MlpI8(gu, gus, dn, ds)
    x, xs = q4.quant_rows(rows(T, H, I, spread=False).cuda())
    assert torch.equal(q4.mlp_i8(m, x, xs, dtype=F), fp32_formula(m, x, xs))
