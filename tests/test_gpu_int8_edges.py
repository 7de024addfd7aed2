"""The 8-bit integer operators at the edges of what their callers may do."""
import ctypes

import pytest
import torch

import bit_codebook_quantized_router_b200 as q4
from bit_codebook_quantized_router_b200 import _lib
from tests import int8_plain as plain
from tests.test_gpu_int8 import BF, F, gen, int8_rows, mlp_weights, on_gpu, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N,K", [(1, 64, 1000), (8, 300, 2048), (16, 48, 129), (24, 200, 1024), (40, 64, 2000)])
def test_weights_written_by_the_kernel_in_front(T, N, K):
    # quant_rows lets the product start before it has written the weights: the
    # product, resident beside it, may only see what it wrote in the end
    w = [rows(N, K, i, spread=False).cuda() for i in range(3)]
    x, xs = q4.quant_rows(rows(T, K, 9, spread=False).cuda())
    q, s = q4.quant_rows(w[0])
    want = []
    for v in w:
        q4.quant_rows(v, q=q, scale=s)
        torch.cuda.synchronize()
        want.append(q4.linear_i8(x, xs, q, s, dtype=F))
        torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])

    def run():
        got = []
        for i in range(60):
            q4.quant_rows(w[i % 3], q=q, scale=s)
            got.append(q4.linear_i8(x, xs, q, s, dtype=F))
        return got

    eager = run()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        captured = run()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for got in (eager, captured):
        for i, y in enumerate(got):
            assert torch.equal(y, want[i % 3]), i


@pytest.mark.parametrize("T,N,K", [(300, 400, 512), (200, 400, 2600), (200, 100, 5200), (64, 512, 2048), (8, 512, 2048)])
def test_limits_do_not_count_the_kernel_in_front(T, N, K):
    # the kernel in front lets the product start and then runs for longer than
    # any of the product's waits may take
    x, xs = q4.quant_rows(rows(T, K, 1, spread=False).cuda())
    w, ws = q4.quant_rows(rows(N, K, 2, spread=False).cuda())
    m = mlp_weights(K, 128, 3)
    want, want_mlp = q4.linear_i8(x, xs, w, ws, dtype=F), q4.mlp_i8(m, x, xs, dtype=F)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got, got_mlp = torch.zeros_like(want), torch.zeros_like(want_mlp)
    ws_mlp = q4.alloc_workspace(q4.mlp_i8_workspace(m, T))
    torch.cuda.synchronize()
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert q4.lib().moe_q4_selftest_hold(2300000, stream) == _lib.OK  # the limit is 2 s
    q4.linear_i8(x, xs, w, ws, out=got, status=status)
    assert q4.lib().moe_q4_selftest_hold(2300000, stream) == _lib.OK
    q4.mlp_i8(m, x, xs, out=got_mlp, ws=ws_mlp, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    assert torch.equal(got, want) and torch.equal(got_mlp, want_mlp)


@pytest.mark.parametrize("dtype,bias", [(F, False), (F, True), (BF, False)])
@pytest.mark.parametrize("T,N,K", [(11, 100, 4096), (40, 200, 4096), (100, 130, 4000), (200, 300, 1000), (200, 130, 4000), (200, 60, 6000)])
def test_scales_at_both_ends_of_fp32(T, N, K, dtype, bias):
    # every pair of scales from 2^-149 to 2^127: the products by themselves leave
    # fp32's range where the result does not
    ends = torch.tensor([2.0 ** -149, 3e-44, 1e-40, 1.1e-38, 1e-25, 1e-16, 1e-3, 1.0, 1e7, 1e20, 2.0 ** 95 * 1.99, 2.0 ** 96, 1e30, 3e38],
                        dtype=torch.float64).float()
    x, _ = int8_rows(T, K, 1)
    w, _ = int8_rows(N, K, 2)
    w[::7] = 0
    xs, ws = ends[torch.arange(T) % len(ends)], ends[torch.arange(N) % 13 + torch.arange(N) // 13 % 2]
    b = torch.randn(N, generator=gen(3)) if bias else None
    got = q4.linear_i8(on_gpu(x), xs.cuda(), on_gpu(w), ws.cuda(), bias=None if b is None else b.cuda(), dtype=dtype).cpu()
    want, bound = plain.linear(x, xs, w, ws, b), plain.linear_bound(x, xs, w, ws, b, dtype)
    # (the bound's 1e-38 is for results below fp32's normal range: there half a unit of 2^-149, or bf16's 2^-133, is lost)
    bound = bound - 1e-38 + 2.0 ** -133
    top = torch.finfo(dtype).max
    inside, outside = want.abs() + bound <= top, want.abs() - bound > top
    assert bool(((got.double() - want).abs() <= bound)[inside].all())
    assert torch.equal(got.double()[outside], want[outside].sign() * float("inf"))
    assert not torch.isnan(got).any() and inside.any() and outside.any()


@pytest.mark.parametrize("T,H,I", [(5, 300, 70), (40, 6144, 100), (100, 1600, 70), (200, 640, 90), (200, 2600, 90), (200, 5200, 60)])
@pytest.mark.parametrize("e", [100, -100])
def test_mlp_with_the_scales_shifted_by_a_power_of_two(T, H, I, e):
    m = mlp_weights(H, I, 4)
    gu, gus, dn, ds = m.tensors
    x, xs = q4.quant_rows(rows(T, H, 5, spread=False).cuda())
    moved = q4.MlpI8(gu, gus * 2.0 ** -e, dn, ds)
    assert torch.equal(q4.mlp_i8(moved, x, xs * 2.0 ** e, dtype=F), q4.mlp_i8(m, x, xs, dtype=F))


def test_residual_is_the_fp32_sum_rounded_to_its_type():
    # sums next to a tie of bf16: 1 + 2^-8 + 2^-30 is 1 + 2^-8 in fp32, a tie
    # that goes to 1, and 1 + 3 2^-8 - 2^-30 one that goes to 1 + 2^-6; rounded
    # once to bf16 they would be 1 + 2^-7
    x = torch.tensor([2.0 ** -8 + 2.0 ** -30, 3 * 2.0 ** -8 - 2.0 ** -30, 2.0 ** -8 + 2.0 ** -23, 0.5], dtype=torch.float64)
    want = torch.tensor([1.0, 1 + 2.0 ** -6, 1 + 2.0 ** -7, 1.5])
    for T, pad in ((1, 4), (3, 5), (300, 4)):
        row = torch.cat([x.float(), torch.zeros(pad)]).repeat(T, 1).cuda()
        res = torch.ones((T, 4 + pad), dtype=BF, device="cuda")
        r = q4.add_norm(row, None, residual=res)[0]
        assert torch.equal(r[:, :4].float().cpu(), want.expand(T, 4))
