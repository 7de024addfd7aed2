"""The layer behind int8 kernels that let it start early, and captured calls
that meet from two streams."""
import pytest
import torch

import bit_codebook_quantized_router_b200 as q4
from tests.test_gpu_int8 import BF, F, gen, mlp_weights, rows
from tests.test_gpu_int8_layer import parts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T", [1, 8, 40, 300])
def test_layer_on_rows_that_add_norm_has_just_written(T, gated):
    w, dev, _, lg = parts(T, 33)
    m = mlp_weights(dev.H, 256, 8)
    gate = (0.05 * torch.randn((dev.E, dev.H), generator=gen(1))).to(BF).cuda()
    res = [rows(T, dev.H, 40 + i, F, spread=False).cuda() for i in range(3)]
    zero = torch.zeros((T, dev.H), dtype=BF, device="cuda")
    h, o32 = torch.empty_like(zero), [torch.empty((T, dev.H), device="cuda") for _ in range(30)]
    q, s = q4.quant_rows(zero)
    ro = torch.empty_like(res[0])
    ws = q4.alloc_workspace(max(q4.forward_gated_workspace(dev, m, T, 2), q4.forward_ex_workspace(dev, m, T, 2)))

    def step(i, to):
        q4.add_norm(zero, None, residual=res[i], residual_out=ro, out=h, q=q, scale=s)
        if gated:
            q4.forward_gated(dev, m, gate, h, 2, out_f32=to, ws=ws, xq=q, x_scale=s)
        else:
            q4.forward_ex(dev, m, h, lg, 2, out_f32=to, ws=ws, xq=q, x_scale=s)

    want = []
    for i in range(3):
        torch.cuda.synchronize()
        step(i, o32[i])
        torch.cuda.synchronize()
        want.append(o32[i].clone())
    assert not torch.equal(want[0], want[1])
    for i, to in enumerate(o32):
        step(i % 3, to)
    torch.cuda.synchronize()
    for i, got in enumerate(o32):
        assert torch.equal(got, want[i % 3]), i
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i, to in enumerate(o32):
            step(i % 3, to.zero_())
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for i, got in enumerate(o32):
        assert torch.equal(got, want[i % 3]), i


@pytest.mark.parametrize("T", [1, 40, 100, 300])
def test_two_streams_that_meet_in_a_capture(T):
    # weights to codes on one stream, rows on another, the product where both are
    # done, and the next turn's codes only after it
    N, K = 300, 2048
    xs = [rows(T, K, i, spread=False).cuda() for i in range(3)]
    ws = [rows(N, K, 10 + i, spread=False).cuda() for i in range(3)]
    x, w = q4.quant_rows(xs[0]), q4.quant_rows(ws[0])
    outs = [torch.empty((T, N), device="cuda") for _ in range(12)]
    want = []
    for i in range(3):
        torch.cuda.synchronize()
        want.append(q4.linear_i8(*q4.quant_rows(xs[i]), *q4.quant_rows(ws[i]), dtype=F))
    side = torch.cuda.Stream()

    def run():
        main = torch.cuda.current_stream()
        for i, out in enumerate(outs):
            side.wait_stream(main)
            q4.quant_rows(ws[i % 3], q=w[0], scale=w[1], stream=side)
            q4.quant_rows(xs[i % 3], q=x[0], scale=x[1])
            main.wait_stream(side)
            q4.linear_i8(*x, *w, out=out)

    def check():
        torch.cuda.synchronize()
        for i, out in enumerate(outs):
            assert torch.equal(out, want[i % 3]), i
            out.zero_()

    run()
    check()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        run()
    for _ in range(3):
        g.replay()
        check()
