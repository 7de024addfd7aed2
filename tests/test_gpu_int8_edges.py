"""The 8-bit integer operators at the edges of what their callers may do."""
import ctypes

import pytest
import torch

import bit_codebook_quantized_router_b200 as q4
from bit_codebook_quantized_router_b200 import _lib
from tests.test_gpu_int8 import F, mlp_weights, rows

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
