"""The 8-bit integer operators at the edges of what their callers may do."""
import pytest
import torch

import bit_codebook_quantized_router_b200 as q4
from tests.test_gpu_int8 import F, rows

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
