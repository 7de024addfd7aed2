"""The MoE layer with an int8 shared expert, behind the residual and norm: the
operators together, as a model runs them."""
import pytest
import torch

import bit_codebook_quantized_router_b200 as q4
from bit_codebook_quantized_router_b200 import inputs
from tests.gpu_support import Guarded
from tests.test_gpu_forward import _small_device_layer
from tests.test_gpu_int8 import mlp_weights

pytestmark = pytest.mark.gpu


def parts(T, seed=31):
    w = inputs.Workload("int8_shared", seed, T, inputs.TINY)
    _, dev = _small_device_layer(w)
    return w, dev, inputs.activations(w).cuda(), inputs.router_logits(w).cuda()


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("T,k", [(1, 2), (4, 2), (16, 2), (17, 1), (300, 3)])
def test_shared_expert_in_int8(T, k, given):
    w, dev, x, lg = parts(T)
    m = mlp_weights(dev.H, 256, 7)
    q, s = q4.quant_rows(x)
    out, o32 = Guarded((T, dev.H), torch.bfloat16), Guarded((T, dev.H), torch.float32)
    ws = Guarded((q4.forward_ex_workspace(dev, m, T, k),), torch.uint8)
    q4.forward_ex(dev, m, x, lg, k, out=out.view, out_f32=o32.view, ws=ws.view, xq=q if given else None,
                  x_scale=s if given else None)
    assert q4.forward_status(ws.view) == 0
    for b in (out, o32, ws):
        b.check()
    base = torch.empty_like(o32.view)
    q4.forward(dev, x, lg, k, out_f32=base)
    # the routed sum first, then the MLP's result, added in fp32
    assert torch.equal(o32.view, base + q4.mlp_i8(m, q, s, dtype=torch.float32))
    assert torch.equal(out.view, o32.view.to(torch.bfloat16))


@pytest.mark.parametrize("T", [1, 8, 40])
def test_block_from_residual_to_layer(T):
    w, dev, x, _ = parts(T, 32)
    m = mlp_weights(dev.H, 384, 8)
    gate = (0.05 * torch.randn((dev.E, dev.H), generator=torch.Generator().manual_seed(1))).to(torch.bfloat16).cuda()
    norm = (1 + 0.1 * torch.randn(dev.H, generator=torch.Generator().manual_seed(2))).to(torch.bfloat16).cuda()
    res = (2 * inputs.activations(w).float()).cuda()
    attn, ascale = q4.quant_rows(x)
    proj, pscale = q4.quant_rows((0.05 * torch.randn((dev.H, dev.H), generator=torch.Generator().manual_seed(3)))
                                 .to(torch.bfloat16).cuda())
    y = q4.linear_i8(attn, ascale, proj, pscale, dtype=torch.float32)
    r, h, q, s = q4.add_norm(y, norm, residual=res)
    o32, lg = torch.empty((T, dev.H), device="cuda"), torch.empty((T, dev.E), device="cuda")
    ws = q4.alloc_workspace(q4.forward_gated_workspace(dev, m, T, 2))
    out = q4.forward_gated(dev, m, gate, h, 2, out_f32=o32, logits=lg, ws=ws, xq=q, x_scale=s)
    assert q4.forward_status(ws) == 0
    base, lg0 = torch.empty_like(o32), torch.empty_like(lg)
    q4.forward_gated(dev, None, gate, h, 2, out_f32=base, logits=lg0)
    assert torch.equal(lg, lg0)
    assert torch.equal(o32, base + q4.mlp_i8(m, q, s, dtype=torch.float32))
    r2, h2, _, _ = q4.add_norm(o32, norm, residual=r)  # the next block's input
    assert torch.equal(out, o32.to(torch.bfloat16)) and torch.isfinite(h2).all() and r2.dtype == torch.float32


def test_refusals():
    w, dev, x, lg = parts(4)
    m = mlp_weights(dev.H, 256, 7)
    q, s = q4.quant_rows(x)
    with pytest.raises(ValueError):
        q4.forward_ex(dev, m, x, lg, 2, xq=q)
    with pytest.raises(ValueError):
        q4.forward_ex(dev, None, x, lg, 2, xq=q, x_scale=s)
    with pytest.raises(ValueError):
        q4.forward_ex(dev, m, x, lg, 2, xq=q[:3], x_scale=s[:3])
    with pytest.raises(q4.MoeQ4Error):
        q4.forward_ex(dev, mlp_weights(128, 64, 9), x, lg, 2)
