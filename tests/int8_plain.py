"""Plain 64-bit forms of the 8-bit integer operators, on the CPU."""
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # of a rounding, relative


def quant(p):
    """Codes and row maxima of fp64 rows; zeros and NaN of a row that is not finite."""
    m = p.abs().amax(1)
    fine = torch.isfinite(m)
    top = torch.where(fine & (m > 0), m, torch.ones_like(m))
    codes = torch.where(fine[:, None], (p * 127 / top[:, None]).round(), torch.zeros_like(p))
    return codes, torch.where(fine, m, torch.full_like(m, float("nan")))


def add_norm(x, weight, eps, residual=None):
    """(r, f64 norm rows, codes, scales) of CPU tensors of the operator's types."""
    r = x if residual is None else (x.double() + residual.double()).float().to(residual.dtype)
    # the fp32 sum is rounded before the residual's type, as the operator adds in fp32
    z = r.double()
    p = z if weight is None else (z.float() * weight.float()).double()
    f = 1 / ((z * z).mean(1) + eps).sqrt()
    codes, m = quant(p)
    return r, p * f[:, None], codes, m * f / 127


def linear(x, xs, w, ws, bias=None):
    y = (x.double() @ w.double().T) * xs.double()[:, None] * ws.double()
    return y if bias is None else y + bias.double()


def linear_bound(x, xs, w, ws, bias, dtype):
    """|result - linear()| at most: the sum's conversion, the scales' product,
    theirs and the bias's addition are an fp32 rounding each, then the type's."""
    y = linear(x, xs, w, ws)
    total = y.abs() if bias is None else y.abs() + bias.double().abs()
    bound = 4 * HALF_STEP[torch.float32] * total
    if dtype == torch.bfloat16:
        bound = bound + HALF_STEP[dtype] * (total + bound)
    return bound + 1e-38


def mlp(x, xs, gate_up, gus, down, ds):
    """(result, 64-bit h) with h rounded to bf16 and brought to codes between
    the products, as the operator does."""
    g, u = linear(x, xs, gate_up, gus).chunk(2, 1)
    h = g / (1 + torch.exp(-g)) * u
    codes, m = quant(h.to(torch.bfloat16).double())
    return linear(codes, m / 127, down, ds), h
