"""What is measured of the 8-bit integer operators: rows to int8 codes with one
scale a row, the residual's addition with the root-mean-square norm and its
int8 output, the int8 linear layer, and the int8 SwiGLU MLP made of them.

An int8 row r stands for codes[r] * scale[r], codes in [-127, 127], with
scale = max|row| / 127 and codes = the nearest whole number to
127 * row / max|row| (a tie to the even one); a row of zeros has the scale 0.
Codes depend on exact quotients, so the plain form takes them in 64 bits.
"""
import torch

own = False  # run(): False the plain form, True the framework's calls

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _q4():
    import bit_codebook_quantized_router_b200 as q4
    return q4


def listed():
    return [
        # one token of a decode step, H of the framework's layer: launch latency
        {"name": "add_norm_t1", "op": "add_norm", "T": 1, "H": 6144, "x": "bf16", "res": "bf16"},
        # a ragged batch whose residual stream is kept in fp32 and takes the layer's fp32 result
        {"name": "add_norm_t777_f32", "op": "add_norm", "T": 777, "H": 1021, "x": "f32", "res": "f32"},
        # a prefill batch: bandwidth
        {"name": "add_norm_t8192", "op": "add_norm", "T": 8192, "H": 6144, "x": "bf16", "res": "bf16"},
        # activations of a small decode batch ahead of a down projection
        {"name": "quant_rows_t8", "op": "quant_rows", "T": 8, "H": 2048, "x": "bf16"},
        # the rows of a gate/up weight matrix, brought to int8 when a model is loaded
        {"name": "quant_rows_4096x6144", "op": "quant_rows", "T": 4096, "H": 6144, "x": "bf16"},
        # one token through a square projection: the weights' bytes
        {"name": "linear_t1", "op": "linear", "T": 1, "N": 6144, "K": 6144, "out": "bf16", "bias": False},
        # a decode batch at odd sizes, with a bias and fp32 results
        {"name": "linear_t45_odd", "op": "linear", "T": 45, "N": 1003, "K": 1990, "out": "f32", "bias": True},
        # a large decode batch or a short prompt
        {"name": "linear_t256", "op": "linear", "T": 256, "N": 6144, "K": 2048, "out": "bf16", "bias": False},
        # a prefill batch: the tensor cores
        {"name": "linear_t8192", "op": "linear", "T": 8192, "N": 6144, "K": 6144, "out": "bf16", "bias": False},
        # the shared expert's MLP for one token
        {"name": "mlp_t1", "op": "mlp", "T": 1, "H": 6144, "I": 2048},
        # a decode batch through a small MLP of odd sizes
        {"name": "mlp_t33_odd", "op": "mlp", "T": 33, "H": 1000, "I": 523},
        # a prefill batch through the shared expert's MLP
        {"name": "mlp_t2048", "op": "mlp", "T": 2048, "H": 6144, "I": 2048},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["add_norm", "quant_rows", "linear", "mlp"])
    T = _log(rng, 1, 8192)
    size = lambda lo, hi: (lambda v: v if rng.random() < 0.5 else max(64, v // 64 * 64))(_log(rng, lo, hi))  # noqa: E731
    if op == "add_norm":
        return {"op": op, "T": T, "H": size(64, 6144), "x": rng.choice(["bf16", "f32"]), "res": rng.choice(["bf16", "f32"])}
    if op == "quant_rows":
        return {"op": op, "T": T, "H": size(64, 6144), "x": rng.choice(["bf16", "f32"])}
    if op == "linear":
        return {"op": op, "T": T, "N": size(64, 6144), "K": size(64, 6144), "out": rng.choice(["bf16", "f32"]), "bias": rng.random() < 0.5}
    return {"op": op, "T": min(T, 2048), "H": size(64, 6144), "I": size(64, 2048)}


def _codes(p, amax):
    """Codes of the rows p (as floats) for the rows' largest magnitudes."""
    top = torch.where(amax > 0, amax, torch.ones_like(amax)).double()
    return (p.double() * 127 / top[:, None]).round()


def _int8(v):
    """fp32 rows as int8 codes, each row on a 16-byte boundary, and their scales."""
    amax = v.abs().amax(1)
    T, K = v.shape
    q = torch.zeros((T, -(-K // 16) * 16), dtype=torch.int8, device=v.device)[:, :K]
    q.copy_(_codes(v, amax))
    return q, amax / 127


def _activations(T, H, g):
    """Hidden states as a layer meets them: normal, a channel in 61 an outlier, and a padding row of zeros in longer batches."""
    x = torch.randn((T, H), generator=g, device="cuda")
    x[:, 7::61] *= 8
    if T > 4:
        x[T // 2] = 0
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, T = case["op"], case["T"]
    s = {"op": op}
    if op in ("add_norm", "quant_rows"):
        H = case["H"]
        s["x"] = _activations(T, H, g).to(TYPES[case["x"]])
        s["q"] = torch.empty((T, -(-H // 16) * 16), dtype=torch.int8, device="cuda")[:, :H]
        s["scale"] = torch.empty(T, device="cuda")
        if op == "add_norm":
            s["residual"] = (4 * _activations(T, H, g)).to(TYPES[case["res"]])
            s["weight"] = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
            s["residual_out"] = torch.empty_like(s["residual"])
            s["out"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    elif op == "linear":
        N, K = case["N"], case["K"]
        s["x"], s["x_scale"] = _int8(_activations(T, K, g))
        s["w"], s["w_scale"] = _int8(0.02 * torch.randn((N, K), generator=g, device="cuda"))
        s["bias"] = 0.5 * torch.randn(N, generator=g, device="cuda") if case["bias"] else None
        s["out"] = torch.empty((T, N), dtype=TYPES[case["out"]], device="cuda")
    else:
        H, I = case["H"], case["I"]
        s["x"], s["x_scale"] = _int8(_activations(T, H, g))
        s["gate_up"], s["gate_up_scale"] = _int8(0.02 * torch.randn((2 * I, H), generator=g, device="cuda"))
        s["down"], s["down_scale"] = _int8(0.02 * torch.randn((H, I), generator=g, device="cuda"))
        s["out"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        if own:  # the handle and the workspace that a program keeps
            q4 = _q4()
            s["mlp"] = q4.MlpI8(s["gate_up"], s["gate_up_scale"], s["down"], s["down_scale"])
            s["ws"] = q4.alloc_workspace(q4.mlp_i8_workspace(s["mlp"], T))
    return s


def _values(q, scale):
    """What int8 codes stand for."""
    return q * scale[:, None]


def _run_own(s):
    q4 = _q4()
    if s["op"] == "add_norm":
        r, out, q, scale = q4.add_norm(s["x"], s["weight"], EPS, residual=s["residual"], residual_out=s["residual_out"], out=s["out"], q=s["q"], scale=s["scale"])
        return r, out, _values(q, scale), scale
    if s["op"] == "quant_rows":
        q, scale = q4.quant_rows(s["x"], q=s["q"], scale=s["scale"])
        return _values(q, scale), scale
    if s["op"] == "linear":
        return q4.linear_i8(s["x"], s["x_scale"], s["w"], s["w_scale"], bias=s["bias"], out=s["out"])
    return q4.mlp_i8(s["mlp"], s["x"], s["x_scale"], out=s["out"], ws=s["ws"])


def _plain_linear(x, x_scale, w, w_scale):
    return (x.float() @ w.float().T) * x_scale[:, None] * w_scale


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "add_norm":
        # the norm is taken of the residual as it is stored
        r = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
        z = r.float()
        p = z * s["weight"].float()
        rstd = torch.rsqrt(z.square().mean(1) + EPS)
        amax = p.abs().amax(1)
        scale = amax * rstd / 127
        return r, (p * rstd[:, None]).to(torch.bfloat16), _codes(p, amax).float() * scale[:, None], scale
    if s["op"] == "quant_rows":
        x = s["x"].float()
        amax = x.abs().amax(1)
        scale = amax / 127
        return _codes(x, amax).float() * scale[:, None], scale
    if s["op"] == "linear":
        y = _plain_linear(s["x"], s["x_scale"], s["w"], s["w_scale"])
        return (y if s["bias"] is None else y + s["bias"]).to(s["out"].dtype)
    g, u = _plain_linear(s["x"], s["x_scale"], s["gate_up"], s["gate_up_scale"]).chunk(2, 1)
    # between the products the operator holds bf16 rows and their int8 codes
    h = (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16).float()
    amax = h.abs().amax(1)
    return _plain_linear(_codes(h, amax), amax / 127, s["down"], s["down_scale"]).to(torch.bfloat16)


def work(case):
    op, T = case["op"], case["T"]
    size = {"bf16": 2, "f32": 4}
    if op == "add_norm":
        H = case["H"]
        return {"bytes": T * H * (size[case["x"]] + 2 * size[case["res"]] + 2 + 1) + 2 * H + 4 * T, "flops": 8 * T * H}
    if op == "quant_rows":
        H = case["H"]
        return {"bytes": T * H * (size[case["x"]] + 1) + 4 * T, "flops": 3 * T * H}
    if op == "linear":
        N, K = case["N"], case["K"]
        return {"bytes": (T + N) * (K + 4) + (4 * N if case["bias"] else 0) + T * N * size[case["out"]], "flops": 2 * T * N * K}
    H, I = case["H"], case["I"]
    return {"bytes": T * (H + 4) + 3 * H * I + 4 * (2 * I + H) + 2 * T * H, "flops": 6 * T * H * I}


def _exact_rows(p):
    """Codes of 64-bit rows: the whole number n with |127 p - n m| least, m the row's largest magnitude."""
    m = p.abs().max(dim=1, keepdim=True).values
    t = 127 * p / m.clamp_min(torch.finfo(torch.float64).tiny)
    return torch.round(t), m[:, 0]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "quant_rows":
        n, m = _exact_rows(s["x"].double())
        return n * (m / 127)[:, None], m / 127
    if op == "add_norm":
        r = (s["x"].double() + s["residual"].double()).to(s["residual"].dtype).double()
        v = r * s["weight"].double()
        # the codes are those of the fp32 products, which decide the ties
        n, m = _exact_rows(v.float().double())
        inv = 1 / (torch.sum(r * r, dim=1) / case["H"] + EPS).sqrt()
        step = m * inv / 127
        return r, v * inv[:, None], n * step[:, None], step
    if op == "linear":
        y = torch.mm(s["x"].double(), s["w"].double().t())
        y = y * torch.outer(s["x_scale"].double(), s["w_scale"].double())
        return y if s["bias"] is None else y + s["bias"].double()
    a = torch.mm(s["x"].double(), s["gate_up"].double().t()) * torch.outer(s["x_scale"].double(), s["gate_up_scale"].double())
    I = case["I"]
    h = a[:, :I] * torch.sigmoid(a[:, :I]) * a[:, I:]
    n, m = _exact_rows(h.to(torch.bfloat16).double())
    return torch.mm(n, s["down"].double().t()) * torch.outer(m / 127, s["down_scale"].double())
