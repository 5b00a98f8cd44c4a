"""The FP8 (e4m3, one scale per block of 128) feed-forward operators, as they are measured.

Four operators that follow one another in a feed-forward block held in 8-bit floating point:

``norm``   s = x + residual; q, d = e4m3(RMSNorm(s) * gamma)     -> q, d, s
``act``    q, d = e4m3(x)                                        -> q, d
``up``     q, d = e4m3(SiLU(g) * u), (g | u) = x_hat (gate | up)^T  -> q, d
``mm``     y = x_hat W^T (+ residual)                            -> y

Quantization, per row and block of 128 columns (the last one may be shorter): with
a = max(max|v|, 2^-100), the code of v is e4m3(v * fl32(448 / a)), rounded to nearest even, and the
block's scale is fl32(a / 448).  Weights have one scale per 128 x 128 block.

``run`` gives each operator in elementary torch operations, or, where ``own`` is set, through this
package's entry points.  Codes are returned as float8_e4m3fn tensors and scales as float32.
"""

import math

import torch

own = False

BLOCK = 128
EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one token of a 0.8B-shaped decoder entering its feed-forward block
        {"name": "norm-token", "op": "norm", "rows": 1, "k": 1024, "type": "f32"},
        # a 512-row prompt of a 2560-wide model
        {"name": "norm-prompt", "op": "norm", "rows": 512, "k": 2560, "type": "bf16"},
        # a long batch of prompts, f32 residual stream, a width that ends inside a block
        {"name": "norm-long", "op": "norm", "rows": 16383, "k": 4112, "type": "f32"},
        # the input of an output projection for a few dozen sequences decoded together
        {"name": "act-batch", "op": "act", "rows": 33, "k": 3584, "type": "f32"},
        # the same for a long prompt
        {"name": "act-prompt", "op": "act", "rows": 8192, "k": 9216, "type": "bf16"},
        # gate|up of one token, 0.8B shape
        {"name": "up-token", "op": "up", "rows": 1, "n": 3584, "k": 1024},
        # gate|up of a 512-row prompt, 0.8B shape
        {"name": "up-512", "op": "up", "rows": 512, "n": 3584, "k": 1024},
        # gate|up of a long prompt, 2560-wide model
        {"name": "up-prompt", "op": "up", "rows": 8192, "n": 9216, "k": 2560},
        # down projection of one token with the residual, 0.8B shape
        {"name": "mm-token", "op": "mm", "rows": 1, "n": 1024, "k": 3584, "residual": True, "type": "f32"},
        # down projection of a few sequences decoded together, 2560-wide model
        {"name": "mm-batch", "op": "mm", "rows": 7, "n": 2560, "k": 9216, "residual": True, "type": "bf16"},
        # a ragged chunk through a projection whose sides end inside a block
        {"name": "mm-ragged", "op": "mm", "rows": 100, "n": 2727, "k": 3600, "residual": False, "type": "f32"},
        # down projection of a long prompt, 2560-wide model
        {"name": "mm-prompt", "op": "mm", "rows": 4096, "n": 2560, "k": 9216, "residual": True, "type": "bf16"},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "act", "up", "mm"])
    k = 16 * _log_between(rng, 16, 576)
    if op in ("norm", "act"):
        rows = _log_between(rng, 1, min(16384, (1 << 26) // k))
        return {"op": op, "rows": rows, "k": k, "type": rng.choice(["f32", "bf16"])}
    rows = _log_between(rng, 1, 8192)
    if op == "up":
        return {"op": op, "rows": rows, "n": 16 * _log_between(rng, 8, 576), "k": min(k, 4096)}
    return {"op": op, "rows": rows, "n": _log_between(rng, 100, 9216), "k": k, "residual": rng.random() < 0.5,
            "type": rng.choice(["f32", "bf16"])}


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


# ---------------------------------------------------------------------------
# the operators in elementary operations
# ---------------------------------------------------------------------------

def _quantize(v):
    """f32 [rows, k] -> (e4m3 [rows, k], f32 [rows, ceil(k / 128)])."""
    rows, k = v.shape
    kb = _blocks(k)
    p = torch.nn.functional.pad(v, (0, kb * BLOCK - k)).view(rows, kb, BLOCK)
    a = p.abs().amax(dim=2).clamp_min(2.0 ** -100)
    # true divisions of tensors: a division by a Python number may become a product with its reciprocal
    top = torch.full_like(a, 448.0)
    q = (p * (top / a).unsqueeze(2)).to(torch.float8_e4m3fn).view(rows, kb * BLOCK)[:, :k]
    return q.contiguous(), a / top


def _activations(q, d):
    return q.float() * d.repeat_interleave(BLOCK, dim=1)[:, :q.shape[1]]


def _weights(q, d):
    n, k = q.shape
    return q.float() * d.repeat_interleave(BLOCK, dim=0)[:n].repeat_interleave(BLOCK, dim=1)[:, :k]


def _plain_norm(x, residual, gamma):
    s = x + residual  # one rounding to the stream's type
    f = s.double()
    r = (1.0 / torch.sqrt(f.square().mean(dim=1, keepdim=True) + EPS)).float()
    q, d = _quantize(s.float() * r * gamma.float())
    return q, d, s


def _plain_up(s):
    n = s["n"]
    x = _activations(s["xq"], s["xd"])
    g = x @ _weights(s["wq"][:n], s["wd"][:_blocks(n)]).t()
    u = x @ _weights(s["wq"][n:], s["wd"][_blocks(n):]).t()
    return _quantize(g / (1.0 + torch.exp(-g)) * u)


def _plain_mm(s):
    y = _activations(s["xq"], s["xd"]) @ _weights(s["wq"], s["wd"]).t()
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["type"])


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _stream(rows, k, gen):
    """Hidden states: unit normal, a few channels far larger than the rest."""
    x = torch.randn((rows, k), generator=gen, device="cuda")
    loud = torch.randperm(k, generator=gen, device="cuda")[: max(1, k // 256)]
    x[:, loud] *= 16.0
    return x


def _weight(n, k, gen):
    """N(0, 0.02) weights with one scale for each 128 x 128 block, both sides padded with zeros to quantize."""
    nb, kb = _blocks(n), _blocks(k)
    w = torch.zeros((nb * BLOCK, kb * BLOCK), device="cuda")
    w[:n, :k] = 0.02 * torch.randn((n, k), generator=gen, device="cuda")
    w = w.view(nb, BLOCK, kb, BLOCK)
    a = w.abs().amax(dim=(1, 3)).clamp_min(2.0 ** -100)
    q = (w * (448.0 / a)[:, None, :, None]).to(torch.float8_e4m3fn).view(nb * BLOCK, kb * BLOCK)
    return q[:n, :k].contiguous(), a / 448.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, rows, k = case["op"], case["rows"], case["k"]
    s = {"op": op, "rows": rows, "k": k}
    x = _stream(rows, k, gen)
    if rows > 4:
        x[-1] = 0.0  # the padding row of a batch
    if op == "act":
        s["x"] = x.to(TYPES[case["type"]])
    elif op == "norm":
        t = TYPES[case["type"]]
        s["x"] = x.to(t)
        s["residual"] = (0.5 * torch.randn((rows, k), generator=gen, device="cuda")).to(t)
        s["gamma"] = (1.0 + 0.1 * torch.randn((k,), generator=gen, device="cuda")).to(t)
        if rows > 4:
            s["residual"][-1] = 0.0
    else:
        s["xq"], s["xd"] = _quantize(x)
        n = s["n"] = case["n"]
        if op == "up":
            halves = [_weight(n, k, gen) for _ in range(2)]
            s["wq"] = torch.cat([h[0].view(torch.uint8) for h in halves]).view(torch.float8_e4m3fn)
            s["wd"] = torch.cat([h[1] for h in halves])
        else:
            s["wq"], s["wd"] = _weight(n, k, gen)
            s["type"] = TYPES[case["type"]]
            s["residual"] = torch.randn((rows, n), generator=gen, device="cuda").to(s["type"]) \
                if case["residual"] else None
    return s


def run(state):
    s = state
    if not own:
        if s["op"] == "norm":
            return _plain_norm(s["x"], s["residual"], s["gamma"])
        if s["op"] == "act":
            return _quantize(s["x"].float())
        return _plain_up(s) if s["op"] == "up" else _plain_mm(s)

    import block_quantized_decode_rmsnorm_gb300 as qg

    if s["op"] == "norm":
        return qg.rmsnorm_add_quantize_e4m3(s["x"], s["gamma"], s["residual"], EPS)
    if s["op"] == "act":
        return qg.quantize_act_e4m3(s["x"])
    w = qg.E4M3Weight(s["wq"], s["wd"])
    if s["op"] == "up":
        return qg.qg_ffn_up_e4m3(w, s["xq"], s["xd"])
    return qg.qgemm_e4m3(w, s["xq"], s["xd"], epilogue="none" if s["residual"] is None else "residual",
                         residual=s["residual"], out_dtype=s["type"])


def work(case):
    op, rows, k = case["op"], case["rows"], case["k"]
    size = {"f32": 4, "bf16": 2}.get(case.get("type"), 0)
    codes = lambda r, c: r * c + 4 * r * _blocks(c)  # noqa: E731
    if op == "act":
        return {"bytes": size * rows * k + codes(rows, k), "flops": 3 * rows * k}
    if op == "norm":
        return {"bytes": 3 * size * rows * k + size * k + codes(rows, k), "flops": 8 * rows * k}
    n = case["n"]
    if op == "up":
        return {"bytes": 2 * n * k + 8 * _blocks(n) * _blocks(k) + codes(rows, k) + codes(rows, n),
                "flops": 4 * rows * n * k}
    moved = n * k + 4 * _blocks(n) * _blocks(k) + codes(rows, k) + size * rows * n * (2 if case["residual"] else 1)
    return {"bytes": moved, "flops": 2 * rows * n * k}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_round_e4m3(v):
    """f64 -> the nearest value of 4 significant bits down to 2^-6, multiples of 2^-9 below; ties to even."""
    exponent = torch.frexp(v).exponent.sub(1).clamp_min(-6)
    step = torch.ldexp(torch.ones_like(v), exponent - 3)
    return torch.round(v / step) * step


def _exact_codes(v):
    """f64 [rows, k] -> (the codes' values, the scales) in f64, block by block."""
    codes, scales = torch.empty_like(v), []
    for c in range(0, v.shape[1], BLOCK):
        b = v[:, c:c + BLOCK]
        a = b.abs().max(dim=1).values.clamp_min(2.0 ** -100)
        inverse = (448.0 / a).float().double()  # the definition's one f32 rounding
        codes[:, c:c + BLOCK] = _exact_round_e4m3((b * inverse[:, None]).float().double())
        scales.append((a / 448.0).float().double())
    return codes, torch.stack(scales, dim=1)


def _exact_product(xq, xd, wq, wd):
    x, w = xq.double(), wq.double()
    y = torch.zeros((x.shape[0], w.shape[0]), dtype=torch.float64, device=x.device)
    rows_of = torch.arange(w.shape[0], device=x.device) // BLOCK
    for j, c in enumerate(range(0, x.shape[1], BLOCK)):
        part = x[:, c:c + BLOCK] @ w[:, c:c + BLOCK].t()
        y += part * xd[:, j].double()[:, None] * wd[:, j].double()[rows_of][None, :]
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "act":
        return _exact_codes(s["x"].double())
    if s["op"] == "norm":
        t = (s["x"].double() + s["residual"].double()).to(s["x"].dtype).double()
        r = t.square().mean(dim=1).add(EPS).sqrt().reciprocal().float().double()
        # two f32 products, as the operator is defined
        v = ((t * r[:, None]).float().double() * s["gamma"].double()).float().double()
        q, d = _exact_codes(v)
        return q, d, t
    if s["op"] == "up":
        n, nb = s["n"], _blocks(s["n"])
        g = _exact_product(s["xq"], s["xd"], s["wq"][:n], s["wd"][:nb])
        u = _exact_product(s["xq"], s["xd"], s["wq"][n:], s["wd"][nb:])
        return _exact_codes(g * torch.sigmoid(g) * u)
    y = _exact_product(s["xq"], s["xd"], s["wq"], s["wd"])
    return y if s["residual"] is None else y + s["residual"].double()
