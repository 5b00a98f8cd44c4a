"""The paged, block-quantized key-value cache and the attention that reads it, as they are measured.

Three operators of a decode step between its projections:

``write``  k, v [rows, heads, dim] quantized into the cache at given slots   -> the cache's codes and scales
``read``   the cached rows at given slots, dequantized                       -> k, v [rows, heads, dim]
``attn``   o = softmax(scale q K^T) V of one new token per sequence          -> o [batch, q_heads, dim]

The cache holds pages of ``page`` tokens: codes [pages, heads, page, dim] and scales [pages, heads, page, blocks];
slot s is token s % page of page s // page.  Two formats, by row of ``dim`` values:

``q8_0``  blocks of 32: d = fl32(max|v| / 127), code = fl32(v / d) rounded half away from zero, scale binary16(d)
``e4m3``  blocks of 128 (the last may be shorter): a = max(max|v|, 2^-100), code = e4m3(v * fl32(448 / a)),
          scale fl32(a / 448)

``run`` gives each operator in elementary torch operations, or, where ``own`` is set, through this
package's entry points.
"""

import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BLOCK = {"q8_0": 32, "e4m3": 128}


def listed():
    return [
        # one token's key and value of a small model, two heads
        {"name": "write-token", "op": "write", "format": "q8_0", "rows": 1, "heads": 2, "dim": 128, "page": 16,
         "prompt": False, "type": "f32"},
        # the new tokens of a batch of sequences decoded together, a few rows of it padding
        {"name": "write-batch", "op": "write", "format": "e4m3", "rows": 67, "heads": 8, "dim": 128, "page": 64,
         "prompt": False, "type": "bf16"},
        # a long prompt
        {"name": "write-prompt", "op": "write", "format": "q8_0", "rows": 8192, "heads": 8, "dim": 128, "page": 16,
         "prompt": True, "type": "bf16"},
        # a ragged chunk of a model with an odd number of narrower heads
        {"name": "read-ragged", "op": "read", "format": "e4m3", "rows": 777, "heads": 5, "dim": 96, "page": 48,
         "prompt": True, "type": "f32"},
        # a cached prefix brought back for a chunk of prompt that attends to it
        {"name": "read-prompt", "op": "read", "format": "q8_0", "rows": 16384, "heads": 8, "dim": 128, "page": 16,
         "prompt": True, "type": "bf16"},
        # one sequence, a short context, a small model
        {"name": "attn-token", "op": "attn", "format": "q8_0", "batch": 1, "length": 700, "heads": 2, "group": 4,
         "dim": 128, "page": 16, "window": 0, "type": "f32"},
        # one sequence, a long document
        {"name": "attn-document", "op": "attn", "format": "q8_0", "batch": 1, "length": 131072, "heads": 8, "group": 4,
         "dim": 128, "page": 64, "window": 0, "type": "bf16"},
        # serving: sequences of very different lengths
        {"name": "attn-serving", "op": "attn", "format": "q8_0", "batch": 64, "length": 8192, "heads": 8, "group": 8,
         "dim": 128, "page": 16, "window": 0, "type": "bf16"},
        # the same in 8-bit floating point, more query heads to a key head
        {"name": "attn-serving-e4m3", "op": "attn", "format": "e4m3", "batch": 48, "length": 6000, "heads": 4,
         "group": 16, "dim": 128, "page": 32, "window": 0, "type": "bf16"},
        # many short conversations, every query head with a key head of its own
        {"name": "attn-chats", "op": "attn", "format": "q8_0", "batch": 256, "length": 1000, "heads": 16, "group": 1,
         "dim": 64, "page": 16, "window": 0, "type": "bf16"},
        # layers that look back over a window, wide heads
        {"name": "attn-window", "op": "attn", "format": "e4m3", "batch": 32, "length": 16384, "heads": 4, "group": 2,
         "dim": 256, "page": 64, "window": 1024, "type": "f32"},
        # odd everything: heads, group, dim, page
        {"name": "attn-odd", "op": "attn", "format": "q8_0", "batch": 7, "length": 4999, "heads": 3, "group": 5,
         "dim": 96, "page": 48, "window": 0, "type": "f32"},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn"])
    c = {"op": op, "format": rng.choice(["q8_0", "e4m3"]), "heads": _log_between(rng, 1, 16),
         "dim": rng.choice([64, 96, 128, 192, 256]), "page": 16 * _log_between(rng, 1, 16),
         "type": rng.choice(["f32", "bf16"])}
    if op != "attn":
        c["rows"] = _log_between(rng, 1, min(16384, (1 << 24) // (c["heads"] * c["dim"])))
        c["prompt"] = c["rows"] > 256 or rng.random() < 0.5
        return c
    c["group"] = _log_between(rng, 1, 32)
    c["batch"] = _log_between(rng, 1, 256)
    room = (1 << 27) // (c["heads"] * c["dim"] * c["batch"])
    c["length"] = _log_between(rng, 1, max(2, min(131072, room)))
    c["window"] = _log_between(rng, 1, c["length"]) if rng.random() < 0.3 else 0
    return c


def _blocks(c):
    return -(-c["dim"] // BLOCK[c["format"]])


def _lengths(c):
    """The sequences' lengths: the longest first, the others spread below it, one slot of a batch unused."""
    n = [max(1, int(c["length"] * ((i * 0.6180339887498949) % 1.0))) for i in range(c["batch"])]
    n[0] = c["length"]
    if c["batch"] > 4:
        n[3] = 0
    return n


# ---------------------------------------------------------------------------
# the operators in elementary operations
# ---------------------------------------------------------------------------

def _quantize(v, fmt):
    """f32 [..., dim] -> (codes [..., dim], scales [..., blocks])."""
    dim, block = v.shape[-1], BLOCK[fmt]
    nb = -(-dim // block)
    p = torch.nn.functional.pad(v, (0, nb * block - dim)).unflatten(-1, (nb, block))
    a = p.abs().amax(dim=-1)
    if fmt == "q8_0":
        d = a / torch.full_like(a, 127.0)  # true divisions of tensors
        t = p / torch.where(d == 0, torch.ones_like(d), d).unsqueeze(-1)
        t = torch.sign(t) * torch.floor(t.abs().double() + 0.5).float()  # half away from zero
        return t.clamp(-127, 127).to(torch.int8).flatten(-2)[..., :dim], d.half()
    a = a.clamp_min(2.0 ** -100)
    top = torch.full_like(a, 448.0)
    q = (p * (top / a).unsqueeze(-1)).to(torch.float8_e4m3fn).flatten(-2)[..., :dim]
    return q, a / top


def _values(q, d, fmt):
    return q.float() * d.float().repeat_interleave(BLOCK[fmt], dim=-1)[..., :q.shape[-1]]


def _bytes(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t  # indexing 8-bit floats by their bits


def _plain_write(s):
    page, at = s["page"], s["slots"] >= 0
    where = s["slots"][at]
    for x, codes, scales in ((s["k"], s["kq"], s["kd"]), (s["v"], s["vq"], s["vd"])):
        q, d = _quantize(x[at].float(), s["format"])
        _bytes(codes)[where // page, :, where % page] = _bytes(q)
        scales[where // page, :, where % page] = d
    return s["kq"], s["kd"], s["vq"], s["vd"]


def _plain_read(s):
    page, slots = s["page"], s["slots"]
    out = []
    for codes, scales in ((s["kq"], s["kd"]), (s["vq"], s["vd"])):
        q = _bytes(codes)[slots // page, :, slots % page].view(codes.dtype)
        out.append(_values(q, scales[slots // page, :, slots % page], s["format"]).to(s["type"]))
    return tuple(out)


def _gathered(codes, scales, pages, fmt):
    """The sequences' rows, [batch, heads, pages * page, dim]."""
    q, d = _bytes(codes)[pages].view(codes.dtype), scales[pages]  # [batch, pages, heads, page, .]
    return _values(q, d, fmt).transpose(1, 2).flatten(2, 3)


def _plain_attn(s):
    q, lengths, pages = s["q"].float(), s["lengths"].long(), s["pages"].long()
    page = s["page"]
    batch, q_heads, dim = q.shape
    column = torch.arange(pages.shape[1], device=q.device).expand(batch, -1)
    if s["window"]:  # the columns of the page table that the window may touch
        column = column[:, :-(-s["window"] // page) + 1] + ((lengths - s["window"]).clamp_min(0) // page)[:, None]
        pages = pages.gather(1, column.clamp_max(pages.shape[1] - 1))
    t = (column[:, :, None] * page + torch.arange(page, device=q.device)).flatten(1)  # the rows' positions
    seen = t < lengths[:, None]
    if s["window"]:
        seen &= t >= lengths[:, None] - s["window"]
    k = _gathered(s["kq"], s["kd"], pages, s["format"])
    heads = k.shape[1]
    score = q.view(batch, heads, q_heads // heads, dim) @ k.transpose(2, 3) * (1.0 / math.sqrt(dim))
    del k
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(dim=-1, keepdim=True)
    o = p @ _gathered(s["vq"], s["vd"], pages, s["format"])
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.reshape(batch, q_heads, dim).to(s["type"])


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _rows(shape, gen):
    """Keys or values: unit normal, a few channels of every head far larger than the rest."""
    x = torch.randn(shape, generator=gen, device="cuda")
    loud = torch.randperm(shape[-1], generator=gen, device="cuda")[: max(1, shape[-1] // 48)]
    x[..., loud] *= 6.0
    return x


def _fill(s, pages, c, gen):
    shape = (pages, c["heads"], c["page"], c["dim"])
    s["kq"], s["kd"] = _quantize(_rows(shape, gen), c["format"])
    s["vq"], s["vd"] = _quantize(_rows(shape, gen), c["format"])
    for name in ("kq", "kd", "vq", "vd"):
        s[name] = s[name].contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = case
    op, heads, dim, page = c["op"], c["heads"], c["dim"], c["page"]
    s = {"op": op, "format": c["format"], "page": page, "type": TYPES[c["type"]]}
    if op == "attn":
        lengths = _lengths(c)
        held = [-(-n // page) for n in lengths]
        total, most = sum(held), max(held)
        pool = torch.randperm(total + 3, generator=gen, device="cuda")[:total].int()  # pages in any order
        s["pages"] = torch.zeros((c["batch"], most), dtype=torch.int32, device="cuda")
        used = torch.arange(most, device="cuda") < torch.tensor(held, device="cuda")[:, None]
        s["pages"][used] = pool
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        _fill(s, total + 3, c, gen)
        s["q"] = torch.randn((c["batch"], heads * c["group"], dim), generator=gen, device="cuda").to(s["type"])
        s["window"] = c["window"]
    else:
        rows = c["rows"]
        pages = -(-rows // page) + 2
        if c["prompt"]:  # runs of consecutive tokens over pages in any order
            order = torch.randperm(pages, generator=gen, device="cuda")
            at = torch.arange(rows, device="cuda")
            s["slots"] = order[at // page] * page + at % page
        else:  # one token of many sequences
            s["slots"] = torch.randperm(pages * page, generator=gen, device="cuda")[:rows]
        _fill(s, pages, c, gen)
        if op == "write":
            if rows > 64:
                s["slots"][-2:] = -1  # the padding rows of a batch
            # keys and values are parts of a stacked projection's rows
            qkv = _rows((rows, 4 * heads, dim), gen).to(s["type"])
            s["k"], s["v"] = qkv[:, 2 * heads:3 * heads], qkv[:, 3 * heads:]
    if own:
        import block_quantized_decode_rmsnorm_gb300 as qg

        s["cache"] = qg.KVCache(s["kq"], s["kd"], s["vq"], s["vd"])
        if op == "attn":
            s["work"] = qg.AttnWork.allocate(heads * c["group"], heads, dim, "cuda")
    return s


def run(state):
    s = state
    if not own:
        if s["op"] == "write":
            return _plain_write(s)
        return _plain_read(s) if s["op"] == "read" else _plain_attn(s)

    import block_quantized_decode_rmsnorm_gb300 as qg

    if s["op"] == "write":
        qg.qg_kv_write(s["cache"], s["k"], s["v"], s["slots"])
        return s["kq"], s["kd"], s["vq"], s["vd"]
    if s["op"] == "read":
        return qg.qg_kv_read(s["cache"], s["slots"], s["type"])
    return qg.qg_attn_decode(s["q"], s["cache"], s["pages"], s["lengths"], window=s["window"], work=s["work"])


def work(case):
    c = case
    size = {"f32": 4, "bf16": 2}[c["type"]]
    row = c["dim"] + _blocks(c) * (2 if c["format"] == "q8_0" else 4)  # a cached row's codes and scales
    if c["op"] != "attn":
        n = 2 * c["rows"] * c["heads"]
        return {"bytes": n * (row + size * c["dim"]) + 8 * c["rows"],
                "flops": n * c["dim"] * (4 if c["op"] == "write" else 1)}
    seen = [min(n, c["window"]) if c["window"] else n for n in _lengths(c)]
    q = c["batch"] * c["heads"] * c["group"] * c["dim"]
    return {"bytes": 2 * sum(seen) * c["heads"] * row + 2 * size * q + 4 * sum(-(-n // c["page"]) for n in seen),
            "flops": 4 * sum(seen) * c["heads"] * c["group"] * c["dim"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_e4m3(v):
    """f64 -> the nearest value of 4 significant bits down to 2^-6, multiples of 2^-9 below; ties to even."""
    exponent = torch.frexp(v).exponent.sub(1).clamp(-6, 8)
    steps = torch.tensor([2.0 ** (e - 3) for e in range(-6, 9)], dtype=torch.float64, device=v.device)
    step = steps[exponent.long() + 6]
    return torch.round(v / step) * step


def _exact_row(x, fmt):
    """f64 [rows, heads, dim] -> codes' values and scales, block by block."""
    codes, scales = torch.empty_like(x), []
    for c in range(0, x.shape[-1], BLOCK[fmt]):
        b = x[..., c:c + BLOCK[fmt]]
        a = b.abs().max(dim=-1).values
        if fmt == "q8_0":
            d = (a / 127).float().double()  # the definition's f32 roundings
            t = (b / torch.where(d > 0, d, torch.ones_like(d))[..., None]).float().double()
            codes[..., c:c + BLOCK[fmt]] = torch.where(t < 0, -(0.5 - t).floor(), (t + 0.5).floor()).clamp(-127, 127)
            scales.append(d.half().double())
        else:
            a = a.clamp_min(2.0 ** -100)
            inverse = (448.0 / a).float().double()
            codes[..., c:c + BLOCK[fmt]] = _exact_e4m3((b * inverse[..., None]).float().double())
            scales.append((a / 448.0).float().double())
    return codes, torch.stack(scales, dim=-1)


def _exact_values(codes, scales, fmt):
    v = codes.double()
    for j in range(scales.shape[-1]):
        at = slice(j * BLOCK[fmt], min((j + 1) * BLOCK[fmt], v.shape[-1]))
        v[..., at] *= scales[..., j:j + 1].double()
    return v


def exact(case, seed):
    s = prepare(case, seed)
    fmt, page = s["format"], s["page"]
    if s["op"] == "write":
        out = []
        keep = (s["slots"] >= 0).nonzero()[:, 0]
        p, o = s["slots"][keep] // page, s["slots"][keep] % page
        for x, codes, scales in ((s["k"], s["kq"], s["kd"]), (s["v"], s["vq"], s["vd"])):
            q, d = _exact_row(x[keep].double(), fmt)
            all_q, all_d = codes.double(), scales.double()
            all_q[p, :, o], all_d[p, :, o] = q, d
            out += [all_q.to(torch.int8) if fmt == "q8_0" else all_q, all_d]
        return tuple(out)
    if s["op"] == "read":
        out = []
        for codes, scales in ((s["kq"], s["kd"]), (s["vq"], s["vd"])):
            flat_q, flat_d = codes.transpose(1, 2).flatten(0, 1), scales.transpose(1, 2).flatten(0, 1)
            q = flat_q.view(torch.uint8)[s["slots"]].view(codes.dtype)
            out.append(_exact_values(q, flat_d[s["slots"]], fmt))
        return tuple(out)
    q, lengths = s["q"].double(), s["lengths"].tolist()
    heads = s["kq"].shape[1]
    o = torch.zeros_like(q)
    for b, n in enumerate(lengths):
        first = max(0, n - s["window"]) if s["window"] else 0
        if n == 0:
            continue
        at = torch.arange(first, n, device=q.device)
        p = s["pages"][b].long()[at // page]
        rows = []
        for codes, scales in ((s["kq"], s["kd"]), (s["vq"], s["vd"])):
            picked = codes.view(torch.uint8)[p, :, at % page].view(codes.dtype)
            rows.append(_exact_values(picked, scales[p, :, at % page], fmt))  # [tokens, heads, dim]
        x = torch.einsum("hgd,thd->hgt", q[b].unflatten(0, (heads, -1)), rows[0]) / math.sqrt(q.shape[2])
        o[b] = torch.einsum("hgt,thd->hgd", torch.softmax(x, dim=-1), rows[1]).flatten(0, 1)
    return o
