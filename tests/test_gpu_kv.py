"""GPU parity of the key-value cache and its attention against the numpy oracle.

Writing: codes and scales bit for bit (their f32 roundings are part of the definition).
Reading: one f32 product, exact for Q8_0 (8 + 11 bits), then half a step of a bf16 output.

Attention.  A score is a sum of dim products in up to 8 blocks: the tensor core's additions of
a block (at most 8 of them, 2^-22 of the terms each, its own alignment), the split of q (2^-22), the blocks'
additions and the scale's product (10 2^-24): within 2^-18 of the sum of |terms|.  A weight moves by what its score
moves, by the exponent's own rounding (3 2^-24 of |s_t - m|, taken as 2^-22) and by 2^-20 for the exponential, the
product with V's scale and the split to 22 bits; for bf16 outputs instead of the split one rounding to f16, 2^-11.
Weights under 2^-29 of the largest lose bits below f16's range: 2^-36 of the largest, with room.  The sum over
tokens has a depth of n / 64 steps of a warp, the warps' and the splits' sums (64 with room), 2^-24 each; the result is
rounded once, by half a step of its type.
"""

import threading

import numpy as np
import pytest

from oracle import kv as K
from tests._gpu import Guarded, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return need_gpu()


@pytest.fixture(scope="module")
def qg():
    import block_quantized_decode_rmsnorm_gb300 as m

    return m


def types(torch):
    return {"f32": torch.float32, "bf16": torch.bfloat16}


def dev(torch, a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def upload(torch, qg, c):
    """An oracle cache on the device."""
    code = torch.int8 if c["format"] == "q8_0" else torch.float8_e4m3fn
    return qg.KVCache(*(dev(torch, c[n].view(np.uint8)).view(code) if n in "kv" else dev(torch, c[n])
                        for n in ("k", "kd", "v", "vd")))


def download(cache, fmt):
    """The device cache as the oracle holds one."""
    u8 = __import__("torch").uint8
    q = np.int8 if fmt == "q8_0" else np.uint8
    return {"format": fmt, "k": cache.k.view(u8).cpu().numpy().view(q), "kd": cache.k_scales.cpu().numpy(),
            "v": cache.v.view(u8).cpu().numpy().view(q), "vd": cache.v_scales.cpu().numpy()}


def random_cache(rng, fmt, pages, heads, page, dim, spread=0.5):
    """Every code, scales over a few powers of two."""
    c = {"format": fmt}
    for n in "kv":
        shape = (pages, heads, page, dim)
        if fmt == "q8_0":
            c[n] = rng.integers(-127, 128, shape, dtype=np.int8)
            d = np.exp2(spread * rng.standard_normal((*shape[:3], dim // 32))) / 64
            c[n + "d"] = d.astype(np.float16)
        else:
            c[n] = rng.integers(0, 256, shape, dtype=np.uint8)
            c[n][(c[n] & 0x7F) == 0x7F] = 0x30
            d = np.exp2(spread * rng.standard_normal((*shape[:3], K.blocks(dim, fmt)))) / 128
            c[n + "d"] = d.astype(np.float32)
    return c


def tables(rng, lengths, page, pages, extra=1):
    """Page tables of distinct pages in any order; entries past a sequence's tokens are garbage."""
    held = [-(-max(n, 0) // page) for n in lengths]
    pool = rng.permutation(pages)[: sum(held)]
    t = np.full((len(lengths), max(held + [0]) + extra), 2 ** 31 - 1, np.int32)
    i = 0
    for b, n in enumerate(held):
        t[b, :n] = pool[i: i + n]
        i += n
    return t


FORMATS = ["q8_0", "e4m3"]
DIMS = [64, 96, 128, 192, 256]


# ---------------------------------------------------------------- write

def check_write(torch, qg, fmt, kind, x, slots, pages, page, strides="packed"):
    """x: numpy f32 [2, rows, heads, dim]; every slot of the cache is compared, the untouched ones too."""
    rng = np.random.default_rng(9)
    _, rows, heads, dim = x.shape
    before = random_cache(rng, fmt, pages, heads, page, dim)
    cache = upload(torch, qg, before)
    t = torch.from_numpy(x).to(types(torch)[kind])
    if strides == "packed":
        k, v = t[0].cuda(), t[1].cuda()
    elif strides == "stacked":  # parts of a stacked projection's rows
        qkv = torch.full((rows, 4 * heads + 1, dim), float("nan"), dtype=t.dtype, device="cuda")
        k, v = qkv[:, 2 * heads: 3 * heads], qkv[:, 3 * heads: 4 * heads]
        k.copy_(t[0]), v.copy_(t[1])
    else:  # heads outermost
        k, v = (t[i].transpose(0, 1).contiguous().cuda().transpose(0, 1) for i in range(2))
    qg.qg_kv_write(cache, k, v, dev(torch, np.asarray(slots, np.int64)))
    got, want = download(cache, fmt), {n: a.copy() if n != "format" else a for n, a in before.items()}
    xf = t.float().numpy()
    for i, n in enumerate("kv"):
        q, d = K.quantize(xf[i], fmt)
        for r, s in enumerate(slots):
            if 0 <= s < pages * page:
                want[n][s // page, :, s % page], want[n + "d"][s // page, :, s % page] = q[r], d[r]
    for n in ("k", "v"):
        w, g = want[n], got[n]
        if fmt == "e4m3":
            nan = (w & 0x7F) == 0x7F
            assert np.array_equal((g & 0x7F) == 0x7F, nan)
            w, g = np.where(nan, 0, w), np.where(nan, 0, g)
        assert np.array_equal(g, w), (n, np.argwhere(g != w)[:4])
        assert np.array_equal(got[n + "d"], want[n + "d"], equal_nan=True), n


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("rows,heads,page,strides", [(1, 1, 16, "packed"), (1, 2, 16, "stacked"), (5, 3, 48, "packed"),
                                                     (70, 2, 64, "stacked"), (33, 7, 16, "heads"), (130, 1, 112, "heads")])
def test_write(torch, qg, fmt, kind, dim, rows, heads, page, strides):
    rng = np.random.default_rng(rows * 1000 + dim)
    x = (rng.standard_normal((2, rows, heads, dim)) * np.exp(2 * rng.standard_normal((2, rows, heads, 1)))).astype(np.float32)
    x[:, -1, :, : dim // 2] = 0
    pages = -(-rows // page) + 3
    slots = rng.permutation(pages * page)[:rows]
    if rows > 4:
        slots[1], slots[3] = -1, -(2 ** 40)
    if rows > 8:
        slots[6], slots[7], slots[8] = pages * page, 2 ** 32 + 5, 2 ** 62
    check_write(torch, qg, fmt, kind, x, slots, pages, page, strides)


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_many_rows(torch, qg, fmt):
    """Enough rows for the form that takes several a thread, and an end inside its last group."""
    rng = np.random.default_rng(3)
    rows, heads, dim, page = 9999, 4, 128, 16
    x = rng.standard_normal((2, rows, heads, dim)).astype(np.float32)
    pages = -(-rows // page) + 1
    check_write(torch, qg, fmt, "bf16", x, rng.permutation(pages * page)[:rows], pages, page, "stacked")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", FORMATS)
def test_write_special_values(torch, qg, fmt, kind):
    x = np.zeros((2, 8, 1, 128), np.float32)
    x[:, 1, 0, 3] = np.float32(3.3e38)
    x[:, 2, 0] = 1e-35
    x[:, 3, 0, ::2] = 1e-40
    x[:, 4, 0] = (np.arange(128) - 63.5)       # ties
    x[:, 4, 0, ::32] = 127
    x[:, 5, 0, 0], x[:, 5, 0, 1:] = 448, np.tile([0.5, 1.5, 2.5, 17, 19, 416, 432], 19)[:127]
    x[:, 6, 0] = -0.0
    x[:, 7, 0, 5] = 65504 * 127                # the largest binary16 scale
    if fmt == "e4m3":
        x[0, 0, 0, 7], x[1, 0, 0, 9] = np.nan, np.inf
    check_write(torch, qg, fmt, kind, x, np.arange(8), 1, 16)


@pytest.mark.parametrize("exponent", [-101, -100, -99, -60, -7, 0, 60, 119])
def test_write_q8_0_near_ties(torch, qg, exponent):
    """Values within two floats of a half-integer multiple of their block's scale, at scales over the whole range, those for
    which each of the two ways to a code is taken among them."""
    rng = np.random.default_rng(exponent + 200)
    rows, dim = 2048, 256
    top = np.ldexp(rng.uniform(127, 254, (2, rows, 1, dim // 32)), exponent).astype(np.float32)
    d = (top / np.float32(127)).astype(np.float64)[..., None]
    v = ((rng.integers(0, 127, (2, rows, 1, dim // 32, 32)) + 0.5) * d).astype(np.float32)
    for _ in range(2):
        v = np.where(rng.random(v.shape) < 0.4, np.nextafter(v, np.float32(0)), v)
        v = np.where(rng.random(v.shape) < 0.4, np.nextafter(v, np.float32(np.inf)), v)
    v = np.minimum(v, top[..., None]) * rng.choice(np.float32([-1, 1]), v.shape)
    v[..., 9] = top
    check_write(torch, qg, "q8_0", "f32", v.reshape(2, rows, 1, dim), rng.permutation(2064)[:rows], 129, 16)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("dim,rows", [(64, 19999), (96, 13007), (192, 6999), (256, 5003)])
def test_many_rows_of_every_width(torch, qg, fmt, kind, dim, rows):
    """The form that takes two rows a thread, written and read, three heads: rows whose threads do not divide a CTA."""
    rng = np.random.default_rng(rows)
    page, heads = 16, 3
    pages = -(-rows // page) + 1
    slots = rng.permutation(pages * page)[:rows]
    x = rng.standard_normal((2, rows, heads, dim)).astype(np.float32)
    check_write(torch, qg, fmt, kind, x, slots, pages, page, "stacked")
    c = random_cache(rng, fmt, 64, heads, page, dim, spread=3.0)
    slots = rng.integers(-3, 64 * page, 3 * rows)
    out = [Guarded(torch, (3 * rows, heads, dim), types(torch)[kind]) for _ in range(2)]
    qg.qg_kv_read(upload(torch, qg, c), dev(torch, slots), None, out[0].view, out[1].view)
    for o, n in zip(out, "kv"):
        o.check()
        want = torch.from_numpy(K.rows(c, slots, n).astype(np.float32)).to(types(torch)[kind])
        assert torch.equal(o.view.cpu(), want)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("dim", DIMS)
def test_write_q8_0_keeps_nan(torch, qg, dim, kind):
    """A NaN or an infinity in a block of a Q8_0 row: scale NaN or infinity, codes 0, the block reads as NaN; the other blocks
    of the row, the other rows and heads are as they are without it."""
    rng = np.random.default_rng(dim)
    x = rng.standard_normal((2, 9, 2, dim)).astype(np.float32)
    x = torch.from_numpy(x).to(types(torch)[kind]).float().numpy()
    odd = np.zeros((2, 9, 2, dim // 32), bool)
    y, scale = x.copy(), np.zeros(odd.shape)
    for i, (row, block, at, value) in enumerate([(1, 0, 5, np.nan), (2, 1, 31, np.inf), (3, 0, 0, -np.inf), (4, 1, slice(None), np.nan),
                                                 (5, 0, slice(None), np.inf), (6, 1, 16, np.nan), (7, 1, 3, -np.nan)]):
        which, head = i % 2, i // 2 % 2
        y[which, row, head, 32 * block: 32 * block + 32][at] = value
        odd[which, row, head, block], scale[which, row, head, block] = True, abs(value)
    y[0, 8, 1, 33], y[0, 8, 1, 49] = np.inf, np.nan  # in two lanes of one block
    odd[0, 8, 1, 1], scale[0, 8, 1, 1] = True, np.nan
    cache = qg.KVCache.allocate(1, 16, 2, dim)
    t = torch.from_numpy(y).to(types(torch)[kind]).cuda()
    qg.qg_kv_write(cache, t[0], t[1], torch.arange(9, device="cuda"))
    back = qg.qg_kv_read(cache, torch.arange(9, device="cuda"))
    held = download(cache, "q8_0")
    for i, n in enumerate("kv"):
        q, d = K.quantize(x[i], "q8_0")
        at = odd[i]
        d = np.where(at, scale[i], d.astype(np.float64))
        q = np.where(np.repeat(at, 32, axis=-1), 0, q)
        assert np.array_equal(held[n][0, :, :9].swapaxes(0, 1), q)
        assert np.array_equal(held[n + "d"][0, :, :9].swapaxes(0, 1).astype(np.float64), d, equal_nan=True)
        assert np.array_equal(torch.isnan(back[i]).cpu().numpy(), np.repeat(at, 32, axis=-1))


def test_write_nothing(torch, qg):
    cache = qg.KVCache.allocate(2, 16, 2, 64)
    empty = torch.empty((0, 2, 64), device="cuda")
    qg.qg_kv_write(cache, empty, empty, torch.empty(0, dtype=torch.int64, device="cuda"))
    none = qg.KVCache.allocate(0, 16, 2, 64)
    one = torch.ones((1, 2, 64), device="cuda")
    qg.qg_kv_write(none, one, one, torch.zeros(1, dtype=torch.int64, device="cuda"))
    k, v = qg.qg_kv_read(none, torch.zeros(1, dtype=torch.int64, device="cuda"))
    assert not k.any() and not v.any()
    o = qg.qg_attn_decode(one, none, torch.zeros((1, 0), dtype=torch.int32, device="cuda"),
                          torch.full((1,), 5, dtype=torch.int32, device="cuda"))
    assert not o.any()
    for columns in (1, 600):  # pages of an empty pool: none of them exists
        o = qg.qg_attn_decode(one, none, torch.zeros((1, columns), dtype=torch.int32, device="cuda"),
                              torch.full((1,), 5, dtype=torch.int32, device="cuda"))
        assert torch.isnan(o).all()


# ---------------------------------------------------------------- read

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("rows,heads,page", [(1, 1, 16), (7, 3, 48), (65, 2, 64), (300, 5, 32)])
def test_read(torch, qg, fmt, kind, dim, rows, heads, page):
    rng = np.random.default_rng(rows * 100 + dim)
    pages = 9
    c = random_cache(rng, fmt, pages, heads, page, dim, spread=3.0)
    slots = rng.integers(0, pages * page, rows)  # some of them more than once
    if rows > 4:
        slots[2], slots[3], slots[4] = -1, pages * page, 2 ** 33
    out = [Guarded(torch, (rows, heads, dim), types(torch)[kind]) for _ in range(2)]
    qg.qg_kv_read(upload(torch, qg, c), dev(torch, slots), None, out[0].view, out[1].view)
    for o, n in zip(out, "kv"):
        o.check()
        want = K.rows(c, slots, n).astype(np.float32)  # the definition's rounding
        got = o.view.float().cpu().numpy()
        if kind == "bf16":
            want = torch.from_numpy(want).bfloat16().float().numpy()
        assert np.array_equal(got, want), np.argwhere(got != want)[:4]


@pytest.mark.parametrize("fmt", FORMATS)
def test_read_many_rows(torch, qg, fmt):
    rng = np.random.default_rng(4)
    c = random_cache(rng, fmt, 40, 4, 16, 64)
    slots = rng.integers(-5, 40 * 16, 30011)
    k, v = qg.qg_kv_read(upload(torch, qg, c), dev(torch, slots))
    assert k.dtype == torch.float32
    assert np.array_equal(k.cpu().numpy(), K.rows(c, slots, "k").astype(np.float32))
    assert np.array_equal(v.cpu().numpy(), K.rows(c, slots, "v").astype(np.float32))


def test_read_special_scales(torch, qg):
    """Infinite and NaN scales and e4m3's NaN codes come back as such."""
    for fmt in FORMATS:
        c = random_cache(np.random.default_rng(5), fmt, 1, 1, 16, 64)
        c["kd"][0, 0, 1], c["kd"][0, 0, 2] = np.inf, np.nan
        c["k"][0, 0, 1] = np.where(c["k"][0, 0, 1] == 0, 1, c["k"][0, 0, 1])
        if fmt == "e4m3":
            c["v"][0, 0, 3, 5] = 0xFF
        k, v = qg.qg_kv_read(upload(torch, qg, c), torch.arange(16, device="cuda"))
        for got, n in ((k, "k"), (v, "v")):
            with np.errstate(all="ignore"):
                want = K.rows(c, np.arange(16), n).astype(np.float32)
            assert np.array_equal(got.cpu().numpy(), want, equal_nan=True)


# ---------------------------------------------------------------- attention

def bounds(part, n, out_bf16):
    each = 2.0 ** -20 + (2.0 ** -11 if out_bf16 else 0.0) + (n / 64 + 64) * 2.0 ** -24
    return K.moved(part, each, 2.0 ** -18, 2.0 ** -22, 2.0 ** -36)


def assert_attention(got, got_lse, want, what=""):
    """want: the oracle's (o, lse, parts); got a torch tensor."""
    o, lse, parts = want
    bf16 = "bfloat16" in str(got.dtype)
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    for b, part in enumerate(parts):
        if part is None:
            assert not got[b].any(), (what, b)
            assert got_lse is None or np.all(np.isneginf(got_lse[b].cpu().numpy())), (what, b)
            continue
        off, off_lse = bounds(part, part[0].shape[-1], bf16)
        lim = off + (np.abs(o[b]) + off) * (2.0 ** -8 if bf16 else 2.0 ** -23) + 2.0 ** -133
        err = np.abs(got[b] - o[b])
        assert np.all(err <= lim), (what, b, np.argwhere(err > lim)[:4], float((err / lim).max()))
        if got_lse is not None:
            _, off_lse = bounds(part, part[0].shape[-1], False)
            e = np.abs(got_lse[b].double().cpu().numpy() - lse[b])
            lim = off_lse + 2.0 ** -21 * (1 + np.abs(lse[b]))
            assert np.all(e <= lim), (what, b, float((e / lim).max()))


def run_attention(torch, qg, fmt, dim, heads, group, page, lengths, window=0, kinds=("f32", "f32"), seed=0, scale=None,
                  gain=1.0, lse=True, q_view="packed", spread=0.5, wide=False):
    """wide: page tables for 5000 tokens more, with which calls on few short sequences take the form for long ones."""
    rng = np.random.default_rng(seed + dim * 7 + heads * 31 + group * 101 + page)
    pages = sum(-(-max(n, 0) // page) for n in lengths) + 2
    c = random_cache(rng, fmt, pages, heads, page, dim, spread)
    t = tables(rng, lengths, page, pages, extra=5000 // page + 1 if wide else 1)
    batch, hq = len(lengths), heads * group
    q = torch.from_numpy((gain * rng.standard_normal((batch, hq, dim))).astype(np.float32)).to(types(torch)[kinds[0]])
    scale64 = dim ** -0.5 if scale is None else float(np.float32(scale))
    want = K.attention(q.float().numpy(), c, t, lengths, float(np.float32(scale64)), window)
    qd = q.cuda()
    if q_view == "stacked":
        qkv = torch.full((batch, hq + 2 * heads, dim), float("nan"), dtype=q.dtype, device="cuda")
        qkv[:, :hq] = qd
        qd = qkv[:, :hq]
    elif q_view == "heads":
        qd = qd.transpose(0, 1).contiguous().transpose(0, 1)
    cache, td, ld = upload(torch, qg, c), dev(torch, t), dev(torch, np.asarray(lengths, np.int32))
    out = Guarded(torch, (batch, hq, dim), types(torch)[kinds[1]])
    ls = Guarded(torch, (batch, hq), torch.float32) if lse else None
    work = qg.AttnWork.allocate(hq, heads, dim)
    got = qg.qg_attn_decode(qd, cache, td, ld, scale, window, out=out.view, lse=ls.view if lse else None, work=work)
    out.check()
    if lse:
        ls.check()
    assert_attention(got, ls.view if lse else None, want, (fmt, dim, heads, group, page, lengths, window, kinds))
    # the same bits again, from the same workspace and from a new one
    a = qg.qg_attn_decode(qd, cache, td, ld, scale, window, out_dtype=types(torch)[kinds[1]], work=work)
    b = qg.qg_attn_decode(qd, cache, td, ld, scale, window, out_dtype=types(torch)[kinds[1]])
    assert torch.equal(a, got) and torch.equal(b, got)
    assert not work.buf[:256].any()  # the counters are zero again


WIDE = pytest.mark.parametrize("wide", [False, True])


@WIDE
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("kinds", [("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("group", [1, 2, 3, 8, 9, 16, 17, 40])
def test_attention_heads(torch, qg, fmt, dim, kinds, group, wide):
    run_attention(torch, qg, fmt, dim, 2, group, 16, [277, 1, 600], kinds=kinds, wide=wide)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kinds", [("f32", "bf16"), ("bf16", "f32")])
def test_attention_mixed_types(torch, qg, fmt, kinds):
    run_attention(torch, qg, fmt, 128, 2, 4, 16, [277, 1, 600], kinds=kinds)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kinds", [("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("lengths", [[1], [2], [15], [16], [17], [31, 32, 33], [63, 64, 65], [127, 128, 129], [0], [0, 0, 5, 0],
                                     [1000], [4097], [9000, 1, 0, 300, 12], [-3, 7, -2 ** 31]])
@WIDE
def test_attention_lengths(torch, qg, fmt, kinds, lengths, wide):
    run_attention(torch, qg, fmt, 128, 2, 4, 16, lengths, kinds=kinds, wide=wide)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page", [16, 32, 48, 80, 128, 256, 4096])
@WIDE
def test_attention_pages(torch, qg, fmt, page, wide):
    run_attention(torch, qg, fmt, 64, 3, 2, page, [500, 33, 0, 777], q_view="stacked", wide=wide)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 7, 16, 17, 100, 128, 700, 10 ** 6, 2 ** 62])
@WIDE
def test_attention_window(torch, qg, fmt, dim, window, wide):
    run_attention(torch, qg, fmt, dim, 2, 3, 48, [900, 16, 0, 1, 129, 640], window=window, q_view="heads", wide=wide)


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_many_sequences(torch, qg, fmt):
    """More sequences than CTAs, most of them short, some empty; heads of one sequence on several CTAs."""
    rng = np.random.default_rng(11)
    lengths = [int(n) for n in rng.integers(0, 60, 700)]
    lengths[100], lengths[699] = 1500, 0
    run_attention(torch, qg, fmt, 64, 2, 2, 16, lengths, kinds=("bf16", "bf16"))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("group,kinds", [(1, ("f32", "f32")), (7, ("bf16", "bf16")), (13, ("f32", "f32")), (20, ("bf16", "bf16"))])
@pytest.mark.parametrize("longest,window", [(31, 0), (200, 0), (500, 40)])
def test_attention_many_short(torch, qg, fmt, dim, group, kinds, longest, window):
    """More heads than CTAs find room for, all of them short: a warp to each."""
    rng = np.random.default_rng(longest)
    lengths = [int(n) for n in rng.integers(0, longest + 1, 320)]
    lengths[0], lengths[-1] = longest, 0
    run_attention(torch, qg, fmt, dim, 2, group, 16, lengths, window=window, kinds=kinds)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,batch,tokens", [(128, 170, 256), (128, 170, 257), (128, 460, 512), (128, 460, 513), (128, 450, 512),
                                              (256, 170, 128), (256, 170, 144), (256, 460, 256), (64, 920, 512)])
def test_attention_limits_of_the_warps(torch, qg, fmt, dim, batch, tokens):
    """Both sides of the limits between the warps' form and the line: steps to an item, items to a GPU's room."""
    rng = np.random.default_rng(batch + tokens)
    lengths = [int(n) for n in rng.integers(0, 90, batch)]
    lengths[3], lengths[-1] = tokens, tokens - 1
    c = random_cache(rng, fmt, sum(-(-n // 16) for n in lengths) + 1, 2, 16, dim)
    t = tables(rng, lengths, 16, len(c["k"]), extra=0)
    q = rng.standard_normal((batch, 4, dim)).astype(np.float32)
    got = qg.qg_attn_decode(dev(torch, q), upload(torch, qg, c), dev(torch, t), dev(torch, np.array(lengths, np.int32)))
    assert_attention(got, None, K.attention(q, c, t, lengths, float(np.float32(dim ** -0.5))))


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_bad_page_many_short(torch, qg, fmt):
    rng = np.random.default_rng(23)
    lengths, dim, pages = [40] * 400, 64, 1300
    c = random_cache(rng, fmt, pages, 2, 16, dim)
    t = tables(rng, lengths, 16, pages)
    q = rng.standard_normal((400, 4, dim)).astype(np.float32)
    want = K.attention(q, c, t, lengths, dim ** -0.5)
    t[7, 1], t[200, 2], t[399, 0] = -1, pages, 2 ** 31 - 1
    got = qg.qg_attn_decode(dev(torch, q), upload(torch, qg, c), dev(torch, t), dev(torch, np.array(lengths, np.int32)))
    bad = [7, 200, 399]
    assert torch.isnan(got[bad]).all()
    keep = [i for i in range(400) if i not in bad]
    assert_attention(got[keep], None, (want[0][keep], want[1][keep], [want[2][i] for i in keep]))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("batch", [32, 33, 127, 128, 129, 300])
def test_attention_batches(torch, qg, fmt, batch):
    """Both sides of the scans' limits: rows of 32 sequences, up to four of them by every warp for itself."""
    rng = np.random.default_rng(batch)
    lengths = [int(n) for n in rng.integers(0, 300, batch)]
    lengths[rng.integers(batch)] = 1700
    run_attention(torch, qg, fmt, 64, 1, 3, 16, lengths, kinds=("f32", "f32"))


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_widest_tables(torch, qg, fmt):
    """Page tables of 2^30 tokens for 128 heads: a line of 2^30 and more places, of which few are used."""
    run = np.random.default_rng(21)
    heads, dim, page, n = 128, 64, 4096, [300, 0, 7]
    c = random_cache(run, fmt, 3, heads, page, dim)
    t = np.zeros((3, (1 << 30) // page), np.int32)
    t[0, 0], t[2, 0] = 2, 1
    q = run.standard_normal((3, heads, dim)).astype(np.float32)
    want = K.attention(q, c, t, n, 0.125)
    got = qg.qg_attn_decode(dev(torch, q), upload(torch, qg, c), dev(torch, t), dev(torch, np.array(n, np.int32)))
    assert_attention(got, None, want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("exponent", [-90, -24, 0])
def test_attention_longest(torch, qg, fmt, exponent):
    """2^30 tokens, one page over and over, of equal scores and values: o is the value, lse 30 ln 2.  The sum of weights stays
    in range, whatever the values' scale.  Each of four warps in 608 CTAs adds its 13797 steps one after another, and their
    sums are joined in 608 more: 2^14 roundings of 2^-24 in each of the two sums, 2^-20 for a weight."""
    if fmt == "q8_0" and exponent < -24:
        exponent = -25  # no binary16: the scale is zero
    run = np.random.default_rng(37)
    page, dim = 4096, 64
    c = random_cache(run, fmt, 1, 1, page, dim)
    code = run.integers(0, 0x7F, dim)
    c["v"][...] = code.astype(c["v"].dtype)
    c["vd"][...] = 2.0 ** exponent
    t = np.zeros((1, (1 << 30) // page), np.int32)
    lse = torch.empty((1, 1), device="cuda")
    got = qg.qg_attn_decode(torch.zeros((1, 1, dim), device="cuda"), upload(torch, qg, c), dev(torch, t),
                            dev(torch, np.array([1 << 30], np.int32)), lse=lse)
    want = torch.from_numpy(code.astype(np.uint8))
    want = (want.double() if fmt == "q8_0" else want.view(torch.float8_e4m3fn).double()) * float(c["vd"].flat[0])
    each = 2.0 ** -10 + 2.0 ** -20 + 2.0 ** -23
    assert ((got.double().cpu() - want).abs() <= 2 * each * want.abs()).all()
    assert abs(lse.item() - 30 * np.log(2.0)) <= each


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("heads", [1, 5, 24])
def test_attention_long(torch, qg, fmt, heads):
    run_attention(torch, qg, fmt, 128, heads, 2, 64, [30011 // heads * 2, 5], kinds=("f32", "f32"))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("gain,scale", [(0.0, None), (1e-20, None), (30.0, None), (1.0, 0.0), (1.0, -0.2), (1e6, 1e-7), (1.0, 3.0)])
@WIDE
def test_attention_scores(torch, qg, fmt, gain, scale, wide):
    """Flat and peaked softmaxes, small and large queries, odd scales."""
    run_attention(torch, qg, fmt, 128, 2, 4, 32, [300, 65], gain=gain, scale=scale, wide=wide)
    run_attention(torch, qg, fmt, 128, 2, 4, 32, [300, 65], gain=gain, scale=scale, wide=wide, kinds=("bf16", "bf16"))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [3.4e38, -3.4e38, 2.4e38, 1e38, 1e-44])
@pytest.mark.parametrize("lengths,columns", [([70, 3], 1), ([300, 1, 650], 400), ([37] * 330, 1)])
def test_attention_largest_scales(torch, qg, fmt, kind, scale, lengths, columns):
    """Scales up to f32's ends: scores of zero stay zero, and keys and queries that are as small come out right."""
    rng = np.random.default_rng(41)
    pages, scale = sum(-(-n // 16) for n in lengths) + 1, float(np.float32(scale))
    c = random_cache(rng, fmt, pages, 2, 16, 128)
    t = tables(rng, lengths, 16, pages, extra=columns)
    args = dev(torch, t), dev(torch, np.array(lengths, np.int32)), scale
    zero = torch.zeros((len(lengths), 6, 128), dtype=types(torch)[kind])
    want = K.attention(zero.float().numpy(), c, t, lengths, scale)
    assert_attention(qg.qg_attn_decode(zero.cuda(), upload(torch, qg, c), *args), None, want)
    if fmt == "e4m3" and abs(scale) > 1:  # scores of some units
        c["kd"] *= np.float32(2.0 ** -63)
        q = torch.from_numpy((1e-20 * rng.standard_normal(zero.shape)).astype(np.float32)).to(types(torch)[kind])
        want = K.attention(q.float().numpy(), c, t, lengths, scale)
        assert 1 < max(np.abs(p[1]).max() for p in want[2]) < 60
        assert_attention(qg.qg_attn_decode(q.cuda(), upload(torch, qg, c), *args), None, want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kinds", [("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("dim,group", [(64, 3), (128, 12), (256, 16)])
@pytest.mark.parametrize("lengths,wide", [([70, 3], False), ([300, 1, 650], True), ([20] * 330, False)])
def test_attention_mixed_types_of_each_form(torch, qg, fmt, kinds, dim, group, lengths, wide):
    run_attention(torch, qg, fmt, dim, 2, group, 16, lengths, kinds=kinds, wide=wide)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("lengths,columns", [([70, 3], 1), ([300, 5, 650], 400), ([37] * 330, 1)])
def test_attention_scale_not_finite(torch, qg, kind, scale, lengths, columns):
    """No number comes of a scale that is none."""
    rng = np.random.default_rng(47)
    pages = sum(-(-n // 16) for n in lengths) + 1
    c = random_cache(rng, "q8_0", pages, 2, 16, 128)
    q = torch.from_numpy(rng.standard_normal((len(lengths), 6, 128)).astype(np.float32)).to(types(torch)[kind]).cuda()
    lse = torch.empty((len(lengths), 6), device="cuda")
    got = qg.qg_attn_decode(q, upload(torch, qg, c), dev(torch, tables(rng, lengths, 16, pages, extra=columns)),
                            dev(torch, np.array(lengths, np.int32)), scale, lse=lse)
    assert torch.isnan(got).all() and not torch.isfinite(lse).any()


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_small_beside_large_query(torch, qg, fmt):
    """A query's values 2^-16 and 2^-24 of the head's largest, which meets keys of zero: held to 22 bits or 2^-39 of the largest."""
    rng = np.random.default_rng(43)
    lengths, dim, heads, group = [400, 33], 128, 2, 3
    pages = sum(-(-n // 16) for n in lengths) + 1
    c = random_cache(rng, fmt, pages, heads, 16, dim)
    c["k"][..., 7] = 0
    t = tables(rng, lengths, 16, pages)
    for ratio in (16, 24):
        q = rng.standard_normal((2, heads * group, dim)).astype(np.float32)
        q[..., 7] = 2.0 ** ratio
        want = K.attention(q, c, t, lengths, float(np.float32(dim ** -0.5)))
        got = qg.qg_attn_decode(dev(torch, q), upload(torch, qg, c), dev(torch, t), dev(torch, np.array(lengths, np.int32)))
        for b, part in enumerate(want[2]):
            # each value off by 2^-39 of the largest: scores by that times the keys' sums
            n = part[0].shape[-1]
            k = np.abs(K.rows(c, t[b, np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16, "k")).sum(axis=-1).max()
            each = 2.0 ** -20 + (n / 64 + 64) * 2.0 ** -24 + dim ** -0.5 * k * 2.0 ** (ratio - 39)
            off, _ = K.moved(part, each, 2.0 ** -18, 2.0 ** -22, 2.0 ** -36)
            lim = off + (np.abs(want[0][b]) + off) * 2.0 ** -23
            err = np.abs(got[b].double().cpu().numpy() - want[0][b])
            assert np.all(err <= lim), (ratio, b, float((err / lim).max()))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,group", [(128, 6), (64, 1), (96, 12)])
@pytest.mark.parametrize("lengths,columns", [([2, 6], 1), ([100, 36, 1500], 600), ([20] * 400, 2)])
def test_attention_bf16_weights(torch, qg, fmt, dim, group, lengths, columns):
    """Pairs of tokens of opposite values and nearly the same weight, in each form (a CTA or cluster, the line, warps): the
    outputs are what is left of the weights' last bits, so that bf16 outputs hold them to 22 bits like f32 ones.  The
    limit is that of f32 outputs and half a step of bf16; one rounding of each weight to 11 bits leaves up to 2^-12 of each
    term, some 2^-4 of these outputs."""
    rng = np.random.default_rng(dim + len(lengths))
    page, heads = 16, 2
    pages = sum(-(-n // page) for n in lengths) + 1
    c = random_cache(rng, fmt, pages, heads, page, dim)
    c["vd"][...] = c["vd"].flat[0]
    c["v"][:, :, 1::2] = -c["v"][:, :, ::2] if fmt == "q8_0" else c["v"][:, :, ::2] ^ 0x80
    t = tables(rng, lengths, page, pages, extra=columns)
    q = torch.from_numpy((2e-3 * rng.standard_normal((len(lengths), heads * group, dim))).astype(np.float32)).bfloat16()
    want, _, parts = K.attention(q.float().numpy(), c, t, lengths, float(np.float32(dim ** -0.5)))
    got = qg.qg_attn_decode(q.cuda(), upload(torch, qg, c), dev(torch, t), dev(torch, np.array(lengths, np.int32)))
    assert got.dtype == torch.bfloat16
    got = got.double().cpu().numpy()
    for b, part in enumerate(parts):
        off, _ = bounds(part, part[0].shape[-1], False)
        lim = off + (np.abs(want[b]) + off) * 2.0 ** -8
        err = np.abs(got[b] - want[b])
        assert np.all(err <= lim), (b, np.argwhere(err > lim)[:4], float((err / lim).max()))


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_scales_far_apart(torch, qg, fmt):
    """Tokens whose values' scales differ by many powers of two: none is lost to the weights' 16 bits."""
    run_attention(torch, qg, fmt, 128, 2, 4, 32, [300, 65], spread=4.0, gain=0.01)
    run_attention(torch, qg, fmt, 128, 2, 4, 32, [300, 65], spread=4.0, gain=0.01, kinds=("bf16", "bf16"))


def assert_by_blocks(got, c, t, lengths, want, what=""):
    """As assert_attention, each block of values by itself: a weight keeps 22 bits, or 2^-31 of the largest weight times scale
    of its own block of the head's values, whatever the other blocks hold (each of n tokens' codes is at most 127 or 448)."""
    o, _, parts = want
    bf16 = "bfloat16" in str(got.dtype)
    got = got.double().cpu().numpy()
    page, block = c["v"].shape[2], K.BLOCK[c["format"]]
    for b, part in enumerate(parts):
        if part is None:
            assert not got[b].any(), (what, b)
            continue
        p = part[0]
        n, dim = p.shape[-1], got.shape[-1]
        at = np.arange(lengths[b] - n, lengths[b])
        d = np.abs(c["vd"][t[b, at // page], :, at % page].astype(np.float64))  # [tokens, heads, blocks]
        each = 2.0 ** -20 + (n / 64 + 64) * 2.0 ** -24
        with np.errstate(all="ignore"):
            off, _ = K.moved((*part[:3], np.where(np.isfinite(part[3]), part[3], 0.0)), each, 2.0 ** -18, 2.0 ** -22, 0.0)
            top = np.einsum("hgt,thb->hgtb", p, d).max(axis=2) * (n * 2.0 ** -31 * (127 if block == 32 else 448))
            off = off + np.repeat(top, block, axis=-1)[..., :dim].reshape(-1, dim)
            lim = off + (np.abs(o[b]) + off) * (2.0 ** -8 if bf16 else 2.0 ** -23) + 2.0 ** -133
            odd = ~np.isfinite(o[b])
            assert np.array_equal(got[b][odd], o[b][odd], equal_nan=True), (what, b)
            err = np.where(odd, 0.0, np.abs(got[b] - o[b]))
            lim = np.where(odd, 0.0, lim)
        assert np.all(err <= lim), (what, b, np.argwhere(~(err <= lim))[:4], float(np.nanmax(err / np.maximum(lim, 1e-300))))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim,group,kind", [(64, 2, "bf16"), (96, 3, "f32"), (128, 12, "f32"), (192, 4, "bf16"), (256, 9, "f32")])
@pytest.mark.parametrize("scales", ["steps", "any", "late", "early", "silent", "least", "most", "infinite"])
@pytest.mark.parametrize("lengths,columns", [([70, 3], 1), ([300, 1, 650], 400), ([37] * 330, 1)])
def test_attention_blocks_far_apart(torch, qg, fmt, dim, group, kind, scales, lengths, columns):
    """Scales of one token's blocks of values many powers of two apart, in each form (a CTA or cluster, the line, warps):
    every block comes out as if it were alone."""
    rng = np.random.default_rng(dim + 17 * len(scales) + lengths[0])
    page, heads = 16, 2
    pages = sum(-(-n // page) for n in lengths) + 1
    c = random_cache(rng, fmt, pages, heads, page, dim)
    t = tables(rng, lengths, page, pages, extra=columns)
    vd, nb = c["vd"], c["vd"].shape[-1]
    low, high = (-24, 15) if fmt == "q8_0" else (-45, 45)
    x = np.exp2(0.5 * rng.standard_normal(vd.shape))
    anywhere = np.exp2(rng.uniform(low, high, vd.shape))
    step = np.exp2(np.linspace(high - 2, low + 2, nb)) if nb > 1 else np.exp2([high])
    if scales == "steps":
        vd[...] = x * step
    elif scales == "any":
        vd[...] = anywhere
        vd[rng.random(vd.shape) < 0.1] = 0
    elif scales in ("late", "early"):  # in the last or the first page of each sequence
        vd[...] = x / 64
        for b, n in enumerate(lengths):
            i = (n - 1) // page if scales == "late" else 0
            vd[t[b, i]] = (x * step)[t[b, i]]
    elif scales == "silent":  # a token without values has most of the weight
        for b, n in enumerate(lengths):
            at = n // 2
            vd[t[b, at // page], :, at % page] = 0
            c["k"][t[b, at // page], :, at % page] = 0x7F if fmt == "q8_0" else 0x7E
            c["kd"][t[b, at // page], :, at % page] = (2.0 if fmt == "q8_0" else 0.5) * 24 / np.sqrt(dim) / 127
    elif scales in ("least", "most"):
        vd[...] = x * (2.0 ** -22 if fmt == "q8_0" else 2.0 ** -106) if scales == "least" else np.minimum(
            x * (2.0 ** 15 if fmt == "q8_0" else 2.0 ** 116), 65504 if fmt == "q8_0" else 2.0 ** 118)
    else:
        at = lengths[0] // 2
        vd[t[0, at // page], 1, at % page, nb // 2] = np.inf
    q = rng.standard_normal((len(lengths), heads * group, dim)).astype(np.float32)
    if scales == "silent":
        q = np.abs(q)
    q = torch.from_numpy(q).to(types(torch)[kind])
    with np.errstate(all="ignore"):
        want = K.attention(q.float().numpy(), c, t, lengths, float(np.float32(dim ** -0.5)))
    got = qg.qg_attn_decode(q.cuda(), upload(torch, qg, c), dev(torch, t), dev(torch, np.array(lengths, np.int32)))
    assert_by_blocks(got, c, t, lengths, want, scales)


@pytest.mark.parametrize("fmt,exponent", [("q8_0", 15), ("e4m3", 15), ("e4m3", 42), ("e4m3", 50), ("e4m3", 80), ("e4m3", 118)])
@pytest.mark.parametrize("kind,dim,group", [("f32", 128, 4), ("bf16", 96, 9), ("f32", 256, 3)])
@pytest.mark.parametrize("where", ["first", "last"])
@pytest.mark.parametrize("lengths,columns", [([70, 33, 17], 1), ([300, 33, 650], 400), ([33] * 330, 1)])
def test_attention_without_values_beside_large_ones(torch, qg, fmt, exponent, kind, dim, group, where, lengths, columns):
    """The first 32 tokens have no values, or the last alone: what they have of the softmax's sum counts beside tokens of the
    largest values, met later by the same warp or by another."""
    rng = np.random.default_rng(exponent + dim)
    page, heads = 16, 2
    pages = sum(-(-n // page) for n in lengths) + 1
    c = random_cache(rng, fmt, pages, heads, page, dim)
    t = tables(rng, lengths, page, pages, extra=columns)
    c["vd"][...] = 2.0 ** exponent
    for b, n in enumerate(lengths):
        silent = np.arange(min(32, n - 1)) if where == "first" else np.array([n - 1])
        c["v"][t[b, silent // page], :, silent % page] = 0
        c["vd"][t[b, silent // page], :, silent % page] = 0 if fmt == "q8_0" else 2.0 ** -108
    q = torch.from_numpy(rng.standard_normal((len(lengths), heads * group, dim)).astype(np.float32)).to(types(torch)[kind])
    want = K.attention(q.float().numpy(), c, t, lengths, float(np.float32(dim ** -0.5)))
    got = qg.qg_attn_decode(q.cuda(), upload(torch, qg, c), dev(torch, t), dev(torch, np.array(lengths, np.int32)))
    assert_by_blocks(got, c, t, lengths, want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[2], [100, 3, 1500], [20] * 400])
def test_attention_small_beside_large(torch, qg, fmt, kind, lengths):
    """One large channel to a block of values: the others, small or zero, come out as exactly as if it were not there."""
    rng = np.random.default_rng(29)
    pages = sum(-(-n // 16) for n in lengths) + 1
    c = random_cache(rng, fmt, pages, 2, 16, 128)
    c["v"][..., 1::2] = rng.integers(0, 3, c["v"][..., 1::2].shape)
    c["v"][..., ::32] = 0x7F if fmt == "q8_0" else 0x7E
    c["v"][..., 5::16] = 0
    t = tables(rng, lengths, 16, pages)
    q = torch.from_numpy(rng.standard_normal((len(lengths), 6, 128)).astype(np.float32)).to(types(torch)[kind])
    want = K.attention(q.float().numpy(), c, t, lengths, float(np.float32(128 ** -0.5)))
    got = qg.qg_attn_decode(q.cuda(), upload(torch, qg, c), dev(torch, t), dev(torch, np.array(lengths, np.int32)))
    assert_attention(got, None, want)
    assert not got[..., 5::16].any()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", [96, 128])
@pytest.mark.parametrize("n,window", [(0, 0), (1, 0), (37, 0), (130, 0), (200, 50), (300, 130)])
@WIDE
def test_attention_ignores_what_is_not_seen(torch, qg, fmt, dim, n, window, wide):
    """NaN and infinite scales and NaN codes in every token outside the ones seen, in all pages."""
    rng = np.random.default_rng(n + 5)
    page, heads, group = 48, 2, 3
    pages = 12
    c = random_cache(rng, fmt, pages, heads, page, dim)
    t = tables(rng, [n], page, pages, extra=120 if wide else 1)
    seen = np.zeros((pages, page), bool)
    for i in range(max(0, n - window) if window else 0, n):
        seen[t[0, i // page], i % page] = True
    for name in "kv":
        hidden = np.broadcast_to(~seen[:, None, :], (pages, heads, page))
        c[name + "d"][hidden] = rng.choice(np.array([np.nan, np.inf, -np.inf], c[name + "d"].dtype), c[name + "d"][hidden].shape)
        c[name][hidden] = -128 if fmt == "q8_0" else 0x7F
    q = rng.standard_normal((1, heads * group, dim)).astype(np.float32)
    t[t == 2 ** 31 - 1] = rng.choice([-1, 2 ** 31 - 1, pages, -2 ** 31])
    if window:
        t[0, : (n - window) // page] = -7  # pages given back
    want = K.attention(q, c, np.where((t < 0) | (t >= pages), 0, t), [n], float(np.float32(dim ** -0.5)), window)
    lse = torch.empty((1, heads * group), device="cuda")
    got = qg.qg_attn_decode(dev(torch, q), upload(torch, qg, c), dev(torch, t), dev(torch, np.array([n], np.int32)),
                            window=window, lse=lse)
    assert_attention(got, lse, want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("bad", [-1, 20, 2 ** 31 - 1, -2 ** 31])
@WIDE
def test_attention_bad_page(torch, qg, fmt, bad, wide):
    """A page outside the cache makes its sequence NaN and leaves the others alone."""
    rng = np.random.default_rng(6)
    lengths, page, heads, group, dim, pages = [100, 300, 40], 16, 2, 2, 64, 32
    c = random_cache(rng, fmt, pages, heads, page, dim)
    t = tables(rng, lengths, page, pages, extra=400 if wide else 1)
    q = rng.standard_normal((3, 4, dim)).astype(np.float32)
    want = K.attention(q, c, t, lengths, dim ** -0.5)
    if bad == 20:
        bad = pages
    t[1, 7] = bad
    lse = torch.empty((3, 4), device="cuda")
    got = qg.qg_attn_decode(dev(torch, q), upload(torch, qg, c), dev(torch, t), dev(torch, np.array(lengths, np.int32)), lse=lse)
    assert torch.isnan(got[1]).all() and torch.isnan(lse[1]).all()
    keep = [0, 2]
    assert_attention(got[keep], lse[keep], (want[0][keep], want[1][keep], [want[2][i] for i in keep]))


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_nan_of_a_token_seen(torch, qg, fmt):
    """NaN in a seen token's value reaches the dimensions that it has a part in, in its key all of them."""
    rng = np.random.default_rng(7)
    c = random_cache(rng, fmt, 8, 1, 16, 128)
    t = tables(rng, [100, 20], 16, 8)
    q = rng.standard_normal((2, 2, 128)).astype(np.float32)
    p, off = t[0, 50 // 16], 50 % 16
    if fmt == "q8_0":
        c["vd"][p, 0, off, 1] = np.nan
    else:
        c["v"][p, 0, off, 40] = 0x7F
    args = dev(torch, t), dev(torch, np.array([100, 20], np.int32))
    got = qg.qg_attn_decode(dev(torch, q), upload(torch, qg, c), *args)
    bad = torch.isnan(got[0]).all(dim=0)
    assert bool(bad[40]) and torch.isfinite(got[1]).all()
    if fmt == "q8_0":
        assert torch.equal(bad.cpu(), torch.arange(128) // 32 == 1) and not torch.isnan(got[0][:, ~bad]).any()
    c["kd"][p, 0, off] = np.nan
    got = qg.qg_attn_decode(dev(torch, q), upload(torch, qg, c), *args)
    assert torch.isnan(got[0]).all() and torch.isfinite(got[1]).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("odd", [np.nan, np.inf])
@pytest.mark.parametrize("group", [3, 12])
def test_attention_odd_query_head(torch, qg, fmt, kind, odd, group):
    """NaN or an infinity in one query head leaves the other heads' bits alone."""
    rng = np.random.default_rng(17)
    c = random_cache(rng, fmt, 40, 2, 16, 128)
    args = upload(torch, qg, c), dev(torch, tables(rng, [500, 70], 16, 40)), dev(torch, np.array([500, 70], np.int32))
    q = torch.from_numpy(rng.standard_normal((2, 2 * group, 128)).astype(np.float32)).to(types(torch)[kind]).cuda()
    plain = qg.qg_attn_decode(q, *args)
    q2 = q.clone()
    q2[0, 1, 77] = odd
    got = qg.qg_attn_decode(q2, *args)
    assert torch.isnan(got[0, 1]).all()
    got[0, 1] = plain[0, 1]
    assert torch.equal(got, plain)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("columns", [3, 40, 600])
def test_attention_replayed(torch, qg, fmt, columns):
    """A captured call replayed as lengths, pages and queries change, for tables that lead to each form (one CTA, a cluster,
    the line), beside eager calls on another workspace."""
    rng = np.random.default_rng(columns)
    heads, group, dim, page, batch = 2, 4, 128, 16, 3
    pages = 3 * columns
    c = random_cache(rng, fmt, pages, heads, page, dim)
    cache = upload(torch, qg, c)
    q = torch.zeros((batch, heads * group, dim), device="cuda")
    t = torch.zeros((batch, columns), dtype=torch.int32, device="cuda")
    n = torch.zeros(batch, dtype=torch.int32, device="cuda")
    out, lse, work = torch.empty_like(q), torch.empty((batch, heads * group), device="cuda"), qg.AttnWork.allocate(heads * group, heads, dim)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        qg.qg_attn_decode(q, cache, t, n, out=out, lse=lse, work=work)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qg.qg_attn_decode(q, cache, t, n, out=out, lse=lse, work=work)
        inner = qg.qg_attn_decode(q, cache, t, n)  # a workspace of the capture's own
    for lengths in ([1, columns * 16, 5], [0, 17, columns * 7], [columns * 16] * 3, [0, 0, 0]):
        tn = rng.permutation(pages).reshape(batch, columns).astype(np.int32)
        qn = rng.standard_normal(q.shape).astype(np.float32)
        q.copy_(torch.from_numpy(qn)), t.copy_(torch.from_numpy(tn)), n.copy_(torch.tensor(lengths, dtype=torch.int32))
        g.replay()
        want = K.attention(qn, c, tn, lengths, float(np.float32(dim ** -0.5)))
        assert_attention(out, lse, want, lengths)
        assert torch.equal(inner, out) and torch.equal(qg.qg_attn_decode(q, cache, t, n), out)


def test_attention_length_beyond_the_table(torch, qg):
    """A length beyond what the page table holds counts as that."""
    rng = np.random.default_rng(8)
    c = random_cache(rng, "q8_0", 4, 1, 16, 64)
    t = np.array([[2, 0, 3]], np.int32)
    q = rng.standard_normal((1, 1, 64)).astype(np.float32)
    want = K.attention(q, c, t, [48], 0.125)
    cache = upload(torch, qg, c)
    for n in (48, 49, 2 ** 31 - 1):
        assert_attention(qg.qg_attn_decode(dev(torch, q), cache, dev(torch, t), dev(torch, np.array([n], np.int32))), None, want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_far_offsets(torch, qg, fmt):
    """Pages whose codes lie past 2^32 bytes of their plane: written, read and attended to."""
    heads, page, dim = 8, 64, 128
    pages = (1 << 32) // (heads * page * dim) + 9
    cache = qg.KVCache.allocate(pages, page, heads, dim, format=fmt)
    rng = np.random.default_rng(10)
    n = 200
    t = np.array([[pages - 1, 0, pages - 5, pages - 2]], np.int32)
    slots = t[0, np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page
    x = rng.standard_normal((2, n, heads, dim)).astype(np.float32)
    qg.qg_kv_write(cache, dev(torch, x[0]), dev(torch, x[1]), dev(torch, slots))
    k, v = qg.qg_kv_read(cache, dev(torch, slots))
    small = {"format": fmt}
    for i, name in enumerate("kv"):
        q, d = K.quantize(x[i], fmt)
        assert np.array_equal((k, v)[i].cpu().numpy(), K.values(q, d, fmt).astype(np.float32))
        pad = 4 * page - n
        small[name] = np.concatenate([q, np.zeros((pad, heads, dim), q.dtype)]).reshape(4, page, heads, dim).swapaxes(1, 2)
        small[name + "d"] = np.concatenate([d, np.zeros((pad, *d.shape[1:]), d.dtype)]).reshape(4, page, heads, -1).swapaxes(1, 2)
    q = rng.standard_normal((1, heads, dim)).astype(np.float32)
    want = K.attention(q, small, np.arange(4, dtype=np.int32)[None], [n], float(np.float32(dim ** -0.5)))
    assert_attention(qg.qg_attn_decode(dev(torch, q), cache, dev(torch, t), dev(torch, np.array([n], np.int32))), None, want)


# ---------------------------------------------------------------- used together

@pytest.mark.parametrize("fmt", FORMATS)
def test_decode_steps(torch, qg, fmt):
    """A prompt written at once, then tokens one by one, as a captured step that is replayed: the new
    token's slot and the lengths advance on the device."""
    rng = np.random.default_rng(12)
    batch, heads, group, dim, page, prompt, steps = 3, 2, 4, 128, 16, [30, 5, 47], 6
    cache = qg.KVCache.allocate(24, page, heads, dim, format=fmt)
    work = qg.AttnWork.allocate(heads * group, heads, dim)
    t = rng.permutation(24)[: batch * 5].reshape(batch, 5).astype(np.int32)
    slot = lambda b, i: int(t[b, i // page]) * page + i % page
    history = [rng.standard_normal((2, n, heads, dim)).astype(np.float32) for n in prompt]
    flat = np.concatenate(history, axis=1)
    qg.qg_kv_write(cache, dev(torch, flat[0]), dev(torch, flat[1]),
                   dev(torch, np.array([slot(b, i) for b in range(batch) for i in range(prompt[b])], np.int64)))
    qkv = torch.zeros((batch, heads * (group + 2), dim), dtype=torch.bfloat16, device="cuda")
    q, k, v = qkv[:, : heads * group], qkv[:, heads * group: heads * (group + 1)], qkv[:, heads * (group + 1):]
    td, ld = dev(torch, t), dev(torch, np.array(prompt, np.int32))
    out = torch.empty((batch, heads * group, dim), dtype=torch.bfloat16, device="cuda")

    def step():
        at = ld.long()
        slots = td.gather(1, (at // page)[:, None])[:, 0].long() * page + at % page
        ld.add_(1)
        qg.qg_kv_write(cache, k, v, slots)
        qg.qg_attn_decode(q, cache, td, ld, out=out, work=work)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()  # a first run of every kernel outside the capture; its token is written again below
        ld.sub_(1)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(steps):
        x = torch.from_numpy(rng.standard_normal(qkv.shape).astype(np.float32)).bfloat16()
        qkv.copy_(x)
        g.replay()
        x = x.float().numpy()
        for b in range(batch):
            new = np.stack([x[b, heads * group: heads * (group + 1)], x[b, heads * (group + 1):]])[:, None]
            history[b] = np.concatenate([history[b], new], axis=1)
        pages_of = {"format": fmt}
        for j, name in enumerate("kv"):
            q8, d8 = zip(*(K.quantize(h[j], fmt) for h in history))
            pages_of[name] = np.zeros((24, heads, page, dim), q8[0].dtype)
            pages_of[name + "d"] = np.zeros((24, heads, page, d8[0].shape[-1]), d8[0].dtype)
            for b in range(batch):
                for n in range(q8[b].shape[0]):
                    p, o = divmod(slot(b, n), page)
                    pages_of[name][p, :, o], pages_of[name + "d"][p, :, o] = q8[b][n], d8[b][n]
        lengths = [n + i + 1 for n in prompt]
        assert ld.tolist() == lengths
        want = K.attention(x[:, : heads * group], pages_of, t, lengths, float(np.float32(dim ** -0.5)))
        assert_attention(out, None, want, i)


@pytest.mark.parametrize("columns", [96, 600])
def test_two_streams_and_threads(torch, qg, columns):
    """Calls at once on streams of their own, each with its own workspace, against calls one by one."""
    rng = np.random.default_rng(13)
    c = random_cache(rng, "q8_0", 400, 2, 16, 128)
    cache = upload(torch, qg, c)
    t = rng.permutation(400)[:384].reshape(4, 96).astype(np.int32)
    t = dev(torch, np.pad(t, ((0, 0), (0, columns - 96))))
    n = dev(torch, np.array([1500, 1, 700, 1536], np.int32))
    qs = [torch.randn((4, 8, 128), device="cuda") for _ in range(4)]
    alone = [qg.qg_attn_decode(q, cache, t, n) for q in qs]
    torch.cuda.synchronize()
    got, failed = [None] * 4, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            w = qg.AttnWork.allocate(8, 2, 128)
            torch.cuda.synchronize()
            for _ in range(50):
                got[i] = qg.qg_attn_decode(qs[i], cache, t, n, work=w, stream=s)
            s.synchronize()
        except Exception as e:  # shown by the assertion below
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [x.start() for x in threads], [x.join() for x in threads]
    assert not failed and all(torch.equal(a, b) for a, b in zip(got, alone))


@pytest.mark.parametrize("columns", [4, 600])
def test_first_call_inside_a_capture(torch, columns):
    """A process whose first calls of all are captured, and its workspace allocated there too."""
    import subprocess
    import sys

    code = f"""
import torch
import block_quantized_decode_rmsnorm_gb300 as qg
cache = qg.KVCache.allocate(40, 16, 2, 128)
k, v = torch.randn((2, 50, 2, 128), device='cuda')
q = torch.randn((1, 8, 128), device='cuda')
slots = torch.arange(50, device='cuda') + 32
pages = (torch.arange({columns}, dtype=torch.int32, device='cuda') + 2)[None]
n = torch.full((1,), 50, dtype=torch.int32, device='cuda')
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    qg.qg_kv_write(cache, k, v, slots)
    back = qg.qg_kv_read(cache, slots)
    o = qg.qg_attn_decode(q, cache, pages, n)
g.replay()
again = qg.qg_attn_decode(q, cache, pages, n)
assert torch.equal(o, again) and bool(o.isfinite().all()) and torch.equal(back[0], qg.qg_kv_read(cache, slots)[0])
assert (back[0] - k).abs().max() < 0.05
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_decode_layer(torch, qg):
    """The decode step around the cache - norm, stacked qkv product, cache, attention, output product with the residual -
    each call against f64 from what the calls before it left."""
    rng = np.random.default_rng(31)
    hidden, heads, group, dim, n = 256, 2, 2, 64, 21
    hq = heads * group
    from oracle import quantize_q8_0

    def weight(rows, k):
        w = (0.06 * rng.standard_normal((rows, k))).astype(np.float32)
        q, d = quantize_q8_0(w)
        return qg.Q8Weight(dev(torch, q), dev(torch, d).view(torch.float16)), q.astype(np.float64) * np.repeat(
            d.view(np.float16).astype(np.float64), 32, axis=1)

    def q8(x):
        q, d = quantize_q8_0(np.ascontiguousarray(x, np.float32))
        return q.astype(np.float64) * np.repeat(d.view(np.float16).astype(np.float64), 32, axis=1)

    (wqkv, fqkv), (wo, fo) = weight((hq + 2 * heads) * dim, hidden), weight(hidden, hq * dim)
    gamma = torch.ones(hidden, device="cuda")
    cache = qg.KVCache.allocate(3, 16, heads, dim)
    pages = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    past = rng.standard_normal((2, n - 1, heads, dim)).astype(np.float32)
    slots = np.array([2 * 16 + i if i < 16 else i - 16 for i in range(n)], np.int64)
    qg.qg_kv_write(cache, dev(torch, past[0]), dev(torch, past[1]), dev(torch, slots[:-1]))
    x = torch.from_numpy(rng.standard_normal((1, hidden)).astype(np.float32)).cuda()
    xq, xd, _ = qg.rmsnorm_quantize(x, gamma, 1e-6)
    qkv = qg.qgemv_q8_0(wqkv, xq, xd).view(1, hq + 2 * heads, dim)
    qg.qg_kv_write(cache, qkv[:, hq: hq + heads], qkv[:, hq + heads:], dev(torch, slots[-1:]))
    o = qg.qg_attn_decode(qkv[:, :hq], cache, pages, torch.tensor([n], dtype=torch.int32, device="cuda"))
    oq, od = qg.quantize_act_q8_0(o.view(1, -1))
    y = qg.qgemv_q8_0(wo, oq, od, epilogue="residual", residual=x)
    want_qkv = (xq.double().cpu().numpy() * np.repeat(xd.double().cpu().numpy(), 32, axis=1)) @ fqkv.T
    assert np.allclose(qkv.cpu().numpy().reshape(1, -1), want_qkv, rtol=0, atol=1e-5 * np.abs(want_qkv).max())
    held = download(cache, "q8_0")
    want, _, parts = K.attention(qkv[:, :hq].cpu().numpy(), held, pages.cpu().numpy(), [n], float(np.float32(dim ** -0.5)))
    assert_attention(o, None, (want, None, parts))
    new = K.rows(held, slots[-1:], "k")[0]
    assert np.array_equal(new, K.values(*K.quantize(qkv[0, hq: hq + heads].cpu().numpy(), "q8_0"), "q8_0"))
    want_y = q8(o.cpu().numpy().reshape(1, -1)) @ fo.T + x.double().cpu().numpy()
    assert np.allclose(y.cpu().numpy(), want_y, rtol=0, atol=1e-5 * np.abs(want_y).max())


def test_one_workspace_for_several_shapes(torch, qg):
    """A workspace of the largest need serves smaller calls in turn, and is left zeroed where it has to be."""
    work = qg.AttnWork.allocate(32, 2, 256)
    rng = np.random.default_rng(14)
    first = None
    for rounds in range(2):
        for dim, heads, group, lengths in [(256, 2, 16, [3000, 40]), (64, 4, 1, [5000, 0, 7]), (128, 1, 8, [20000]), (96, 2, 3, [1] * 300)]:
            rng = np.random.default_rng(dim)
            pages = sum(-(-x // 16) for x in lengths) + 1
            c = random_cache(rng, "e4m3", pages, heads, 16, dim)
            t = tables(rng, lengths, 16, pages)
            q = rng.standard_normal((len(lengths), heads * group, dim)).astype(np.float32)
            args = dev(torch, q), upload(torch, qg, c), dev(torch, t), dev(torch, np.array(lengths, np.int32))
            assert torch.equal(qg.qg_attn_decode(*args, work=work), qg.qg_attn_decode(*args))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("group", [1, 8, 16])
def test_workspace_bounds_and_counters(torch, qg, fmt, dim, group):
    """A workspace of exactly the reported size between guard bands: every CTA's counter is zero again after calls whose items
    lie on two CTAs, on many and on one, and nothing is written outside."""
    rng = np.random.default_rng(dim + group)
    heads = 2
    ws = Guarded(torch, (qg.qg_attn_decode_workspace_bytes(heads * group, heads, dim),), torch.uint8)
    work = qg.AttnWork(ws.view.zero_())
    counters = 4 * 4 * torch.cuda.get_device_properties(0).multi_processor_count  # four CTAs an SM at most
    for lengths in ([9000], [700, 0, 5200, 31, 1], [int(n) for n in rng.integers(0, 1200, 400)]):
        c = random_cache(rng, fmt, 700, heads, 16, dim)
        t = rng.integers(0, 700, (len(lengths), -(-max(lengths) // 16) + 300)).astype(np.int32)  # pages shared by sequences
        q = rng.standard_normal((len(lengths), heads * group, dim)).astype(np.float32)
        args = dev(torch, q), upload(torch, qg, c), dev(torch, t), dev(torch, np.array(lengths, np.int32))
        got = qg.qg_attn_decode(*args, work=work)
        ws.check()
        assert not ws.view[:counters].any()
        assert ws.view[counters:].any()  # the line's records
        if len(lengths) < 10:
            assert_attention(got, None, K.attention(q, c, t, lengths, float(np.float32(dim ** -0.5))))
        assert torch.equal(qg.qg_attn_decode(*args, work=work), got)


def test_binding_refusals(torch, qg):
    cache = qg.KVCache.allocate(4, 16, 2, 64)
    x, slots = torch.zeros((3, 2, 64), device="cuda"), torch.arange(3, device="cuda")
    pages, n = torch.zeros((3, 2), dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")
    work = qg.AttnWork.allocate(2, 2, 64)
    for bad in (lambda: qg.qg_kv_write(cache, x[:, :1], x, slots), lambda: qg.qg_kv_write(cache, x, x[:2], slots),
                lambda: qg.qg_kv_write(cache, x, x.bfloat16(), slots), lambda: qg.qg_kv_write(cache, x, x, slots.int()),
                lambda: qg.qg_kv_write(cache, x, x, slots[:2]), lambda: qg.qg_kv_write(cache, x.half(), x.half(), slots),
                lambda: qg.qg_kv_write(cache, torch.zeros((3, 64, 2), device="cuda").transpose(1, 2), x, slots),
                lambda: qg.qg_kv_write(qg.KVCache(cache.k, cache.k_scales.float(), cache.v, cache.v_scales), x, x, slots),
                lambda: qg.qg_kv_write(qg.KVCache(cache.k[:, :, ::2], cache.k_scales, cache.v, cache.v_scales), x, x, slots),
                lambda: qg.qg_kv_write(qg.KVCache(cache.k.short(), cache.k_scales, cache.v, cache.v_scales), x, x, slots),
                lambda: qg.qg_kv_read(cache, slots.int()), lambda: qg.qg_kv_read(cache, slots[None]),
                lambda: qg.qg_kv_read(cache, slots, torch.float32, x.bfloat16(), x.bfloat16()),
                lambda: qg.qg_kv_read(cache, slots, None, x[:2], x), lambda: qg.qg_kv_read(cache, slots, torch.float16),
                lambda: qg.qg_attn_decode(x[:, :1], cache, pages, n), lambda: qg.qg_attn_decode(x[0], cache, pages, n),
                lambda: qg.qg_attn_decode(x, cache, pages[:2], n), lambda: qg.qg_attn_decode(x, cache, pages.long(), n),
                lambda: qg.qg_attn_decode(x, cache, pages, n[:2]), lambda: qg.qg_attn_decode(x, cache, pages, n.long()),
                lambda: qg.qg_attn_decode(x, cache, pages, n, out=x[:2]), lambda: qg.qg_attn_decode(x, cache, pages, n, out_dtype=torch.half),
                lambda: qg.qg_attn_decode(x, cache, pages, n, lse=x[:, :, 0]), lambda: qg.qg_attn_decode(x, cache, pages, n, scale="a"),
                lambda: qg.qg_attn_decode(x, cache, pages.t().contiguous().t(), n),
                lambda: qg.qg_attn_decode(x, cache, pages, n, work=qg.AttnWork(work.buf.int()))):
        with pytest.raises((ValueError, TypeError)):
            bad()
    from block_quantized_decode_rmsnorm_gb300._lib import QGError

    for bad in (lambda: qg.qg_attn_decode(x, cache, pages, n, window=-1), lambda: qg.qg_attn_decode(x, cache, pages, n, out=x),
                lambda: qg.qg_attn_decode(x, cache, pages, n, work=qg.AttnWork(work.buf[:-16])),
                lambda: qg.qg_kv_read(cache, slots, None, x, x),
                lambda: qg.qg_kv_write(cache, torch.zeros(3 * 2 * 64 + 1, device="cuda")[1:].view(3, 2, 64), x, slots)):
        with pytest.raises(QGError):
            bad()
    torch.cuda.synchronize()
