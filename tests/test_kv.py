"""The key-value cache on the CPU: its oracle against brute force, the C boundary's refusals, the binding's."""

import ctypes

import numpy as np
import pytest

from oracle import kv as K

OK, NULL, ALIGN, SHAPE, UNSUPPORTED = range(5)
F32, BF16 = 0, 1
Q8_0, E4M3 = 0, 1


@pytest.fixture(scope="module")
def lib():
    from block_quantized_decode_rmsnorm_gb300 import _lib, build

    build()
    return _lib.load()


def at(i, off=0):
    """Well aligned addresses far from one another, never dereferenced."""
    return (1 << 44) + (i << 40) + off


def desc(**kw):
    from block_quantized_decode_rmsnorm_gb300._lib import KVCacheDesc

    c = dict(k_codes=at(1), k_scales=at(2), v_codes=at(3), v_scales=at(4), n_pages=10, page_size=16, heads=2,
             head_dim=128, format=Q8_0)
    c.update(kw)
    return KVCacheDesc(**c)


# ---------------------------------------------------------------- the oracle

def test_quantize_agrees_with_the_q8_0_oracle(orc):
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((5, 3, 96)) * np.exp(2 * rng.standard_normal((5, 3, 1)))).astype(np.float32)
    x[0, 0, :32] = 0
    x[1, 1, 0], x[1, 1, 1] = 127.0, 0.5  # a tie, if the block's largest is 127
    x[1, 1, 2:32] = np.arange(30) - 14.5
    q, d = K.quantize(x, "q8_0")
    wq, wd = orc.quantize_q8_0(x.reshape(15, 96))
    assert np.array_equal(q.reshape(15, 96), wq) and np.array_equal(d.view(np.uint16).reshape(15, 3), wd.view(np.uint16))
    assert list(q[1, 1, :4]) == [127, 1, -15, -14]  # half away from zero


@pytest.mark.parametrize("fmt", ["q8_0", "e4m3"])
def test_attention_by_hand(fmt):
    """One head, three tokens over two pages in reverse order, against sums written out."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((2, 3, 1, 64)).astype(np.float32)
    cache = {"format": fmt}
    for i, name in enumerate("kv"):
        q, d = K.quantize(x[i], fmt)
        plane = np.zeros((2, 1, 2, 64), q.dtype), np.zeros((2, 1, 2, d.shape[-1]), d.dtype)
        for t, (page, off) in enumerate([(1, 0), (1, 1), (0, 0)]):
            plane[0][page, 0, off], plane[1][page, 0, off] = q[t, 0], d[t, 0]
        cache[name], cache[name + "d"] = plane
    query = rng.standard_normal((1, 2, 64)).astype(np.float32)
    o, lse, parts = K.attention(query, cache, np.array([[1, 0]], np.int32), [3], 0.125)
    for h in range(2):
        val = [[K.values(*K.quantize(x[i, t], fmt), fmt)[0] for t in range(3)] for i in range(2)]
        w = [np.exp(0.125 * sum(query[0, h, i].astype(np.float64) * val[0][t][i] for i in range(64))) for t in range(3)]
        want = sum(w[t] * val[1][t] for t in range(3)) / sum(w)
        assert np.allclose(o[0, h], want, rtol=1e-12, atol=1e-14) and np.isclose(lse[0, h], np.log(sum(w)), rtol=1e-12)
    last, _, _ = K.attention(query, cache, np.array([[1, 0]], np.int32), [3], 0.125, window=1)
    assert np.allclose(last[0, 0], val[1][2], rtol=1e-12)
    none, l0, _ = K.attention(query, cache, np.array([[1, 0]], np.int32), [0], 0.125)
    assert not none.any() and np.all(np.isneginf(l0))


def test_moved_covers_a_change_of_the_weights():
    """The bound that the GPU tests use, against weights really changed that far."""
    rng = np.random.default_rng(2)
    p = rng.random((1, 1, 40))
    s = np.log(p)
    v = rng.standard_normal((40, 1, 8))
    part = (p / p.sum(), s - s.max(), np.ones_like(p), v)
    off, lse = K.moved(part, 1e-3, 0.0, 0.0, 0.0)
    for _ in range(200):
        w = p * (1 + 1e-3 * rng.choice([-1, 1], p.shape))
        o = np.einsum("hgt,thd->hgd", w / w.sum(), v) - np.einsum("hgt,thd->hgd", part[0], v)
        assert np.all(np.abs(o.reshape(1, 8)) <= off * 1.01)
        assert abs(np.log(w.sum() / p.sum())) <= lse[0] * 1.01


# ---------------------------------------------------------------- the kernel's arithmetic

@pytest.mark.parametrize("exponent", [-100, -24, 0, 120])
def test_corrected_quotients_give_the_divisions_codes(orc, exponent):
    """Every 4099th mantissa of a block's scale, at both ends of the exponents for which the cache's writing takes the
    corrected quotient; all 2^23 of them (5.3e9 quotients, some minutes) with QG_ALL_QUOTIENTS=1."""
    import os

    from oracle import _load

    count = _load().orc_corrected_quotients_off
    count.restype, count.argtypes = ctypes.c_int64, [ctypes.c_int64] * 3 + [ctypes.c_int]
    assert count(0, 1 << 23, 1 if os.environ.get("QG_ALL_QUOTIENTS") else 4099, exponent) == 0
    assert count((1 << 23) - 64, 1 << 23, 1, exponent) == 0 and count(0, 64, 1, exponent) == 0


# ---------------------------------------------------------------- C refusals

BAD_CACHES = [(dict(format=2), UNSUPPORTED), (dict(format=-1), UNSUPPORTED), (dict(head_dim=80), UNSUPPORTED),
              (dict(head_dim=0), UNSUPPORTED), (dict(head_dim=32), UNSUPPORTED), (dict(head_dim=512), UNSUPPORTED),
              (dict(heads=0), SHAPE), (dict(heads=-1), SHAPE), (dict(heads=1025), SHAPE), (dict(page_size=0), SHAPE),
              (dict(page_size=8), SHAPE), (dict(page_size=24), SHAPE), (dict(page_size=-16), SHAPE),
              (dict(page_size=4112), SHAPE), (dict(n_pages=-1), SHAPE), (dict(n_pages=1 << 31), SHAPE),
              (dict(k_codes=None), NULL), (dict(k_scales=None), NULL), (dict(v_codes=None), NULL),
              (dict(v_scales=None), NULL), (dict(k_codes=at(1, 8)), ALIGN), (dict(k_scales=at(2, 4)), ALIGN),
              (dict(v_codes=at(3, 1)), ALIGN), (dict(v_scales=at(4, 8)), ALIGN), (dict(v_codes=at(1)), SHAPE),
              (dict(v_codes=at(1, 10 * 16 * 2 * 128 - 16)), SHAPE), (dict(k_scales=at(1, 16)), SHAPE),
              (dict(v_scales=at(2)), SHAPE), (dict(format=E4M3, v_scales=at(2, 10 * 16 * 2 * 4 - 16)), SHAPE)]


def calls(lib):
    write = lambda c, **kw: lib.qg_kv_write(c, *{**dict(k=at(5), kr=256, kh=128, v=at(6), vr=256, vh=128, t=F32, s=at(7), n=3, st=None), **kw}.values())
    read = lambda c, **kw: lib.qg_kv_read(c, *{**dict(s=at(7), n=3, k=at(5), v=at(6), t=F32, st=None), **kw}.values())
    wb = lib.qg_attn_decode_workspace_bytes(8, 2, 128)
    attn = lambda c, **kw: lib.qg_attn_decode(c, *{**dict(q=at(5), qr=1024, qh=128, qt=F32, b=3, hq=8, p=at(6), mp=4, n=at(7), scale=0.1, w=0, o=at(8), ot=F32, lse=at(9), ws=at(10), wb=wb, st=None), **kw}.values())
    return write, read, attn


@pytest.mark.parametrize("i", range(len(BAD_CACHES)))
def test_cache_refusals(lib, i):
    kw, want = BAD_CACHES[i]
    for f in calls(lib):
        assert f(ctypes.byref(desc(**kw))) == want, kw
        assert f(None) == NULL


def test_write_refusals(lib):
    write, _, _ = calls(lib)
    c = ctypes.byref(desc())
    for kw, want in [(dict(t=2), UNSUPPORTED), (dict(n=-1), SHAPE), (dict(n=1 << 31), SHAPE), (dict(kr=-256), SHAPE),
                     (dict(kh=-128), SHAPE), (dict(vr=-4), SHAPE), (dict(vh=-4), SHAPE), (dict(k=None), NULL),
                     (dict(v=None), NULL), (dict(s=None), NULL), (dict(k=at(5, 8)), ALIGN), (dict(v=at(6, 4)), ALIGN),
                     (dict(s=at(7, 4)), ALIGN), (dict(kr=258), ALIGN), (dict(kh=130), ALIGN), (dict(vr=257), ALIGN),
                     (dict(vh=2), ALIGN), (dict(t=BF16, kr=260), ALIGN), (dict(kr=1 << 62), SHAPE),
                     (dict(k=at(1)), SHAPE), (dict(v=at(4, 16)), SHAPE), (dict(s=at(2)), SHAPE),
                     (dict(k=at(1, -(2 * 256 + 128 + 128) * 4 + 16)), SHAPE)]:
        assert write(c, **kw) == want, kw
    assert write(ctypes.byref(desc(k_codes=None)), n=0, k=None, v=None, s=None) == OK


def test_read_refusals(lib):
    _, read, _ = calls(lib)
    c = ctypes.byref(desc())
    for kw, want in [(dict(t=-1), UNSUPPORTED), (dict(n=-1), SHAPE), (dict(n=1 << 31), SHAPE), (dict(k=None), NULL),
                     (dict(v=None), NULL), (dict(s=None), NULL), (dict(k=at(5, 8)), ALIGN), (dict(v=at(6, 2)), ALIGN),
                     (dict(s=at(7, 4)), ALIGN), (dict(k=at(1)), SHAPE), (dict(v=at(2, 16)), SHAPE), (dict(v=at(5)), SHAPE),
                     (dict(v=at(5, 3 * 2 * 128 * 4 - 16)), SHAPE), (dict(k=at(7, 16)), SHAPE), (dict(s=at(6)), SHAPE)]:
        assert read(c, **kw) == want, kw
    assert read(ctypes.byref(desc(v_scales=None)), n=0, k=None, v=None, s=None) == OK


def test_attention_refusals(lib):
    _, _, attn = calls(lib)
    c = ctypes.byref(desc())
    wb = lib.qg_attn_decode_workspace_bytes(8, 2, 128)
    assert wb > 0
    for kw, want in [(dict(qt=2), UNSUPPORTED), (dict(ot=-1), UNSUPPORTED), (dict(b=-1), SHAPE),
                     (dict(b=(1 << 20) + 1), SHAPE), (dict(hq=0), SHAPE), (dict(hq=1), SHAPE), (dict(hq=7), SHAPE),
                     (dict(hq=16386), SHAPE), (dict(qr=-8), SHAPE), (dict(qh=-8), SHAPE), (dict(mp=-1), SHAPE),
                     (dict(mp=1 << 27), SHAPE), (dict(mp=(1 << 26) + 1), SHAPE), (dict(w=-1), SHAPE),
                     (dict(mp=1 << 26, b=1 << 20, qr=0), UNSUPPORTED), (dict(q=None), NULL), (dict(p=None), NULL),
                     (dict(n=None), NULL), (dict(o=None), NULL), (dict(ws=None), NULL), (dict(q=at(5, 8)), ALIGN),
                     (dict(p=at(6, 2)), ALIGN), (dict(n=at(7, 1)), ALIGN), (dict(o=at(8, 8)), ALIGN),
                     (dict(lse=at(9, 2)), ALIGN), (dict(ws=at(10, 8)), ALIGN), (dict(qr=1026), ALIGN),
                     (dict(qh=130), ALIGN), (dict(qt=BF16, qr=1028), ALIGN), (dict(wb=wb - 1), SHAPE), (dict(wb=0), SHAPE),
                     (dict(qr=1 << 62), SHAPE), (dict(o=at(5)), SHAPE), (dict(o=at(3)), SHAPE), (dict(lse=at(8, 16)), SHAPE),
                     (dict(lse=at(7)), SHAPE), (dict(ws=at(2)), SHAPE), (dict(ws=at(8)), SHAPE), (dict(lse=at(10)), SHAPE),
                     (dict(o=at(6)), SHAPE)]:
        assert attn(c, **kw) == want, kw
    assert attn(ctypes.byref(desc(k_codes=None)), b=0, q=None, p=None, n=None, o=None, ws=None) == OK


def test_workspace_sizes(lib):
    f = lib.qg_attn_decode_workspace_bytes
    for bad in [(0, 1, 128), (8, 0, 128), (8, 3, 128), (1, 2, 128), (8, 2, 100), (16385, 1, 64), (2048, 1025, 64)]:
        assert f(*bad) == -1, bad
    assert f(8, 8, 64) > 0 and f(16384, 1, 256) > 0


# ---------------------------------------------------------------- binding refusals

def test_binding_refuses_cpu_tensors(lib):
    torch = pytest.importorskip("torch")
    import block_quantized_decode_rmsnorm_gb300 as qg

    for fmt in ("q8_0", "e4m3"):
        cache = qg.KVCache.allocate(3, 16, 2, 64, "cpu", fmt)
        assert (cache.n_pages, cache.heads, cache.page_size, cache.head_dim) == (3, 2, 16, 64)
        assert cache.nbytes == 2 * 3 * 2 * 16 * (64 + 4)
        k = torch.zeros(4, 2, 64)
        slots = torch.zeros(4, dtype=torch.int64)
        pages = torch.zeros((4, 1), dtype=torch.int32)
        for call in (lambda: qg.qg_kv_write(cache, k, k, slots), lambda: qg.qg_kv_read(cache, slots),
                     lambda: qg.qg_attn_decode(k, cache, pages, pages[:, 0]),
                     lambda: qg.qg_attn_decode(k, cache, pages, pages[:, 0], work=qg.AttnWork(torch.zeros(16, dtype=torch.uint8)))):
            with pytest.raises(ValueError, match="CUDA"):
                call()
        with pytest.raises(TypeError):
            qg.qg_kv_write(cache, np.zeros((4, 2, 64), np.float32), k, slots)
        with pytest.raises(TypeError):
            qg.qg_kv_read(cache, slots, torch.float16)


def test_allocate_refusals():
    pytest.importorskip("torch")
    import block_quantized_decode_rmsnorm_gb300 as qg

    for bad in [(3, 8, 2, 64, "cpu"), (3, 24, 2, 64, "cpu"), (3, 8192, 2, 64, "cpu"), (3, 16, 2, 72, "cpu"),
                (3, 16, 2, 64, "cpu", "bf16")]:
        with pytest.raises(ValueError):
            qg.KVCache.allocate(*bad)
    with pytest.raises(ValueError):
        qg.qg_attn_decode_workspace_bytes(7, 2, 64)
