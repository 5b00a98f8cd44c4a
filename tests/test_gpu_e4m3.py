"""GPU parity of the 8-bit floating point path against the numpy oracle.

Quantizers: codes and scales bit for bit (their f32 roundings are part of the
definition).  Products: an f32 sum of KB = ceil(k/128) block terms, each block sum
made of at most 4 rounded accumulations (2^-22 of the terms allowed each, the
tensor core's own alignment), its scale of one rounding, its addition of one, then
at most 8 partial sums joined and the residual added: within
(KB + 32) 2^-24 of the sum of |terms|, and half a step of y's type.
h = SiLU(g) u: those bounds through the formula's derivatives, and 2^-20 of |h| for
the exponential, the quotient and the products; a code lies between the codes of
the two ends of the interval that leaves.
"""

import numpy as np
import pytest

from oracle import e4m3 as E
from tests._gpu import Guarded, need_gpu

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def torch():
    return need_gpu()


@pytest.fixture(scope="module")
def qg():
    import block_quantized_decode_rmsnorm_gb300 as m

    return m


def types(torch):
    return {"f32": torch.float32, "bf16": torch.bfloat16}


def bits(t):
    return t.cpu().view(__import__("torch").uint8).numpy()


def codes_dev(torch, q):
    return torch.from_numpy(np.ascontiguousarray(q)).cuda().view(torch.float8_e4m3fn)


def dev(torch, a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def same_codes(got, want, what=""):
    nan = (want & 0x7F) == 0x7F
    assert np.array_equal((got & 0x7F) == 0x7F, nan), what
    bad = (got != want) & ~nan
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


def same_floats(got, want, what=""):
    assert np.array_equal(got, want, equal_nan=True), (what, np.argwhere(got != want)[:4])


# ---------------------------------------------------------------- quantize

@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows,k", [(1, 16), (1, 128), (2, 112), (3, 144), (33, 1024), (5, 3600), (129, 272), (1, 9216),
                                    (2, 1 << 20)])
def test_quantize(torch, qg, kind, rows, k):
    rng = np.random.default_rng(rows * 7919 + k)
    x = torch.from_numpy((rng.standard_normal((rows, k)) * np.exp(2 * rng.standard_normal((rows, k)))).astype(np.float32))
    x[-1, : k // 2] = 0
    x = x.to(types(torch)[kind])
    q, d = Guarded(torch, (rows, k), torch.float8_e4m3fn), Guarded(torch, (rows, E.blocks(k)), torch.float32)
    qg.quantize_act_e4m3(x.cuda(), q.view, d.view)
    q.check(), d.check()
    want_q, want_d = E.quantize(x.float().numpy())
    same_floats(d.view.cpu().numpy(), want_d)
    same_codes(bits(q.view), want_q)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_quantize_special_values(torch, qg, kind):
    x = np.zeros((10, 272), np.float32)
    x[1, 3], x[1, 140] = np.nan, -3.0
    x[2, 7], x[2, 200] = np.inf, -np.inf
    x[3] = np.nan
    x[4] = 1e-35          # below the floor
    x[5, ::2] = 1e-40     # subnormal
    x[6] = np.float32(3.3e38)
    x[7, 100] = 2.0 ** -100
    x[8, :127] = E.decode(np.arange(127))  # every code, then every middle of two: amax 448, factor 1
    x[9, :126] = (E.decode(np.arange(126)) + E.decode(np.arange(1, 127))) / 2
    x[9, 127], x[9, 128:254], x[9, 255] = 448, -x[9, :126], -448
    t = torch.from_numpy(x).to(types(torch)[kind])
    q, d = qg.quantize_act_e4m3(t.cuda())
    want_q, want_d = E.quantize(t.float().numpy())
    same_floats(d.cpu().numpy(), want_d)
    same_codes(bits(q), want_q)


def test_quantize_one_row_and_none(torch, qg):
    x = torch.randn(144, device="cuda")
    q, d = qg.quantize_act_e4m3(x)
    q2, d2 = qg.quantize_act_e4m3(x[None])
    assert q.shape == (1, 144) and np.array_equal(bits(q), bits(q2)) and torch.equal(d, d2)
    q, d = qg.quantize_act_e4m3(torch.empty((0, 144), device="cuda"))
    assert q.shape == (0, 144) and d.shape == (0, 2)


# ---------------------------------------------------------------- norm

NORM_SHAPES = [(1, 16), (1, 1024), (3, 144), (2, 1040), (257, 256), (5, 2560), (3, 4112), (4, 8192), (2, 8208),
               (2, 16384), (2, 16400), (1, 65536),
               (310, 1024), (311, 1536), (312, 2448), (313, 4096), (314, 4112)]  # rows that fill the SMs


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("place", ["none", "new", "x", "residual"])
@pytest.mark.parametrize("rows,k", NORM_SHAPES)
def test_norm(torch, qg, kind, place, rows, k):
    t = types(torch)[kind]
    gen = torch.Generator().manual_seed(rows * 31 + k)
    x, res = torch.randn((rows, k), generator=gen).mul(3).to(t), torch.randn((rows, k), generator=gen).to(t)
    x[-1, 1:], res[-1, 1:] = 0, 0  # one lone value
    if rows > 2:
        x[1], res[1] = 0, 0
    gamma = (1 + 0.1 * torch.randn(k, generator=gen)).to(t)
    s = x if place == "none" else (x.float() + res.float()).to(t)
    xd = x.cuda()
    rd = None if place == "none" else res.cuda()
    q, d = Guarded(torch, (rows, k), torch.float8_e4m3fn), Guarded(torch, (rows, E.blocks(k)), torch.float32)
    new = Guarded(torch, (rows, k), t)
    out = {"none": None, "new": new.view, "x": xd, "residual": rd}[place]
    _, _, got = qg.rmsnorm_add_quantize_e4m3(xd, gamma.cuda(), rd, EPS, out, q.view, d.view)
    q.check(), d.check(), new.check()
    assert torch.equal(got.cpu(), s)
    if place in ("none", "new"):
        assert torch.equal(xd.cpu(), x)
    if place in ("x", "new"):
        assert torch.equal(rd.cpu(), res)
    want_q, want_d = E.quantize(E.norm(s.float().numpy(), gamma.float().numpy(), EPS))
    same_floats(d.view.cpu().numpy(), want_d)
    same_codes(bits(q.view), want_q)


def test_norm_special_values(torch, qg):
    x = torch.randn(4, 384)
    x[0, 5], x[1, 200], x[2] = float("nan"), float("inf"), 0.0
    q, d, s = qg.rmsnorm_add_quantize_e4m3(x.cuda(), torch.ones(384, device="cuda"), torch.zeros(4, 384, device="cuda"))
    q, d = bits(q), d.cpu().numpy()
    assert np.all((q[0] & 0x7F) == 0x7F)      # NaN is in the row's mean
    assert (q[1, 200] & 0x7F) == 0x7F         # inf * (1 / inf)
    assert np.all(q[2] == 0)
    want_q, want_d = E.quantize(E.norm(x[3:].numpy(), np.ones(384), EPS))
    same_codes(q[3:], want_q), same_floats(d[3:], want_d)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("place", ["none", "new"])
@pytest.mark.parametrize("eps", [EPS, 0.0, float("inf")])
@pytest.mark.parametrize("rows,k", [(11, 144), (11, 4112), (11, 8192), (11, 16400), (310, 1024), (310, 4096)])
def test_norm_whole_range(torch, qg, kind, place, eps, rows, k):
    """Rows whose squares leave f32 at either end, with infinities and NaN among them: the
    mean is the formula's all the same, and rows beside them are what they are alone."""
    t = types(torch)[kind]
    gen = torch.Generator().manual_seed(rows + k)
    x = torch.randn((rows, k), generator=gen)
    x[0] *= 1e20
    x[1] = torch.where(x[1] > 0, 3.3e38, 1.5e38)
    x[2, k // 2] = float("inf")
    x[3, 5], x[3, k - 1] = float("-inf"), float("inf")
    x[4] *= 1e-25
    x[5] *= 1e-41
    x[6, 3] = float("nan")
    x[7], x[7, 9] = 0, 2e19
    x[8] = 0
    x[9] *= 2.0 ** -50
    x = x.to(t)
    res = (torch.randn((rows, k), generator=gen) * x.float().abs().clamp(max=1e37) * 0.25).nan_to_num(0.0).to(t)
    res[1:4] = 0
    gamma = (1 + 0.1 * torch.randn(k, generator=gen)).to(t)
    s = x if place == "none" else (x.float() + res.float()).to(t)
    q, d, got = qg.rmsnorm_add_quantize_e4m3(x.cuda(), gamma.cuda(), None if place == "none" else res.cuda(), eps)
    same_floats(got.float().cpu().numpy(), s.float().numpy())
    with np.errstate(all="ignore"):
        want_q, want_d = E.quantize(E.norm(s.float().numpy(), gamma.float().numpy(), eps))
    same_floats(d.cpu().numpy(), want_d)
    same_codes(bits(q), want_q)


# ---------------------------------------------------------------- product

def tol(k):
    return (E.blocks(k) + 32) * 2.0 ** -24


def acts(rng, m, k):
    return E.quantize((rng.standard_normal((m, k)) * np.where(rng.random(k) < 0.02, 16, 1)).astype(np.float32))


def check_product(torch, qg, rng, m, n, k, kind="f32", residual=None, weight=None, act=None):
    """residual: None, "apart" or "place" (y's own buffer)."""
    t = types(torch)[kind]
    wq, wd = weight or E.weight(rng, n, k)
    xq, xd = act or acts(rng, m, k)
    res = torch.from_numpy(rng.standard_normal((m, n)).astype(np.float32)).to(t)
    y = Guarded(torch, (m, n), t)
    rdev = None
    if residual:
        rdev = y.view if residual == "place" else res.cuda()
        rdev.copy_(res)
    qg.qgemm_e4m3(qg.E4M3Weight(codes_dev(torch, wq), dev(torch, wd)), codes_dev(torch, xq), dev(torch, xd),
                  "residual" if residual else "none", rdev, y.view)
    y.check()
    got = y.view.float().cpu().numpy().astype(np.float64)
    y64, a = E.product(wq, wd, xq, xd)
    if residual:
        r64 = res.double().numpy()
        y64, a = y64 + r64, a + np.abs(r64)
    half = torch.finfo(t).eps / 2
    bound = tol(k) * a + half * np.abs(y64) * (1 + 2.0 ** -6) + 2.0 ** -133
    bad = ~(np.abs(got - y64) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], y64[bad][:4], bound[bad][:4])


@pytest.mark.parametrize("m", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 64, 100, 127, 128, 129, 257])
def test_product_rows(torch, qg, m):
    check_product(torch, qg, np.random.default_rng(m), m, 272, 400)


@pytest.mark.parametrize("m", [1, 12, 40, 150])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000])
def test_product_columns(torch, qg, m, n):
    check_product(torch, qg, np.random.default_rng(n), m, n, 272, kind="bf16" if n % 2 else "f32",
                  residual=[None, "apart", "place"][n % 3])


@pytest.mark.parametrize("m", [1, 12, 40, 150])
@pytest.mark.parametrize("k", [16, 48, 112, 128, 144, 240, 256, 1024, 1040, 3600, 9216])
def test_product_depths(torch, qg, m, k):
    check_product(torch, qg, np.random.default_rng(k), m, 144, k, kind="bf16" if k % 64 else "f32",
                  residual=["place", None, "apart"][k % 3])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("residual", [None, "apart", "place"])
@pytest.mark.parametrize("m", [1, 7, 16, 100, 300])
def test_product_epilogues(torch, qg, m, kind, residual):
    check_product(torch, qg, np.random.default_rng(m), m, 328, 1168, kind, residual)


# few rows over more 16-row tiles than CTAs find room: two, three, and a ragged last of each
@pytest.mark.parametrize("m,n,k,kind,residual", [(1, 5001, 272, "f32", None), (8, 9744, 1040, "bf16", "place"),
                                                 (5, 14600, 144, "bf16", "apart"), (3, 9729, 2576, "f32", "apart")])
def test_product_few_rows_many_columns(torch, qg, m, n, k, kind, residual):
    check_product(torch, qg, np.random.default_rng(n), m, n, k, kind, residual)


def test_product_many_tiles(torch, qg):
    check_product(torch, qg, np.random.default_rng(5), 700, 2727, 656, "bf16", "apart")
    check_product(torch, qg, np.random.default_rng(6), 17, 5001, 1040, "f32", None)


# tiles walked by one CTA per SM: 256, 192 and 128 columns wide
@pytest.mark.parametrize("m,n,kind", [(4800, 1024, "bf16"), (2600, 999, "f32"), (2601, 1000, "bf16"), (5100, 1400, "bf16"),
                                      (5100, 1401, "bf16")])
def test_product_prompts(torch, qg, m, n, kind):
    check_product(torch, qg, np.random.default_rng(n), m, n, 272, kind, "place" if n % 2 else None)


# the same with y's rows on 32 bytes and not, with and without a residual
@pytest.mark.parametrize("residual", [None, "apart", "place"])
@pytest.mark.parametrize("m,n,kind", [(m, n, kind) for m, n0 in ((2601, 1408), (1701, 1408), (1701, 1040))
                                      for n, kind in ((n0, "f32"), (n0, "bf16"), (n0 + 1, "f32"), (n0 - 7, "bf16"))])
def test_product_stores(torch, qg, m, n, kind, residual):
    check_product(torch, qg, np.random.default_rng(m + n), m, n, 160, kind, residual)


def test_product_largest_codes(torch, qg):
    """Every code 448 or -448: the largest block sums; exact in f32 where they do not cancel."""
    for m in (3, 140):
        k, n = 384, 130
        wq, xq = np.full((n, k), 0x7E, np.uint8), np.full((m, k), 0x7E, np.uint8)
        xq[1] = 0xFE
        wd, xd = np.ones((2, 3), np.float32), np.full((m, 3), 0.5, np.float32)
        y = qg.qgemm_e4m3(qg.E4M3Weight(codes_dev(torch, wq), dev(torch, wd)), codes_dev(torch, xq), dev(torch, xd))
        want = np.full((m, n), 448.0 * 448 * k / 2)
        want[1] *= -1
        assert np.array_equal(y.cpu().numpy(), want)


def test_product_nan_stays_in_its_row_and_column(torch, qg):
    for m in (5, 150):
        rng = np.random.default_rng(m)
        n, k = 200, 272
        (wq, wd), (xq, xd) = E.weight(rng, n, k), acts(rng, m, k)
        xq[3, 270], wq[150, 0] = 0x7F, 0xFF
        xd[4, 1] = np.inf
        y = qg.qgemm_e4m3(qg.E4M3Weight(codes_dev(torch, wq), dev(torch, wd)), codes_dev(torch, xq),
                          dev(torch, xd)).cpu().numpy()
        assert np.isnan(y[3]).all() and np.isnan(y[:, 150]).all()
        assert not np.isfinite(y[4]).any()
        keep = np.ones(m, bool)
        keep[[3, 4]] = False
        assert np.isfinite(np.delete(y[keep], 150, axis=1)).all()


def test_product_zero_rows(torch, qg):
    w = qg.E4M3Weight(torch.zeros((32, 64), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                      torch.zeros((1, 1), device="cuda"))
    q, d = qg.quantize_act_e4m3(torch.empty((0, 64), device="cuda"))
    assert qg.qgemm_e4m3(w, q, d).shape == (0, 32)
    stacked = qg.E4M3Weight(w.codes, torch.zeros((2, 1), device="cuda"))
    assert qg.qg_ffn_up_e4m3(stacked, q, d)[0].shape == (0, 16)


# ---------------------------------------------------------------- gate|up

def check_up(torch, qg, rng, m, f, k, big=1.0):
    halves = [E.weight(rng, f, k, 0.05 * big) for _ in range(2)]
    wq, wd = np.concatenate([h[0] for h in halves]), np.concatenate([h[1] for h in halves])
    xq, xd = acts(rng, m, k)
    hq, hd = Guarded(torch, (m, f), torch.float8_e4m3fn), Guarded(torch, (m, E.blocks(f)), torch.float32)
    qg.qg_ffn_up_e4m3(qg.E4M3Weight(codes_dev(torch, wq), dev(torch, wd)), codes_dev(torch, xq), dev(torch, xd),
                      hq.view, hd.view)
    hq.check(), hd.check()
    (g, ag), (u, au) = (E.product(q, d, xq, xd) for q, d in halves)
    sig = 1 / (1 + np.exp(-g))
    h = g * sig * u
    eg, eu = tol(k) * ag, tol(k) * au
    eh = (np.abs(sig * (1 + g * (1 - sig))) * np.abs(u) + eu) * eg + np.abs(g * sig) * eu + eg * eg * np.abs(u) \
        + 2.0 ** -20 * np.abs(h) + 2.0 ** -140
    lo, hi = np.abs(h) - eh, np.abs(h) + eh
    a_lo, a_hi = E.block_top(np.maximum(lo, 0)), E.block_top(hi)
    d = hd.view.cpu().numpy().astype(np.float64)
    assert np.all(d >= a_lo / 448 * (1 - 2.0 ** -23)) and np.all(d <= a_hi / 448 * (1 + 2.0 ** -23))
    # the factor is 1/d to two roundings; the product is rounded once more
    f64 = 1 / E.spread(d, f)
    t, dt = h * f64, eh * f64 + np.abs(h) * f64 * 2.0 ** -21
    got = E.decode(bits(hq.view))
    c_lo, c_hi = E.decode(E.round_codes(t - dt)), E.decode(E.round_codes(t + dt))
    bad = ~((got >= c_lo) & (got <= c_hi))
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], t[bad][:4], dt[bad][:4])


@pytest.mark.parametrize("m", [1, 2, 8, 9, 16, 17, 33, 64, 100, 128, 129, 257])
def test_up_rows(torch, qg, m):
    check_up(torch, qg, np.random.default_rng(m), m, 272, 400)


@pytest.mark.parametrize("m", [1, 10, 40, 140])
@pytest.mark.parametrize("f", [16, 48, 112, 128, 144, 240, 256, 400, 1040])
def test_up_columns(torch, qg, m, f):
    check_up(torch, qg, np.random.default_rng(f), m, f, 256)


@pytest.mark.parametrize("m", [1, 10, 40, 140])
@pytest.mark.parametrize("k", [16, 112, 128, 144, 1024, 2560, 4112])
def test_up_depths(torch, qg, m, k):
    check_up(torch, qg, np.random.default_rng(k), m, 144, k)


@pytest.mark.parametrize("m,f,k", [(2500, 1040, 272), (2433, 1072, 656)])
def test_up_prompts(torch, qg, m, f, k):
    check_up(torch, qg, np.random.default_rng(f), m, f, k)


# few rows: eight and four warps a CTA, blocks within the ring, behind it, and behind what goes to L2
@pytest.mark.parametrize("m,f,k", [(1, 3648, 272), (8, 3664, 272), (3, 5008, 1168), (8, 512, 9216), (2, 400, 3088),
                                   (5, 144, 6160)])
def test_up_few_rows(torch, qg, m, f, k):
    check_up(torch, qg, np.random.default_rng(f + k), m, f, k)


@pytest.mark.parametrize("m,n,k", [(1, 272, 6144), (8, 400, 6160), (3, 144, 12304), (2, 272, 18448), (7, 2560, 9216)])
def test_product_few_rows_deep(torch, qg, m, n, k):
    check_product(torch, qg, np.random.default_rng(n + k), m, n, k, "bf16" if m % 2 else "f32", "apart")


def test_up_large_arguments(torch, qg):
    """Gates far into both tails of the SiLU."""
    for m in (4, 130):
        check_up(torch, qg, np.random.default_rng(m), m, 256, 512, big=40.0)


def test_up_padding_row(torch, qg):
    """A row of zeros gives zero codes and the floor's scale."""
    rng = np.random.default_rng(1)
    halves = [E.weight(rng, 144, 256) for _ in range(2)]
    w = qg.E4M3Weight(codes_dev(torch, np.concatenate([h[0] for h in halves])),
                      dev(torch, np.concatenate([h[1] for h in halves])))
    for m in (3, 140):
        x = torch.randn((m, 256), device="cuda")
        x[1] = 0
        hq, hd = qg.qg_ffn_up_e4m3(w, *qg.quantize_act_e4m3(x))
        assert np.all(bits(hq)[1] & 0x7F == 0)
        assert np.all(hd[1].cpu().numpy() == np.float32(2.0 ** -100) / np.float32(448))


@pytest.mark.parametrize("m", [4, 30, 2500])
@pytest.mark.parametrize("scale", [1e-3, 1.0, 1e6])
def test_up_negative_gates(torch, qg, m, scale):
    """SiLU of a large negative gate is zero, however large the gate and the up value are:
    nothing but zeros in a block of them, and the floor's scale."""
    f, k = 272, 256
    wq = np.concatenate([np.full((f, k), 0xFE, np.uint8), np.full((f, k), 0x7E, np.uint8)])  # -448 and 448
    wd = np.full((2 * E.blocks(f), 2), scale, np.float32)
    hq, hd = qg.qg_ffn_up_e4m3(qg.E4M3Weight(codes_dev(torch, wq), dev(torch, wd)),
                               codes_dev(torch, np.full((m, k), 0x7E, np.uint8)),
                               dev(torch, np.ones((m, 2), np.float32)))
    assert np.all(bits(hq) & 0x7F == 0)
    assert np.all(hd.cpu().numpy() == np.float32(2.0 ** -100) / np.float32(448))


@pytest.mark.parametrize("m", [4, 30, 2500])
def test_up_tail_of_the_silu(torch, qg, m):
    """Gates from -80 to -88.7, where e^-g nears f32's end, with up values large enough for h
    to count; from -88.75 on h is zero.  One term a sum: g and u have three roundings each (to f32
    of the scales' product and of its product with the term), which moves h by 88.7 * 3 * 2^-24
    (g) and 3 * 2^-24 (u) of itself, and a code's half step is 2^-4; 2^-12 on top of that for h."""
    g = np.append(np.linspace(-80.0, -88.7, m - 1), -88.75)
    xd = (g / -448.0).astype(np.float32)[:, None]
    xq, wq = np.zeros((m, 128), np.uint8), np.zeros((2 * 256, 128), np.uint8)
    xq[:, 5], wq[:256, 5], wq[256:, 5] = 0x38, 0xFE, 0x7E  # 1, -448, 448
    wd = np.array([1, 1, 1e30, 1e30], np.float32)[:, None]
    hq, hd = qg.qg_ffn_up_e4m3(qg.E4M3Weight(codes_dev(torch, wq), dev(torch, wd)), codes_dev(torch, xq), dev(torch, xd))
    got = E.decode(bits(hq)) * E.spread(hd.cpu().numpy().astype(np.float64), 256)
    g64, u64 = -448.0 * xd.astype(np.float64), 448.0 * xd.astype(np.float64) * np.float64(np.float32(1e30))
    h = np.repeat(g64 / (1 + np.exp(-g64)) * u64, 256, axis=1)
    assert np.all(np.abs(h) > 1e-6)
    assert np.all(np.abs(got[:-1] - h[:-1]) <= (2.0 ** -4 + 2.0 ** -12) * np.abs(h[:-1]))
    assert np.all(got[-1] == 0)


@pytest.mark.parametrize("m", [4, 30, 2500])
def test_up_nan_row(torch, qg, m):
    """A NaN activation makes its own row's codes NaN, with the floor's scale, and leaves
    the other rows alone; a NaN weight its own column's."""
    rng = np.random.default_rng(m)
    f = 1040
    halves = [E.weight(rng, f, 256) for _ in range(2)]
    wq = np.concatenate([h[0] for h in halves])
    w = qg.E4M3Weight(codes_dev(torch, wq), dev(torch, np.concatenate([h[1] for h in halves])))
    xq, xd = acts(rng, m, 256)
    clean = qg.qg_ffn_up_e4m3(w, codes_dev(torch, xq), dev(torch, xd))
    xq[2, 77] = 0x7F
    hq, hd = qg.qg_ffn_up_e4m3(w, codes_dev(torch, xq), dev(torch, xd))
    assert np.all(bits(hq)[2] & 0x7F == 0x7F)
    assert np.all(hd[2].cpu().numpy() == np.float32(2.0 ** -100) / np.float32(448))
    rest = np.arange(m) != 2
    assert np.array_equal(bits(hq)[rest], bits(clean[0])[rest]) and torch.equal(hd[rest], clean[1][rest])
    wq[f + 500, 3] = 0x7F
    hq, hd = qg.qg_ffn_up_e4m3(qg.E4M3Weight(codes_dev(torch, wq), w.scales), codes_dev(torch, xq), dev(torch, xd))
    assert np.all(bits(hq)[:, 500] & 0x7F == 0x7F)
    assert not np.any(np.delete(bits(hq)[rest], 500, axis=1) & 0x7F == 0x7F)


# ---------------------------------------------------------------- together

def make_layer(torch, qg, rng, hidden, ffn, t):
    halves = [E.weight(rng, ffn, hidden, 0.05) for _ in range(2)]
    dq, dd = E.weight(rng, hidden, ffn, 0.05)
    gamma = (1 + 0.1 * torch.randn(hidden, generator=torch.Generator().manual_seed(3))).to(t).cuda()
    return qg.E4M3Layer(gamma, qg.E4M3Weight(codes_dev(torch, np.concatenate([h[0] for h in halves])),
                                             dev(torch, np.concatenate([h[1] for h in halves]))),
                        qg.E4M3Weight(codes_dev(torch, dq), dev(torch, dd)))


def chain(qg, x, layer, residual, eps=EPS):
    q, d, s = qg.rmsnorm_add_quantize_e4m3(x, layer.gamma, residual, eps)
    hq, hd = qg.qg_ffn_up_e4m3(layer.gate_up, q, d)
    return qg.qgemm_e4m3(layer.down, hq, hd, "residual", s)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("m", [1, 5, 16, 40, 200])
def test_ffn_is_its_three_calls(torch, qg, kind, m):
    t = types(torch)[kind]
    rng = np.random.default_rng(m)
    layer = make_layer(torch, qg, rng, 400, 272, t)
    x, res = torch.randn((m, 400), device="cuda").to(t), torch.randn((m, 400), device="cuda").to(t)
    want, want0 = chain(qg, x, layer, res), chain(qg, x, layer, None)
    assert torch.equal(qg.qg_ffn_e4m3(x, layer, res, EPS), want)
    assert torch.equal(qg.qg_ffn_e4m3(x, layer, None, EPS), want0)
    buf = qg.E4M3Buffers.allocate(m, 400, 272, "cuda")
    x2 = x.clone()
    assert torch.equal(qg.qg_ffn_e4m3(x2, layer, res, EPS, buf, x2), want) and torch.equal(x2, want)
    x2, r2 = x.clone(), res.clone()
    qg.qg_ffn_e4m3(x2, layer, r2, EPS, buf, r2)
    assert torch.equal(r2, want) and torch.equal(x2, x)
    x2 = x.clone()
    qg.qg_ffn_e4m3(x2, layer, None, EPS, buf, x2)
    assert torch.equal(x2, want0)


def test_layers_against_f64(torch, qg):
    """Three layers over a padded batch: each stage against the formula on the
    GPU's own input to it, as the stages' tests do, here through the chain."""
    t = torch.float32
    layers = [make_layer(torch, qg, np.random.default_rng(i), 256, 400, t) for i in range(3)]
    x = torch.randn((6, 256), device="cuda")
    x[4:] = 0
    for layer in layers:
        y = qg.qg_ffn_e4m3(x, layer, None, EPS)
        q, d = E.quantize(E.norm(x.cpu().numpy(), layer.gamma.cpu().numpy(), EPS))
        gq, gd = bits(layer.gate_up.codes), layer.gate_up.scales.cpu().numpy()
        g, _ = E.product(gq[:400], gd[:4], q, d)
        u, _ = E.product(gq[400:], gd[4:], q, d)
        h = g / (1 + np.exp(-g)) * u
        hq, hd = E.quantize(h.astype(np.float32))
        y64, a = E.product(bits(layer.down.codes), layer.down.scales.cpu().numpy(), hq, hd)
        # a code of h may fall on the other side of a middle: a step (2^-3 of a value) in a few of
        # the 400 terms; one in a hundred of the terms' sum is far beyond that
        want = x.cpu().numpy() + y64
        assert np.all(np.abs(y.cpu().numpy() - want) <= 0.01 * a + 1e-6 * np.abs(want))
        assert torch.equal(y[4:], x[4:])
        x = y


@pytest.mark.parametrize("m", [1, 12, 140])
def test_graph_replay(torch, qg, m):
    layer = make_layer(torch, qg, np.random.default_rng(m), 256, 272, torch.bfloat16)
    x, res = (torch.randn((m, 256), device="cuda").bfloat16() for _ in range(2))
    buf, y = qg.E4M3Buffers.allocate(m, 256, 272, "cuda"), torch.empty_like(x)
    qg.qg_ffn_e4m3(x, layer, res, EPS, buf, y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(2):
            qg.qg_ffn_e4m3(x, layer, res, EPS, buf, y)
    for seed in range(3):
        x.copy_(torch.randn((m, 256), generator=torch.Generator().manual_seed(seed)))
        y.zero_()
        g.replay()
        assert torch.equal(y, chain(qg, x, layer, res))


def test_streams_at_once(torch, qg):
    """Two streams run different calls at the same time; outputs are those of one after the other."""
    layers = [make_layer(torch, qg, np.random.default_rng(i), 512, 400, torch.float32) for i in range(2)]
    xs = [torch.randn((m, 512), device="cuda") for m in (3, 170)]
    want = [chain(qg, x, ly, None) for x, ly in zip(xs, layers)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(qg.qg_ffn_e4m3(xs[i], layers[i], None, EPS, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


@pytest.mark.parametrize("m", [1, 40, 300])
def test_streams_by_handle(torch, qg, m):
    """stream= as a torch stream, its raw handle, and the legacy default stream's."""
    layer = make_layer(torch, qg, np.random.default_rng(m), 256, 272, torch.float32)
    x = torch.randn((m, 256), device="cuda")
    want = chain(qg, x, layer, None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, torch.cuda.default_stream(), 0):
        q, d, s = qg.rmsnorm_add_quantize_e4m3(x, layer.gamma, None, EPS, stream=stream)
        h = qg.qg_ffn_up_e4m3(layer.gate_up, q, d, stream=stream)
        y = qg.qgemm_e4m3(layer.down, *h, "residual", s, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        q2, d2 = qg.quantize_act_e4m3(x, stream=stream)
        torch.cuda.synchronize()
        same_codes(bits(q2), E.quantize(x.cpu().numpy())[0])


def test_threads_at_once(torch, qg):
    """Host threads with a stream each: the library's per-device caches are filled under a lock."""
    import threading

    layer = make_layer(torch, qg, np.random.default_rng(0), 384, 272, torch.bfloat16)
    xs = [torch.randn((m, 384), device="cuda").bfloat16() for m in (1, 9, 70, 200)]
    want = [chain(qg, x, layer, None) for x in xs]
    torch.cuda.synchronize()
    got, errors = [[] for _ in xs], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(10):
                got[i].append(qg.qg_ffn_e4m3(xs[i], layer, None, EPS, stream=stream))
            stream.synchronize()
        except Exception as e:  # noqa: BLE001 - handed to the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
    [t.start() for t in threads], [t.join() for t in threads]
    assert not errors, errors
    assert all(torch.equal(y, want[i]) for i in range(len(xs)) for y in got[i])


@pytest.mark.parametrize("m", [1, 30, 2500])
def test_first_call_inside_a_capture(torch, m):
    """A process whose first call of all is captured: nothing that the call asks the
    driver for on first use breaks the capture."""
    import subprocess
    import sys

    code = f"""
import torch
import block_quantized_decode_rmsnorm_gb300 as qg
f8 = torch.float8_e4m3fn
x = torch.randn(({m}, 256), device='cuda')
w = lambda n, k: torch.randint(0, 120, (n, k), device='cuda').to(torch.uint8).view(f8)
layer = qg.E4M3Layer(torch.ones(256, device='cuda'), qg.E4M3Weight(w(2 * 1040, 256), torch.full((18, 2), 1e-4, device='cuda')),
                     qg.E4M3Weight(w(256, 1040), torch.full((2, 9), 1e-4, device='cuda')))
buf, y = qg.E4M3Buffers.allocate({m}, 256, 1040, 'cuda'), torch.empty_like(x)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    qg.qg_ffn_e4m3(x, layer, x, 1e-6, buf, y)
y.zero_()
g.replay()
assert torch.equal(y, qg.qg_ffn_e4m3(x, layer, x, 1e-6)) and bool(y.isfinite().all())
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("m", [1, 40, 300])
def test_weights_replaced_in_stream_order(torch, qg, m):
    """Weights written by a kernel of another library just before the call: that one has
    ended when this one starts (the library's own kernels do not write weights that the
    next call reads)."""
    rng = np.random.default_rng(m)
    ws = [E.weight(rng, 400, 1024) for _ in range(2)]
    codes, scales = [codes_dev(torch, w[0]) for w in ws], [dev(torch, w[1]) for w in ws]
    xq, xd = qg.quantize_act_e4m3(torch.randn((m, 1024), device="cuda"))
    want = [qg.qgemm_e4m3(qg.E4M3Weight(c, s), xq, xd) for c, s in zip(codes, scales)]
    w = qg.E4M3Weight(codes[0].clone(), scales[0].clone())
    got = []
    for i in range(20):
        w.codes.view(torch.uint8).copy_(codes[i % 2].view(torch.uint8))
        w.scales.copy_(scales[i % 2])
        got.append(qg.qgemm_e4m3(w, xq, xd))
    assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(got))


@pytest.mark.parametrize("m", [1, 40, 300])
@pytest.mark.parametrize("wait", ["host", "event"])
def test_codes_of_a_quantizer_as_a_weight(torch, qg, m, wait):
    """One row's codes and scales are a weight of one row, once the call that writes them has
    been waited for (which the documentation asks for)."""
    gen = torch.Generator().manual_seed(m)
    row, x = torch.randn((1, 4112), generator=gen), torch.randn((m, 4112), generator=gen)
    xq, xd = qg.quantize_act_e4m3(x.cuda())
    rows = [row.cuda() * (i + 1) for i in range(4)]
    q, d = qg.quantize_act_e4m3(rows[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for r in rows:
        qg.quantize_act_e4m3(r, q, d)
        if wait == "host":
            torch.cuda.synchronize()
            y = qg.qgemm_e4m3(qg.E4M3Weight(q, d), xq, xd)
        else:
            side.wait_stream(torch.cuda.current_stream())
            y = qg.qgemm_e4m3(qg.E4M3Weight(q, d), xq, xd, stream=side)
            torch.cuda.current_stream().wait_stream(side)
        want, a = E.product(*E.quantize(r.cpu().numpy()), bits(xq), xd.cpu().numpy())
        assert np.all(np.abs(y.cpu().numpy() - want) <= tol(4112) * a + 2.0 ** -23 * np.abs(want))


def test_rows_past_the_last(torch, qg):
    """The first rows of a larger batch: what lies behind them is neither read into the
    results nor written."""
    rng = np.random.default_rng(2)
    w = E.weight(rng, 144, 512)
    w = qg.E4M3Weight(codes_dev(torch, w[0]), dev(torch, w[1]))
    x = torch.randn((300, 512), device="cuda")
    q, d = qg.quantize_act_e4m3(x)
    for m in (1, 8, 9, 33, 129):
        q2, d2 = q.clone(), d.clone()
        q2.view(torch.uint8)[m:] = 0x7F
        d2[m:] = float("nan")
        y = torch.full((300, 144), -7.0, device="cuda")
        qg.qgemm_e4m3(w, q2[:m], d2[:m], y=y[:m])
        assert torch.equal(y[:m], qg.qgemm_e4m3(w, q[:m], d[:m]))
        assert bool((y[m:] == -7.0).all())


def test_results_repeat(torch, qg):
    rng = np.random.default_rng(0)
    for m, n, k in [(1, 1000, 4112), (12, 300, 2560), (60, 1000, 4112), (300, 500, 1024)]:
        w = E.weight(rng, n, k)
        w = qg.E4M3Weight(codes_dev(torch, w[0]), dev(torch, w[1]))
        q, d = qg.quantize_act_e4m3(torch.randn((m, k), device="cuda"))
        first = qg.qgemm_e4m3(w, q, d)
        assert all(torch.equal(first, qg.qgemm_e4m3(w, q, d)) for _ in range(5))


def test_refusals(torch, qg):
    x = torch.randn((4, 256), device="cuda")
    q, d = qg.quantize_act_e4m3(x)
    w = qg.E4M3Weight(torch.zeros((64, 256), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                      torch.zeros((1, 2), device="cuda"))
    bad = [
        (TypeError, lambda: qg.quantize_act_e4m3(x.half())),
        (ValueError, lambda: qg.quantize_act_e4m3(x[:, ::2])),
        (ValueError, lambda: qg.quantize_act_e4m3(x[None])),
        (qg_error(qg), lambda: qg.quantize_act_e4m3(x[:, :24].contiguous())),
        (qg_error(qg), lambda: qg.quantize_act_e4m3(x.view(-1)[1:513])),       # not on 16 bytes
        (TypeError, lambda: qg.quantize_act_e4m3(x, q.view(torch.uint8))),
        (ValueError, lambda: qg.quantize_act_e4m3(x, q, d[:, :1].contiguous())),
        (TypeError, lambda: qg.rmsnorm_add_quantize_e4m3(x, x[0].bfloat16())),
        (ValueError, lambda: qg.rmsnorm_add_quantize_e4m3(x, x[0], x[:2])),
        (ValueError, lambda: qg.rmsnorm_add_quantize_e4m3(x, x[0], None, EPS, torch.empty_like(x))),
        (qg_error(qg), lambda: qg.rmsnorm_add_quantize_e4m3(x, x[0].clone(), None, -1.0)),
        (ValueError, lambda: qg.qgemm_e4m3(w, q, d[:2])),
        (ValueError, lambda: qg.qgemm_e4m3(w, q[:, :128].contiguous(), d)),
        (ValueError, lambda: qg.qgemm_e4m3(w, q, d, "residual")),
        (ValueError, lambda: qg.qgemm_e4m3(w, q, d, "none", x[:, :64].contiguous())),
        (TypeError, lambda: qg.qgemm_e4m3(w, q, d, out_dtype=torch.float16)),
        (ValueError, lambda: qg.qgemm_e4m3(w, q, d, y=torch.empty((4, 63), device="cuda"))),
        (ValueError, lambda: qg.qgemm_e4m3(qg.E4M3Weight(w.codes, d), q, d)),
        (qg_error(qg), lambda: qg.qgemm_e4m3(w, q, d, "silu_mul")),
        (ValueError, lambda: qg.qg_ffn_up_e4m3(qg.E4M3Weight(w.codes[:48], w.scales), q, d)),
        (ValueError, lambda: qg.qg_ffn_up_e4m3(qg.E4M3Weight(w.codes[:32], w.scales), q, d)),  # one scale row, not two
        (ValueError, lambda: qg.quantize_act_e4m3(x, q.cpu(), d)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()


def qg_error(qg):
    from block_quantized_decode_rmsnorm_gb300._lib import QGError

    return QGError
