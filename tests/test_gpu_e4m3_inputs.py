"""The 8-bit floating point path on inputs that lie, count or begin otherwise than in its other
tests: the smallest alignments that the calls allow, tensors of more than 2^31 values, the two
sides of each rule that chooses a kernel, a process's first calls from several threads, and
repeated calls.  Bounds are those of test_gpu_e4m3."""

import subprocess
import sys

import numpy as np
import pytest

from oracle import e4m3 as E
from tests._gpu import need_gpu
from tests.test_gpu_e4m3 import acts, bits, check_product, check_up, codes_dev, dev, same_codes, same_floats, tol

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def torch():
    return need_gpu()


@pytest.fixture(scope="module")
def qg():
    import block_quantized_decode_rmsnorm_gb300 as m

    return m


def off(t, by):
    """A copy of t that starts `by` bytes behind a multiple of 256."""
    import torch

    raw = torch.zeros(t.numel() * t.element_size() + 512, dtype=torch.uint8, device="cuda")
    start = (-raw.data_ptr()) % 256 + by
    copy = raw[start:start + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
    copy.copy_(t)
    assert copy.data_ptr() % 256 == by
    return copy


def same(a, b):
    import torch

    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---------------------------------------------------------------- alignment

# few rows; clusters sharing k; the walk (a multiple of four blocks of k, and not)
ALIGN_SHAPES = [(3, 272, 1024), (9, 272, 1024), (100, 400, 2048), (129, 144, 4096), (2601, 1408, 512), (2601, 1408, 656)]


@pytest.mark.parametrize("m,n,k", ALIGN_SHAPES)
def test_scales_on_four_bytes(torch, qg, m, n, k):
    rng = np.random.default_rng(m + k)
    halves = [E.weight(rng, n, k) for _ in range(2)]
    w = qg.E4M3Weight(codes_dev(torch, halves[0][0]), dev(torch, halves[0][1]))
    gu = qg.E4M3Weight(codes_dev(torch, np.concatenate([h[0] for h in halves])),
                       dev(torch, np.concatenate([h[1] for h in halves])))
    xq, xd = qg.quantize_act_e4m3(torch.randn((m, k), device="cuda"))
    want, (want_q, want_d) = qg.qgemm_e4m3(w, xq, xd), qg.qg_ffn_up_e4m3(gu, xq, xd)
    for a, b in ((4, 0), (0, 4), (8, 12), (12, 8)):
        assert same(qg.qgemm_e4m3(qg.E4M3Weight(w.codes, off(w.scales, b)), xq, off(xd, a)), want)
        hd = off(torch.zeros_like(want_d), a)
        hq, _ = qg.qg_ffn_up_e4m3(qg.E4M3Weight(gu.codes, off(gu.scales, b)), xq, off(xd, a), None, hd)
        assert same(hq, want_q) and same(hd, want_d)


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
@pytest.mark.parametrize("m,n,k", ALIGN_SHAPES)
def test_outputs_and_codes_on_sixteen_bytes(torch, qg, m, n, k, kind):
    t = getattr(torch, kind)
    rng = np.random.default_rng(m + k)
    w = qg.E4M3Weight(*(f(torch, a) for f, a in zip((codes_dev, dev), E.weight(rng, n, k))))
    xq, xd = qg.quantize_act_e4m3(torch.randn((m, k), device="cuda"))
    res = torch.randn((m, n), device="cuda").to(t)
    plain, added = qg.qgemm_e4m3(w, xq, xd, out_dtype=t), qg.qgemm_e4m3(w, xq, xd, "residual", res)
    w16, x16 = qg.E4M3Weight(off(w.codes, 16), w.scales), off(xq, 48)
    for a, b in ((16, 0), (0, 16), (16, 16), (48, 32)):
        y = off(torch.zeros_like(res), a)
        assert same(qg.qgemm_e4m3(w16, x16, xd, y=y), plain)
        assert same(qg.qgemm_e4m3(w16, x16, xd, "residual", off(res, b), y), added)
        y = off(res, a)
        assert same(qg.qgemm_e4m3(w16, x16, xd, "residual", y, y), added)


@pytest.mark.parametrize("m,n,k", ALIGN_SHAPES)
def test_codes_of_h_on_sixteen_bytes(torch, qg, m, n, k):
    rng = np.random.default_rng(m + k)
    halves = [E.weight(rng, n, k) for _ in range(2)]
    w = qg.E4M3Weight(codes_dev(torch, np.concatenate([h[0] for h in halves])),
                      dev(torch, np.concatenate([h[1] for h in halves])))
    xq, xd = qg.quantize_act_e4m3(torch.randn((m, k), device="cuda"))
    want_q, want_d = qg.qg_ffn_up_e4m3(w, xq, xd)
    hq = off(torch.zeros_like(want_q), 16)
    _, hd = qg.qg_ffn_up_e4m3(qg.E4M3Weight(off(w.codes, 112), w.scales), off(xq, 16), xd, hq)
    assert same(hq, want_q) and same(hd, want_d)


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,k", [(1, 1024), (3, 144), (400, 1024), (400, 4112), (3, 8192), (3, 16400)])
def test_quantizers_on_sixteen_bytes(torch, qg, rows, k, kind):
    t = getattr(torch, kind)
    x, res = (torch.randn((rows, k), device="cuda").to(t) for _ in range(2))
    gamma = torch.randn(k, device="cuda").to(t)
    (q0, d0), (q1, d1, s1) = qg.quantize_act_e4m3(x), qg.rmsnorm_add_quantize_e4m3(x, gamma, res, EPS)
    q, d = off(q0, 16), off(d0, 4)
    q.view(torch.uint8).zero_(), d.zero_()
    qg.quantize_act_e4m3(off(x, 16), q, d)
    assert same(q, q0) and same(d, d0)
    q, d, s = off(q1, 48), off(d1, 12), off(s1, 16)
    q.view(torch.uint8).zero_(), d.zero_(), s.zero_()
    qg.rmsnorm_add_quantize_e4m3(off(x, 16), off(gamma, 16), off(res, 112), EPS, s, q, d)
    assert same(q, q1) and same(d, d1) and same(s, s1)


# ---------------------------------------------------------------- more than 2^31 values

BIG = 2 ** 31


def ends(rows, width):
    """A few rows at the start, where the values' count passes 2^31, and at the end."""
    mid = BIG // width
    return np.r_[0:3, mid - 2:mid + 2, rows - 3:rows]


@pytest.mark.parametrize("rows,k", [(32769 + 2, 65536), (32769 + 2, 65520 + 32)])
def test_quantize_past_2_31(torch, qg, rows, k):
    assert rows * k > BIG
    x = torch.randn((rows, k), device="cuda", dtype=torch.bfloat16)
    q, d = qg.quantize_act_e4m3(x)
    at = ends(rows, k)
    want_q, want_d = E.quantize(x[at].float().cpu().numpy())
    same_floats(d[at].cpu().numpy(), want_d)
    same_codes(bits(q.view(torch.uint8)[at]), want_q)


@pytest.mark.parametrize("k", [65536, 8192])
def test_norm_past_2_31(torch, qg, k):
    rows = BIG // k + 3
    x = torch.randn((rows, k), device="cuda", dtype=torch.bfloat16)
    res = x.flip(0)
    gamma = torch.ones(k, device="cuda", dtype=torch.bfloat16)
    q, d, s = qg.rmsnorm_add_quantize_e4m3(x, gamma, res, EPS)
    at = ends(rows, k)
    want = (x[at].float() + res[at].float()).bfloat16()
    assert torch.equal(s[at], want)
    want_q, want_d = E.quantize(E.norm(want.float().cpu().numpy(), np.ones(k), EPS))
    same_floats(d[at].cpu().numpy(), want_d)
    same_codes(bits(q.view(torch.uint8)[at]), want_q)


def random_codes(torch, n, k, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(0, 256, (n, k), dtype=torch.uint8, device="cuda", generator=gen)
    c.bitwise_and_(0xF7)  # the lowest bit of the exponent cleared: no NaN
    return c


def random_scales(torch, n, k, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand((n, k), device="cuda", generator=gen).mul_(1e-3)


def rows_of(wd, at):
    """The scales of single weight rows, as a weight of as many blocks of rows would have them."""
    return wd.cpu().numpy()[at // 128]


def product_of_rows(wq, wd, at, xq, xd):
    """(y, sum of |terms|) for weight rows `at`, in f64."""
    w = E.decode(wq[at].cpu().numpy()) * E.spread(rows_of(wd, at).astype(np.float64), wq.shape[1])
    x = E.decode(xq) * E.spread(xd.astype(np.float64), xq.shape[1])
    return x @ w.T, np.abs(x) @ np.abs(w).T


@pytest.mark.parametrize("m", [1, 8, 20, 300])
def test_product_weights_past_2_31(torch, qg, m):
    n, k = 32784, 65552
    assert n * k > BIG
    wq, wd = random_codes(torch, n, k, 1), random_scales(torch, E.blocks(n), E.blocks(k), 2)
    xq, xd = acts(np.random.default_rng(m), m, k)
    y = qg.qgemm_e4m3(qg.E4M3Weight(wq.view(torch.float8_e4m3fn), wd), codes_dev(torch, xq), dev(torch, xd)).cpu().numpy()
    at = ends(n, k)
    want, a = product_of_rows(wq, wd, at, xq, xd)
    assert np.all(np.abs(y[:, at] - want) <= tol(k) * a + 2.0 ** -24 * np.abs(want))


@pytest.mark.parametrize("n", [16, 144])
def test_product_activations_past_2_31(torch, qg, n):
    m, k = 32784, 65552
    xq, xd = random_codes(torch, m, k, 3), random_scales(torch, m, E.blocks(k), 4)
    wq, wd = E.weight(np.random.default_rng(n), n, k)
    y = qg.qgemm_e4m3(qg.E4M3Weight(codes_dev(torch, wq), dev(torch, wd)), xq.view(torch.float8_e4m3fn), xd).cpu().numpy()
    at = ends(m, k)
    want, a = E.product(wq, wd, xq[at].cpu().numpy(), xd[at].cpu().numpy())
    assert np.all(np.abs(y[at] - want) <= tol(k) * a + 2.0 ** -24 * np.abs(want))


@pytest.mark.parametrize("n,residual", [(16400, False), (16400, True), (16401, False), (16401, True)])
def test_product_outputs_past_2_31(torch, qg, n, residual):
    m, k = 131077, 144
    xq, xd = random_codes(torch, m, k, 5), random_scales(torch, m, E.blocks(k), 6)
    wq, wd = E.weight(np.random.default_rng(n), n, k)
    at = ends(m, n)
    y = torch.randn((m, n), device="cuda", dtype=torch.bfloat16) if residual else None
    r64 = y[at].double().cpu().numpy() if residual else 0.0
    y = qg.qgemm_e4m3(qg.E4M3Weight(codes_dev(torch, wq), dev(torch, wd)), xq.view(torch.float8_e4m3fn), xd,
                      "residual" if residual else "none", y, y, torch.bfloat16)
    want, a = E.product(wq, wd, xq[at].cpu().numpy(), xd[at].cpu().numpy())
    want, a = want + r64, a + np.abs(r64)
    got = y[at].double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol(k) * a + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -6))


def check_block(got, d, g, ag, u, au, k):
    """Codes and scales [rows, cols <= 128], [rows] of one block of h, as check_up has them."""
    sig = 1 / (1 + np.exp(-g))
    h = g * sig * u
    eg, eu = tol(k) * ag, tol(k) * au
    eh = (np.abs(sig * (1 + g * (1 - sig))) * np.abs(u) + eu) * eg + np.abs(g * sig) * eu + eg * eg * np.abs(u) \
        + 2.0 ** -20 * np.abs(h) + 2.0 ** -140
    d = d.astype(np.float64)[:, None]
    assert np.all(d >= E.block_top(np.maximum(np.abs(h) - eh, 0)) / 448 * (1 - 2.0 ** -23))
    assert np.all(d <= E.block_top(np.abs(h) + eh) / 448 * (1 + 2.0 ** -23))
    t, dt = h / d, eh / d + np.abs(h) / d * 2.0 ** -21
    assert np.all((E.decode(got) >= E.decode(E.round_codes(t - dt))) & (E.decode(got) <= E.decode(E.round_codes(t + dt))))


@pytest.mark.parametrize("m", [1, 8, 20, 300])
def test_up_weights_past_2_31(torch, qg, m):
    f, k = 16400, 65552
    assert 2 * f * k > BIG
    wq, wd = random_codes(torch, 2 * f, k, 7), random_scales(torch, 2 * E.blocks(f), E.blocks(k), 8)
    wd.mul_(1e-2)
    xq, xd = acts(np.random.default_rng(m), m, k)
    hq, hd = qg.qg_ffn_up_e4m3(qg.E4M3Weight(wq.view(torch.float8_e4m3fn), wd), codes_dev(torch, xq), dev(torch, xd))
    got, d = bits(hq), hd.cpu().numpy()
    for c in (0, f // 128 * 128):  # the first block, and the last, of 16
        at = np.arange(c, min(c + 128, f))
        gate = product_of_rows(wq, wd[:E.blocks(f)], at, xq, xd)
        up = product_of_rows(wq[f:], wd[E.blocks(f):], at, xq, xd)
        check_block(got[:, at], d[:, c // 128], *gate, *up, k)


def test_up_outputs_past_2_31(torch, qg):
    m, f, k = 131077, 16400, 144
    xq, xd = random_codes(torch, m, k, 9), random_scales(torch, m, E.blocks(k), 10)
    rng = np.random.default_rng(0)
    halves = [E.weight(rng, f, k) for _ in range(2)]
    hq, hd = qg.qg_ffn_up_e4m3(qg.E4M3Weight(codes_dev(torch, np.concatenate([h[0] for h in halves])),
                                             dev(torch, np.concatenate([h[1] for h in halves]))),
                               xq.view(torch.float8_e4m3fn), xd)
    at = ends(m, f)
    got, d = bits(hq.view(torch.uint8)[at]), hd[at].cpu().numpy()
    x = xq[at].cpu().numpy(), xd[at].cpu().numpy()
    (g, ag), (u, au) = (E.product(q, s, *x) for q, s in halves)
    for b in range(E.blocks(f)):
        c = slice(128 * b, min(128 * b + 128, f))
        check_block(got[:, c], d[:, b], g[:, c], ag[:, c], u[:, c], au[:, c], k)


# ---------------------------------------------------------------- the largest sizes

@pytest.mark.parametrize("m", [1, 9, 20])
def test_largest_depth(torch, qg, m):
    k, f = 1 << 20, 16
    wq, wd = random_codes(torch, 2 * f, k, 15), random_scales(torch, 2, E.blocks(k), 16)
    x, xd = random_codes(torch, m, k, 17), random_scales(torch, m, E.blocks(k), 18)
    wd.mul_(1e-2)
    xq, at = x.view(torch.float8_e4m3fn), np.arange(f)
    y = qg.qgemm_e4m3(qg.E4M3Weight(wq[:f].view(torch.float8_e4m3fn), wd[:1]), xq, xd).cpu().numpy()
    hq, hd = qg.qg_ffn_up_e4m3(qg.E4M3Weight(wq.view(torch.float8_e4m3fn), wd), xq, xd)
    acts64 = x.cpu().numpy(), xd.cpu().numpy()
    g, ag = product_of_rows(wq, wd[:1], at, *acts64)
    u, au = product_of_rows(wq[f:], wd[1:], at, *acts64)
    assert np.all(np.abs(y - g) <= tol(k) * ag + 2.0 ** -24 * np.abs(g))
    check_block(bits(hq), hd[:, 0].cpu().numpy(), g, ag, u, au, k)


def test_most_rows(torch, qg):
    """2^24 activation rows, and one more refused."""
    m, k, n = 1 << 24, 16, 16
    xq, xd = random_codes(torch, m + 1, k, 11), random_scales(torch, m + 1, 1, 12)
    xq = xq.view(torch.float8_e4m3fn)
    halves = [E.weight(np.random.default_rng(i), n, k) for i in range(2)]
    w = qg.E4M3Weight(codes_dev(torch, halves[0][0]), dev(torch, halves[0][1]))
    gu = qg.E4M3Weight(codes_dev(torch, np.concatenate([h[0] for h in halves])),
                       dev(torch, np.concatenate([h[1] for h in halves])))
    y = qg.qgemm_e4m3(w, xq[:m], xd[:m])
    hq, hd = qg.qg_ffn_up_e4m3(gu, xq[:m], xd[:m])
    at = np.r_[0:130, m - 130:m]
    x = bits(xq.view(torch.uint8)[at]), xd[at].cpu().numpy()
    (g, ag), (u, au) = (E.product(*h, *x) for h in halves)
    assert np.all(np.abs(y[at].cpu().numpy() - g) <= tol(k) * ag + 2.0 ** -24 * np.abs(g))
    check_block(bits(hq.view(torch.uint8)[at]), hd[at, 0].cpu().numpy(), g, ag, u, au, k)
    from block_quantized_decode_rmsnorm_gb300._lib import QGError

    with pytest.raises(QGError):
        qg.qgemm_e4m3(w, xq, xd)
    with pytest.raises(QGError):
        qg.qg_ffn_up_e4m3(gu, xq, xd)


@pytest.mark.parametrize("m", [1, 9])
def test_many_columns(torch, qg, m):
    n, k = (1 << 27) + 1, 16
    wq, wd = random_codes(torch, n, k, 13), random_scales(torch, E.blocks(n), 1, 14)
    xq, xd = acts(np.random.default_rng(m), m, k)
    y = qg.qgemm_e4m3(qg.E4M3Weight(wq.view(torch.float8_e4m3fn), wd), codes_dev(torch, xq), dev(torch, xd),
                      out_dtype=torch.bfloat16)
    at = np.r_[0:3, n // 2 - 2:n // 2 + 2, n - 3:n]
    want, a = product_of_rows(wq, wd, at, xq, xd)
    got = y[:, torch.from_numpy(at).cuda()].double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol(k) * a + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -6))


def test_most_norm_rows(torch, qg):
    rows, k = (1 << 24) + 5, 16
    x = torch.randn((rows, k), device="cuda", dtype=torch.bfloat16)
    gamma = torch.ones(k, device="cuda", dtype=torch.bfloat16)
    q, d, _ = qg.rmsnorm_add_quantize_e4m3(x, gamma, None, EPS)
    at = np.r_[0:5, rows - 5:rows]
    want_q, want_d = E.quantize(E.norm(x[at].float().cpu().numpy(), np.ones(k), EPS))
    same_floats(d[at].cpu().numpy(), want_d)
    same_codes(bits(q.view(torch.uint8)[at]), want_q)


# ---------------------------------------------------------------- both sides of the rules

# few rows of gate|up: eight warps a CTA up to 228 CTAs of 16 columns on 152 SMs, four beyond
@pytest.mark.parametrize("m", [1, 8])
@pytest.mark.parametrize("f", [3568, 3584, 3600])
def test_up_warps_of_a_few_row_cta(torch, qg, m, f):
    check_up(torch, qg, np.random.default_rng(f), m, f, 2576)


# few rows of the product: a CTA to each 16 columns up to 304 of them, several to a CTA beyond
@pytest.mark.parametrize("m,n", [(1, 4864), (8, 4864), (1, 4865), (8, 4880), (3, 9728), (3, 9744)])
def test_product_tiles_of_a_few_row_cta(torch, qg, m, n):
    check_product(torch, qg, np.random.default_rng(n), m, n, 1040, "bf16", "apart")


# ---------------------------------------------------------------- no memory left

NO_MEMORY = """
import torch
import block_quantized_decode_rmsnorm_gb300 as qg

x = torch.ones((1 << 14, 1 << 14), device='cuda')
limit = torch.cuda.memory_reserved() + (1 << 26)  # not enough for the 2^28 codes
torch.cuda.set_per_process_memory_fraction(limit / torch.cuda.mem_get_info()[1])
try:
    qg.quantize_act_e4m3(x)
except torch.OutOfMemoryError:
    pass
else:
    raise AssertionError(torch.cuda.memory_summary())
torch.cuda.set_per_process_memory_fraction(1.0)
q, d = qg.quantize_act_e4m3(x)
assert bool((q.view(torch.uint8) == 0x7E).all()) and bool((d * 448 == 1).all())
"""


def test_no_memory_for_an_output():
    """torch's own error, which programs catch to try again, and the next call as ever."""
    need_gpu()
    r = subprocess.run([sys.executable, "-c", NO_MEMORY], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]


# ---------------------------------------------------------------- first calls, repeated calls

FIRST_CALLS = """
import threading
import torch
import block_quantized_decode_rmsnorm_gb300 as qg

f8, dev = torch.float8_e4m3fn, 'cuda'
codes = lambda n, k: torch.randint(0, 120, (n, k), device=dev).to(torch.uint8).view(f8)
layer = qg.E4M3Layer(torch.ones(1152, device=dev), qg.E4M3Weight(codes(2 * 1040, 1152), torch.full((18, 9), 1e-5, device=dev)),
                     qg.E4M3Weight(codes(1152, 1040), torch.full((9, 9), 1e-4, device=dev)))
xs = [torch.randn((m, 1152), device=dev) for m in (1, 9, 9, 70, 200, 2500, 2500, 1)]
torch.cuda.synchronize()
together, got, errors = threading.Barrier(len(xs)), [None] * len(xs), []

def work(i):
    try:
        stream = torch.cuda.Stream()
        together.wait()
        got[i] = [qg.qg_ffn_e4m3(xs[i], layer, xs[i], 1e-6, stream=stream) for _ in range(3)]
        stream.synchronize()
    except Exception as e:
        errors.append(e)

threads = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
[t.start() for t in threads]
[t.join() for t in threads]
assert not errors, errors
for x, ys in zip(xs, got):
    want = qg.qg_ffn_e4m3(x, layer, x, 1e-6)
    assert bool(want.isfinite().all()) and all(torch.equal(y, want) for y in ys)
"""


def test_first_calls_from_several_threads(torch):
    """A process whose first calls of all come from eight threads at the same time: the per-device
    caches (shared memory opted in to, SMs, clusters that find room, the front end itself) are
    filled by whoever is first."""
    for _ in range(2):
        r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("m,f,k", [(1, 3584, 1024), (8, 5008, 1168), (12, 400, 2560), (100, 1040, 4112), (512, 3584, 1024),
                                   (2500, 1040, 1168)])
def test_up_repeats(torch, qg, m, f, k):
    """Bit for bit, whatever ran between."""
    rng = np.random.default_rng(m)
    halves = [E.weight(rng, f, k) for _ in range(2)]
    w = qg.E4M3Weight(codes_dev(torch, np.concatenate([h[0] for h in halves])),
                      dev(torch, np.concatenate([h[1] for h in halves])))
    x, other = (qg.quantize_act_e4m3(torch.randn((m, k), device="cuda")) for _ in range(2))
    first_q, first_d = qg.qg_ffn_up_e4m3(w, *x)
    for _ in range(10):
        qg.qg_ffn_up_e4m3(w, *other)
        hq, hd = qg.qg_ffn_up_e4m3(w, *x)
        assert same(hq, first_q) and same(hd, first_d)
