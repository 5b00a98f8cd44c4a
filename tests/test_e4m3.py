"""CPU checks of the 8-bit floating point path: the oracle's format against the
definition and against torch's cast, and every refusal of the C entry points and
of the binding (argument errors are found before any CUDA call)."""

import ctypes

import numpy as np
import pytest

from oracle import e4m3 as E

FAKE = 1 << 20  # well aligned, never dereferenced
G = 1 << 32     # operands this far apart do not overlap
EPS = ctypes.c_float(1e-6)
OK, NULL, ALIGN, SHAPE, UNSUPPORTED = range(5)
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    from block_quantized_decode_rmsnorm_gb300 import _lib, build

    build()
    return _lib.load()


def at(i, off=0):
    return FAKE + i * G + off


# ---------------------------------------------------------------- the oracle

def test_table():
    assert E.VALUE[0x7E] == 448 and np.isnan(E.VALUE[0x7F]) and E.VALUE[1] == 2.0 ** -9
    assert E.VALUE[0x38] == 1 and E.VALUE[0xB8] == -1 and E.VALUE[8] == 2.0 ** -6
    assert np.all(np.diff(E.VALUE[:127]) > 0)


def test_rounding_matches_torch():
    torch = pytest.importorskip("torch")
    codes = np.arange(127, dtype=np.uint8)
    v = E.decode(codes)
    mid = (v[1:] + v[:-1]) / 2
    eps = np.spacing(mid.astype(np.float32)).astype(np.float64)
    t = np.concatenate([v, mid, mid - eps, mid + eps, [0.0, 2.0 ** -20]])
    t = np.concatenate([t, -t]).astype(np.float32)
    want = torch.from_numpy(t).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(E.round_codes(t), want)
    assert E.round_codes(np.array([1e30, -1e30, np.nan])).tolist() == [0x7E, 0xFE, 0x7F]


def test_quantize_error_bound():
    rng = np.random.default_rng(0)
    v = (rng.standard_normal((5, 304)) * np.exp(3 * rng.standard_normal((5, 304)))).astype(np.float32)
    q, d = E.quantize(v)
    back = E.decode(q) * E.spread(d.astype(np.float64), 304)
    # a half step: 2^-4 of the value, or 2^-10 codes; the two f32 roundings of factor and scale on top
    bound = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * E.spread(d, 304)) * (1 + 2.0 ** -21) + 2.0 ** -21 * np.abs(v)
    assert np.all(np.abs(back - v) <= bound)


def test_quantize_special_blocks():
    v = np.zeros((4, 256), np.float32)
    v[1, 0], v[1, 130] = np.nan, 2.0
    v[2, 5] = np.inf
    v[3, :128] = 1e-33
    q, d = E.quantize(v)
    assert np.all(q[0] == 0) and np.all(d[0] == np.float32(2.0 ** -100) / np.float32(448))
    assert q[1, 0] & 0x7F == 0x7F and q[1, 130] == 0x7E and d[1, 1] == np.float32(2) / np.float32(448)
    assert np.isinf(d[2, 0]) and q[2, 5] & 0x7F == 0x7F and np.all(q[2, :5] == 0)
    assert E.decode(q[3, 0]) * d[3, 0] == pytest.approx(1e-33, rel=0.07)


# ---------------------------------------------------------------- C refusals

def test_quantize_refusals(lib):
    f = lib.quantize_act_e4m3
    good = [at(0), F32, 3, 144, at(1), at(2), None]
    for i, v, want in [(1, 2, UNSUPPORTED), (1, -1, UNSUPPORTED), (2, -1, SHAPE), (2, 1 << 40, SHAPE), (3, 0, SHAPE),
                       (3, 24, SHAPE), (3, (1 << 20) + 16, SHAPE), (0, None, NULL), (4, None, NULL), (5, None, NULL),
                       (0, at(0, 8), ALIGN), (4, at(1, 8), ALIGN), (5, at(2, 2), ALIGN), (4, at(0, 16), SHAPE),
                       (5, at(0, 3 * 144 * 4 - 4), SHAPE), (5, at(1, 16), SHAPE)]:
        a = list(good)
        a[i] = v
        assert f(*a) == want, (i, v)
    assert f(None, BF16, 0, 16, None, None, None) == OK


def test_norm_refusals(lib):
    f = lib.rmsnorm_add_quantize_e4m3
    good = [at(0), at(1), at(2), BF16, 3, 144, EPS, at(3), at(4), at(5), None]
    for i, v, want in [(3, 7, UNSUPPORTED), (4, -1, SHAPE), (4, 1 << 31, SHAPE), (5, 136, SHAPE), (5, 65552, SHAPE),
                       (6, ctypes.c_float(-1.0), SHAPE), (6, ctypes.c_float(float("nan")), SHAPE), (0, None, NULL),
                       (2, None, NULL), (7, None, NULL), (8, None, NULL), (9, None, NULL), (0, at(0, 2), ALIGN),
                       (1, at(1, 8), ALIGN), (2, at(2, 4), ALIGN), (7, at(3, 8), ALIGN), (8, at(4, 1), ALIGN),
                       (9, at(5, 2), ALIGN), (7, at(0, 16), SHAPE), (7, at(1, 32), SHAPE), (7, at(2), SHAPE),
                       (8, at(0), SHAPE), (9, at(4, 16), SHAPE), (8, at(3, 16), SHAPE)]:
        a = list(good)
        a[i] = v
        assert f(*a) == want, (i, v)
    assert f(None, None, None, F32, 0, 16, EPS, None, None, None, None) == OK


def test_product_refusals(lib):
    f = lib.qgemm_e4m3
    good = [at(0), at(1), 300, 144, at(2), at(3), 5, 2, at(4), at(5), F32, None]
    for i, v, want in [(10, 2, UNSUPPORTED), (7, 1, UNSUPPORTED), (7, 9, UNSUPPORTED), (3, 0, SHAPE), (3, 8, SHAPE),
                       (3, (1 << 20) + 16, SHAPE), (6, -1, SHAPE), (6, (1 << 24) + 1, SHAPE), (2, -1, SHAPE),
                       (2, 1 << 31, SHAPE), (0, None, NULL), (1, None, NULL), (4, None, NULL), (5, None, NULL),
                       (8, None, NULL), (9, None, NULL), (0, at(0, 8), ALIGN), (1, at(1, 2), ALIGN),
                       (4, at(2, 8), ALIGN), (5, at(3, 1), ALIGN), (8, at(4, 8), ALIGN), (9, at(5, 4), ALIGN),
                       (9, at(0), SHAPE), (9, at(1), SHAPE), (9, at(2), SHAPE), (9, at(3), SHAPE),
                       (9, at(4, 16), SHAPE)]:
        a = list(good)
        a[i] = v
        assert f(*a) == want, (i, v)
    assert f(None, None, 0, 16, None, None, 4, 0, None, None, F32, None) == OK
    assert f(None, None, 4, 16, None, None, 0, 0, None, None, F32, None) == OK


def test_up_refusals(lib):
    f = lib.qg_ffn_up_e4m3
    good = [at(0), at(1), 144, 256, at(2), at(3), 5, at(4), at(5), None]
    for i, v, want in [(2, 24, SHAPE), (2, -16, SHAPE), (2, 1 << 30, SHAPE), (3, 8, SHAPE), (6, -1, SHAPE),
                       (6, (1 << 24) + 1, SHAPE), (0, None, NULL), (1, None, NULL), (4, None, NULL), (5, None, NULL),
                       (7, None, NULL), (8, None, NULL), (0, at(0, 4), ALIGN), (1, at(1, 2), ALIGN),
                       (4, at(2, 8), ALIGN), (7, at(4, 8), ALIGN), (8, at(5, 2), ALIGN), (7, at(2), SHAPE),
                       (8, at(3), SHAPE), (8, at(4, 16), SHAPE), (7, at(0, 2 * 144 * 256 - 16), SHAPE)]:
        a = list(good)
        a[i] = v
        assert f(*a) == want, (i, v)
    assert f(None, None, 0, 16, None, None, 4, None, None, None) == OK
    assert f(None, None, 16, 16, None, None, 0, None, None, None) == OK


def test_ffn_refusals(lib):
    f = lib.qg_ffn_e4m3
    good = [at(0), at(1), at(2), F32, 5, 256, 144, EPS] + [at(i) for i in range(3, 12)] + [None]
    y = 16
    for i, v, want in [(3, 3, UNSUPPORTED), (4, -1, SHAPE), (5, 24, SHAPE), (5, 65552, SHAPE), (6, 8, SHAPE),
                       (6, (1 << 20) + 16, SHAPE), (7, ctypes.c_float(-1.0), SHAPE), (0, None, NULL), (2, None, NULL),
                       (8, None, NULL), (11, None, NULL), (12, None, NULL), (15, None, NULL), (y, None, NULL),
                       (12, at(7, 8), ALIGN), (y, at(11, 8), ALIGN), (y, at(0, 16), SHAPE), (y, at(7), SHAPE),
                       (14, at(7, 16), SHAPE), (12, at(3), SHAPE)]:
        a = list(good)
        a[i] = v
        assert f(*a) == want, (i, v)
    assert f(None, None, None, F32, 0, 16, 16, EPS, *([None] * 10)) == OK


def test_stalled_refusals(lib):
    f = lib.qg_debug_stalled_e4m3
    good = [at(0), at(1), 144, 256, at(2), at(3), 9, at(4), at(5), 0, 0, None]
    for i, v, want in [(2, 0, SHAPE), (2, 24, SHAPE), (2, 1 << 30, SHAPE), (3, 24, SHAPE), (6, 8, SHAPE),
                       (6, (1 << 24) + 1, SHAPE), (9, -1, SHAPE), (10, -1, SHAPE), (0, None, NULL), (1, None, NULL),
                       (4, None, NULL), (5, None, NULL), (7, None, NULL), (0, at(0, 8), ALIGN), (7, at(4, 8), ALIGN),
                       (8, at(5, 2), ALIGN), (7, at(2), SHAPE), (8, at(3), SHAPE), (8, at(4, 16), SHAPE),
                       (7, at(0, 2 * 144 * 256 - 16), SHAPE)]:
        a = list(good)
        a[i] = v
        assert f(*a) == want, (i, v)
    assert f(*good[:7], at(0, 144 * 256 - 16), None, *good[9:]) == SHAPE  # a product's f32 y over its weight


# ---------------------------------------------------------------- binding refusals

def test_binding_refuses_cpu_tensors(lib):
    torch = pytest.importorskip("torch")
    import block_quantized_decode_rmsnorm_gb300 as qg

    x = torch.zeros(2, 128)
    q, d = torch.zeros(2, 128, dtype=torch.float8_e4m3fn), torch.zeros(2, 1)
    w = qg.E4M3Weight(torch.zeros(256, 128, dtype=torch.float8_e4m3fn), torch.zeros(2, 1))
    layer = qg.E4M3Layer(torch.zeros(128), w, w)
    for call in (lambda: qg.quantize_act_e4m3(x), lambda: qg.rmsnorm_add_quantize_e4m3(x, x[0]),
                 lambda: qg.qgemm_e4m3(w, q, d), lambda: qg.qg_ffn_up_e4m3(w, q, d), lambda: qg.qg_ffn_e4m3(x, layer)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        qg.quantize_act_e4m3(np.zeros((2, 128), np.float32))


def need_front():
    from block_quantized_decode_rmsnorm_gb300 import builder

    if builder._torch_dir() is None:
        pytest.skip("torch with CUDA is not installed")


def test_binding_calls_the_library_that_was_loaded(lib, tmp_path):
    """_lib.load(path) decides for the e4m3 calls on torch tensors too."""
    import shutil
    import subprocess
    import sys

    need_front()
    from block_quantized_decode_rmsnorm_gb300 import _lib

    other = str(tmp_path / "other.so")
    shutil.copy(_lib.LIB_PATH, other)
    code = f"""
import torch
from block_quantized_decode_rmsnorm_gb300 import _lib, api
_lib.load({other!r})
front = api._load_front()
maps = open('/proc/self/maps').read()
assert {other!r} in maps and {_lib.LIB_PATH!r} not in maps
try:
    front.bind(_lib.QGError, 0, 0, 0, 0, 0, 0)
except ValueError:
    pass
else:
    raise AssertionError('a missing entry point was taken')
try:
    api.quantize_act_e4m3(torch.zeros(2, 128))
except ValueError as e:
    assert 'CUDA' in str(e)
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_binding_refuses_before_a_library_is_bound():
    import subprocess
    import sys

    need_front()
    code = """
import torch
from block_quantized_decode_rmsnorm_gb300 import _qg_torch
try:
    _qg_torch.quantize_act(torch.zeros(2, 128), None, None)
except RuntimeError as e:
    assert 'bound' in str(e)
else:
    raise AssertionError
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
