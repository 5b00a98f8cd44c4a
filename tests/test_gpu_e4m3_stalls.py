"""A copy that stalls, in the e4m3 tile kernels: the waits give up, the CTA waits for what
it has issued, its tiles are NaN, every other tile is as it always is, and the calls after it
are.  qg_debug_stalled_e4m3 makes the stall: one CTA holds one block's copies back for longer
than the waits last."""

import numpy as np
import pytest

from oracle import e4m3 as E
from tests._gpu import Guarded, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    return need_gpu()


@pytest.fixture(scope="module")
def qg():
    import block_quantized_decode_rmsnorm_gb300 as m

    return m


def stalled(torch, w, xq, xd, n, out, out_d, cta, block):
    from block_quantized_decode_rmsnorm_gb300 import _lib

    _lib.call("qg_debug_stalled_e4m3", w.codes.data_ptr(), w.scales.data_ptr(), n, w.codes.shape[1], xq.data_ptr(),
              xd.data_ptr(), xq.shape[0], out.data_ptr(), out_d.data_ptr() if out_d is not None else None, cta, block,
              torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()


def operands(torch, qg, seed, m, n, k, halves):
    rng = np.random.default_rng(seed)
    parts = [E.weight(rng, n, k) for _ in range(halves)]
    w = qg.E4M3Weight(torch.from_numpy(np.concatenate([p[0] for p in parts])).cuda().view(torch.float8_e4m3fn),
                      torch.from_numpy(np.concatenate([p[1] for p in parts])).cuda())
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return w, *qg.quantize_act_e4m3(torch.randn((m, k), generator=gen, device="cuda"))


def cells(bad, width):
    """Which cells of 128 rows by `width` columns are bad throughout; each is, or is not at all."""
    m, n = bad.shape
    found = []
    for r in range(0, m, 128):
        for c in range(0, n, width):
            cell = bad[r:r + 128, c:c + width]
            assert cell.all() or not cell.any(), (r, c)
            if cell.all():
                found.append((r, c))
    return found


# clusters sharing k: as many blocks a CTA as stages, more, the first block held back, one in
# the first use of the stages, one in the second; then the walk: in a CTA's first tile and in
# its second, 128, 192 and 256 columns wide
@pytest.mark.parametrize("m,n,k,cta,block,most", [
    (100, 300, 1040, 1, 0, 1), (100, 300, 1040, 0, 3, 1), (40, 144, 9216, 3, 0, 1), (40, 144, 9216, 4, 4, 1),
    (40, 144, 9216, 1, 9, 1), (129, 300, 2560, 2, 1, 1), (2601, 1000, 1168, 5, 2, 4), (5100, 1400, 1168, 3, 13, 4),
    (2601, 1408, 1168, 100, 7, 8), (5100, 1401, 1168, 0, 0, 8)])
def test_product(torch, qg, m, n, k, cta, block, most):
    w, xq, xd = operands(torch, qg, m + n, m, n, k, 1)
    want = qg.qgemm_e4m3(w, xq, xd)
    y = Guarded(torch, (m, n), torch.float32)
    stalled(torch, w, xq, xd, n, y.view, None, cta, block)
    y.check()
    bad = torch.isnan(y.view).cpu().numpy()
    assert 1 <= len(cells(bad, 64)) <= most
    keep = torch.from_numpy(~bad).cuda()
    assert torch.equal(y.view[keep], want[keep])
    assert torch.equal(qg.qgemm_e4m3(w, xq, xd), want)


@pytest.mark.parametrize("m,f,k,cta,block,most", [(40, 272, 2560, 1, 0, 1), (40, 272, 2560, 2, 1, 1), (140, 400, 4112, 3, 5, 1),
                                                  (2500, 1040, 1168, 2, 4, 2), (2500, 1040, 1168, 2, 12, 1)])
def test_gate_up(torch, qg, m, f, k, cta, block, most):
    w, xq, xd = operands(torch, qg, m + f, m, f, k, 2)
    want, want_d = qg.qg_ffn_up_e4m3(w, xq, xd)
    hq, hd = Guarded(torch, (m, f), torch.float8_e4m3fn), Guarded(torch, (m, E.blocks(f)), torch.float32)
    stalled(torch, w, xq, xd, f, hq.view, hd.view, cta, block)
    hq.check(), hd.check()
    got, ref = (t.cpu().view(torch.uint8).numpy() for t in (hq.view, want))
    bad = got & 0x7F == 0x7F
    found = cells(bad, 128)
    assert 1 <= len(found) <= most
    assert np.array_equal(got[~bad], ref[~bad])
    d, ref_d = hd.view.cpu().numpy(), want_d.cpu().numpy()
    for r, c in found:
        assert np.all(d[r:r + 128, c // 128] == np.float32(2.0 ** -100) / np.float32(448))
        d[r:r + 128, c // 128] = ref_d[r:r + 128, c // 128]
    assert np.array_equal(d, ref_d)
    again, again_d = qg.qg_ffn_up_e4m3(w, xq, xd)
    assert torch.equal(again.view(torch.uint8), want.view(torch.uint8)) and torch.equal(again_d, want_d)


def test_nothing_held(torch, qg):
    """A block that no CTA has: the shorter waits alone change nothing."""
    for m in (100, 2601):
        w, xq, xd = operands(torch, qg, m, m, 1000, 1168, 1)
        y = torch.empty((m, 1000), device="cuda")
        stalled(torch, w, xq, xd, 1000, y, None, 0, 1 << 40)
        assert torch.equal(y, qg.qgemm_e4m3(w, xq, xd))
