"""4-bit pools where values lie next to the borders between codes, and beside values that are no numbers."""
import numpy as np
import pytest
import torch

import paged_kv_cache_112_gb300 as pkv
from tests import window_ref as R
from tests.test_gpu_fp4 import DT, pool, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load(build_if_missing=True)


def head_scale_for(z):
    """A float32 whose reciprocal, rounded to float32, is z: rows of 1 are then z."""
    near = np.float32(1) / np.float32(z)
    for h in (near, *(np.nextafter(near, np.float32(t)) for t in (0, np.inf))):
        if np.float32(1) / h == np.float32(z):
            return h
    return None


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_borders_beside_infinities(dt, D):
    """One float32 step below, on and above each border between codes, in a group whose largest value is infinite
    (its scale is 448) and, for comparison, in one where it is 6 * 448."""
    borders = (R.E2M1[1:8] + R.E2M1[:7]) / 2 * 448
    at = [np.float32(b) for b in borders]
    zs = [z for b in at for z in (np.nextafter(b, np.float32(0)), b, np.nextafter(b, np.float32(np.inf)))]
    found = [(z, head_scale_for(z)) for z in zs]
    found = [(z, h) for z, h in found if h is not None]
    assert len(found) >= 10 and sum(z < b for b in at for z, _ in found if np.nextafter(b, np.float32(0)) == z) >= 3
    H, T, B = len(found), 6, 16
    hs = np.array([h for _, h in found], np.float32)
    x = torch.ones(T, H, D, dtype=DT[dt])
    x[1] = -1
    x[:, :, 1::3] *= 0.5
    x[:3, :, ::16] = float("inf")
    x[2, :, 5::16] = -float("inf")
    # a finite value of 6 * 448 and more in every group, by the head's own scale
    x[3:, :, ::16] = torch.from_numpy(2.0 ** np.ceil(np.log2(6.5 * 448 * hs)))[None, :, None].to(DT[dt])
    kp, vp, st = pool(2, H, B, D), pool(2, H, B, D), status()
    d = torch.from_numpy(hs).cuda()
    pkv.write_cache_fp4(x.cuda(), x.cuda(), kp, vp, d, d, torch.arange(T, dtype=torch.int32, device="cuda"), status=st)
    assert int(st) == 0
    want, want_sc = R.quantise(x.float().numpy(), hs)
    assert np.all(want_sc[:3] == 126)
    for p in (kp, vp):
        code, sc = R.unpack(p.cpu().numpy(), D)
        assert np.array_equal(sc[0, :, :T].transpose(1, 0, 2), want_sc)
        assert np.array_equal(R.E2M1[code[0, :, :T].transpose(1, 0, 2)], R.E2M1[want])
