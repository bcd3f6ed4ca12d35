"""Sparse decode where warps diverge, data is hostile or magnitudes lie far
apart: more of test_gpu_sparse.py, against the same float64 statements."""
import numpy as np
import pytest
import torch

import paged_kv_cache_112_gb300 as pkv
from tests import layer_ref as R
from tests.test_gpu_sparse import Attend, Select, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load(build_if_missing=True)


@pytest.mark.parametrize("lens", [[900], [900, 20, 0], [333] * 18])
@pytest.mark.parametrize("D", [64, 128])
def test_one_head_over_a_cluster(lens, D):
    """A group of one head: the rows that a CTA sends and receives occupy part of a warp, whose lanes are
    together again at the cluster's barriers."""
    a = Attend(lens, Hq=1, Hkv=1, D=D, keep=50, seed=3)
    for _ in range(3):
        a.call()
        a.check()


@pytest.mark.parametrize("keep", [45, 131, 250])
@pytest.mark.parametrize("Hq", [2, 16])
def test_whole_lists_over_a_cluster(keep, Hq):
    """Lists that need no choice, of lengths that end inside a warp, beside one that does, on clusters."""
    s = Select([4000, 600, 16 * keep, 0, 3, 16 * 131], Hq=Hq, Hkv=2, keep=keep, seed=keep)
    for _ in range(3):
        s.call()
        s.check()


@pytest.mark.parametrize("n", [20, 200, 700, 1024, 3000])
@pytest.mark.parametrize("zero_query", [False, True])
def test_scales_that_no_summary_has(n, zero_query):
    """Negative, infinite and NaN scales (memory that no summary was written to) and unusable table entries:
    those blocks come last, the lowest first, whatever their codes and the query -- zeros among them, whose
    product with an infinite scale is no number."""
    keep = n // 2
    s = Select([16 * n], keep=keep, first=1, last=2, seed=n)
    phys = s.tables[0, :n].long()
    rng = np.random.default_rng(n)
    odd = torch.from_numpy(rng.permutation(n)[:3 * n // 4])
    for i, x in enumerate((float("inf"), float("nan"), -1.0, -float("inf"))):
        s.scale[phys[odd[i::4].cuda()]] = x
    s.summary[phys[odd[::2].cuda()]] = 0
    s.tables[0, odd[:n // 10].cuda()] = -3
    if zero_query:
        s.q.zero_()
    usable = torch.isfinite(s.scale) & (s.scale >= 0)
    s.call()
    torch.cuda.synchronize()
    assert int(s.status.item()) == pkv.DEV_ERR_BLOCK
    q, codes, tables = f64(s.q), s.summary.cpu().numpy(), s.tables.cpu().numpy()[0, :n]
    for g in range(s.Hkv):
        at = np.maximum(tables, 0)
        ok = (tables >= 0) & usable[:, g].cpu().numpy()[at]
        unit = np.where(ok, f64(s.scale)[at, g], 0.0)
        sc = R.scores(q[0, 4 * g:4 * g + 4], codes[at, g], unit, 3.3895313892515355e38)
        want = R.select(np.where(ok, sc, -np.inf), n, keep, 1, 2)
        assert s.sel[0, g].tolist() == want and int(s.cnt[0, g]) == keep
