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
