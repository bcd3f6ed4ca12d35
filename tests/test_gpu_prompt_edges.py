"""Prompt attention where its arguments and inputs end."""
import numpy as np
import pytest
import torch

import paged_kv_cache_112_gb300 as pkv
from tests import window_ref as R
from tests.test_gpu_prefill import STEP, Prompt

pytestmark = pytest.mark.gpu
LAST = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load(build_if_missing=True)


@pytest.mark.parametrize("Hkv", [2, 40])  # over clusters and on a whole grid
@pytest.mark.parametrize("window,sinks", [(LAST, 0), (LAST, LAST), (LAST - 10, 3), (30, LAST), (1, 0)])
def test_more_new_tokens_than_history_in_the_widest_windows(Hkv, window, sinks):
    """Rows before the history's first token see nothing, the others what they always do: a pair's positions less the
    window need not fit 32 bits."""
    p = Prompt([40, 300, 5], [0, 20, 0], 4 * Hkv, Hkv, seed=17)
    for i, L in enumerate((25, 200, 1)):
        p.d_lens[i] = L
        p.lens[i] = L
    p.call(window, sinks)
    p.check(window, sinks, want_status=pkv.DEV_ERR_LENGTH, rows=40)
    assert torch.all(p.out[:15] == 0) and not torch.all(p.out[15:40] == 0)
