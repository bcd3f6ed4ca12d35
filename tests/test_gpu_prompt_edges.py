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


@pytest.mark.parametrize("Hq,Hkv,D,B,dt,out", [(8, 2, 128, 16, "bf16", None), (1, 1, 64, 8, "f16", torch.float32),
                                               (80, 40, 128, 32, "f16", None), (200, 40, 64, 64, "bf16", torch.float32),
                                               (40, 40, 128, 16, "bf16", None)])
@pytest.mark.parametrize("past,window,sinks", [(100, 0, 0), (0, 0, 0), (700, 90, 5), (150, 60, 170), (9, 300, 40)])
def test_values_that_are_no_numbers_reach_the_rows_that_see_them(Hq, Hkv, D, B, dt, out, past, window, sinks):
    """Infinite and NaN values of single channels: the rows that see their tokens are no numbers in those channels, and
    as with zeros there in the others; rows that do not see them are the same to the bit.  Over clusters and on grids of
    more pairs of tiles than are resident."""
    rng = np.random.default_rng(past + window + D)
    new = [300, 1, 130]
    p = Prompt(new, [past, past + 3, past], Hq, Hkv, D, B, dt, seed=past, out=out)
    poked = []  # sequence, token, KV head, channel
    for i, (L, n) in enumerate(zip(p.lens, new)):
        for t in {int(L) - 1, int(L) - n, max(0, int(L) - 1 - n // 2), min(2, int(L) - 1), *rng.integers(0, L, 12)}:
            poked.append((i, int(t), int(rng.integers(Hkv)), int(rng.integers(D))))
    p.q[5, 0] = 0  # a row of equal weights
    at = [(int(p.tables[i, t // B]), t % B, g, c) for i, t, g, c in poked]
    for x in at:
        p.dev[1][x] = 0
    p.call(window, sinks)
    plain = p.out.clone()
    bad = [float("inf"), -float("inf"), float("nan")]
    for m, x in enumerate(at):
        p.dev[1][x] = bad[m % 3]
    p.call(window, sinks)
    torch.cuda.synchronize()
    assert int(p.st.item()) == 0
    want = torch.zeros(p.out.shape, dtype=torch.bool)
    for i, t, g, c in poked:
        for r in range(new[i]):
            pos = int(p.lens[i]) - new[i] + r
            if R.visible(pos, t + 1, window, sinks)[t]:
                want[p.start[i] + r, g * (Hq // Hkv):(g + 1) * (Hq // Hkv), c] = True
    assert want.any() and not want.all()
    assert torch.equal(~torch.isfinite(p.out).cpu(), want)
    assert torch.equal(p.out.cpu()[~want], plain.cpu()[~want])
