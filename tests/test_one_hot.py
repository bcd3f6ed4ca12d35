"""The histories of tests/one_hot.py show what they are for: a token left out of a row or counted twice lies outside
the bound that the GPU tests hold the row to, at every length that they use (no GPU needed)."""
import numpy as np
import pytest

from tests import one_hot as H
from tests import window_ref as R


def smallest_slip(L, Hq, Hkv, D, chain, part, out_step, first=0):
    """Over tokens first .. L - 1: how far a row moves when the token is left out or counted twice, in units of its
    bound in that channel; the smallest of the largest over the heads of a group."""
    rng = np.random.default_rng(L)
    q = H.queries(1, Hq, D, rng)[0].astype(np.float64)
    t = np.arange(first, L)
    worst = np.inf
    for g in range(Hkv):
        k, v = rng.uniform(-1, 1, len(t)), rng.uniform(0.9, 1.1, len(t))
        at = (t + 5 * g) % D
        for sign in (-1, 1):
            slip = np.zeros(len(t))
            for h in range(g * (Hq // Hkv), (g + 1) * (Hq // Hkv)):
                w = np.exp(q[h, (7 * t + g) % D] * k)
                total, row = w.sum(), np.bincount(at, w * v, D)
                far = H.bound(row / total, chain, part, out_step, 2.0 ** -32 * 1.1 * (L / D + 1))
                moved = np.abs((row[at] + sign * w * v) / (total + sign * w) - row[at] / total)
                slip = np.maximum(slip, moved / far[at])
            worst = min(worst, slip.min())
    return worst


@pytest.mark.parametrize("lens,Hq,Hkv,D,B,dt,ps", H.PARTITIONS)
def test_partitions(lens, Hq, Hkv, D, B, dt, ps):
    for L in set(x for x in lens if x):
        assert smallest_slip(L, Hq, Hkv, D, H.partition_chain(max(lens), ps), 2.0 ** -22, 2.0 ** -24) > 1.2


@pytest.mark.parametrize("bits,S,L,window", H.WINDOWS)
def test_windows(bits, S, L, window):
    assert smallest_slip(window, 4, 1, 128, window + 20, 2.0 ** -22 if bits == 4 else 2.0 ** -17, 2.0 ** -24) > 1.2


@pytest.mark.parametrize("new,past,Hq,Hkv,D", H.PROMPTS)
@pytest.mark.parametrize("dt,out", H.PROMPT_TYPES)
def test_prompts(new, past, Hq, Hkv, D, dt, out):
    L = max(n + p for n, p in zip(new, past))
    step = 2.0 ** -24 if out else 2.0 ** -11
    assert smallest_slip(L, Hq, Hkv, D, L, H.prompt_part(dt, out), step) > 1.2


def test_the_rows_are_as_they_are_counted_here():
    """The closed form above against the plain statement on the histories themselves."""
    rng = np.random.default_rng(0)
    L, Hq, Hkv, D, B = 300, 4, 2, 64, 16
    k, v = H.histories([L], np.arange(20)[None], 20, B, Hkv, D, rng)
    q = H.queries(1, Hq, D, rng)[0]
    k, v = (x.reshape(-1, Hkv, D)[:L].astype(np.float64) for x in (k, v))
    out = H.attend(q, k, v, 1.0, R.visible(L - 1, L, 0, 0))
    for h in range(Hq):
        g, t = h // 2, np.arange(L)
        w = np.exp(q[h, (7 * t + g) % D] * k[t, g, (7 * t + g) % D])
        want = np.bincount((t + 5 * g) % D, w * v[t, g, (t + 5 * g) % D], D) / w.sum()
        assert np.allclose(out[h], want, rtol=1e-12, atol=0)
