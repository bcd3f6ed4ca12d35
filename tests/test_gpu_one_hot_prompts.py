"""Prompt attention on histories where each token's weight shows in the output at its full size."""
import numpy as np
import pytest
import torch

import paged_kv_cache_112_gb300 as pkv
from tests import one_hot as H
from tests import window_ref as R
from tests.test_gpu_prefill import STEP, Prompt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load(build_if_missing=True)


class OneHot(Prompt):
    def __init__(self, new, past=None, Hq=8, Hkv=2, D=128, B=16, dt="bf16", seed=0, out=None):
        super().__init__(new, past, Hq, Hkv, D, B, dt, seed, out)
        rng = np.random.default_rng(seed + 1)
        for i, x in enumerate(H.histories(self.lens, self.tables, self.NB, B, Hkv, D, rng)):
            x = torch.from_numpy(x).to(self.dt)
            self.vals[i], self.dev[i] = x.double().numpy(), x.cuda()
        rows = torch.from_numpy(H.queries(len(self.out), Hq, D, rng)).to(self.dt)
        self.q = rows.cuda()
        self.scale = 1.0
        # Weights in f16 are off by half of its smallest step, times 2^7, too.
        self.part = H.prompt_part(dt, "f32" if out == torch.float32 else None)
        self.floor = 2.0 ** -32 if dt == "f16" else 0.0

    def compare(self, window=0, sinks=0, rows=None):
        torch.cuda.synchronize()
        assert int(self.st.item()) == 0
        got, q = self.out.double().cpu().numpy(), self.q.double().cpu().numpy()
        assert np.all(got[self.start[-1]:] == 77)
        rng = np.random.default_rng(1)
        for i, (L, n) in enumerate(zip(self.lens, self.new)):
            blocks = self.tables[i, :-(-L // self.B)]
            k, v = (x[blocks].reshape(-1, self.Hkv, self.D)[:L] for x in self.vals)
            which = range(n) if rows is None or n <= rows else sorted({0, n - 1, *rng.integers(0, n, rows)})
            for r in which:
                at = self.start[i] + r
                want = H.attend(q[at], k, v, 1.0, R.visible(L - n + r, L, window, sinks))
                far = H.bound(want, L, self.part, STEP[self.out.dtype], self.floor * 1.1 * (L / self.D + 1))
                assert np.all(np.abs(got[at] - want) <= far), (i, r, np.nanmax(np.abs(got[at] - want) / far))


@pytest.mark.parametrize("Hq,Hkv,D,B", [(8, 2, 128, 16), (3, 3, 64, 8), (16, 2, 64, 32), (5, 1, 128, 64)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 7)])
def test_float32_outputs_keep_the_weights_bits(Hq, Hkv, D, B, dt, window, sinks):
    """One 16-bit part a weight would be off by up to 2^-8 and 2^-11; on whole grids and over clusters."""
    p = OneHot([1, 70, 0, 129, 5], [300, 0, 50, 257, 127], Hq, Hkv, D, B, dt, seed=D + Hq, out=torch.float32)
    p.call(window, sinks)
    p.compare(window, sinks, rows=12)
    p = OneHot([500], [900], 16 * Hq, 16 * Hkv, D, B, dt, seed=Hq, out=torch.float32)
    p.call(window, sinks)
    p.compare(window, sinks, rows=6)


@pytest.mark.parametrize("new,past,Hq,Hkv,D", H.PROMPTS)
@pytest.mark.parametrize("dt,out", H.PROMPT_TYPES)
def test_long_histories(new, past, Hq, Hkv, D, dt, out):
    """Over clusters of two to eight CTAs and on whole grids."""
    p = OneHot(new, past, Hq, Hkv, D, dt=dt, seed=sum(new), out=torch.float32 if out else None)
    p.call()
    p.compare(rows=8)
