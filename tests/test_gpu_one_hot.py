"""Attention over 4-bit pools on histories where each token's weight shows in the output at its full size."""
import numpy as np
import pytest
import torch

import paged_kv_cache_112_gb300 as pkv
from tests import one_hot as H
from tests import window_ref as R
from tests.test_gpu_fp4 import DT, STEP, Decode

pytestmark = pytest.mark.gpu
PART = {4: 2.0 ** -22, 16: 2.0 ** -17}  # two f16 parts; at the least two bf16 parts


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load(build_if_missing=True)


class OneHot(Decode):
    """A batch of such histories; `chain`: tokens that one accumulator takes up at the most."""

    def __init__(self, lens, Hq=8, Hkv=2, D=128, B=16, dt="bf16", bits=4, seed=0, out=torch.float32):
        super().__init__(lens, Hq, Hkv, D, B, dt, bits, seed=seed, out=out)
        rng = np.random.default_rng(seed + 1)
        self.seen = {}  # sequences whose tokens are not all visible
        for i, x in enumerate(H.histories(lens, self.tables, self.NB, B, Hkv, D, rng)):
            if bits == 4:
                code, sc = R.quantise(x)
                p = R.pack(code.transpose(0, 2, 1, 3), sc.transpose(0, 2, 1, 3))
                self.vals[i], self.dev[i] = R.values(p, D), torch.from_numpy(p).cuda()
            else:
                x = torch.from_numpy(x).to(DT[dt])
                self.vals[i], self.dev[i] = x.double().numpy(), x.cuda()
        self.q = torch.from_numpy(H.queries(len(lens), Hq, D, rng)).to(DT[dt]).cuda()
        self.scale = 1.0

    def rows(self, i, L):
        return [x[self.tables[i, :-(-L // self.B)]].reshape(-1, *x.shape[2:])[:L] for x in self.vals]

    def compare(self, chain, window=0, sinks=0, lens=None, want_status=0):
        torch.cuda.synchronize()
        assert int(self.st.item()) == want_status
        got, q = self.out.double().cpu().numpy(), self.q.double().cpu().numpy()
        for i, L in enumerate(self.lens if lens is None else lens):
            see = R.visible(L - 1, L, window, sinks) & self.seen.get(i, np.ones(L, bool))
            want = H.attend(q[i], *self.rows(i, L), 1.0, see)
            far = H.bound(want, min(chain, L), PART[self.bits], STEP[self.out.dtype],
                          2.0 ** -33 * 1.1 * (L / self.D + 1))
            assert np.all(np.abs(got[i] - want) <= far), (i, L, np.nanmax(np.abs(got[i] - want) / far))


@pytest.mark.parametrize("Hq,Hkv,D,B", [(2, 2, 128, 16), (6, 2, 64, 32), (8, 2, 128, 64), (4, 1, 64, 16), (5, 1, 128, 16),
                                        (14, 2, 64, 16), (8, 1, 128, 32)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_weights_keep_their_bits(Hq, Hkv, D, B, dt):
    """Weights in f16 alone would be off by up to 2^-11; whole histories, and a window with first tokens."""
    d = OneHot([0, 1, 5, 40, 300, 1000], Hq, Hkv, D, B, dt, seed=D + Hq)
    d.attend()
    d.compare(1000)
    d.window(100, 20)
    d.compare(120, 100, 20)
