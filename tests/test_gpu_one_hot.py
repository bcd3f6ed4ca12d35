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
    """A batch of such histories in scattered blocks; what lies behind them is NaN."""

    def __init__(self, lens, Hq=8, Hkv=2, D=128, B=16, dt="bf16", bits=4, seed=0, out=torch.float32):
        super().__init__([0] * len(lens), Hq, Hkv, D, B, dt, bits, seed=seed, out=out)
        rng = np.random.default_rng(seed + 1)
        self.lens = np.asarray(lens)
        n = -(-self.lens // B)
        self.NB, self.width, self.max_len = int(n.sum()) + 3, int(n.max()) + 1, int(self.lens.max())
        self.tables, perm, at = np.full((len(lens), self.width), -7, np.int32), rng.permutation(self.NB), 0
        for i, m in enumerate(n):
            self.tables[i, :m] = perm[at:at + m]
            at += m
        self.dt_tables = torch.from_numpy(self.tables).cuda()
        self.dt_lens = torch.from_numpy(self.lens.astype(np.int32)).cuda()
        self.seen = {}  # sequences whose tokens are not all visible
        for j, x in enumerate(H.histories(lens, self.tables, self.NB, B, Hkv, D, rng)):
            if bits == 4:
                code, sc = R.quantise(x)
                p = R.pack(code.transpose(0, 2, 1, 3), sc.transpose(0, 2, 1, 3))
                self.vals[j], self.dev[j] = R.values(p, D), torch.from_numpy(p).cuda()
            else:
                x = torch.from_numpy(x).to(DT[dt])
                self.vals[j], self.dev[j] = x.double().numpy(), x.cuda()
        for i, L in enumerate(lens):
            if L % B:
                self.poison(i, L)
        self.q = torch.from_numpy(H.queries(len(lens), Hq, D, rng)).to(DT[dt]).cuda()
        self.scale = 1.0

    def in_partitions(self):
        """Whether the last call went through the workspace."""
        torch.cuda.synchronize()
        return bool((self.ws != 0xFF).any())

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


@pytest.mark.parametrize("lens,Hq,Hkv,D,B,dt,ps", H.PARTITIONS)
def test_partitions(lens, Hq, Hkv, D, B, dt, ps):
    """Histories cut into partitions and joined, twice on the same workspace: every group size, block size and type,
    partitions of an odd number of tiles, whose last step of two holds a tile of the next partition."""
    d = OneHot(lens, Hq, Hkv, D, B, dt, seed=ps)
    d.attend(partition_size=ps)
    assert d.in_partitions()
    d.compare(H.partition_chain(max(lens), ps))
    first = d.out.clone()
    d.out.fill_(0)
    d.attend(partition_size=ps)
    assert torch.equal(d.out, first)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
def test_partitions_of_a_layer_with_bad_entries_and_lengths(out):
    """One layer of an all-layer pool in partitions; entries outside the pool are left out, lengths beyond the table are
    cut, negative ones are none."""
    ps = 1008
    d = OneHot([30000, 20000, 500, 100], 8, 2, 128, 32, "f16", seed=3, out=out)
    whole = [torch.full((d.NB, 3, *p.shape[1:]), 0xFF, dtype=torch.uint8, device="cuda") for p in d.dev]
    for w, p in zip(whole, d.dev):
        w[:, 1] = p
    d.dev = [w[:, 1] for w in whole]
    d.attend(partition_size=ps)
    assert d.in_partitions()
    d.compare(H.partition_chain(30000, ps))
    for i, blk in ((0, 0), (0, 31), (0, 32), (0, 937), (1, 300), (2, 15)):  # 31 and 32: where two partitions meet
        d.dt_tables[i, blk] = d.NB if blk % 2 else -1
        see = d.seen.setdefault(i, np.ones(int(d.lens[i]), bool))
        see[blk * 32:blk * 32 + 32] = False
    d.attend(partition_size=ps)
    assert d.in_partitions()
    d.compare(H.partition_chain(30000, ps), want_status=pkv.DEV_ERR_BLOCK)
    d.st.zero_()
    d.dt_lens[1], d.dt_lens[2], d.dt_lens[3] = 2 ** 31 - 1, -1, 0
    d.seen = {0: d.seen[0]}
    d.dt_tables[1] = d.dt_tables[0]  # as long as the table is, with the first one's entries
    d.tables[1] = d.tables[0]
    d.lens[1] = 30000
    d.max_len = 30000
    d.seen[1] = d.seen[0]
    d.attend(partition_size=ps)
    assert d.in_partitions()
    d.compare(H.partition_chain(30000, ps), lens=[30000, 30000, 0, 0], want_status=pkv.DEV_ERR_BLOCK | pkv.DEV_ERR_LENGTH)


@pytest.mark.parametrize("bits,S,L,window", H.WINDOWS)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_windows(bits, S, L, window, dt):
    """From one sequence on clusters of eight to more units than the device holds."""
    d = OneHot([L - 7 * (i % 5) for i in range(S)], 4, 1, bits=bits, dt=dt, seed=S)
    d.window(window, 20)
    d.compare(window + 20, window, 20)


@pytest.mark.parametrize("lens,ps", [([40000, 400], 1024), ([4000, 900], 256)])
@pytest.mark.parametrize("D", [64, 128])
def test_a_nan_value_stays_in_its_channels(lens, ps, D):
    """The scale of 16 channels of V alone is NaN: they are no numbers in the rows that see the token, all else is as
    ever.  In partitions, whole and in a window."""
    Hkv, G = 4, 2
    d = OneHot(lens, G * Hkv, Hkv, D, seed=ps)
    d.attend(partition_size=ps)
    assert d.in_partitions() == (max(lens) > 10000)
    plain = d.out.clone()
    d.window(300, 4)
    window = d.out.clone()
    t, g, group = lens[0] - 50, 2, 1
    d.dev[1][d.tables[0, t // 16], g, 0, 8 * D + t % 16 * (D // 16) + group] = 0x7F
    want = torch.zeros_like(plain, dtype=torch.bool)
    want[0, G * g:G * g + G, 16 * group:16 * group + 16] = True
    for before, call in ((plain, lambda: d.attend(partition_size=ps)), (window, lambda: d.window(300, 4))):
        call()
        assert torch.equal(torch.isnan(d.out), want)
        assert torch.equal(d.out[~want], before[~want])
