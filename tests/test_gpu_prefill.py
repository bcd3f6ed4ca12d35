"""Prompt attention on the GPU against float64."""
import numpy as np
import pytest
import torch

import paged_kv_cache_112_gb300 as pkv
from tests import window_ref as R

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load(build_if_missing=True)


class Prompt:
    """New tokens `new` behind `past` of each sequence; scattered blocks, rows of a wider projection."""

    def __init__(self, new, past=None, Hq=8, Hkv=2, D=128, B=16, dt="bf16", seed=0, out=None, loud=1.0, behind=3):
        rng = np.random.default_rng(seed)
        self.new = np.asarray(new)
        self.lens = self.new + np.asarray(past if past is not None else [0] * len(new))
        self.Hq, self.Hkv, self.D, self.B, self.dt = Hq, Hkv, D, B, DT[dt]
        n = -(-self.lens // B)
        self.NB = int(n.sum()) + 2
        perm = rng.permutation(self.NB)
        self.tables, at = np.full((len(new), max(1, int(n.max()))), -9, np.int32), 0
        for i, m in enumerate(n):
            self.tables[i, :m] = perm[at:at + m]
            at += m
        pools = [torch.from_numpy(rng.normal(size=(self.NB, B, Hkv, D))).to(self.dt) for _ in range(2)]
        self.vals = [p.double().numpy() for p in pools]
        self.dev = [p.cuda() for p in pools]
        T = int(self.new.sum())
        rows = torch.from_numpy(rng.normal(size=(T + behind, Hq + 2, D)) * loud).to(self.dt).cuda()
        self.q = rows[:, :Hq] if T + behind > 1 else rows[:, :Hq].contiguous()
        self.start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.out = torch.full((T + behind, Hq, D), 77.0, dtype=self.dt if out is None else out, device="cuda")
        self.st, self.scale = torch.zeros(1, dtype=torch.int32, device="cuda"), D ** -0.5
        self.d_tables, self.d_lens, self.d_start = (torch.from_numpy(x.astype(np.int32)).cuda() for x in (
            self.tables, self.lens, self.start))
        self.max_len = max(1, int(self.lens.max()))

    def poison(self, window=0, sinks=0):
        """What no new token sees becomes NaN and infinite, entries of blocks without a visible token no blocks."""
        for i, (L, n) in enumerate(zip(self.lens, self.new)):
            wide = -(-L // self.B) * self.B
            see = np.zeros(wide, bool)
            if n:
                low = max(0, L - n - window + 1) if window else 0
                t = np.arange(wide)
                see = (t < L) & ((t >= low) | (t < (sinks if window else 0)))
            for t in np.nonzero(~see)[0]:
                for p in self.dev:
                    p[self.tables[i, t // self.B], t % self.B] = float("nan") if t % 3 else float("inf")
            dead = ~see.reshape(-1, self.B).any(1) if wide else np.zeros(0, bool)
            self.d_tables[i, :len(dead)][torch.from_numpy(dead).cuda()] = 2 ** 31 - 1

    def call(self, window=0, sinks=0, **kw):
        pkv.prefill_attention(self.out, self.q, *self.dev, self.d_tables, self.d_lens, self.d_start, self.scale,
                              window=window, sinks=sinks, max_context_len=kw.pop("max_len", self.max_len),
                              status=self.st, **kw)

    def check(self, window=0, sinks=0, want_status=0, rows=None):
        torch.cuda.synchronize()
        assert int(self.st.item()) == want_status
        got, q = self.out.double().cpu().numpy(), self.q.double().cpu().numpy()
        assert np.all(got[self.start[-1]:] == 77)
        rng = np.random.default_rng(1)
        for i, (L, n) in enumerate(zip(self.lens, self.new)):
            blocks = self.tables[i, :-(-L // self.B)]
            k, v = (x[blocks].reshape(-1, self.Hkv, self.D)[:L] for x in self.vals)
            which = range(n) if rows is None or n <= rows else sorted({0, n - 1, *rng.integers(0, n, rows)})
            for r in which:
                at = self.start[i] + r
                want, extra = R.attend(q[at], k, v, self.scale, R.visible(L - n + r, L, window, sinks))
                far = R.bound(want, extra, self.D, L, STEP[self.dt], STEP[self.out.dtype], 2.0 ** -32)
                assert np.all(np.abs(got[at] - want) <= far), (i, r, np.nanmax(np.abs(got[at] - want) / far))


@pytest.mark.parametrize("n", [1, 2, 16, 31, 32, 33, 63, 64, 65, 130, 300])
@pytest.mark.parametrize("D", [64, 128])
def test_one_prompt(n, D):
    p = Prompt([n], D=D, seed=n)
    p.poison()
    p.call()
    p.check()


@pytest.mark.parametrize("Hq,Hkv,D,B", [(8, 2, 128, 16), (3, 3, 64, 8), (16, 2, 64, 32), (5, 1, 128, 64), (7, 1, 128, 16),
                                        (6, 1, 64, 64), (6, 3, 128, 8)])
@pytest.mark.parametrize("dt,out", [("bf16", None), ("f16", torch.float32), ("f16", None), ("bf16", torch.float32)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (40, 3), (128, 0), (200, 150), (100000, 9)])
def test_ragged(Hq, Hkv, D, B, dt, out, window, sinks):
    """Prompts, chunks behind histories, single tokens and idle sequences in one call."""
    p = Prompt([0, 1, 70, 0, 129, 5, 0], [0, 300, 0, 50, 257, 127, 0], Hq, Hkv, D, B, dt, seed=window, out=out)
    p.poison(window, sinks)
    p.call(window, sinks)
    p.check(window, sinks, rows=12)


@pytest.mark.parametrize("n,past", [(1, 5000), (37, 2000), (64, 129), (65, 4000), (200, 900), (7, 20000)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 5)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_few_rows_over_clusters(n, past, window, sinks, dt):
    p = Prompt([n], [past], 4, 1, seed=n, dt=dt)
    p.poison(window, sinks)
    for _ in range(2):
        p.call(window, sinks)
        p.check(window, sinks, rows=20)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,past,Hkv", [([5, 1, 30, 0, 2], [3000, 0, 4, 9, 130], 2), ([65] * 6, [2000] * 6, 3),
                                          ([33, 129, 1], [0, 0, 4000], 8)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (2500, 70)])
def test_uneven_sequences_over_clusters(D, new, past, Hkv, window, sinks):
    """CTAs of a cluster without a tile of a short history, pairs of a single row, more of them than are resident."""
    p = Prompt(new, past, 4 * Hkv, Hkv, D, 32, seed=sum(new))
    p.poison(window, sinks)
    p.call(window, sinks, max_len=4200)
    p.check(window, sinks, rows=12)


@pytest.mark.parametrize("window", [0, 1000])
def test_long_prompt(window):
    p = Prompt([6000, 2100], [100, 0], 8, 2, seed=3)
    p.call(window, 4)
    p.check(window, 4, rows=40)


def test_many_sequences():
    """More sequences than a CTA has threads."""
    rng = np.random.default_rng(0)
    p = Prompt(rng.integers(0, 40, 700), rng.integers(0, 60, 700), 4, 2, 64, seed=8)
    p.call()
    p.check(rows=2)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 4.0])
def test_scales_and_growing_maxima(scale):
    """Scores that grow along the history by far more than the lazy reference allows, of either sign; none at all."""
    p = Prompt([150], [800], 4, 1, seed=6, loud=3.0)
    ramp = torch.linspace(0.05, 3.0, p.NB * 16).view(p.NB, 16, 1, 1)
    order = torch.from_numpy(p.tables[0].astype(np.int64))
    k = p.dev[0].cpu()
    k[order] = (k[order].double() * ramp[: len(order)].double()).to(p.dt)
    p.dev[0].copy_(k)
    p.vals[0] = k.double().numpy()
    p.scale = scale
    p.call()
    p.check()


def test_layers_view_and_other_streams():
    p = Prompt([90, 20], [30, 400], seed=4)
    whole = [torch.zeros(p.NB, 3, *x.shape[1:], dtype=p.dt, device="cuda") for x in p.dev]
    for w, x in zip(whole, p.dev):
        w[:, 1] = x
    p.dev = [w[:, 1] for w in whole]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    p.call(stream=side)
    other = Prompt([300], seed=5)
    other.call()
    p.check()
    other.check(rows=30)


def test_graph_replay_with_other_lengths():
    p = Prompt([40, 100, 3], [10, 0, 500], seed=9)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        p.call(max_len=512)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        p.call(max_len=512)
    for new, lens in (([40, 100, 3], [50, 100, 503]), ([1, 0, 142], [20, 90, 500]), ([0, 80, 0], [50, 80, 503])):
        p.new, p.lens = np.array(new), np.array(lens)
        p.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        p.d_start.copy_(torch.from_numpy(p.start)), p.d_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        p.out.fill_(77)
        g.replay()
        p.check(rows=20)


@pytest.mark.parametrize("past,Hkv", [(0, 20), (3000, 1)])
@pytest.mark.parametrize("out", [None, torch.float32])
def test_what_is_no_number_stays_so(past, Hkv, out):
    """A NaN query, and a NaN or infinite key: the rows that meet them are no numbers, the others are as ever (on
    whole grids and over clusters)."""
    n, G = 200, 4
    p = Prompt([n], [past], G * Hkv, Hkv, seed=41, out=out)
    p.q[50, 1] = float("nan")
    at = past + 120
    blk, off = p.tables[0, at // p.B], at % p.B
    p.dev[0][blk, off, 0] = float("nan")
    p.call()
    torch.cuda.synchronize()
    assert int(p.st.item()) == 0
    bad = torch.isnan(p.out[:n]).all(-1).cpu()
    want = torch.zeros(n, G * Hkv, dtype=torch.bool)
    want[50, 1] = True
    want[120:, :G] = True
    assert torch.equal(bad, want) and torch.equal(torch.isnan(p.out[:n]).any(-1).cpu(), want)
    got, q = p.out.double().cpu().numpy(), p.q.double().cpu().numpy()
    k, v = (x[p.tables[0]].reshape(-1, Hkv, p.D)[:n + past] for x in p.vals)
    for r in (0, 49, 51, 119, n - 1):
        ok = ~want[r].numpy()
        ref, extra = R.attend(q[r], np.nan_to_num(k), v, p.scale, R.visible(past + r, n + past, 0, 0))
        far = R.bound(ref, extra, p.D, n + past, STEP[p.dt], STEP[p.out.dtype], 2.0 ** -32)
        assert np.all(np.abs(got[r] - ref)[ok] <= far[ok])


def test_two_streams_and_graphs_of_whole_grids():
    """Calls that fill the device, of both head sizes, side by side on two streams, eagerly and from two graphs, with
    an output that is 16-byte aligned alone."""
    a, b = Prompt([3000, 2500], [0, 400], 8, 2, seed=21), Prompt([4000, 700, 60], [5, 0, 300], 8, 2, 64, dt="f16", seed=22)
    flat = torch.full((a.out.numel() + 8,), 77.0, dtype=a.dt, device="cuda")
    a.out = flat[8:].view(a.out.shape)
    assert a.out.data_ptr() % 32 == 16
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for p, st in zip((a, b), streams):
            p.call(stream=st)
    for p in (a, b):
        p.check(rows=20)
        p.out.fill_(77)
    graphs = []
    for p, st, w in zip((a, b), streams, (0, 600)):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(2):
                p.call(w, 3)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    a.check(0, 0, rows=20)
    b.check(600, 3, rows=20)


def test_pools_past_four_gigabytes():
    """Blocks whose bytes lie past 2^32, for prompts and windowed decode."""
    H, D, B, n = 8, 128, 16, 300
    NB = (1 << 32) // (B * H * D * 2) + 40
    pools = [torch.zeros(NB, B, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    p = Prompt([n], Hq=8, Hkv=8, seed=31)
    far = torch.arange(NB - 1, NB - 1 - p.tables.shape[1], -1, dtype=torch.int32)
    for whole, small in zip(pools, p.dev):
        whole[far.cuda().long()] = small[torch.from_numpy(p.tables[0]).cuda().long()]
    p.dev, p.d_tables = pools, far[None].cuda()
    p.call()
    p.check(rows=20)
    one = torch.zeros(1, 8, D, device="cuda")
    pkv.decode_window(one, p.q[n - 1:n].contiguous(), *pools, p.d_tables, p.d_lens, p.scale, window=100, sinks=2,
                      max_context_len=n, status=p.st)
    k, v = (x[p.tables[0]].reshape(-1, H, D)[:n] for x in p.vals)
    want, extra = R.attend(p.q[n - 1].double().cpu().numpy(), k, v, p.scale, R.visible(n - 1, n, 100, 2))
    assert np.all(np.abs(one[0].double().cpu().numpy() - want) <= R.bound(want, extra, D, n, 2.0 ** -16, 2.0 ** -24))


def test_flags():
    p = Prompt([40, 30], [0, 10], seed=2)
    p.d_tables[1, 1] = p.NB
    p.vals = [v.copy() for v in p.vals]
    spare = int(p.tables[1, 1])
    p.vals[0][spare] = p.vals[1][spare] = 0.0  # the block outside the pool counts as zeros
    p.call()
    p.check(want_status=pkv.DEV_ERR_BLOCK)
    # more new tokens than the sequence has: those before its start see nothing
    p = Prompt([40, 30], [0, 10], seed=2)
    p.d_lens[0] = 25
    p.lens[0] = 25
    p.call()
    p.check(want_status=pkv.DEV_ERR_LENGTH)
    assert torch.all(p.out[:15] == 0)
    # a length beyond the caller's bound is cut, a negative one is none
    p = Prompt([40, 30], [100, 10], seed=2)
    p.call(max_len=128)
    p.lens[0] = 128
    p.check(want_status=pkv.DEV_ERR_LENGTH)
    p = Prompt([40, 30], seed=2)
    p.d_lens[1] = -4
    p.call()
    p.lens[1] = 0
    p.check(want_status=pkv.DEV_ERR_LENGTH)
    # a descent that leaves a sequence without rows: alone, behind many others, and of no rows at all
    for start in ([0, 5, 3, 8], [0] * 40 + [4, 3] + [8] * 40, [8, 8, 2], [-3, 0, 8], [20, 20, 20]):
        S = len(start) - 1
        p = Prompt([4] * S, seed=2)
        p.q, p.out = p.q[:8], p.out[:8]
        p.d_start = torch.tensor(start, dtype=torch.int32, device="cuda")
        p.d_lens[:] = 16
        p.call(max_len=16)
        torch.cuda.synchronize()
        assert int(p.st.item()) == pkv.DEV_ERR_LENGTH, start
    # starts that descend or lie outside
    p = Prompt([40, 30], [0, 10], seed=2)
    p.d_start[2] = 1000
    p.call()
    torch.cuda.synchronize()
    assert int(p.st.item()) == pkv.DEV_ERR_LENGTH


def test_prompt_then_decode_agree():
    """A prompt in two chunks, then single tokens: the last rows are what decode gives, windowed and not."""
    rng = np.random.default_rng(3)
    H, Hq, D, B, NB, n = 2, 8, 128, 16, 30, 200
    kp, vp = (torch.zeros(NB, B, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bm = pkv.BlockManager(NB, B)
    _, slots = bm.add_sequence(0, rng.integers(0, 100, n))
    qkv = torch.from_numpy(rng.normal(size=(n, Hq + 2 * H, D))).bfloat16().cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    qo, out = (torch.zeros(n, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.from_numpy(bm.block_table(0))[None].cuda()
    inv = 10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)
    ang = torch.arange(256, dtype=torch.float64)[:, None] * inv
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    pkv.norm_rope_write(q, k, v, kp, vp, torch.from_numpy(slots).cuda(), q_out=qo, cos_sin=cs,
                        positions=torch.arange(n, dtype=torch.int32, device="cuda"), status=st)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    for window, sinks in ((0, 0), (50, 4)):
        for a, b in ((0, 130), (130, n)):
            pkv.prefill_attention(out[a:b], qo[a:b], kp, vp, table, i32(b), i32(0, b - a), D ** -0.5, window=window,
                                  sinks=sinks, max_context_len=n, status=st)
        for last in (1, 17, 129, 130, 131, n):
            one, ref = out[last - 1:last], torch.zeros(1, Hq, D, device="cuda")
            if window:
                pkv.decode_window(ref, qo[last - 1:last].contiguous(), kp, vp, table, i32(last), D ** -0.5,
                                  window=window, sinks=sinks, max_context_len=n, status=st)
            else:
                pkv.decode_attention(ref, qo[last - 1:last].contiguous(), kp, vp, table, i32(last), D ** -0.5,
                                     max_context_len=n, status=st)
            mass = vp.float().abs().max()
            assert float((one.float() - ref).abs().max()) <= float(mass) * 3 * 2.0 ** -8
    assert int(st.item()) == 0


def test_refusals_of_tensors():
    p = Prompt([40], seed=1)
    call = lambda **kw: pkv.prefill_attention(
        kw.get("out", p.out), kw.get("q", p.q), kw.get("k", p.dev[0]), p.dev[1], kw.get("bt", p.d_tables),
        kw.get("cl", p.d_lens), kw.get("qs", p.d_start), 0.1, window=kw.get("window", 0), max_context_len=40)
    call()
    for bad in (dict(out=p.out[:-1]), dict(q=p.q[:, :, :64]), dict(q=p.q.float()), dict(q=p.q.half()),
                dict(k=p.dev[0].cpu()), dict(bt=p.d_tables.long()), dict(bt=p.d_tables[0]), dict(cl=p.d_lens[:0]),
                dict(qs=p.d_start[:1]), dict(qs=p.d_start.float()), dict(window=-1), dict(q=p.q.transpose(0, 1)),
                dict(out=p.out.transpose(1, 2))):
        with pytest.raises(pkv.PkvError):
            call(**bad)
