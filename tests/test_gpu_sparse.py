"""Block summaries, block selection and sparse decode against their float64
statements.  Summaries and selections are whole numbers from exact arithmetic
and must be equal; attention is held to layer_ref.attend_bound plus half a
step of the output type."""
import numpy as np
import pytest
import torch

import paged_kv_cache_112_gb300 as pkv
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
MOST = {"bf16": float(torch.finfo(torch.bfloat16).max), "f16": 65504.0, "fp8": 448.0}
SPLIT = {"bf16": 2.0 ** -16, "f16": 2.0 ** -20, "fp8": 2.0 ** -20}  # hi + lo weights


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load(build_if_missing=True)


def f64(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------ summaries


def summarize(pool, ids, k_scale=None, NB=None, Hkv=None, D=None, stream=None):
    NB, _, Hkv, D = pool.shape
    summary = torch.full((NB, Hkv, 2, D), 77, dtype=torch.int8, device="cuda")
    scale = torch.full((NB, Hkv), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids = torch.as_tensor(ids, dtype=torch.int32).cuda()
    if k_scale is not None:
        pkv.summarize_blocks_fp8(summary, scale, pool, k_scale, ids, status=status, stream=stream)
    else:
        pkv.summarize_blocks(summary, scale, pool, ids, status=status, stream=stream)
    torch.cuda.synchronize()
    return summary.cpu().numpy(), scale.cpu().numpy(), int(status.item())


def check_summary(keys64, ids, got, most):
    """keys64 [NB, B, H, D] as float64; rows of blocks not listed stay 77 / 7."""
    summary, scale, _ = got
    for b in range(keys64.shape[0]):
        for g in range(keys64.shape[2]):
            if b in ids:
                codes, unit = R.summarize(keys64[b, :, g], most)
                assert np.array_equal(summary[b, g], codes) and scale[b, g] == unit
            else:
                assert np.all(summary[b, g] == 77) and scale[b, g] == 7.0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hkv,D,B", [(8, 128, 16), (1, 64, 16), (3, 128, 32), (5, 64, 64), (2, 128, 64)])
def test_summaries(dtype, Hkv, D, B):
    g = torch.Generator().manual_seed(B + D)
    pool = torch.randn(13, B, Hkv, D, generator=g)
    pool *= torch.exp(2 * torch.randn(13, 1, Hkv, 1, generator=g))
    pool = pool.to(DT[dtype]).cuda()
    pool[3, :, 0] = 0
    pool[4, :, 0] = -pool[4, :, 0].abs()
    ids = [0, 3, 4, 7, 12, -1, 9]
    got = summarize(pool, ids)
    assert got[2] == 0
    check_summary(f64(pool), ids, got, MOST[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_summaries_at_the_edges(dtype):
    """NaN keys, channels of NaN alone, infinities, subnormals, signed zeros, bounds of exactly 127 steps
    and one above, duplicate and repeated -1 entries."""
    pool = torch.zeros(9, 16, 2, 64, dtype=DT[dtype])
    pool[0] = torch.randn(16, 2, 64).to(DT[dtype])
    pool[0, 3, 0, 5] = pool[0, 7, 1, :] = float("nan")
    pool[0, :, 0, 9] = float("nan")
    pool[1, :, 0] = float("nan")
    pool[2, 4, 0, 3], pool[2, 5, 1, 4] = float("inf"), float("-inf")
    pool[3, 1, 0, 1] = torch.finfo(DT[dtype]).tiny / 64
    pool[3, 1, 1, 1] = -torch.finfo(DT[dtype]).tiny / 64
    pool[4, 1, 0, 1], pool[4, 2, 0, 2], pool[4, 3, 1, 3] = -0.0, 127.0, 127.5
    pool[5, 1, 0, 1], pool[5, 1, 0, 2], pool[5, 2, 1, 0] = MOST[dtype], 6e-5, -127.0 / 64
    pool[6] = 1.0
    pool[7] = -3.0
    pool = pool.cuda()
    ids = [0, 1, 2, 3, 4, 5, 6, 7, 4, -1, -1]
    got = summarize(pool, ids)
    assert got[2] == 0
    check_summary(f64(pool), ids, got, MOST[dtype])


def test_summaries_of_a_layer_view_and_bad_ids():
    pool = torch.randn(6, 3, 16, 2, 128).bfloat16().cuda()
    got = summarize(pool[:, 1], [5, 6, -2, 0])
    assert got[2] == pkv.DEV_ERR_BLOCK
    check_summary(f64(pool[:, 1]), [5, 0], got, MOST["bf16"])
    assert summarize(pool[:, 1], [])[2] == 0


@pytest.mark.parametrize("Hkv,D,layers", [(8, 128, 1), (3, 64, 1), (2, 128, 2)])
def test_summaries_fp8(Hkv, D, layers):
    g = torch.Generator().manual_seed(D)
    whole = torch.randint(0, 256, (11, layers, 16, Hkv, D), generator=g, dtype=torch.uint8).cuda()  # NaN codes too
    sc = torch.exp(3 * torch.randn(11, layers, Hkv, generator=g)).cuda()
    sc[2, :, 0], sc[3, :, 0], sc[4, :, 0], sc[5, :, 0] = 0.0, -1.0, float("nan"), float("inf")
    sc[6, :, 0], sc[7, :, 0], sc[8, :, 0] = 2.0 ** -140, 3e38, 127.0 / 448
    whole[9, :, :, 0] = 0x7F
    pool, scale = whole[:, layers - 1], sc[:, layers - 1]
    got = summarize(pool, list(range(11)), scale)
    assert got[2] == 0
    s64 = f64(scale)
    s64[~((s64 > 0) & np.isfinite(s64))] = 0.0
    keys = R.E4M3[pool.cpu().numpy()] * s64[:, None, :, None]
    # products above float32 are cut at its largest value
    check_summary(keys, range(11), got, 3.4028234663852886e38)


# ------------------------------------------------------------------ selection


class Select:
    def __init__(self, lens, Hq=8, Hkv=2, D=128, B=16, keep=8, first=1, last=1, dtype="bf16", seed=0, ties=False,
                 negative=False, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.__dict__.update(Hq=Hq, Hkv=Hkv, D=D, B=B, keep=keep, first=first, last=last, dtype=dtype)
        self.lens = np.asarray(lens)
        n = -(-self.lens // B)
        NB = int(n.sum()) + 5
        self.NB = NB
        S, width = len(lens), int(max(1, n.max())) + 2
        perm = torch.randperm(NB, generator=g).int()
        tables, at = torch.full((S, width), -1, dtype=torch.int32), 0
        for s in range(S):
            tables[s, :n[s]] = perm[at:at + n[s]]
            at += int(n[s])
        a, b = torch.randint(-127, 128, (2, NB, Hkv, D), generator=g)
        codes = torch.stack([torch.minimum(a, b), torch.maximum(a, b)], 2)
        if ties:  # few different blocks
            codes = codes[torch.randint(0, 3, (NB,), generator=g)]
        if negative:  # every score below zero
            codes = torch.full_like(codes, -1)
        scale = torch.exp2(torch.randint(-3, 3, (NB, Hkv), generator=g).float())
        q = torch.randn(S, Hq, D, generator=g) * spread
        if negative:
            q = q.abs()
        if ties:
            scale.fill_(0.5)
        self.q, self.summary, self.scale = q.to(DT[dtype]).cuda(), codes.to(torch.int8).cuda(), scale.cuda()
        self.tables, self.cl = tables.cuda(), torch.from_numpy(self.lens).int().cuda()
        self.sel = torch.full((S, Hkv, keep), 55, dtype=torch.int32, device="cuda")
        self.cnt = torch.full((S, Hkv), 55, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.max_len = int(max(1, self.lens.max()))

    def call(self, stream=None):
        pkv.select_blocks(self.sel, self.cnt, self.q, self.summary, self.scale, self.tables, self.cl,
                          block_size=self.B, first_blocks=self.first, last_blocks=self.last,
                          max_context_len=self.max_len, status=self.status, stream=stream)

    def check(self, status=0, lens=None):
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        q, codes, scale = f64(self.q), self.summary.cpu().numpy(), f64(self.scale)
        sel, cnt, tables = self.sel.cpu().numpy(), self.cnt.cpu().numpy(), self.tables.cpu().numpy()
        G = self.Hq // self.Hkv
        for s, L in enumerate(self.lens if lens is None else lens):
            n = -(-int(L) // self.B)
            blocks = tables[s, :n]
            inside = (blocks >= 0) & (blocks < self.NB)
            for g in range(self.Hkv):
                sc = R.scores(q[s, g * G:(g + 1) * G], codes[np.where(inside, blocks, 0), g],
                              scale[np.where(inside, blocks, 0), g], MOST[self.dtype])
                want = R.select(np.where(inside, sc, -np.inf), n, self.keep, self.first, self.last)
                assert cnt[s, g] == len(want), (s, g)
                assert sel[s, g].tolist() == want + [-1] * (self.keep - len(want)), (s, g)


SELECT = [
    dict(lens=[0, 1, 15, 16, 17, 127, 128, 129, 400]), dict(lens=[1]), dict(lens=[0, 0]),
    dict(lens=[3000, 700, 5000], keep=64, first=2, last=2), dict(lens=[2000] * 3, Hq=64, Hkv=8, keep=17, dtype="f16"),
    dict(lens=[999, 1500], Hq=5, Hkv=5, keep=3, first=0, last=1), dict(lens=[999, 1500], Hq=4, Hkv=2, D=64, keep=20),
    dict(lens=[800, 811], Hq=15, Hkv=5, D=64, keep=9, dtype="f16"), dict(lens=[800, 811], Hq=14, Hkv=2, D=64, keep=9),
    dict(lens=[5000, 64, 65], B=64, keep=30), dict(lens=[5000, 33], B=32, keep=155, first=3, last=4),
    dict(lens=[4096, 4097], keep=255, Hq=6, Hkv=1), dict(lens=[600, 601], keep=2), dict(lens=[600], keep=36, last=35),
    dict(lens=[600, 900], keep=10, ties=True), dict(lens=[6000], keep=300, ties=True, first=0, last=1),
    dict(lens=[600, 900], keep=10, negative=True), dict(lens=[900], keep=10, spread=1e-30),
    dict(lens=[900], keep=10, spread=1e30), dict(lens=[70000, 131072, 20], keep=128, Hq=8, Hkv=2),
    dict(lens=[3000] * 40, Hq=16, Hkv=4, keep=33),
]


@pytest.mark.parametrize("kw", SELECT)
def test_selection(kw):
    s = Select(seed=7, **kw)
    s.call()
    s.check()


def test_selection_of_odd_queries():
    """Zero queries (all scores 0: the lowest blocks), NaN and infinities in a query."""
    s = Select([500, 500, 500], keep=9)
    s.q[0] = 0
    s.q[1, 2, 7], s.q[1, 5] = float("nan"), float("nan")
    s.q[2, 0, 3], s.q[2, 6, 4] = float("inf"), float("-inf")
    s.call()
    s.check()


def test_selection_flags_bad_lengths_and_entries():
    s = Select([500, 600, 700], keep=9)
    s.cl[1] = -4
    s.cl[2] = 100000
    s.tables[0, 5], s.tables[0, 31] = s.NB, -7
    s.call()
    wide = s.tables.shape[1] * 16
    s.check(pkv.DEV_ERR_LENGTH | pkv.DEV_ERR_BLOCK, lens=[500, 0, min(700, wide)])


def test_selection_on_streams_and_in_graphs():
    a, b = Select([3000, 20], seed=1), Select([2500, 4000], seed=2)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a.call(sa)
    b.call(sb)
    a.check()
    b.check()
    s, t = Select([3000, 900], seed=3), Select([3000, 900], seed=4)
    g, h = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.call()
    with torch.cuda.graph(h):
        t.call()
    for _ in range(2):
        s.q.copy_(torch.randn(s.q.shape).to(s.q.dtype))
        g.replay()
        h.replay()
        s.check()
        t.check()


# ------------------------------------------------------------------ attention


class Attend:
    def __init__(self, lens, Hq=8, Hkv=2, D=128, B=16, keep=8, dtype="bf16", out=torch.float32, seed=0, fp8=False,
                 layers=1, poison=True, mag=1.0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.__dict__.update(Hq=Hq, Hkv=Hkv, D=D, B=B, keep=keep, dtype=dtype, fp8=fp8)
        self.lens = np.asarray(lens)
        n = -(-self.lens // B)
        S, NB = len(lens), int(n.sum()) + 5
        self.NB = NB
        perm = torch.randperm(NB, generator=g).int()
        tables, at = torch.full((S, int(max(1, n.max())) + 1), -1, dtype=torch.int32), 0
        for s in range(S):
            tables[s, :n[s]] = perm[at:at + n[s]]
            at += int(n[s])
        shape = (NB, B, Hkv, D) if layers == 1 else (NB, layers, B, Hkv, D)
        pick = (slice(None),) if layers == 1 else (slice(None), 0)
        if fp8:
            kv = [(torch.randn(*shape, generator=g) * 40).to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2)]
            sc = [torch.exp2(torch.randint(-7, -3, shape[:-3] + (Hkv,), generator=g).float()) * 1.1 for _ in range(2)]
            self.ks, self.vs = (x.cuda()[pick] for x in sc)
            nan = 0x7F
        else:
            kv = [(torch.randn(*shape, generator=g) * mag).to(DT[dtype]) for _ in range(2)]
            nan = float("nan")
        if poison:  # rows no sequence owns
            owned = torch.zeros(NB, B, dtype=torch.bool)
            for s in range(S):
                for i in range(n[s]):
                    owned[tables[s, i], :min(B, int(lens[s]) - i * B)] = True
            for x in kv:
                x[pick][~owned] = nan
        self.kp, self.vp = (x.cuda()[pick] for x in kv)
        self.q = torch.randn(S, Hq, D, generator=g).to(DT[dtype]).cuda()
        self.tables, self.cl = tables.cuda(), torch.from_numpy(self.lens).int().cuda()
        sel, cnt = np.full((S, Hkv, keep), -1), np.zeros((S, Hkv), int)
        for s in range(S):
            for h in range(Hkv):
                m = int(min(n[s], keep))
                cnt[s, h] = m
                if m:
                    rest = np.sort(rng.permutation(n[s] - 1)[:m - 1])
                    sel[s, h, :m] = np.append(rest, n[s] - 1)
        self.sel, self.cnt = torch.from_numpy(sel).int().cuda(), torch.from_numpy(cnt).int().cuda()
        self.out = torch.full((S, Hq, D), 9.0, dtype=out, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.max_len, self.scale = int(max(1, self.lens.max())), D ** -0.5

    def call(self, stream=None):
        kw = dict(max_context_len=self.max_len, status=self.status, stream=stream)
        if self.fp8:
            pkv.decode_sparse_fp8(self.out, self.q, self.kp, self.vp, self.ks, self.vs, self.tables, self.cl, self.sel,
                                  self.cnt, self.scale, **kw)
        else:
            pkv.decode_sparse(self.out, self.q, self.kp, self.vp, self.tables, self.cl, self.sel, self.cnt, self.scale,
                              **kw)

    def values(self, pool, scale, phys, g):
        if self.fp8:
            return R.E4M3[pool[phys, :, g].cpu().numpy()] * float(scale[phys, g])
        return f64(pool[phys, :, g])

    def check(self, status=0, lists=None):
        """lists: {(s, g): blocks that count}, where they are not the lists as given."""
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        got, q = f64(self.out), f64(self.q)
        sel, cnt, tables = self.sel.cpu().numpy(), self.cnt.cpu().numpy(), self.tables.cpu().numpy()
        G = self.Hq // self.Hkv
        half = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[self.out.dtype]
        for s, L in enumerate(self.lens):
            for g in range(self.Hkv):
                blocks = (lists or {}).get((s, g), sel[s, g, :cnt[s, g]].tolist())
                k, v = ([self.values(p, sc, int(tables[s, b]), g)[:max(0, min(self.B, int(L) - b * self.B))]
                         for b in blocks] for p, sc in ((self.kp, getattr(self, "ks", None)),
                                                        (self.vp, getattr(self, "vs", None))))
                k = np.concatenate(k) if k else np.zeros((0, self.D))
                v = np.concatenate(v) if v else np.zeros((0, self.D))
                rows = slice(g * G, (g + 1) * G)
                want = R.attend(q[s, rows], k, v, self.scale)
                tol = R.attend_bound(q[s, rows], k, v, self.scale, SPLIT["fp8" if self.fp8 else self.dtype])
                err = np.abs(got[s, rows] - want)
                assert np.all(err <= tol + half * (np.abs(want) + tol) + 2.0 ** -25), (s, g, err.max(), tol)


ATTEND = [
    dict(lens=[0, 1, 15, 16, 17, 127, 128, 129, 400]), dict(lens=[1], Hq=1, Hkv=1, D=64), dict(lens=[0, 0]),
    dict(lens=[3000, 700, 5000], keep=64, dtype="f16"), dict(lens=[2000] * 3, Hq=64, Hkv=8, keep=17, dtype="f16"),
    dict(lens=[999, 1500], Hq=5, Hkv=5, keep=3, out=torch.bfloat16), dict(lens=[999, 1500], Hq=4, Hkv=2, D=64, keep=20),
    dict(lens=[800, 811], Hq=15, Hkv=5, D=64, keep=9, dtype="f16", out=torch.float16),
    dict(lens=[800, 811], Hq=14, Hkv=2, D=64, keep=1), dict(lens=[5000, 64, 65], B=64, keep=30),
    dict(lens=[5000, 33], B=32, keep=155), dict(lens=[9000, 40], B=64, keep=100, D=64, dtype="f16"),
    dict(lens=[4097], keep=256, Hq=6, Hkv=1), dict(lens=[40000], keep=1000, Hq=8, Hkv=1),
    dict(lens=[300] * 70, Hq=8, Hkv=4, keep=12), dict(lens=[600, 900], layers=3), dict(lens=[500], mag=8.0),
    dict(lens=[500], mag=8.0, dtype="f16"),
]


@pytest.mark.parametrize("kw", ATTEND)
def test_attention(kw):
    a = Attend(seed=11, **kw)
    a.call()
    a.check()


@pytest.mark.parametrize("kw", [dict(lens=[0, 1, 15, 16, 17, 33, 400]), dict(lens=[3000, 700], keep=64, dtype="f16"),
                                dict(lens=[2000] * 3, Hq=64, Hkv=8, keep=17), dict(lens=[999], Hq=5, Hkv=5, keep=3),
                                dict(lens=[5000, 600], layers=2, keep=131, out=torch.bfloat16),
                                dict(lens=[300] * 70, Hq=8, Hkv=4, keep=12), dict(lens=[40000], keep=700, Hkv=1)])
def test_attention_fp8(kw):
    a = Attend(seed=13, fp8=True, **kw)
    a.call()
    a.check()


def test_attention_fp8_with_far_apart_scales():
    a = Attend([700], keep=40, fp8=True)
    a.vs[:] = torch.exp2(torch.linspace(-100, 20, a.NB)).cuda()[torch.randperm(a.NB).cuda()][:, None]
    a.call()
    a.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_lists(fp8):
    """Entries out of order, repeated, negative or past the sequence, bad counts and table entries are
    passed over; the rest of the row is right."""
    a = Attend([800, 800, 800], keep=8, fp8=fp8)
    a.sel[0, 0] = torch.tensor([1, 5, 5, 4, 9, 50, -1, 20])
    a.cnt[0, 1], a.cnt[1, 0] = 9, -1
    a.tables[2, 49] = a.NB + 3
    a.call()
    sel = a.sel.cpu().numpy()
    lists = {(0, 0): [1, 5, 9, 20], (1, 0): [], (2, 0): sel[2, 0, :-1].tolist(), (2, 1): sel[2, 1, :-1].tolist()}
    a.check(pkv.DEV_ERR_SELECT | pkv.DEV_ERR_BLOCK, lists)


def test_all_blocks_selected_is_decode_attention():
    a = Attend([333, 1200, 16], Hq=32, Hkv=8, keep=75)
    a.call()
    full = torch.empty_like(a.out)
    pkv.decode_attention(full, a.q, a.kp, a.vp, a.tables, a.cl, a.scale, max_context_len=a.max_len)
    a.check()
    assert float((a.out - full).abs().max()) <= 2e-3


def test_infinite_and_masked_scores():
    """Keys so far apart that all weight falls on one token, and a row of equal scores."""
    a = Attend([200, 200], keep=13)
    a.q[0] = 50.0
    a.kp[a.tables[0, 3], 2] = 20.0
    a.q[1] = 0.0
    a.call()
    a.check()


def test_attention_on_streams_and_in_graphs():
    a, b = Attend([3000, 20], seed=1, keep=60), Attend([2500, 4000], seed=2, keep=90)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a.call(sa)
    b.call(sb)
    a.check()
    b.check()
    g, h = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.call()
    with torch.cuda.graph(h):
        b.call()
    for _ in range(2):
        a.q.copy_(torch.randn(a.q.shape).to(a.q.dtype))
        g.replay()
        h.replay()
        a.check()
        b.check()


def test_refusals():
    a, s = Attend([300]), Select([300])
    for kw in (dict(sel=a.sel.long()), dict(cnt=a.cnt[:, :1]), dict(q=a.q.half()), dict(out=a.out[:, :4]),
               dict(tables=a.tables.cpu()), dict(cl=a.cl.long()), dict(sel=a.sel.expand(2, -1, -1))):
        f = lambda n: kw.get(n, getattr(a, n))
        with pytest.raises(pkv.PkvError):
            pkv.decode_sparse(f("out"), f("q"), a.kp, a.vp, f("tables"), f("cl"), f("sel"), f("cnt"), 0.1,
                              max_context_len=300)
    for kw in (dict(sel=s.sel.long()), dict(cnt=s.cnt[:, :1]), dict(q=s.q[..., :64]), dict(summary=s.summary.float()),
               dict(scale=s.scale.half()), dict(tables=s.tables.cpu()), dict(cl=s.cl.long())):
        f = lambda n: kw.get(n, getattr(s, n))
        with pytest.raises(pkv.PkvError):
            pkv.select_blocks(f("sel"), f("cnt"), f("q"), f("summary"), f("scale"), f("tables"), f("cl"), block_size=16,
                              max_context_len=300)
    ids = torch.zeros(3, dtype=torch.int32, device="cuda")
    for kw in (dict(ids=ids.long()), dict(summary=s.summary[:3]), dict(scale=s.scale[:, :1]), dict(ids=ids.cpu())):
        with pytest.raises(pkv.PkvError):
            pool = torch.zeros(s.NB, 16, 2, 128, dtype=torch.bfloat16, device="cuda")
            pkv.summarize_blocks(kw.get("summary", s.summary), kw.get("scale", s.scale), pool, kw.get("ids", ids))


@pytest.mark.parametrize("n,keep", [(300, 8), (300, 200), (2500, 100), (9000, 700)])
def test_selection_among_unusable_entries(n, keep):
    """Blocks whose table entries lie outside the pool are taken last, the lowest first, when there are not
    enough others; never in place of a usable one."""
    s = Select([n * 16], keep=keep, first=1, last=2, seed=n)
    bad = torch.randperm(n, generator=torch.Generator().manual_seed(n))[:n - keep // 2]
    s.tables[0, bad[bad < n].cuda()] = -5
    s.call()
    s.check(pkv.DEV_ERR_BLOCK)


@pytest.mark.parametrize("seed", range(6))
def test_selection_on_random_shapes(seed):
    rng = np.random.default_rng(100 + seed)
    for _ in range(6):
        Hkv = int(rng.integers(1, 5))
        keep = int(rng.integers(3, 200))
        kw = dict(Hq=Hkv * int(rng.integers(1, 9)), Hkv=Hkv, D=int(rng.choice([64, 128])), B=int(rng.choice([16, 32, 64])),
                  keep=keep, first=int(rng.integers(0, 2)), last=int(rng.integers(1, 3)),
                  dtype=str(rng.choice(["bf16", "f16"])), ties=bool(rng.random() < 0.3))
        lens = rng.integers(0, int(np.exp(rng.uniform(3, 11))), size=int(rng.integers(1, 5)))
        s = Select(lens, seed=int(rng.integers(1 << 30)), **kw)
        s.call()
        s.check()


def test_selection_at_the_block_limit():
    """49152 blocks of one sequence are scored and searched; one more is refused."""
    n = 49152
    s = Select([n * 16], Hq=2, Hkv=1, D=64, keep=300)
    s.tables = s.tables[:, :n].contiguous()
    s.call()
    s.check()
    s.tables = torch.nn.functional.pad(s.tables, (0, 1), value=-1)
    s.max_len += 1
    with pytest.raises(pkv.PkvError):
        s.call()


@pytest.mark.parametrize("fp8", [False, True])
def test_pools_and_summaries_past_four_gigabytes(fp8):
    """Blocks beyond 2^32 bytes and 2^31 elements of the pools (and 2^31 bytes of the summaries)."""
    Hkv, D, B = 8, 128, 16
    NB = 290000 if fp8 else 140000
    ids = torch.tensor([NB - 1, 5, NB - 7, NB // 2, 131071, 131072], dtype=torch.int32).cuda()
    n = len(ids)
    a = Attend([n * B - 3], Hq=8, Hkv=Hkv, keep=n, fp8=fp8, poison=False)
    make = lambda: torch.empty((NB, B, Hkv, D), dtype=a.kp.dtype, device="cuda")
    kp, vp = make(), make()
    own = a.tables[0, :n].long()
    kp[ids.long()], vp[ids.long()] = a.kp[own], a.vp[own]
    if fp8:
        ks, vs = (torch.empty((NB, Hkv), device="cuda") for _ in range(2))
        ks[ids.long()], vs[ids.long()] = a.ks[own], a.vs[own]
    summary = torch.empty((NB, Hkv, 2, D), dtype=torch.int8, device="cuda")
    scale = torch.empty((NB, Hkv), device="cuda")
    if fp8:
        pkv.summarize_blocks_fp8(summary, scale, kp, ks, ids, status=a.status)
    else:
        pkv.summarize_blocks(summary, scale, kp, ids, status=a.status)
    torch.cuda.synchronize()
    keys = R.E4M3[a.kp.cpu().numpy()] * f64(a.ks)[:, None, :, None] if fp8 else f64(a.kp)
    for i in range(n):
        for g in range(Hkv):
            codes, unit = R.summarize(keys[int(own[i]), :, g], MOST["fp8" if fp8 else "bf16"] if not fp8 else 3.4e38)
            assert np.array_equal(summary[int(ids[i]), g].cpu().numpy(), codes) and float(scale[int(ids[i]), g]) == unit
    sel = torch.empty((1, Hkv, 4), dtype=torch.int32, device="cuda")
    cnt = torch.empty((1, Hkv), dtype=torch.int32, device="cuda")
    pkv.select_blocks(sel, cnt, a.q, summary, scale, ids[None].contiguous(), a.cl, block_size=B, max_context_len=n * B,
                      status=a.status)
    torch.cuda.synchronize()
    q = f64(a.q)
    for g in range(Hkv):
        sc = R.scores(q[0, g:g + 1], summary[ids.long(), g].cpu().numpy(), f64(scale)[ids.cpu().numpy(), g], MOST["bf16"])
        assert sel[0, g].tolist() == R.select(sc, n, 4, 1, 1)
    a.tables, a.kp, a.vp, own_tables = ids[None].contiguous(), kp, vp, a.tables
    if fp8:
        a.ks, a.vs = ks, vs
    a.call()
    a.check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", [dict(lens=[100, 17, 230, 90, 1] * 26, Hq=8, Hkv=4, keep=6),
                                dict(lens=[1000, 300, 0, 65] * 12, Hq=12, Hkv=4, keep=50),
                                dict(lens=[700] * 19, Hq=64, Hkv=8, keep=20, dtype="f16"),
                                dict(lens=[400, 900] * 10, Hq=16, Hkv=16, keep=40, D=64, B=32)])
def test_attention_of_many_units(kw, fp8):
    """As many (sequence, KV head) units as SMs and more, short and long."""
    if fp8 and kw.get("D") == 64:
        kw = dict(kw, D=128, B=16)
    a = Attend(seed=17, fp8=fp8, **kw)
    a.call()
    a.check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [0.0, -0.05, 3.0])
def test_attention_with_other_scales(scale, fp8):
    a = Attend([300, 50], keep=10, fp8=fp8)
    a.scale = scale
    a.call()
    a.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_a_query_that_is_not_finite_stays_in_its_row(fp8):
    a, b = Attend([700, 90], keep=30, fp8=fp8), Attend([700, 90], keep=30, fp8=fp8)
    a.q[0, 3, 7], a.q[1, 4, 0] = float("nan"), float("inf")
    a.call()
    b.call()
    torch.cuda.synchronize()
    rest = torch.ones(2, 8, dtype=torch.bool, device="cuda")
    rest[0, 3] = rest[1, 4] = False
    assert torch.equal(a.out[rest], b.out[rest]) and not torch.isfinite(a.out[0, 3]).any()


def test_tables_of_no_blocks():
    """A table of width 0 holds no token: zero rows and empty lists; a length above it is reported."""
    s, a = Select([0, 0]), Attend([0, 0])
    s.tables, a.tables = s.tables[:, :0].contiguous(), a.tables[:, :0].contiguous()
    s.call()
    s.check()
    a.call()
    a.check()
    s.cl[1] = a.cl[1] = 5
    s.call()
    s.check(pkv.DEV_ERR_LENGTH)
    a.call()
    a.check(pkv.DEV_ERR_LENGTH)


def test_equal_inputs_give_equal_bits():
    """Repeated calls, alone and beside another stream's, agree bit for bit."""
    s, a = Select([60000, 9000, 33], keep=99), Attend([20000, 300], keep=500)
    busy = torch.cuda.Stream()
    noise = Attend([5000] * 8, keep=200)
    torch.cuda.synchronize()
    first = None
    for i in range(20):
        if i % 2:
            noise.call(busy)
        s.call()
        a.call()
        torch.cuda.synchronize()
        got = (s.sel.clone(), a.out.clone())
        first = first or got
        assert all(torch.equal(x, y) for x, y in zip(first, got))


@pytest.mark.parametrize("fp8", [False, True])
def test_heads_of_far_apart_magnitudes(fp8):
    """Each head is as exact as beside heads of its own size."""
    a = Attend([500, 60], Hq=8, Hkv=1, keep=30, fp8=fp8)
    a.q *= torch.exp2(torch.tensor([0.0, 60, -40, 17, -20, 100, 3, 30]))[:, None].to(a.q)
    a.call()
    torch.cuda.synchronize()
    got, q = f64(a.out), f64(a.q)
    for s, L in enumerate(a.lens):
        blocks = a.tables[s].cpu().numpy()[a.sel[s, 0, :a.cnt[s, 0]].cpu().numpy()]
        k, v = (np.concatenate([a.values(p, sc, int(b), 0) for b in blocks])
                for p, sc in ((a.kp, getattr(a, "ks", None)), (a.vp, getattr(a, "vs", None))))
        ok = ~np.isnan(k).any(1)  # the poisoned rows behind the sequence
        for h in range(8):
            want = R.attend(q[s, h:h + 1], k[ok], v[ok], a.scale)
            tol = R.attend_bound(q[s, h:h + 1], k[ok], v[ok], a.scale, SPLIT["fp8" if fp8 else a.dtype])
            assert np.all(np.abs(got[s, h] - want) <= tol + 2.0 ** -24 * np.abs(want) + 2.0 ** -25), (s, h)


@pytest.mark.parametrize("kind", [dict(), dict(fp8=True), dict(D=64, dtype="f16")])
@pytest.mark.parametrize("units,tiles", [(1, 3), (1, 10), (1, 24), (2, 48), (3, 100), (40, 9), (153, 18), (77, 33),
                                         (38, 49), (330, 3), (330, 30), (700, 2), (1300, 4), (2100, 1)])
def test_attention_by_number_and_length_of_lists(units, tiles, kind):
    """Every number of warps a CTA and of CTAs a list, with tiles that do not fill the last round."""
    a = Attend([16 * tiles - i % 16 for i in range(units)], Hq=2, Hkv=1, keep=tiles, seed=units, **kind)
    a.call()
    a.check()
