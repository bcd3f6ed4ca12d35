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


def check_channels(a, split, floor):
    """a's rows against the float64 statement, each channel to the magnitudes that meet in it.

    A weight p_t (the largest of the row is 1) is off by 2 eps_t of itself for its score's error eps_t
    (layer_ref.attend_bound, of this token), by `split` for the two parts that hold it, and by `floor`, of the
    largest weight times value scale, where the parts' subnormals end (c: the values without their scale u).  Sums
    lose at most 2^-23 a token and merge, above and below the line:
        |err_d| <= sum_t p_t (r_t + r) |v_td| / l + floor max_t(p_t u_t) sum_t |c_td| / l,
        r_t = 2 eps_t + split + (n + 64) 2^-23,  r = sum_t p_t r_t / l."""
    torch.cuda.synchronize()
    assert int(a.status.item()) == 0
    got, q, tables = f64(a.out), f64(a.q), a.tables.cpu().numpy()
    G, worst = a.Hq // a.Hkv, 0.0
    for s, L in enumerate(a.lens):
        for g in range(a.Hkv):
            blocks = a.sel[s, g, :int(a.cnt[s, g])].tolist()
            k, v = (np.concatenate([a.values(p, sc, int(tables[s, b]), g)[:min(a.B, int(L) - b * a.B)]
                                    for b in blocks])
                    for p, sc in ((a.kp, getattr(a, "ks", None)), (a.vp, getattr(a, "vs", None))))
            u, c = np.ones(k.shape[0]), v
            if a.fp8:
                u = np.repeat(f64(a.vs)[tables[s, blocks], g], a.B)[:k.shape[0]]
                c = np.where(u[:, None] > 0, v / np.where(u > 0, u, 1)[:, None], 448.0)
            for h in range(g * G, (g + 1) * G):
                logit = a.scale * (k @ q[s, h])
                p = np.exp(logit - logit.max())
                eps = a.D * 2.0 ** -23 * a.scale * (np.abs(k) @ np.abs(q[s, h]))
                want, l = p @ v / p.sum(), p.sum()
                r = 2 * eps + split + (k.shape[0] + 64) * 2.0 ** -23
                tol = (p * (r + p @ r / l)) @ np.abs(v) / l + floor * (p * u).max() * np.abs(c).sum(0) / l
                err = np.abs(got[s, h] - want)
                tol = tol + 2.0 ** -24 * np.abs(want)
                worst = max(worst, float((err / tol).max()))
    assert worst <= 1.0, worst


def _scored(a, blocks, code):
    """Gives the keys of sequence 0's listed blocks `code` (FP8) or its value in channel 0, other keys 0 there."""
    phys = a.tables[0].long()
    a.kp[..., 0] = 0
    for b in blocks:
        a.kp[phys[b], :, :, 0] = code


# Two f16 parts of a weight (times value scale) times 2^14: half a step of the second part, and half of f16's
# smallest number, in a unit at most twice the largest.
F16_PARTS = dict(split=2.0 ** -22, floor=2.0 ** -38)


@pytest.mark.parametrize("e", [0, 8, 12, 16, 20, 40])
@pytest.mark.parametrize("low", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_weights_under_far_apart_value_scales(dtype, low, e):
    """low: the first half of the blocks has values 2^e times as large and next to no weight, in every warp's
    first tiles.  Else: the first block has most of the weight and values 2^e times smaller than the rest."""
    a = Attend([2048], Hq=8, Hkv=2, keep=128, fp8=True, dtype=dtype, seed=e)
    phys = a.tables[0, :128].long()
    a.q *= 0.125
    a.vs[:] = 2.0 ** -6
    a.ks[:] = 1 / 32
    if low:  # a score of -448 / 32 * 40 / sqrt(128) = -49.5 in channel 0
        _scored(a, range(64), 0xFE)
        a.q[..., 0] = 40.0
        a.vs[phys[:64]] = 2.0 ** (e - 6)
    else:  # 12.4
        _scored(a, [0], 0x7E)
        a.q[..., 0] = 10.0
        a.vs[phys[0]] = 2.0 ** (-6 - e)
    a.call()
    check_channels(a, **F16_PARTS)


@pytest.mark.parametrize("base", [-90, -6, 100])
@pytest.mark.parametrize("first,zeros", [(True, False), (False, False), (False, True)])
def test_long_lists_under_far_apart_value_scales(first, zeros, base):
    """Some 65 tiles a warp: half of the blocks, the first or the last, has values far larger than the others,
    which are about 2^base, and next to no weight.  zeros: each warp's first two tiles have most of the weight,
    and value scales of zero."""
    a = Attend([67200], Hq=2, Hkv=1, keep=4200, fp8=True, seed=5)
    phys = a.tables[0, :4200].long()
    a.q *= 0.125
    a.vs[:] = 2.0 ** base * (1 + torch.rand(a.vs.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(1)))
    a.ks[:] = 1 / 32
    low = range(2100) if first else range(2100, 4200)
    _scored(a, low, 0xFE)
    a.q[..., 0] = 40.0
    a.vs[phys[low.start:low.stop]] = 2.0 ** min(base + 24, 112)
    if zeros:
        a.kp[phys[:128], :, :, 0] = 0x6C  # 96: e^10.6 times the weight
        a.vs[phys[:128]] = 0
    a.call()
    check_channels(a, **F16_PARTS)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,q0", [(128, 10.0), (64, 11.0), (128, 15.0)])
def test_small_weights_keep_their_bits(dtype, D, q0):
    """16-bit pools: one block has nearly all the weight and no values, so the rows are made of weights
    that are all about exp(-14 q0 / sqrt(D)), 2^-18 to 2^-28."""
    a = Attend([1500, 40], Hq=8, Hkv=2, D=D, keep=94, dtype=dtype, seed=D)
    _scored(a, [2], 14.0)
    a.q *= 0.125
    a.q[0, :, 0] = q0
    a.vp[a.tables[0, 2].long()] = 0
    a.call()
    # bf16 has float32's exponents: a second part of 2^-17 and no floor.
    check_channels(a, **(F16_PARTS if dtype == "f16" else dict(split=2.0 ** -16, floor=0.0)))


def test_heads_scored_far_apart():
    """One head's positive score decides against another's whose queries are 2^120 times smaller, in blocks
    whose summaries are far apart too."""
    s = Select([40 * 16], Hq=2, Hkv=1, keep=4, first=0, last=1)
    phys = s.tables[0, :40].long()
    s.q.zero_()
    s.q[0, 0, 0], s.q[0, 1, 64:] = 1.0, 2.0 ** -120
    s.summary.zero_()
    s.summary[phys, 0, :, 0] = -1  # the first head: negative everywhere,
    s.summary[phys, 0, :, 64:] = 100  # the second: the same positive score in every block
    s.scale[phys] = 1.0
    for b in (11, 23, 38):  # but here the first head's is positive, and larger than the second's elsewhere
        s.summary[phys[b], 0, :, 0] = 1
        s.scale[phys[b]] = 2.0 ** -95
    s.call()
    s.check()
    assert s.sel[0, 0].tolist() == [11, 23, 38, 39]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("given,counted", [([5, 3, 5], [5, 5]), ([5, -1, 5], [5, 5]), ([1, 50, 20], [1]),
                                           ([7, 7, 7], [7]), ([9, 8, 7], [9]), ([2, 4, 3, 4], [2, 4, 4])])
def test_lists_that_do_not_ascend(given, counted, fp8):
    """Flagged, and what counts is what the comparison of neighbours leaves."""
    a = Attend([800, 33], Hq=4, Hkv=1, keep=len(given), fp8=fp8)
    a.sel[0, 0] = torch.tensor(given)
    a.call()
    a.check(pkv.DEV_ERR_SELECT, {(0, 0): counted})


@pytest.mark.parametrize("kind", [dict(), dict(fp8=True), dict(D=64, dtype="f16")])
@pytest.mark.parametrize("units,tiles", [(20, 70), (50, 60), (76, 300), (100, 128), (200, 90)])
def test_attention_of_long_lists_on_small_clusters(units, tiles, kind):
    """From twenty lists to a few more than SMs, long enough that CTAs share them: at head size 128 these are
    8 warps in clusters of 4, 4 of 8, 8 of 2, 4 of 4 and 4 of 2."""
    a = Attend([16 * tiles - i % 16 if i % 5 else 16 for i in range(units)], Hq=2, Hkv=1, keep=tiles, seed=units,
               **kind)
    a.call()
    a.check()
