"""The layer operators' float64 statements, pinned by what must hold of them;
and the entry points' refusals (no GPU needed)."""
import numpy as np
import pytest

import paged_kv_cache_112_gb300 as pkv
from paged_kv_cache_112_gb300 import build as pkv_build
from tests import layer_ref as R


@pytest.fixture(scope="module")
def lib():
    try:
        pkv_build.build()
    except RuntimeError as e:  # no nvcc on this machine
        pytest.skip(str(e))
    return pkv.load()


def test_rotation_keeps_norms_and_relative_angles():
    rng = np.random.default_rng(0)
    x, y = rng.normal(size=(2, 1, 1, 64))
    inv = 10000.0 ** (-np.arange(16) / 16)
    ang = lambda p: np.concatenate([np.cos(p * inv), np.sin(p * inv)])[None]
    for inter in (False, True):
        a, _ = R.norm_rope(x, None, 0, ang(70), inter)
        b, _ = R.norm_rope(y, None, 0, ang(50), inter)
        c, _ = R.norm_rope(x, None, 0, ang(20), inter)
        assert np.isclose((a * a).sum(), (x * x).sum())
        assert np.isclose((a * b).sum(), (c * y).sum())  # only the difference of positions counts
        assert np.array_equal(a[..., 32:], x[..., 32:])


def test_summaries_bound_every_key_and_scores_every_dot_product():
    rng = np.random.default_rng(1)
    keys = rng.normal(size=(40, 16, 64)) * np.exp(rng.normal(size=(40, 1, 64)))
    q = rng.normal(size=(3, 64))
    codes, scale = map(np.array, zip(*(R.summarize(k, 1e30) for k in keys)))
    for k, c, u in zip(keys, codes, scale):
        assert np.all(c[0] * u <= k.min(0)) and np.all(c[1] * u >= k.max(0))
        assert np.all(k.min(0) - c[0] * u < u) and np.abs(c.astype(int)).max() <= 127
        assert max(np.abs(k).max() / u, 64) > 63.5  # the scale is no larger than it has to be
    qr = np.stack([np.rint(r / 2.0 ** R.step_exponent(np.abs(r).max())) * 2.0 ** R.step_exponent(np.abs(r).max())
                   for r in q])
    s = R.scores(q, codes, scale, 1e30)
    assert np.all(s >= np.einsum("gd,btd->bgt", qr, keys).max((1, 2)) - 1e-9)


def test_selection_by_hand():
    sc = np.array([9, 1, 5, 5, 5, 2, 0, 9.0])
    assert R.select(sc, 8, 8, 1, 1) == list(range(8))
    assert R.select(sc, 8, 4, 1, 1) == [0, 2, 3, 7]
    assert R.select(sc, 8, 3, 0, 1) == [0, 2, 7]
    assert R.select(sc, 8, 2, 1, 1) == [0, 7]
    assert R.select(sc, 0, 4, 1, 1) == []


FAKE = 0x10000  # never dereferenced: validation fails before any device work
INV, UNS, OK = 1, 2, 0


def _norm(lib, fp8=False, **kw):
    a = dict(qo=FAKE, qos=0, ko=None, kos=0, q=FAKE + 65536, qs=0, k=FAKE, v=FAKE, kvs=0, qw=None, kw=None, eps=1e-6,
             cs=FAKE, pos=FAKE, top=100, rot=128, inter=0, kp=FAKE, vp=FAKE, bs=0, ks=FAKE, vs=FAKE, slots=FAKE, T=4,
             Hq=8, Hkv=2, D=128, B=16, NB=10, L=1, dt=pkv.PKV_BF16)
    a.update(kw)
    head = (a["qo"], a["qos"], a["ko"], a["kos"], a["q"], a["qs"], a["k"], a["v"], a["kvs"], a["qw"], a["kw"],
            a["eps"], a["cs"], a["pos"], a["top"], a["rot"], a["inter"], a["kp"], a["vp"])
    tail = (a["T"], a["Hq"], a["Hkv"], a["D"], a["B"], a["NB"])
    if fp8:
        return lib.pkv_norm_rope_write_fp8(*head, a["ks"], a["vs"], a["slots"], *tail, a["L"], a["dt"], None, None)
    return lib.pkv_norm_rope_write(*head, a["bs"], a["slots"], *tail, a["dt"], None, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_norm_rope_write_refusals(lib, fp8):
    for want, kw in [
        (INV, dict(T=-1)), (INV, dict(Hq=0)), (INV, dict(NB=0)), (INV, dict(rot=-16)), (INV, dict(rot=144)),
        (INV, dict(inter=2)), (INV, dict(dt=pkv.PKV_F32)), (INV, dict(qw=FAKE, eps=0.0)),
        (INV, dict(kw=FAKE, eps=float("nan"))), (UNS, dict(D=96, rot=96)), (UNS, dict(rot=24)), (UNS, dict(B=24)),
        (INV, dict(qo=None)), (INV, dict(q=None)), (INV, dict(k=None)), (INV, dict(slots=None)), (INV, dict(cs=None)),
        (INV, dict(pos=None)), (INV, dict(top=0)), (INV, dict(q=FAKE + 8)), (INV, dict(cs=FAKE + 4)),
        (INV, dict(qs=8 * 128 - 8)), (INV, dict(qs=8 * 128 + 4)), (INV, dict(kvs=100)), (INV, dict(qos=1000)),
        (INV, dict(ko=FAKE + 32, kos=12)), (INV, dict(qo=FAKE, q=FAKE, qs=4096)), (INV, dict(slots=FAKE + 2)),
        (UNS, dict(T=1 << 30, Hq=64)), (OK, dict(T=0)), (OK, dict(T=0, q=None)),
    ]:
        assert _norm(lib, fp8, **kw) == want, kw
    if fp8:
        assert _norm(lib, True, ks=None) == INV and _norm(lib, True, L=0) == INV and _norm(lib, True, B=32) == UNS
    else:
        assert _norm(lib, bs=16 * 2 * 128 - 8) == INV


def test_summarize_refusals(lib):
    f = lambda **k: lib.pkv_summarize_blocks(k.get("s", FAKE), k.get("sc", FAKE), k.get("kp", FAKE), k.get("bs", 0),
                                             k.get("ids", FAKE), k.get("n", 3), k.get("Hkv", 2), k.get("D", 128),
                                             k.get("B", 16), 10, k.get("dt", pkv.PKV_F16), None, None)
    for want, kw in [(INV, dict(n=-1)), (INV, dict(Hkv=0)), (UNS, dict(D=96)), (UNS, dict(B=8)), (UNS, dict(B=24)),
                     (INV, dict(s=None)), (INV, dict(sc=None)), (INV, dict(ids=None)), (INV, dict(s=FAKE + 8)),
                     (INV, dict(dt=pkv.PKV_F32)), (INV, dict(bs=64)), (OK, dict(n=0))]:
        assert f(**kw) == want, kw
    f8 = lambda **k: lib.pkv_summarize_blocks_fp8(FAKE, FAKE, FAKE, k.get("ks", FAKE), FAKE, k.get("n", 3), 2, 128,
                                                  k.get("B", 16), 10, k.get("L", 1), None, None)
    assert f8(ks=None) == INV and f8(B=32) == UNS and f8(L=0) == INV and f8(n=0) == OK


def test_select_refusals(lib):
    def f(**k):
        return lib.pkv_select_blocks(k.get("sel", FAKE), k.get("cnt", FAKE), k.get("q", FAKE), k.get("sum", FAKE), FAKE,
                                     FAKE, k.get("w", 100), FAKE, k.get("S", 2), k.get("Hq", 8), k.get("Hkv", 2),
                                     k.get("D", 128), k.get("B", 16), 10, k.get("keep", 8), k.get("first", 1),
                                     k.get("last", 1), k.get("L", 1600), k.get("dt", pkv.PKV_BF16), None, None)

    for want, kw in [(INV, dict(S=-1)), (INV, dict(keep=0)), (INV, dict(first=-1)), (INV, dict(last=0)),
                     (INV, dict(first=8)), (INV, dict(dt=pkv.PKV_F32)), (INV, dict(L=-1)), (UNS, dict(D=96)),
                     (UNS, dict(B=8)), (UNS, dict(Hq=18)), (UNS, dict(Hq=7)), (UNS, dict(keep=(1 << 20) + 1)),
                     (INV, dict(sel=None)), (INV, dict(cnt=None)), (INV, dict(q=None)), (INV, dict(q=FAKE + 8)),
                     (INV, dict(sum=FAKE + 8)), (UNS, dict(w=1 << 30)), (OK, dict(S=0))]:
        assert f(**kw) == want, kw


def test_decode_sparse_refusals(lib):
    def f(**k):
        return lib.pkv_decode_sparse(k.get("out", FAKE), k.get("q", FAKE), k.get("kp", FAKE), FAKE, k.get("bs", 0), FAKE,
                                     k.get("w", 100), FAKE, k.get("sel", FAKE), k.get("cnt", FAKE), k.get("keep", 8),
                                     k.get("S", 2), k.get("Hq", 8), k.get("Hkv", 2), k.get("D", 128), k.get("B", 16), 10,
                                     k.get("sc", 0.1), k.get("L", 1600), k.get("dt", pkv.PKV_BF16),
                                     k.get("od", pkv.PKV_F32), None, None)

    for want, kw in [(INV, dict(S=-1)), (INV, dict(keep=0)), (INV, dict(sc=float("inf"))), (INV, dict(L=-1)),
                     (INV, dict(dt=pkv.PKV_F32)), (INV, dict(od=7)), (UNS, dict(D=96)), (UNS, dict(B=8)),
                     (UNS, dict(Hq=18)), (UNS, dict(Hq=7)), (INV, dict(out=None)), (INV, dict(sel=None)),
                     (INV, dict(cnt=None)), (INV, dict(kp=FAKE + 8)), (INV, dict(q=FAKE + 4)), (INV, dict(bs=24)),
                     (UNS, dict(w=1 << 30)), (OK, dict(S=0))]:
        assert f(**kw) == want, kw
    f8 = lambda **k: lib.pkv_decode_sparse_fp8(FAKE, FAKE, FAKE, FAKE, k.get("ks", FAKE), FAKE, FAKE, 100, FAKE, FAKE,
                                               FAKE, 8, k.get("S", 2), 8, 2, k.get("D", 128), k.get("B", 16), 10,
                                               k.get("L", 1), 0.1, 1600, pkv.PKV_BF16, pkv.PKV_F32, None, None)
    assert f8(ks=None) == INV and f8(D=64) == UNS and f8(B=32) == UNS and f8(L=0) == INV and f8(S=0) == OK
