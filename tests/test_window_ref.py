"""The 4-bit and window statements pinned by what must hold of them, and the
entry points' refusals (no GPU needed)."""
import numpy as np
import pytest

import paged_kv_cache_112_gb300 as pkv
from paged_kv_cache_112_gb300 import build as pkv_build
from tests import window_ref as R


@pytest.fixture(scope="module")
def lib():
    try:
        pkv_build.build()
    except RuntimeError as e:  # no nvcc on this machine
        pytest.skip(str(e))
    return pkv.load()


def test_grids():
    assert R.E4M3[1] == 2.0 ** -9 and R.E4M3[126] == 448 and np.isnan(R.E4M3[127])
    assert [R.E2M1[R.nearest(np.array(x), R.E2M1[:8])] for x in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 5.01, 99)] == [
        0, 1, 1, 2, 2, 4, 4, 6, 6]


def test_quantised_rows_are_near_and_pack_and_unpack():
    rng = np.random.default_rng(0)
    x = (rng.normal(size=(3, 32, 2, 64)) * np.exp(rng.normal(size=(3, 32, 2, 1)))).astype(np.float32)
    hs = np.array([0.7, 4.0], np.float32)
    code, scale = R.quantise(x, hs)
    pool = R.pack(code.transpose(0, 2, 1, 3), scale.transpose(0, 2, 1, 3))
    assert pool.shape == (3, 2, 2, 9 * 64)
    y = R.values(pool, 64, hs)
    top = np.abs(x).reshape(3, 32, 2, 4, 16).max(-1).repeat(16, -1)
    # Half the widest step (1 of 6) and the scale's rounding of 2^-4.
    assert np.all(np.abs(y - x) <= top * (1 / 6) * (1 + 2.0 ** -4) + 1e-6)


def test_a_window_of_everything_is_causal_and_sinks_stay():
    assert np.array_equal(R.visible(9, 20, 64, 0), np.arange(20) <= 9)
    assert np.nonzero(R.visible(9, 20, 3, 2))[0].tolist() == [0, 1, 7, 8, 9]
    assert np.nonzero(R.visible(3, 20, 3, 9))[0].tolist() == [0, 1, 2, 3]


FAKE = 0x10000  # never dereferenced: validation fails before any device work


def test_fp4_refusals(lib):
    w = lambda **kw: lib.pkv_write_cache_fp4(kw.get("k", FAKE), FAKE, kw.get("kp", FAKE), FAKE, kw.get("ks", None),
                                             kw.get("vs", None), FAKE, kw.get("T", 4), kw.get("stride", 0),
                                             kw.get("H", 8), kw.get("D", 128), kw.get("B", 16), 100, kw.get("L", 1),
                                             kw.get("dt", pkv.PKV_BF16), None, None)
    assert w(T=0) == pkv.PKV_OK
    assert w(D=96) == w(B=8) == w(B=128) == pkv.PKV_ERR_UNSUPPORTED
    assert w(L=0) == w(L=4097) == w(T=-1) == w(H=0) == w(k=None) == w(kp=FAKE + 8) == pkv.PKV_ERR_INVALID_ARG
    assert w(H=2 ** 20, L=4096) == pkv.PKV_ERR_UNSUPPORTED  # more records than 32 bits number
    assert w(ks=FAKE + 2) == w(vs=FAKE + 1) == w(stride=100) == w(dt=pkv.PKV_F32) == pkv.PKV_ERR_INVALID_ARG

    n = lambda **kw: lib.pkv_norm_rope_write_fp4(
        kw.get("qo", FAKE), 0, None, 0, FAKE, 0, FAKE, FAKE, 0, None, None, 0.0, kw.get("cs", FAKE), FAKE, 10,
        kw.get("rot", 64), kw.get("inter", 0), FAKE, FAKE, kw.get("ks", None), None, FAKE, kw.get("T", 4),
        kw.get("Hq", 8), 2, kw.get("D", 128), kw.get("B", 16), 100, kw.get("L", 1), pkv.PKV_BF16, None, None)
    assert n(T=0) == pkv.PKV_OK
    assert n(B=8) == n(rot=24) == n(D=96) == pkv.PKV_ERR_UNSUPPORTED
    assert n(qo=None) == n(cs=None) == n(Hq=0) == n(inter=2) == n(L=0) == n(ks=FAKE + 2) == pkv.PKV_ERR_INVALID_ARG

    c = lambda **kw: lib.pkv_copy_blocks_fp4(FAKE, FAKE, kw.get("pairs", FAKE), kw.get("P", 3), kw.get("L", 1), 8,
                                             kw.get("D", 128), kw.get("B", 16), 100, None, None)
    assert c(P=0) == pkv.PKV_OK
    assert c(B=8) == c(D=80) == pkv.PKV_ERR_UNSUPPORTED
    assert c(L=0) == c(pairs=None) == c(P=-1) == pkv.PKV_ERR_INVALID_ARG

    d = lambda **kw: lib.pkv_decode_attention_fp4(
        FAKE, kw.get("q", FAKE), FAKE, FAKE, kw.get("ks", None), None, FAKE, kw.get("maxb", 4), FAKE, kw.get("S", 2),
        kw.get("Hq", 8), 2, kw.get("D", 128), kw.get("B", 16), 10, kw.get("L", 1), kw.get("scale", 0.1),
        kw.get("ps", 0), kw.get("maxlen", 64), kw.get("ws", None), kw.get("wsb", 0), kw.get("qd", pkv.PKV_BF16),
        kw.get("od", pkv.PKV_F32), None, None)
    assert d(S=0) == pkv.PKV_OK
    assert d(ps=-1) == d(ps=24) == d(B=8) == d(D=96) == d(Hq=7) == d(Hq=18) == pkv.PKV_ERR_UNSUPPORTED
    assert d(ps=-2) == d(q=None) == d(q=FAKE + 8) == d(ks=FAKE + 2) == d(L=0) == pkv.PKV_ERR_INVALID_ARG
    assert d(scale=float("inf")) == d(qd=pkv.PKV_F32) == d(od=7) == pkv.PKV_ERR_INVALID_ARG
    need = pkv.decode_workspace_bytes(2, 8, 128, 64, 16)
    assert d(ps=16) == d(ps=16, ws=FAKE, wsb=need - 1) == d(ps=16, ws=FAKE + 8, wsb=need) == pkv.PKV_ERR_WORKSPACE


def test_window_refusals(lib):
    d = lambda **kw: lib.pkv_decode_window(
        FAKE, kw.get("q", FAKE), FAKE, FAKE, kw.get("bs", 0), kw.get("bt", FAKE), 4, FAKE, kw.get("S", 2),
        kw.get("Hq", 8), 2, kw.get("D", 128), kw.get("B", 16), 10, kw.get("scale", 0.1), kw.get("window", 16),
        kw.get("sinks", 0), kw.get("maxlen", 64), kw.get("kd", pkv.PKV_BF16), pkv.PKV_F32, None, None)
    f = lambda **kw: lib.pkv_decode_window_fp4(
        FAKE, kw.get("q", FAKE), FAKE, FAKE, None, kw.get("vs", None), kw.get("bt", FAKE), 4, FAKE, kw.get("S", 2),
        kw.get("Hq", 8), 2, kw.get("D", 128), kw.get("B", 16), 10, kw.get("L", 1), kw.get("scale", 0.1),
        kw.get("window", 16), kw.get("sinks", 0), kw.get("maxlen", 64), kw.get("kd", pkv.PKV_BF16), pkv.PKV_F32, None,
        None)
    for call in (d, f):
        assert call(S=0) == pkv.PKV_OK
        assert call(B=8) == call(D=96) == call(Hq=7) == call(Hq=18) == pkv.PKV_ERR_UNSUPPORTED
        assert call(window=0) == call(window=-1) == call(sinks=-1) == call(bt=None) == pkv.PKV_ERR_INVALID_ARG
        assert call(q=FAKE + 4) == call(kd=pkv.PKV_F32) == call(maxlen=-1) == call(S=-1) == pkv.PKV_ERR_INVALID_ARG
    assert d(bs=16 * 2 * 128 - 8) == pkv.PKV_ERR_INVALID_ARG
    assert f(L=0) == f(vs=FAKE + 2) == pkv.PKV_ERR_INVALID_ARG


def test_prefill_refusals(lib):
    def c(**kw):
        a = dict(out=FAKE, q=FAKE, qst=0, k=FAKE, bs=0, bt=FAKE, cl=FAKE, qs=FAKE, S=2, T=10, Hq=8, Hkv=2, D=128, B=16,
                 scale=0.1, window=0, sinks=0, maxlen=64, kd=pkv.PKV_BF16, od=pkv.PKV_F32)
        a.update(kw)
        return lib.pkv_prefill_attention(a["out"], a["q"], a["qst"], a["k"], FAKE, a["bs"], a["bt"], 4, a["cl"], a["qs"],
                                         a["S"], a["T"], a["Hq"], a["Hkv"], a["D"], a["B"], 10, a["scale"], a["window"],
                                         a["sinks"], a["maxlen"], a["kd"], a["od"], None, None)

    assert c(S=0) == c(T=0) == c(T=0, out=None) == pkv.PKV_OK
    assert c(B=12) == c(D=96) == c(Hq=7) == c(Hq=18) == c(T=2 ** 31 - 1, Hkv=8) == pkv.PKV_ERR_UNSUPPORTED
    assert c(window=-1) == c(sinks=-1) == c(T=-1) == c(S=-1) == c(maxlen=-1) == pkv.PKV_ERR_INVALID_ARG
    assert c(q=None) == c(out=None) == c(qs=None) == c(cl=None) == c(bt=None) == pkv.PKV_ERR_INVALID_ARG
    assert c(q=FAKE + 8) == c(out=FAKE + 8) == c(qs=FAKE + 2) == c(k=FAKE + 8) == pkv.PKV_ERR_INVALID_ARG
    assert c(qst=1000) == c(qst=1028) == c(bs=8) == c(kd=pkv.PKV_F32) == pkv.PKV_ERR_INVALID_ARG
    assert c(scale=float("nan")) == pkv.PKV_ERR_INVALID_ARG
