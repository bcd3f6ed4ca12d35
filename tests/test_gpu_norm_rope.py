"""pkv_norm_rope_write(_fp8) against the float64 statement: every element of
q_out, k_out and both pools, rows that must stay as they were among them.

Tolerances.  The float32 path: a sum of D squares, rsqrt (2 ulp), two
products, the rotation's two products and a sum -- fewer than 24 roundings of
2^-24 on terms whose magnitudes add up to m (layer_ref.norm_rope), the norm's
sum included (its D - 1 additions of positive terms form a tree of depth 8 per
lane chain of 16).  So |err| <= 2^-19 m before the one rounding to the output
type, which adds half a step: eps/2 relative, and half the smallest
subnormal.  e4m3: half a step is 2^-4 relative or 2^-10 absolute."""
import numpy as np
import pytest
import torch

import paged_kv_cache_112_gb300 as pkv
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load(build_if_missing=True)


def f64(t):
    return t.detach().double().cpu().numpy()


class Step:
    """Inputs of one call on the GPU and as float64."""

    def __init__(self, seed=0, T=17, Hq=8, Hkv=2, D=128, dtype="bf16", B=16, rot=128, interleaved=False, qw=True,
                 kw=True, fused=False, fp8=False, layers=1, k_out=False, in_place=False, top=4096, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        dt = DT[dtype]
        self.__dict__.update(T=T, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, B=B, rot=rot, interleaved=interleaved, fp8=fp8)
        rand = lambda *s: (torch.randn(*s, generator=g) * scale).to(dt).cuda()
        if fused:
            rows = rand(T, Hq + 2 * Hkv, D)
            self.q, self.k, self.v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        else:
            self.q, self.k, self.v = rand(T, Hq, D), rand(T, Hkv, D), rand(T, Hkv, D)
        self.qw = (1 + 0.3 * torch.randn(D, generator=g)).to(dt).cuda() if qw else None
        self.kw = (1 + 0.3 * torch.randn(D, generator=g)).to(dt).cuda() if kw else None
        self.cs = self.pos = None
        if rot:
            inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
            ang = torch.arange(top, dtype=torch.float64)[:, None] * inv
            self.cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
            self.pos = torch.randint(0, top, (T,), generator=g).to(torch.int32).cuda()
        NB = -(-T // B) + 3
        self.NB = NB
        self.slots = torch.randperm(NB * B, generator=g)[:T].to(torch.int32).cuda()
        shape = (NB, B, Hkv, D) if layers == 1 else (NB, layers, B, Hkv, D)
        at = (slice(None),) if layers == 1 else (slice(None), layers - 1)
        if fp8:
            whole = [torch.randint(0, 255, shape, generator=g, dtype=torch.uint8).cuda() for _ in range(2)]
            ss = shape[:-3] + (Hkv,)
            sc = [(torch.rand(ss, generator=g) * 0.05 + 0.002).cuda() for _ in range(2)]
            self.ks, self.vs = (x[at] for x in sc)
        else:
            whole = [rand(*shape) for _ in range(2)]
        self.whole = whole
        self.kp, self.vp = (x[at] for x in whole)
        self.before = [x.clone() for x in whole]
        self.in64 = [f64(x) for x in (self.q, self.k, self.v)]
        self.q_out = self.q if in_place else torch.full((T, Hq, D), 7.0, dtype=dt, device="cuda")
        self.k_out = (self.k if in_place else torch.full((T, Hkv, D), 7.0, dtype=dt, device="cuda")) if k_out else None
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.at = at

    def call(self, stream=None):
        kw = dict(q_out=self.q_out, k_out=self.k_out, q_weight=self.qw, k_weight=self.kw, eps=1e-5, cos_sin=self.cs,
                  positions=self.pos, interleaved=self.interleaved, status=self.status, stream=stream)
        if self.fp8:
            pkv.norm_rope_write_fp8(self.q, self.k, self.v, self.kp, self.vp, self.ks, self.vs, self.slots, **kw)
        else:
            pkv.norm_rope_write(self.q, self.k, self.v, self.kp, self.vp, self.slots, **kw)

    def check(self, status=0):
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        slots = self.slots.cpu().numpy()
        pos = self.pos.cpu().numpy() if self.rot else np.zeros(self.T, int)
        ok = (pos >= 0) & (pos < (self.cs.shape[0] if self.rot else 1))
        ang = f64(self.cs)[np.where(ok, pos, 0)] if self.rot else None
        q, k, v = self.in64
        w = lambda t: None if t is None else f64(t)
        yq, mq = R.norm_rope(q, w(self.qw), 1e-5, ang, self.interleaved)
        yk, mk = R.norm_rope(k, w(self.kw), 1e-5, ang, self.interleaved)
        half = HALF_STEP[self.dtype]
        for out, y, m, old in ((self.q_out, yq, mq, q if self.q_out is self.q else 7.0),
                               (self.k_out, yk, mk, k if self.k_out is self.k else 7.0)):
            if out is None:
                continue
            got = f64(out)
            tol = half * np.abs(y) + 2.0 ** -19 * m * (1 + half) + TINY[self.dtype]
            assert np.all(np.abs(got - y)[ok] <= tol[ok])
            assert np.array_equal(got[~ok], np.broadcast_to(old, got.shape)[~ok])
        live = ok & (slots >= 0) & (slots < self.NB * self.B)
        b, o = slots[live] // self.B, slots[live] % self.B
        for name, whole, before, y, m in (("k", self.whole[0], self.before[0], yk, mk),
                                          ("v", self.whole[1], self.before[1], v, None)):
            if self.fp8:
                sc = f64(self.ks if name == "k" else self.vs)[b][..., None]
                got = R.E4M3[whole[self.at].cpu().numpy()[b, o]]
                want = np.clip(y[live] / sc, -448, 448)
                err = 2.0 ** -19 * (np.abs(y[live]) if m is None else m[live]) / sc
                assert np.all(np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + err * (1 + 2.0 ** -3))
            elif name == "v":
                bits = lambda t: t.view(torch.int16)
                assert torch.equal(bits(whole)[self.at][torch.from_numpy(b).cuda(), torch.from_numpy(o).cuda()],
                                   torch.from_numpy(v[live]).to(DT[self.dtype]).cuda().view(torch.int16))
            else:
                got = f64(whole[self.at])[b, o]
                tol = half * np.abs(y[live]) + 2.0 ** -19 * m[live] * (1 + half) + TINY[self.dtype]
                assert np.all(np.abs(got - y[live]) <= tol)
            # everything else is as it was
            rest, kept = whole.clone(), before.clone()
            rest[self.at][torch.from_numpy(b).cuda(), torch.from_numpy(o).cuda()] = 0
            kept[self.at][torch.from_numpy(b).cuda(), torch.from_numpy(o).cuda()] = 0
            raw = torch.uint8 if self.fp8 else torch.int16
            assert torch.equal(rest.view(raw), kept.view(raw))


CASES = [
    dict(T=1), dict(T=1, Hq=1, Hkv=1, D=64, rot=64), dict(T=3, Hq=9, Hkv=3, dtype="f16", fused=True),
    dict(T=257, Hq=32, Hkv=8, fused=True), dict(T=64, Hq=64, Hkv=8, dtype="f16", B=32),
    dict(T=33, Hq=15, Hkv=5, D=64, rot=32, interleaved=True, B=64), dict(T=40, rot=16, B=8),
    dict(T=40, rot=64, interleaved=True), dict(T=21, rot=0), dict(T=21, rot=0, qw=False, kw=False),
    dict(T=21, qw=False), dict(T=21, kw=False, dtype="f16"), dict(T=19, k_out=True, fused=True),
    dict(T=19, k_out=True, in_place=True, fused=True, dtype="f16"), dict(T=19, in_place=True, D=64, rot=48),
    dict(T=35, layers=3), dict(T=1025, Hq=5, Hkv=5, D=64, rot=64, fused=True), dict(T=8, scale=1e-4),
    dict(T=8, scale=300.0, dtype="f16", qw=True), dict(T=30, D=128, rot=112, interleaved=True),
]


@pytest.mark.parametrize("kw", CASES)
def test_16_bit_pools(kw):
    s = Step(seed=3, **kw)
    s.call()
    s.check()


@pytest.mark.parametrize("kw", [dict(T=1), dict(T=100, Hq=32, Hkv=8, fused=True), dict(T=45, layers=2, dtype="f16"),
                                dict(T=31, Hq=9, Hkv=3, rot=64, interleaved=True), dict(T=17, D=64, rot=32, Hkv=4),
                                dict(T=17, rot=0, kw=False), dict(T=9, scale=40.0)])
def test_fp8_pools(kw):
    s = Step(seed=5, fp8=True, **kw)
    s.call()
    s.check()


def test_no_tokens():
    s = Step(T=0)
    s.call()
    s.check()


@pytest.mark.parametrize("fp8", [False, True])
def test_padding_and_bad_indices(fp8):
    """Position -1: the token is left alone, whatever its slot; slot -1: the pools are; bad ones set their bits."""
    s = Step(T=24, k_out=True, fp8=fp8)
    s.pos[2] = s.pos[23] = -1
    s.slots[23] = 1 << 30
    s.slots[5] = -1
    s.call()
    s.check()
    s = Step(T=24, k_out=True, fp8=fp8)
    s.pos[3], s.pos[4], s.slots[7], s.slots[8] = 4096, -2, s.NB * 16, -3
    s.call()
    s.check(pkv.DEV_ERR_POSITION | pkv.DEV_ERR_SLOT)


def test_rows_of_zeros_and_non_finite_rows():
    """A row of zeros stays zero; NaN and infinity in one head reach no other head or token."""
    s = Step(T=9, k_out=True)
    s.q[0] = 0
    s.q[4, 3, 5], s.k[6, 1, 9] = float("nan"), float("inf")
    s.call()
    torch.cuda.synchronize()
    assert torch.all(s.q_out[0] == 0)
    bad_q = torch.zeros(9, 8, dtype=torch.bool)
    bad_q[4, 3] = True
    bad_k = torch.zeros(9, 2, dtype=torch.bool)
    bad_k[6, 1] = True
    assert torch.equal(torch.isfinite(s.q_out).all(2).cpu(), ~bad_q)
    assert torch.equal(torch.isfinite(s.k_out).all(2).cpu(), ~bad_k)


def test_equal_to_write_cache_without_norm_and_rotation():
    """rot_dim 0 and no weights: bit for bit what write_cache writes, and q unchanged (16-bit and FP8)."""
    for fp8 in (False, True):
        s = Step(T=50, rot=0, qw=False, kw=False, fp8=fp8)
        o = Step(T=50, rot=0, qw=False, kw=False, fp8=fp8)
        s.call()
        if fp8:
            pkv.write_cache_fp8(o.k, o.v, o.kp, o.vp, o.ks, o.vs, o.slots)
        else:
            pkv.write_cache(o.k, o.v, o.kp, o.vp, o.slots)
        torch.cuda.synchronize()
        raw = torch.uint8 if fp8 else torch.int16
        assert torch.equal(s.kp.view(raw), o.kp.view(raw)) and torch.equal(s.vp.view(raw), o.vp.view(raw))
        assert torch.equal(s.q_out, s.q)


def test_other_streams_and_graph_replays():
    """Two calls on two streams at once; a captured call replayed on new inputs in the same buffers."""
    a, b = Step(seed=1, T=300, Hq=32, Hkv=8), Step(seed=2, T=300, Hq=32, Hkv=8)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a.call(sa)
    b.call(sb)
    a.check()
    b.check()
    s, new = Step(seed=1, T=40, fused=True), Step(seed=9, T=40, fused=True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.call()
    for x, y in ((s.q, new.q), (s.k, new.k), (s.v, new.v), (s.pos, new.pos), (s.slots, new.slots)):
        x.copy_(y)
    s.in64 = new.in64
    g.replay()
    s.check()


def test_refusals():
    s = Step(T=4)
    f = lambda **kw: pkv.norm_rope_write(*[kw.get(n, d) for n, d in (("q", s.q), ("k", s.k), ("v", s.v), ("kp", s.kp),
                                                                      ("vp", s.vp), ("slots", s.slots))],
                                         q_out=kw.get("qo", s.q_out), cos_sin=kw.get("cs", s.cs),
                                         positions=kw.get("pos", s.pos), q_weight=kw.get("qw"))
    for kw in (dict(q=s.q.float()), dict(k=s.k[:, :1]), dict(v=s.v[:3]), dict(qo=s.q_out[:3]), dict(q=s.q.cpu()),
               dict(slots=s.slots.long()), dict(pos=None), dict(pos=s.pos.cpu()), dict(cs=s.cs.double()),
               dict(k=s.k[:1].expand(4, -1, -1)), dict(q=s.q.transpose(0, 1).contiguous().transpose(0, 1)),
               dict(qw=s.qw[:64]), dict(qw=s.qw.float()), dict(kp=s.kp.half()), dict(pos=s.pos[:2]),
               dict(cs=s.cs[:, :100].contiguous()), dict(slots=s.slots[:2])):
        with pytest.raises(pkv.PkvError):
            f(**kw)


def test_arguments_of_the_wrong_kind():
    s = Step(T=4)
    for kw in (dict(interleaved=torch.zeros(2)), dict(eps="small"), dict(eps=None), dict(stream=7),
               dict(status=torch.zeros(1)), dict(q_weight=1.0), dict(eps=float("nan"), q_weight=s.qw)):
        with pytest.raises(pkv.PkvError):
            pkv.norm_rope_write(s.q, s.k, s.v, s.kp, s.vp, s.slots, q_out=s.q_out, cos_sin=s.cs, positions=s.pos, **kw)
    with pytest.raises(pkv.PkvError):
        pkv.norm_rope_write(s.q, s.k, [1.0], s.kp, s.vp, s.slots, q_out=s.q_out, cos_sin=s.cs, positions=s.pos)
    torch.cuda.synchronize()  # nothing was launched and no error is left behind


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_fp8_codes_are_those_of_the_division(dtype):
    """Values and scales whose quotients lie on, next to and far from rounding borders, beyond the largest
    code, among the subnormals, and scales of every size (subnormal, zero, infinite and NaN among them):
    bit for bit write_cache_fp8's codes."""
    g = torch.Generator().manual_seed(3)
    T, Hkv = 512, 8
    s = Step(T=T, Hq=8, Hkv=Hkv, rot=0, qw=False, kw=False, fp8=True, dtype=dtype)
    scales = torch.exp2(torch.randint(-20, 20, s.ks.shape, generator=g).float()) * (
        1 + torch.randint(0, 64, s.ks.shape, generator=g) / 64)
    odd = torch.tensor([1e-39, 2e38, 0.0, float("inf"), float("nan"), 1.0, 3e-38, 2.0 ** 127])
    scales[::3] = odd
    s.ks.copy_(scales)
    s.vs.copy_(scales.flip(0))
    # multiples of half a code step times the block's scale, as near as the type holds them
    b = (s.slots.long() // 16).cpu()
    border = (torch.randint(-127, 128, (T, Hkv, 128), generator=g) / 16) * torch.exp2(
        torch.randint(-8, 8, (T, Hkv, 128), generator=g).float())
    for x, sc in ((s.k, s.ks), (s.v, s.vs)):
        y = border * sc.cpu()[b][..., None]
        x.copy_(torch.nan_to_num(y, nan=1.5, posinf=3.0, neginf=-3.0).clamp(-60000, 60000).to(x.dtype))
    kp, vp = s.kp.clone(), s.vp.clone()
    s.call()
    pkv.write_cache_fp8(s.k, s.v, kp, vp, s.ks, s.vs, s.slots)
    torch.cuda.synchronize()
    assert torch.equal(s.kp, kp) and torch.equal(s.vp, vp)


@pytest.mark.parametrize("T", [24, 3000])
def test_padding_without_rotation(T):
    """Positions count without an angle table too: -1 is padding, other negative ones are reported."""
    s = Step(T=T, rot=0, Hq=32, Hkv=8)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 1000
    pos[5] = pos[T - 1] = -1
    pos[7] = -2
    kp = s.kp.clone()
    pkv.norm_rope_write(s.q, s.k, s.v, s.kp, s.vp, s.slots, q_out=s.q_out, q_weight=s.qw, k_weight=s.kw, eps=1e-5,
                        positions=pos, status=s.status)
    torch.cuda.synchronize()
    assert int(s.status.item()) == pkv.DEV_ERR_POSITION
    left = [5, 7, T - 1]
    assert torch.all(s.q_out[left] == 7.0)
    at = s.slots.long()[left]
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert same(s.kp[at // s.B, at % s.B], kp[at // s.B, at % s.B])
    rest = torch.ones(T, dtype=torch.bool)
    rest[left] = False
    y, m = R.norm_rope(s.in64[0], f64(s.qw), 1e-5, None, False)
    assert np.all((np.abs(f64(s.q_out) - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -18 * m)[rest.numpy()])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw", [dict(T=3001, Hq=32, Hkv=8, fused=True), dict(T=2500, Hq=9, Hkv=3, rot=64, interleaved=True),
                                dict(T=5000, Hq=15, Hkv=5, D=64, rot=48, dtype="f16"),
                                dict(T=1500, Hq=70, Hkv=7, in_place=True, k_out=True, dtype="f16", rot=0, qw=False)])
def test_long_prompts(kw, fp8):
    """Lengths at which rows are streamed, with odd head counts whose last part is ragged, padding tokens and
    bad positions among them."""
    s = Step(seed=7, fp8=fp8, **kw)
    if s.rot:
        s.pos[::501] = -1
        s.pos[17] = 1 << 20
    s.slots[::77] = -1
    s.call()
    s.check(pkv.DEV_ERR_POSITION if s.rot else 0)


def test_pools_past_four_gigabytes():
    """Slots whose rows lie beyond 2^32 bytes and 2^31 elements of the pools."""
    T, Hq, Hkv, D, B, NB = 40, 8, 8, 128, 16, 140000
    s = Step(T=T, Hq=Hq, Hkv=Hkv)
    kp, vp = (torch.empty((NB, B, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = (torch.arange(T, device="cuda") * 55987 + 5).to(torch.int32)
    slots[-1] = NB * B - 1
    pkv.norm_rope_write(s.q, s.k, s.v, kp, vp, slots, q_out=s.q_out, q_weight=s.qw, k_weight=s.kw, cos_sin=s.cs,
                        positions=s.pos, status=s.status)
    pkv.norm_rope_write(s.q, s.k, s.v, s.kp, s.vp, s.slots, q_out=s.q_out, q_weight=s.qw, k_weight=s.kw, cos_sin=s.cs,
                        positions=s.pos, status=s.status)
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    for big, small in ((kp, s.kp), (vp, s.vp)):
        assert torch.equal(big.view(-1, Hkv, D)[slots.long()], small.reshape(-1, Hkv, D)[s.slots.long()])
