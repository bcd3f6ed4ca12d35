"""4-bit pools on the GPU: writes bit for bit, decode against float64."""
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


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def pool(NB, H, B, D, fill=0xA5, layers=0):
    shape = (NB, layers, H, B // 16, 9 * D) if layers else (NB, H, B // 16, 9 * D)
    return torch.full(shape, fill, dtype=torch.uint8, device="cuda")


def random_pool(rng, NB, H, B, D, scale=1.0):
    code, sc = R.quantise((rng.normal(size=(NB, B, H, D)) * scale).astype(np.float32))
    return R.pack(code.transpose(0, 2, 1, 3), sc.transpose(0, 2, 1, 3))


def rows(rng, T, H, D, dt, odd=True):
    """Rows of all magnitudes; with odd ones among them: zeros, subnormal groups, huge ones, infinities and NaN."""
    x = torch.from_numpy(rng.normal(size=(T, H, D)) * np.exp(2 * rng.normal(size=(T, H, 1)))).to(DT[dt])
    if odd:
        x[0, 0, :16] = 0
        x[0, 0, 16:32] *= 1e-4
        x[T // 2, -1, 5] = float("inf")
        x[T // 2, 0, 16:32] = 30000.0
        x[T - 1, 0, 3] = float("nan")
        x[T - 1, -1, :16] = torch.arange(16) * 0.25  # ties: the group's scale is a power of two and more
    return x


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("H,D,B", [(8, 128, 16), (3, 64, 32), (1, 128, 64), (5, 64, 16)])
@pytest.mark.parametrize("scales", [False, True])
@pytest.mark.parametrize("T", [1, 37, 5000])
def test_write_is_exact(dt, H, D, B, scales, T):
    rng = np.random.default_rng(T + D)
    NB = T // B + 3
    fused = torch.cat([rows(rng, T, H, D, dt, T > 1) for _ in range(2)], 1).cuda()
    k, v = fused[:, :H], fused[:, H:]
    hs = [torch.from_numpy(rng.uniform(0.01, 20, H).astype(np.float32)).cuda() if scales else None for _ in range(2)]
    slots = torch.from_numpy(rng.permutation(NB * B)[:T].astype(np.int32)).cuda()
    if T > 2:
        slots[1] = -1
    kp, vp, st = pool(NB, H, B, D), pool(NB, H, B, D), status()
    pkv.write_cache_fp4(k, v, kp, vp, *hs, slots, status=st)
    assert int(st) == 0
    sl = slots.cpu().numpy()
    on = sl >= 0
    for p, x, s in ((kp, k, hs[0]), (vp, v, hs[1])):
        code, sc = R.quantise(x.float().cpu().numpy(), None if s is None else s.cpu().numpy())
        got_code, got_sc = R.unpack(p.cpu().numpy(), D)
        want_code, want_sc = R.unpack(np.full(p.shape, 0xA5, np.uint8), D)
        want_code, want_sc = want_code.copy(), want_sc.copy()
        want_code[sl[on] // B, :, sl[on] % B] = code[on]
        want_sc[sl[on] // B, :, sl[on] % B] = sc[on]
        assert np.array_equal(got_sc, want_sc)
        real = (want_sc != 127).repeat(16, -1)  # the codes of a NaN group say nothing
        assert np.array_equal(R.E2M1[got_code[real]], R.E2M1[want_code[real]])  # a zero's sign is not specified


@pytest.mark.parametrize("rot,inter", [(128, False), (64, True), (16, False), (48, False), (0, False), (96, True)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T", [3, 2500])
def test_norm_and_rotation(rot, inter, dt, T):
    """q and k as the 16-bit operator gives them; the pool's values near the float32 key (within half a code's step
    of the group's scale, which follows the group's largest), v exact."""
    rng = np.random.default_rng(rot + T)
    H, Hq, D, B = 3, 7, 128, 32
    NB = T // B + 2
    q, k, v = (rows(rng, T, h, D, dt, False).cuda() for h in (Hq, H, H))
    qw, kw = (torch.from_numpy(1 + 0.2 * rng.normal(size=D)).to(DT[dt]).cuda() for _ in range(2))
    cs = torch.from_numpy(rng.uniform(-1, 1, (50, rot)).astype(np.float32)).cuda() if rot else None
    pos = torch.from_numpy(rng.integers(0, 50, T).astype(np.int32)).cuda()
    pos[T // 2] = -1
    slots = torch.from_numpy(rng.permutation(NB * B)[:T].astype(np.int32)).cuda()
    kp, vp, st = pool(NB, H, B, D), pool(NB, H, B, D), status()
    qo, ko, qo16, ko16 = (torch.zeros_like(x) for x in (q, k, q, k))
    more = dict(q_weight=qw, k_weight=kw, cos_sin=cs, positions=pos, interleaved=inter, status=st)
    pkv.norm_rope_write_fp4(q, k, v, kp, vp, None, None, slots, q_out=qo, k_out=ko, **more)
    k16, v16 = (torch.zeros(NB, B, H, D, dtype=DT[dt], device="cuda") for _ in range(2))
    pkv.norm_rope_write(q, k, v, k16, v16, slots, q_out=qo16, k_out=ko16, **more)
    assert int(st) == 0
    assert torch.equal(qo, qo16) and torch.equal(ko, ko16)
    sl = slots.cpu().numpy()
    on = np.arange(T) != T // 2
    code, sc = R.unpack(vp.cpu().numpy(), D)
    want, want_sc = R.quantise(v.float().cpu().numpy())
    assert np.array_equal(R.E2M1[code[sl[on] // B, :, sl[on] % B]], R.E2M1[want[on]])
    assert np.array_equal(sc[sl[on] // B, :, sl[on] % B], want_sc[on])
    assert np.all(code[sl[~on] // B, :, sl[~on] % B] == np.array([5, 10] * (D // 2)))  # 0xA5, as it was
    code, sc = R.unpack(kp.cpu().numpy(), D)
    code, sc = code[sl[on] // B, :, sl[on] % B], sc[sl[on] // B, :, sl[on] % B]
    y = ko.double().cpu().numpy()[on]  # the float32 key rounded to 16 bits: off by half a step
    err = STEP[DT[dt]]
    top = np.abs(y).reshape(*y.shape[:-1], -1, 16).max(-1)
    s = R.E4M3[sc]
    # s is top / 6 to half a step of e4m3 (2^-4 of a normal number, 2^-10 below 2^-6) and top's own error
    assert np.all(np.abs(s - top / 6) <= top / 6 * (2.0 ** -4 + 2 * err) + 2.0 ** -10 * (top / 6 < 2.0 ** -6))
    s = s.repeat(16, -1)
    a = np.abs(y) / np.maximum(s, 1e-30)
    half = np.where(a < 2, 0.25, np.where(a < 4, 0.5, 1.0)) * s
    assert np.all(np.abs(R.E2M1[code] * s - y) <= half + 2 * err * np.abs(y) + (a >= 2) * (a < 2.1) * 0.25 * s
                  + (a >= 4) * (a < 4.1) * 0.5 * s)


def test_all_layer_pools_and_copies():
    """A layer's view of an all-layer pool; copy-on-write of whole blocks; swap of the same bytes."""
    rng = np.random.default_rng(4)
    NB, LY, H, B, D = 6, 3, 2, 32, 64
    kp, vp, st = pool(NB, H, B, D, layers=LY), pool(NB, H, B, D, layers=LY), status()
    kp.copy_(torch.from_numpy(rng.integers(0, 256, kp.shape, dtype=np.uint8)))
    before = kp.clone()
    k = rows(rng, 40, H, D, "bf16", False).cuda()
    slots = torch.arange(40, dtype=torch.int32, device="cuda") + 2 * B
    pkv.write_cache_fp4(k, k, kp[:, 1], vp[:, 1], None, None, slots, status=st)
    assert torch.equal(kp[:, 0], before[:, 0]) and torch.equal(kp[:, 2], before[:, 2])
    assert torch.equal(kp[:2], before[:2]) and torch.equal(kp[2:4, 1], vp[2:4, 1]) is False  # 24 rows are not written
    code, _ = R.unpack(kp[:, 1].cpu().numpy(), D)
    want, _ = R.quantise(k.float().cpu().numpy())
    assert np.array_equal(R.E2M1[code[2]].transpose(1, 0, 2), R.E2M1[want[:32]])
    assert np.array_equal(R.E2M1[code[3]].transpose(1, 0, 2)[:8], R.E2M1[want[32:]])
    pairs = torch.tensor([[2, 5], [3, 0]], dtype=torch.int32, device="cuda")
    at = kp.clone()
    pkv.copy_blocks_fp4(kp, vp, pairs, status=st)
    at[5], at[0] = at[2], at[3]
    assert torch.equal(kp, at) and int(st) == 0
    host = torch.zeros(2, LY, H, B // 16, 9 * D, dtype=torch.uint8).pin_memory()
    host_v = torch.zeros_like(host).pin_memory()
    out = torch.tensor([[5, 1]], dtype=torch.int32, device="cuda")
    pkv.swap_blocks(host, host_v, kp, vp, out, status=st)
    torch.cuda.synchronize()
    assert torch.equal(host[1], kp[5].cpu()) and int(st) == 0
    bad = torch.tensor([[2, 6]], dtype=torch.int32, device="cuda")
    pkv.copy_blocks_fp4(kp, vp, bad, status=st)
    assert int(st) == pkv.DEV_ERR_PAIR and torch.equal(kp, at)


class Decode:
    """A batch over 4-bit or 16-bit pools with scattered blocks; whatever no query sees is NaN."""

    def __init__(self, lens, Hq=8, Hkv=2, D=128, B=16, dt="bf16", bits=4, scales=False, seed=0, out=torch.float32,
                 magnitude=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.B, self.D, self.bits = np.asarray(lens), B, D, bits
        n = -(-self.lens // B)
        self.NB = int(n.sum()) + 3
        perm = rng.permutation(self.NB)
        self.width = max(1, int(n.max())) + 1
        tables, at = np.full((len(lens), self.width), -7, np.int32), 0
        for i, m in enumerate(n):
            tables[i, :m] = perm[at:at + m]
            at += m
        self.tables = tables
        self.hs = [rng.uniform(0.3, 3, Hkv).astype(np.float32) if scales else None for _ in range(2)]
        if bits == 4:
            self.pools = [random_pool(rng, self.NB, Hkv, B, D, magnitude) for _ in range(2)]
            self.vals = [R.values(p, D, s) for p, s in zip(self.pools, self.hs)]
            self.dev = [torch.from_numpy(p).cuda() for p in self.pools]
        else:
            t = [torch.from_numpy(rng.normal(size=(self.NB, B, Hkv, D)) * magnitude).to(DT[dt]) for _ in range(2)]
            self.vals = [x.double().numpy() for x in t]
            self.dev = [x.cuda() for x in t]
        self.q = torch.from_numpy(rng.normal(size=(len(lens), Hq, D)) * 1.5).to(DT[dt]).cuda()
        self.dh = [None if s is None else torch.from_numpy(s).cuda() for s in self.hs]
        self.out = torch.full((len(lens), Hq, D), float("nan"), dtype=out, device="cuda")
        self.st, self.scale = status(), D ** -0.5
        self.dt_tables, self.dt_lens = torch.from_numpy(tables).cuda(), torch.from_numpy(
            self.lens.astype(np.int32)).cuda()
        self.max_len = max(1, int(self.lens.max()))
        self.weights = 2.0 ** -11 if bits == 4 else 2.0 ** -16  # of the type that holds a softmax weight

    def poison(self, i, t, value=None):
        """Token t of sequence i becomes NaN (or `value`) in both pools."""
        blk, off = self.tables[i, t // self.B], t % self.B
        for p in self.dev:
            if self.bits == 4:
                p[blk, :, off // 16, 8 * self.D + off % 16 * (self.D // 16):][:, :self.D // 16] = 0x7F
            else:
                p[blk, off] = float("nan") if value is None else value

    def attend(self, **kw):
        ps = kw.pop("partition_size", 0)
        need = pkv.decode_workspace_bytes(*self.q.shape, self.max_len, ps) if ps else 0
        self.ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None
        pkv.decode_attention_fp4(self.out, self.q, *self.dev, *self.dh, self.dt_tables, self.dt_lens, self.scale,
                                 partition_size=ps, max_context_len=self.max_len, workspace=self.ws, status=self.st,
                                 **kw)

    def window(self, window, sinks, **kw):
        more = dict(window=window, sinks=sinks, max_context_len=self.max_len, status=self.st, **kw)
        if self.bits == 4:
            pkv.decode_window_fp4(self.out, self.q, *self.dev, *self.dh, self.dt_tables, self.dt_lens, self.scale,
                                  **more)
        else:
            pkv.decode_window(self.out, self.q, *self.dev, self.dt_tables, self.dt_lens, self.scale, **more)

    def check(self, window=0, sinks=0, lens=None, want_status=0):
        torch.cuda.synchronize()
        assert int(self.st.item()) == want_status
        got, q = self.out.double().cpu().numpy(), self.q.double().cpu().numpy()
        for i, L in enumerate(self.lens if lens is None else lens):
            blocks = self.tables[i, :-(-L // self.B)]
            k, v = (x[blocks].reshape(-1, *x.shape[2:])[:L] for x in self.vals)
            want, extra = R.attend(q[i], k, v, self.scale, R.visible(L - 1, L, window, sinks))
            far = R.bound(want, extra, self.D, L, self.weights, STEP[self.out.dtype],
                          2.0 ** -33 if self.bits == 4 else 2.0 ** -39)
            assert np.all(np.abs(got[i] - want) <= far), (i, L, np.nanmax(np.abs(got[i] - want) / far))


LENS = [0, 1, 15, 16, 17, 31, 33, 64, 100, 257, 1000]


@pytest.mark.parametrize("Hq,Hkv,D,B", [(8, 2, 128, 16), (3, 3, 64, 32), (16, 2, 64, 16), (5, 1, 128, 64),
                                        (14, 2, 128, 32)])
@pytest.mark.parametrize("dt,out", [("bf16", torch.bfloat16), ("f16", torch.float32), ("f16", torch.float16)])
@pytest.mark.parametrize("ps", [0, 16, 48, 256, 1024])
def test_decode(Hq, Hkv, D, B, dt, out, ps):
    d = Decode(LENS, Hq, Hkv, D, B, dt, scales=ps == 48, out=out, seed=ps)
    for i, L in enumerate(LENS):  # rows behind the sequence's end, in its last block
        if L % B:
            d.poison(i, L)
    d.attend(partition_size=ps)
    d.check()


def test_decode_long_and_magnitudes():
    """Long histories over many partitions; head scales that carry the values' magnitude; loud queries."""
    d = Decode([20000, 3], 4, 1, scales=True, seed=9)
    d.hs = [np.float32([1e-4]), np.float32([3e4])]
    d.dh = [torch.from_numpy(s).cuda() for s in d.hs]
    d.vals = [R.values(p, 128, s) for p, s in zip(d.pools, d.hs)]
    d.q *= 20000.0
    d.attend(partition_size=512)
    d.check()


def test_decode_layers_view():
    d = Decode([300, 40], 8, 2, 128, 16, seed=2)
    whole = [torch.zeros(d.NB, 3, *p.shape[1:], dtype=torch.uint8, device="cuda") for p in d.dev]
    for w, p in zip(whole, d.dev):
        w[:, 2] = p
    d.dev = [w[:, 2] for w in whole]
    d.attend(partition_size=64)
    d.check()
    d.window(100, 5)
    d.check(100, 5)


def test_pools_past_four_gigabytes():
    """Records whose bytes lie past 2^32: written, read whole and through a window."""
    H, D, B, n = 8, 128, 16, 100
    NB = (1 << 32) // (B * H * D * 9 // 16) + 50
    kp, vp = (torch.zeros(NB, H, 1, 9 * D, dtype=torch.uint8, device="cuda") for _ in range(2))
    rng = np.random.default_rng(5)
    k, v = rows(rng, n, H, D, "bf16", False), rows(rng, n, H, D, "bf16", False)
    blocks = np.arange(NB - 1, NB - 1 - 7, -1).astype(np.int32)
    slots = blocks[np.arange(n) // B] * B + np.arange(n) % B
    st = status()
    pkv.write_cache_fp4(k.cuda(), v.cuda(), kp, vp, None, None, torch.from_numpy(slots.astype(np.int32)).cuda(), status=st)
    vals = []
    for x in (k, v):
        code, sc = R.quantise(x.float().numpy())
        vals.append(R.E2M1[code] * R.E4M3[sc].repeat(16, -1))
    q = torch.from_numpy(rng.normal(size=(1, 8, D))).bfloat16().cuda()
    out, win = (torch.zeros(1, 8, D, device="cuda") for _ in range(2))
    tables, lens = torch.from_numpy(blocks[None]).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda")
    ws = torch.zeros(pkv.decode_workspace_bytes(1, 8, D, n, 32), dtype=torch.uint8, device="cuda")
    pkv.decode_attention_fp4(out, q, kp, vp, None, None, tables, lens, 0.1, partition_size=32, max_context_len=n,
                             workspace=ws, status=st)
    pkv.decode_window_fp4(win, q, kp, vp, None, None, tables, lens, 0.1, window=30, sinks=1, max_context_len=n, status=st)
    assert int(st.item()) == 0
    for got, w, f in ((out, 0, 0), (win, 30, 1)):
        want, extra = R.attend(q[0].double().cpu().numpy(), *vals, 0.1, R.visible(n - 1, n, w, f))
        far = R.bound(want, extra, D, n, 2.0 ** -11, 2.0 ** -24, 2.0 ** -33)
        assert np.all(np.abs(got[0].double().cpu().numpy() - want) <= far)


@pytest.mark.parametrize("D", [64, 128])
def test_many_units_and_repeated_calls(D):
    """More partitions than the device holds at once, called again on the same workspace."""
    d = Decode([3000 + 37 * (i % 7) for i in range(40)], 8, 4, D, out=torch.bfloat16, seed=8)
    for _ in range(2):
        d.attend(partition_size=128)
    d.check()


@pytest.mark.parametrize("lens,Hkv,D,ps", [([40000, 1, 0, 333], 8, 128, 1024), ([50000, 49999], 4, 64, 1024),
                                           ([4000, 900], 2, 128, 256), ([4000, 900], 2, 64, 256)])
def test_a_visible_nan_stays_one(lens, Hkv, D, ps):
    """In partitions (long histories of many heads) and whole: the heads that meet a NaN scale give no numbers, the
    others are as ever."""
    d = Decode(lens, 2 * Hkv, Hkv, D, seed=ps)
    d.attend(partition_size=ps)
    d.check()
    assert bool((d.ws != 0xFF).any()) == (max(lens) > 10000)  # the workspace holds what the partitions gave
    t = lens[0] // 2
    d.dev[0][d.tables[0, t // 16], 1, 0, 8 * D + t % 16 * (D // 16)] = 0x7F
    before = d.out.clone()
    d.attend(partition_size=ps)
    bad = torch.isnan(d.out)
    assert bool(bad[0, 2:4].all()) and int(bad.sum()) == 2 * D
    assert torch.equal(d.out[~bad], before[~bad])


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_other_scales(bits, scale):
    """A scale of 0 (every visible token alike) and a negative one."""
    d = Decode([0, 1, 100, 700], 8, 2, bits=bits, seed=3)
    d.scale = scale
    d.window(60, 5)
    d.check(60, 5)
    if bits == 4:
        for ps in (0, 64):
            d.attend(partition_size=ps)
            d.check()


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("window", [40, 3900])
def test_a_nan_in_the_window_stays_one(bits, window):
    d = Decode([4000, 900], 8, 4, bits=bits, seed=window)
    d.window(window, 4)
    before = d.out.clone()
    d.poison(0, 3985)
    d.window(window, 4)
    assert bool(torch.isnan(d.out[0]).all()) and torch.equal(d.out[1], before[1])


def test_bad_tables_and_lengths():
    d = Decode([200, 300, 50], 8, 2, seed=5)
    keep = d.tables.copy()
    d.dt_tables[1, 3] = d.NB
    d.attend(partition_size=64)
    assert int(d.st.item()) == pkv.DEV_ERR_BLOCK
    d.st.zero_()
    d.dt_tables.copy_(torch.from_numpy(keep))
    d.dt_lens.copy_(torch.tensor([-5, 10000, 50], dtype=torch.int32))
    d.attend(partition_size=64)
    cap = min(d.max_len, d.width * 16)
    d.check(lens=[0, cap, 50], want_status=pkv.DEV_ERR_LENGTH)


def test_empty_batch_and_no_table():
    d = Decode([0, 0], 8, 2, seed=1)
    d.dt_tables = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    d.attend()
    d.check()
    d.window(4, 4)
    d.check()


@pytest.mark.parametrize("Hq,Hkv,D,B,bits,dt", [(8, 2, 128, 16, 16, "bf16"), (8, 2, 128, 16, 4, "bf16"),
                                                (3, 3, 64, 32, 16, "f16"), (16, 2, 64, 64, 4, "f16"),
                                                (7, 1, 128, 64, 16, "f16")])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (17, 16), (40, 33), (100, 130), (256, 0), (4000, 7),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (3, 260)])
def test_window(Hq, Hkv, D, B, bits, dt, window, sinks):
    """Windows that end anywhere in tiles and blocks; sinks before, beside and across the window; what is not
    seen is NaN, and entries of blocks without a visible token are no blocks at all."""
    d = Decode(LENS, Hq, Hkv, D, B, dt, bits, scales=bits == 4, seed=window % 97)
    for i, L in enumerate(LENS):
        see = R.visible(L - 1, -(-L // B) * B, window, sinks)
        for t in np.nonzero(~see)[0]:
            d.poison(i, int(t), float("inf") if t % 2 else None)
        seen = see.reshape(-1, B).any(1)
        d.dt_tables[i, :len(seen)] = torch.where(torch.from_numpy(seen).cuda(), d.dt_tables[i, :len(seen)], -99)
    d.window(window, sinks)
    d.check(window, sinks)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("S,L,window", [(1, 9000, 8000), (40, 3000, 2000), (200, 500, 300), (3, 30000, 29000)])
def test_window_batches(bits, S, L, window):
    """From one sequence on clusters of eight to more units than the device holds."""
    d = Decode([L - 7 * (i % 5) for i in range(S)], 4, 1, bits=bits, seed=S, out=torch.bfloat16)
    for _ in range(2):
        d.window(window, 20)
        d.check(window, 20)


@pytest.mark.parametrize("bits", [4, 16])
def test_window_bad_entries_and_lengths(bits):
    d = Decode([200, 300], 8, 2, bits=bits, seed=5)
    d.dt_tables[1, 18] = -2
    d.window(32, 4)
    torch.cuda.synchronize()
    assert int(d.st.item()) == pkv.DEV_ERR_BLOCK
    d.st.zero_()
    d.dt_lens[0], d.dt_lens[1] = -1, 0
    d.window(32, 4)
    d.check(32, 4, lens=[0, 0], want_status=pkv.DEV_ERR_LENGTH)


def test_serving_loop_with_graph_replay():
    """Tokens appended one by one across blocks, a copy-on-write in between, decode of all and of a window from one
    captured graph on another stream, against the statement of what was written."""
    rng = np.random.default_rng(7)
    H, Hq, D, B, NB, S = 2, 8, 128, 16, 40, 3
    kp, vp, st = pool(NB, H, B, D, 0xFF), pool(NB, H, B, D, 0xFF), status()
    bm = pkv.BlockManager(NB, B)
    hs = torch.tensor([0.5, 2.0], device="cuda")
    history = {}
    for s, n in enumerate((30, 17)):
        _, slots = bm.add_sequence(s, rng.integers(0, 1000, n))
        k, v = rows(rng, n, H, D, "bf16", False), rows(rng, n, H, D, "bf16", False)
        pkv.write_cache_fp4(k.cuda(), v.cuda(), kp, vp, hs, None, torch.from_numpy(slots).cuda(), status=st)
        history[s] = [k, v]
    bm.fork(0, 2)
    history[2] = [x.clone() for x in history[0]]
    q, k, v = (torch.zeros(S, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hq, H, H))
    qo, out, win = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
    slots, lens = (torch.zeros(S, dtype=torch.int32, device="cuda") for _ in range(2))
    tables = torch.zeros(S, 8, dtype=torch.int32, device="cuda")
    ws = torch.zeros(pkv.decode_workspace_bytes(S, Hq, D, 128, 32), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()

    def step():
        pkv.norm_rope_write_fp4(q, k, v, kp, vp, hs, None, slots, q_out=qo, status=st)
        pkv.decode_attention_fp4(out, qo, kp, vp, hs, None, tables, lens, D ** -0.5, partition_size=32,
                                 max_context_len=128, workspace=ws, status=st)
        pkv.decode_window_fp4(win, qo, kp, vp, hs, None, tables, lens, D ** -0.5, window=20, sinks=3,
                              max_context_len=128, status=st)

    graph = None
    for i in range(20):
        sl, ln, tb, pairs = bm.decode_step([0, 1, 2], rng.integers(0, 1000, 3), 8)
        if len(pairs):
            pkv.copy_blocks_fp4(kp, vp, torch.from_numpy(pairs).cuda(), status=st)
        new = [rows(rng, S, h, D, "bf16", False) for h in (Hq, H, H)]
        for a, b in zip((q, k, v), new):
            a.copy_(b)
        for s in range(S):
            history[s] = [torch.cat([a, b[s:s + 1]]) for a, b in zip(history[s], new[1:])]
        slots.copy_(torch.from_numpy(sl)), lens.copy_(torch.from_numpy(ln)), tables.copy_(torch.from_numpy(tb))
        if i == 2:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                step()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay() if graph else step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        for s in range(S):
            vals = []
            for x, hsc in zip(history[s], (hs.cpu().numpy(), None)):
                code, sc = R.quantise(x.float().numpy(), hsc)
                p = R.pack(code.transpose(1, 0, 2)[None, :, :len(x) // 16 * 16], sc.transpose(1, 0, 2)[
                    None, :, :len(x) // 16 * 16])
                val = R.E2M1[code] * R.E4M3[sc].repeat(16, -1)
                vals.append(val if hsc is None else val * hsc[:, None].astype(np.float64))
                assert np.array_equal(R.values(p, D)[0], val[:len(x) // 16 * 16])
            for got, w, f in ((out, 0, 0), (win, 20, 3)):
                n = len(vals[0])
                want, extra = R.attend(q[s].double().cpu().numpy(), *vals, D ** -0.5, R.visible(n - 1, n, w, f))
                far = R.bound(want, extra, D, n, 2.0 ** -11, 2.0 ** -8, 2.0 ** -33)
                assert np.all(np.abs(got[s].double().cpu().numpy() - want) <= far)


def test_refusals_of_tensors():
    d = Decode([40], 8, 2)
    p = d.dev[0]
    call = lambda **kw: pkv.decode_window_fp4(
        kw.get("out", d.out), kw.get("q", d.q), kw.get("k", p), kw.get("v", d.dev[1]), kw.get("ks"), None,
        kw.get("bt", d.dt_tables), d.dt_lens, 0.1, window=kw.get("window", 4), max_context_len=40)
    call()
    for bad in (dict(k=p[..., :-1]), dict(k=p.cpu()), dict(v=p[:-1]), dict(q=d.q[:, :, :64]), dict(q=d.q.float()),
                dict(ks=torch.ones(3, device="cuda")), dict(ks=torch.ones(2, device="cuda").double()),
                dict(bt=d.dt_tables.long()), dict(bt=d.dt_tables[:0]), dict(window=0), dict(window=1.5),
                dict(out=d.out[:, :4]), dict(k=p.transpose(1, 2))):
        with pytest.raises(pkv.PkvError):
            call(**bad)
    k = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in ((k[:, :1], k, slots), (k, k[:, :, :64], slots), (k.float(), k.float(), slots), (k, k, slots[:3]),
                (k, k.half(), slots), (k, k, slots.long())):
        with pytest.raises(pkv.PkvError):
            pkv.write_cache_fp4(bad[0], bad[1], p, d.dev[1], None, None, bad[2])
