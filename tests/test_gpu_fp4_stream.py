"""Writes of long prompts into 4-bit pools: from 320 groups of heads a SM on, another kernel streams the rows through
shared memory (a group: as many heads as a warp holds, 4 of 128 channels or 8 of 64)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_112_gb300 as pkv
from tests import test_gpu_fp4 as few
from tests import window_ref as R
from tests.test_gpu_fp4 import DT, pool, rows, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load(build_if_missing=True)


def streamed(heads, D, more=37):
    """Tokens that take the streaming kernel: the least, and some more."""
    groups = -(-heads * D // 512)
    return -(-320 * torch.cuda.get_device_properties(0).multi_processor_count // groups) + more


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("H,D,B,scales", [(8, 128, 16, True), (5, 128, 64, False), (5, 64, 32, True), (16, 64, 16, False)])
def test_write_is_exact(dt, H, D, B, scales):
    """Code for code and scale for scale; head counts that do not fill the last group, tokens without a slot, NaN and
    infinite rows, rows of a wider projection."""
    T = streamed(2 * H, D)
    rng = np.random.default_rng(T)
    NB = T // B + 3
    wide = torch.cat([rows(rng, T, H, D, dt) for _ in range(2)] + [torch.full((T, 3, D), float("nan")).to(DT[dt])], 1).cuda()
    k, v = wide[:, :H], wide[:, H:2 * H]
    hs = [torch.from_numpy(rng.uniform(0.01, 20, H).astype(np.float32)).cuda() if scales else None for _ in range(2)]
    slots = torch.from_numpy(rng.permutation(NB * B)[:T].astype(np.int32)).cuda()
    slots[1], slots[T // 3:T // 3 + 200], slots[T - 2] = -1, -1, -1
    kp, vp, st = pool(NB, H, B, D), pool(NB, H, B, D), status()
    pkv.write_cache_fp4(k, v, kp, vp, *hs, slots, status=st)
    assert int(st) == 0
    sl = slots.cpu().numpy()
    on = sl >= 0
    for p, x, s in ((kp, k, hs[0]), (vp, v, hs[1])):
        code, sc = R.quantise(x.float().cpu().numpy(), None if s is None else s.cpu().numpy())
        got_code, got_sc = R.unpack(p.cpu().numpy(), D)
        want_code, want_sc = (a.copy() for a in R.unpack(np.full(p.shape, 0xA5, np.uint8), D))
        want_code[sl[on] // B, :, sl[on] % B] = code[on]
        want_sc[sl[on] // B, :, sl[on] % B] = sc[on]
        assert np.array_equal(got_sc, want_sc)
        real = (want_sc != 127).repeat(16, -1)  # the codes of a NaN group say nothing
        assert np.array_equal(R.E2M1[got_code[real]], R.E2M1[want_code[real]])


@pytest.mark.parametrize("rot,inter", [(128, False), (64, True), (48, False), (0, False)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_norm_and_rotation(rot, inter, dt):
    """The statements that hold of few tokens (13 heads: the last group holds one)."""
    few.test_norm_and_rotation(rot, inter, dt, streamed(13, 128))


@pytest.mark.parametrize("Hq,Hkv,D,B,rot,inter,dt", [(16, 4, 64, 32, 32, True, "f16"), (9, 3, 64, 16, 64, False, "bf16"),
                                                     (32, 8, 128, 16, 128, False, "bf16"), (6, 1, 128, 64, 16, False, "f16")])
def test_the_same_rows_as_in_short_calls(Hq, Hkv, D, B, rot, inter, dt):
    """All of a prompt at once against calls of few tokens, bit for bit: queries, keys and both pools; padding tokens and
    tokens without a slot, single ones and runs of them, in mid-stream; head scales, NaN and infinite rows."""
    T = streamed(Hq + 2 * Hkv, D)
    rng = np.random.default_rng(T + rot)
    NB = T // B + 3
    wide = torch.cat([rows(rng, T, h, D, dt) for h in (Hq, Hkv, Hkv)], 1).cuda()
    q, k, v = wide[:, :Hq], wide[:, Hq:Hq + Hkv], wide[:, Hq + Hkv:]
    qw, kw = (torch.from_numpy(1 + 0.2 * rng.normal(size=D)).to(DT[dt]).cuda() for _ in range(2))
    cs = torch.from_numpy(rng.uniform(-1, 1, (70, rot)).astype(np.float32)).cuda()
    pos = torch.from_numpy(rng.integers(0, 70, T).astype(np.int32)).cuda()
    slots = torch.from_numpy(rng.permutation(NB * B)[:T].astype(np.int32)).cuda()
    pos[torch.from_numpy(rng.random(T) < 0.1).cuda()] = -1
    slots[torch.from_numpy(rng.random(T) < 0.1).cuda()] = -1
    pos[T // 4:T // 4 + 300], slots[T // 2:T // 2 + 300], pos[T - 5:] = -1, -1, -1
    hs = [torch.from_numpy(rng.uniform(0.3, 3, Hkv).astype(np.float32)).cuda() for _ in range(2)]
    res = []
    for step in (T, 700):
        kp, vp, st = pool(NB, Hkv, B, D), pool(NB, Hkv, B, D), status()
        qo, ko = torch.full_like(q, 7.0).contiguous(), torch.full_like(k, 7.0).contiguous()
        for a in range(0, T, step):
            s = slice(a, min(T, a + step))
            pkv.norm_rope_write_fp4(q[s], k[s], v[s], kp, vp, *hs, slots[s], q_out=qo[s], k_out=ko[s], q_weight=qw,
                                    k_weight=kw, cos_sin=cs, positions=pos[s], interleaved=inter, status=st)
        assert int(st) == 0
        res.append([x.view(torch.uint8) if x.dtype == torch.uint8 else x.view(torch.int16) for x in (qo, ko, kp, vp)])
    for a, b in zip(*res):
        assert torch.equal(a, b)
    assert torch.all(res[0][0][T - 5:] == qo.new_tensor(7.0).view(torch.int16))
