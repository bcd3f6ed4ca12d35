"""The layer operators together, as a serving loop uses them: prompts admitted
and decode steps taken through the block manager (prefix sharing, forks with
copy-on-write, a swap to host memory and back), each step one captured graph
of norm + rotation + write, summaries of the blocks it filled, selection and
sparse attention, over a padded batch.  Every step's queries, selection and
attention are compared with the float64 statements over the pools' contents."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_kv_cache_112_gb300 as pkv
from tests import layer_ref as R

pytestmark = pytest.mark.gpu

HQ, HKV, D, B, NB, SLOTS, WIDTH = 8, 2, 128, 16, 160, 5, 40
KEEP, FIRST, LAST = 6, 1, 2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv.load(build_if_missing=True)


def f64(t):
    return t.detach().double().cpu().numpy()


class Layer:
    """One layer's device state and the captured step over SLOTS batch slots."""

    def __init__(self, fp8, seed=0):
        self.fp8, self.g = fp8, torch.Generator().manual_seed(seed)
        self.dt = torch.bfloat16
        if fp8:
            self.kp, self.vp = (torch.full((NB, B, HKV, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
            # the caller's scales; a power of two times 1.25
            self.ks, self.vs = (torch.full((NB, HKV), 1.25 / 64, device="cuda") for _ in range(2))
        else:
            self.kp, self.vp = (torch.full((NB, B, HKV, D), float("nan"), dtype=self.dt, device="cuda")
                                for _ in range(2))
        self.summary = torch.zeros((NB, HKV, 2, D), dtype=torch.int8, device="cuda")
        self.summary_scale = torch.ones((NB, HKV), device="cuda")
        self.qw, self.kw = ((1 + 0.2 * torch.randn(D, generator=self.g)).to(self.dt).cuda() for _ in range(2))
        inv = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
        ang = torch.arange(2048, dtype=torch.float64)[:, None] * inv
        self.cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
        i32 = lambda *s: torch.full(s, -1, dtype=torch.int32, device="cuda")
        self.qkv = torch.zeros((SLOTS, HQ + 2 * HKV, D), dtype=self.dt, device="cuda")
        self.q = torch.zeros((SLOTS, HQ, D), dtype=self.dt, device="cuda")
        self.pos, self.slots, self.filled, self.tables = i32(SLOTS), i32(SLOTS), i32(SLOTS), i32(SLOTS, WIDTH)
        self.lens = torch.zeros(SLOTS, dtype=torch.int32, device="cuda")
        self.sel, self.cnt = i32(SLOTS, HKV, KEEP), i32(SLOTS, HKV)
        self.out = torch.zeros((SLOTS, HQ, D), dtype=torch.float32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.write(self.qkv, self.q, self.pos, self.slots)
            self.summarize(self.filled)
            pkv.select_blocks(self.sel, self.cnt, self.q, self.summary, self.summary_scale, self.tables, self.lens,
                              block_size=B, first_blocks=FIRST, last_blocks=LAST, max_context_len=WIDTH * B,
                              status=self.status)
            a = (self.out, self.q, self.kp, self.vp)
            b = (self.tables, self.lens, self.sel, self.cnt, D ** -0.5)
            kw = dict(max_context_len=WIDTH * B, status=self.status)
            pkv.decode_sparse_fp8(*a, self.ks, self.vs, *b, **kw) if fp8 else pkv.decode_sparse(*a, *b, **kw)

    def rows(self, n):
        return torch.randn(n, HQ + 2 * HKV, D, generator=self.g).to(self.dt).cuda()

    def write(self, qkv, q_out, pos, slots):
        parts = (qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:])
        kw = dict(q_out=q_out, q_weight=self.qw, k_weight=self.kw, cos_sin=self.cs, positions=pos, status=self.status)
        if self.fp8:
            pkv.norm_rope_write_fp8(*parts, self.kp, self.vp, self.ks, self.vs, slots, **kw)
        else:
            pkv.norm_rope_write(*parts, self.kp, self.vp, slots, **kw)

    def summarize(self, ids):
        if self.fp8:
            pkv.summarize_blocks_fp8(self.summary, self.summary_scale, self.kp, self.ks, ids, status=self.status)
        else:
            pkv.summarize_blocks(self.summary, self.summary_scale, self.kp, ids, status=self.status)

    def prompt(self, table, slots):
        """Writes a prompt (slot -1: cached tokens) and summarises its full blocks."""
        n = len(slots)
        q = torch.empty((n, HQ, D), dtype=self.dt, device="cuda")
        i32 = lambda x: torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()
        self.write(self.rows(n), q, i32(np.arange(n)), i32(slots))
        self.summarize(i32(table[:n // B]))

    def step(self, pos, slots, lens, tables, filled):
        """One decode step of len(lens) sequences; the other batch slots stay idle."""
        n = len(lens)
        pad = lambda x, fill: np.concatenate([np.asarray(x), np.full((SLOTS - n,) + np.asarray(x).shape[1:], fill)])
        for dst, src, fill in ((self.pos, pos, -1), (self.slots, slots, -1), (self.lens, lens, 0),
                               (self.tables, tables, -1), (self.filled, filled, -1)):
            dst.copy_(torch.from_numpy(pad(src, fill).astype(np.int32)))
        new = self.rows(SLOTS)
        self.qkv.copy_(new)
        self.q.fill_(3.0)
        self.graph.replay()
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        self.check(new, pos, lens, tables)

    def check(self, new, pos, lens, tables):
        n = len(lens)
        y, m = R.norm_rope(f64(new[:n, :HQ]), f64(self.qw), 1e-6, f64(self.cs)[np.asarray(pos)], False)
        q = f64(self.q)
        assert np.all(np.abs(q[:n] - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -18 * m)
        assert np.all(q[n:] == 3.0)  # idle slots are left alone
        out, sel, cnt = f64(self.out), self.sel.cpu().numpy(), self.cnt.cpu().numpy()
        assert np.all(out[n:] == 0) and np.all(cnt[n:] == 0) and np.all(sel[n:] == -1)
        if self.fp8:
            value = lambda p, sc: R.E4M3[p.cpu().numpy()] * f64(sc)[:, None, :, None]
            kv = [value(self.kp, self.ks), value(self.vp, self.vs)]
        else:
            kv = [f64(self.kp), f64(self.vp)]
        most, G = 3.3895313892515355e38, HQ // HKV
        for s in range(n):
            nblk = -(-int(lens[s]) // B)
            for g in range(HKV):
                heads = slice(g * G, (g + 1) * G)
                codes, unit = np.zeros((nblk, 2, D)), np.ones(nblk)
                for i in range(max(0, nblk - LAST)):  # blocks that are scored: full ones
                    codes[i], unit[i] = R.summarize(kv[0][tables[s][i], :, g], most)
                want = R.select(R.scores(q[s, heads], codes, unit, most), nblk, KEEP, FIRST, LAST)
                assert sel[s, g, :cnt[s, g]].tolist() == want
                k, v = (np.concatenate([x[tables[s][b], :min(B, int(lens[s]) - b * B), g] for b in want]) for x in kv)
                ref = R.attend(q[s, heads], k, v, D ** -0.5)
                tol = R.attend_bound(q[s, heads], k, v, D ** -0.5, 2.0 ** -16)
                assert np.all(np.abs(out[s, heads] - ref) <= tol + 2.0 ** -23 * np.abs(ref) + 2.0 ** -25)


@pytest.mark.parametrize("fp8", [False, True])
def test_serving_loop(fp8):
    rng = np.random.default_rng(5)
    layer = Layer(fp8)
    bm = pkv.BlockManager(NB, B)
    shared = rng.integers(0, 1000, 130)
    # an odd prompt, two that share a prefix of whole blocks, one shorter than a block
    for seq, tokens in ((1, rng.integers(0, 1000, 201)), (2, np.concatenate([shared, [1, 2, 3]])),
                        (3, np.concatenate([shared, rng.integers(0, 1000, 40)])), (4, [7, 8, 9])):
        cached, slots = bm.add_sequence(seq, tokens)
        assert cached == (128 if seq == 3 else 0)
        layer.prompt(bm.block_table(seq), slots)

    def step(seqs):
        pos = [bm.seq_len(s) for s in seqs]
        slots, lens, tables, pairs = bm.decode_step(seqs, rng.integers(0, 1000, len(seqs)), WIDTH)
        if len(pairs):
            p = torch.from_numpy(pairs).cuda()
            if fp8:
                pkv.copy_blocks_fp8(layer.kp, layer.vp, layer.ks, layer.vs, p, status=layer.status)
            else:
                pkv.copy_blocks(layer.kp, layer.vp, p, status=layer.status)
        filled = [t[L // B - 1] if L % B == 0 else -1 for t, L in zip(tables, lens)]
        layer.step(pos, slots, lens, tables, filled)

    for _ in range(9):
        step([1, 2, 3, 4])
    bm.fork(2, 5)  # a shared tail: the first append copies it
    for _ in range(18):
        step([1, 2, 3, 5])
    step([4])
    # Sequence 1 to host memory and back, into other blocks; their summaries are made anew.
    old = bm.swap_out(1)
    keep = [x.cpu().pin_memory() for x in (layer.kp, layer.vp)]  # host pools of the same shape
    n = len(old)
    i32 = lambda a, b: torch.from_numpy(np.stack([a, b], 1).astype(np.int32)).cuda()
    host = np.arange(n)
    pkv.swap_blocks(keep[0], keep[1], layer.kp, layer.vp, i32(old, host))
    step([2, 3, 4])
    back = bm.swap_in(1)
    pkv.swap_blocks(layer.kp, layer.vp, keep[0], keep[1], i32(host, back))
    layer.summarize(torch.from_numpy(back[:bm.seq_len(1) // B].astype(np.int32)).cuda())
    for _ in range(5):
        step([1, 2, 3, 4, 5])
    bm.close()


def test_two_captured_layers_replay_side_by_side():
    """Two layers' graphs, replayed on two streams at once, step after step, with nothing shared."""
    a, b = Layer(False, 1), Layer(False, 2)
    rng = np.random.default_rng(0)
    tables = np.full((2, WIDTH), -1)
    tables[0, :30], tables[1, :30] = np.split(rng.permutation(NB)[:60], 2)
    slots = lambda t, n: [t[i // B] * B + i % B for i in range(n)]
    for layer in (a, b):
        for t, n in ((tables[0], 300), (tables[1], 470)):
            layer.prompt(t, slots(t, n))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(3):
        lens = [301 + i, 471 + i]
        new = []
        for layer in (a, b):
            new.append(layer.rows(SLOTS))
            layer.qkv.copy_(new[-1])
            layer.q.fill_(3.0)
            pad = lambda x, f: torch.tensor(list(x) + [f] * (SLOTS - len(x)), dtype=torch.int32)
            layer.pos.copy_(pad([L - 1 for L in lens], -1))
            layer.lens.copy_(pad(lens, 0))
            layer.slots.copy_(pad([slots(t, L)[-1] for t, L in zip(tables, lens)], -1))
            layer.filled.copy_(pad([t[L // B - 1] if L % B == 0 else -1 for t, L in zip(tables, lens)], -1))
            layer.tables.fill_(-1)
            layer.tables[:2].copy_(torch.from_numpy(tables.astype(np.int32)))
        torch.cuda.synchronize()
        for layer, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                layer.graph.replay()
        torch.cuda.synchronize()
        for layer, rows in zip((a, b), new):
            assert int(layer.status.item()) == 0
            layer.check(rows, [L - 1 for L in lens], lens, tables)


FIRST_CALLS = """
import sys
sys.path.insert(0, sys.argv[1])
import torch
import paged_kv_cache_112_gb300 as pkv
from tests.test_gpu_norm_rope import Step
from tests.test_gpu_sparse import Attend, Select

calls = [Select([70000, 900, 20], keep=40), Attend([700, 900], keep=20), Attend([700, 20], keep=20, fp8=True),
         Step(T=33), Step(T=3000, Hq=32, Hkv=8)]
pool = torch.randn(9, 16, 2, 128, device="cuda").bfloat16()
summary, scale = torch.zeros(9, 2, 2, 128, dtype=torch.int8, device="cuda"), torch.zeros(9, 2, device="cuda")
ids = torch.arange(9, dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for c in calls:
        c.call()
    pkv.summarize_blocks(summary, scale, pool, ids)
g.replay()
torch.cuda.synchronize()
for c in calls:
    c.check()
print("ok")
"""


def test_first_calls_of_a_process_inside_a_capture():
    """Nothing has to run before a capture: attributes, occupancy and descriptors are found within it."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS, root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
