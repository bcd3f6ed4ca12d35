"""Operators of a decode layer over a paged KV cache, as measured cases.

Four operators, each in a plain form (elementary torch operations in 32 bits)
and as the calls that a user makes of the library:

  write      norms of queries and keys per head, position rotation, and the
             scatter of K and V into the pools, in one pass (16-bit and FP8 pools)
  summarize  per (block, KV head) bounds of the keys, int8 with a power-of-two scale
  select     the blocks each sequence and KV head attends to, by those bounds
  attend     single-token attention over the selected blocks (16-bit and FP8 pools)

Every number that decides a choice is exact in 32 bits: summaries and query
codes are small integers with power-of-two scales, a score is an integer below
2^22 times two powers of two, and equal scores go to the lowest block.
"""
import math

import numpy as np
import torch

own = False

# (query heads, KV heads, head dim) of the repository's workloads: the
# 8B-class, the 70B-class, the prefix-sharing and the tiny layer.
H8B, H70B, HPREFIX, HTINY = (32, 8, 128), (64, 8, 128), (32, 4, 128), (4, 2, 64)


def _case(op, heads, **kw):
    c = dict(op=op, hq=heads[0], hkv=heads[1], d=heads[2], dtype="bf16", kv="16", block=16)
    c.update(kw)
    return c


def listed():
    long_ctx = dict(seqs=8, len_lo=32768, len_hi=131072, len_seed=4)
    return [
        # One sequence generates one token: latency alone.
        _case("write", H8B, name="write_1_token", tokens=1, pool_blocks=256, norm=True, rot=128, interleaved=False,
              fused=True),
        # A decode step of a large batch, rows from a fused projection, a captured graph's padding rows among them.
        _case("write", H70B, name="write_256_tokens_f16", dtype="f16", tokens=256, pool_blocks=2048, norm=True,
              rot=128, interleaved=False, fused=True, padding=13),
        # A long prompt written at once.
        _case("write", H8B, name="write_prompt_16384", tokens=16384, pool_blocks=1280, norm=True, rot=128,
              interleaved=False, fused=True),
        # A prompt of odd length into FP8 pools, half of each head rotated in adjacent pairs.
        _case("write", HPREFIX, name="write_prompt_4097_fp8", kv="fp8", tokens=4097, pool_blocks=512, norm=True,
              rot=64, interleaved=True, fused=False),
        # A decode step of 64 sequences: the four whose last block just became full; the others' entries are padding.
        _case("summarize", H8B, name="summarize_step_64", blocks=64, live=4, pool_blocks=1024),
        # The blocks of a prompt of 131072 tokens.
        _case("summarize", H8B, name="summarize_prompt_131072", blocks=8192, live=8192, pool_blocks=8192),
        # The same prompt's blocks in an FP8 pool, 70B-class heads have the same 8 KV heads.
        _case("summarize", H70B, name="summarize_fp8_4001", kv="fp8", blocks=4001, live=4001, pool_blocks=4096),
        # The 8B-class batch: short and middling contexts, an idle slot among them.
        _case("select", H8B, name="select_64_short", seqs=64, len_lo=128, len_hi=2048, len_seed=2, idle=1, keep=32,
              first=1, last=2),
        # The long-context batch: up to 8192 blocks a sequence.
        _case("select", H8B, name="select_8_long", keep=128, first=1, last=2, **long_ctx),
        # One sequence of the long-context range over 128 of its blocks: few rows, latency and splitting.
        _case("attend", H8B, name="attend_1_long", seqs=1, len_lo=100001, len_hi=100001, len_seed=4, keep=128),
        # The 70B-class batch at longer contexts: the largest.
        _case("attend", H70B, name="attend_256_f16", dtype="f16", seqs=256, len_lo=512, len_hi=4096, len_seed=3,
              keep=64, idle=3),
        # The long-context batch over FP8 pools.
        _case("attend", H8B, name="attend_8_long_fp8", kv="fp8", keep=128, **long_ctx),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "write", "summarize", "select", "select", "attend", "attend"])
    kv = rng.choice(["16", "16", "fp8"]) if op != "select" else "16"
    heads = rng.choice([H8B, H70B, HPREFIX, (16, 2, 128), (6, 6, 128), (40, 8, 128), (9, 3, 128)])
    if kv == "16" and rng.random() < 0.3:
        heads = rng.choice([HTINY, (16, 4, 64), (15, 5, 64)])
    c = _case(op, heads, dtype=rng.choice(["bf16", "f16"]), kv=kv,
              block=16 if kv == "fp8" else rng.choice([16, 16, 32, 64]))
    if op == "write":
        t = _log_int(rng, 1, 16384 * H8B[0] // max(H8B[0], heads[0]))
        c.update(tokens=t, pool_blocks=t // c["block"] + rng.randint(2, 200), norm=rng.random() < 0.8,
                 rot=rng.choice([heads[2], heads[2], heads[2] // 2, 16]), interleaved=rng.random() < 0.3,
                 fused=rng.random() < 0.6, padding=rng.choice([0, 0, t // 10]))
    elif op == "summarize":
        n = _log_int(rng, 1, 8192 * 16 // c["block"])
        c.update(blocks=n, live=n if rng.random() < 0.7 else (n + 1) // 2, pool_blocks=n + rng.randint(1, 100))
    else:
        seqs = _log_int(rng, 1, 256)
        # The batch's context in blocks x KV heads stays below the long-context batch's.
        top = min(131072, 8 * 64000 * 8 // (seqs * heads[1]))
        hi = _log_int(rng, 64, max(top, 65))
        c.update(seqs=seqs, len_lo=rng.choice([hi, max(1, hi // 16)]), len_hi=hi, len_seed=rng.randint(0, 9999),
                 idle=rng.choice([0, 0, (seqs + 7) // 8 if seqs > 1 else 0]),
                 keep=_log_int(rng, 4, max(5, min(256, 1900000 // (seqs * heads[1] * c["block"])))))
        if op == "select":  # some sequence has blocks to choose among
            keep = _log_int(rng, 4, max(5, min(256, 1000000 // (seqs * heads[1] * c["block"]))))
            hi = max(hi, rng.randint(2, 4) * keep * c["block"])
            c.update(keep=keep, len_hi=hi, first=rng.randint(0, 2), last=rng.randint(1, 2))
    return c


# ------------------------------------------------------------------ inputs


def _lens(c):
    """Context lengths of the batch; `idle` slots of a captured batch hold no sequence."""
    r = np.random.RandomState(c["len_seed"])
    lens = r.randint(c["len_lo"], c["len_hi"] + 1, size=c["seqs"]).astype(np.int64)
    if c.get("idle"):
        lens[r.permutation(c["seqs"] - 1)[:c["idle"]]] = 0
    lens[-1] = c["len_hi"]
    return lens


def _dtype(c):
    return {"bf16": torch.bfloat16, "f16": torch.float16}[c["dtype"]]


def _tables(c, lens, g):
    """Block tables of scattered physical blocks: int32 [S, widest], -1 past each sequence's end."""
    n = torch.from_numpy((lens + c["block"] - 1) // c["block"]).cuda()
    width = max(1, int(n.max()))
    total = int(n.sum())
    perm = torch.randperm(max(total, 1) + 7, device="cuda", generator=g).to(torch.int32)
    cols = torch.arange(width, device="cuda")
    inside = cols[None, :] < n[:, None]
    order = torch.cumsum(inside.reshape(-1), 0).reshape(inside.shape) - 1
    tables = torch.where(inside, perm[order.clamp(min=0)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    return tables.contiguous(), n, int(perm.numel())


def _normal(shape, dt, g, scale=1.0):
    """Keys, values and queries have unit scale and a few heavy channels."""
    x = torch.empty(shape, dtype=dt, device="cuda").normal_(0.0, scale, generator=g)
    heavy = torch.ones(shape[-1], dtype=dt, device="cuda")
    heavy[:: max(1, shape[-1] // 8)] = 2.5
    return x.mul_(heavy)


def _codes(shape, g):
    """e4m3 codes of normal values of scale 64 (finite, both signs), as bytes."""
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // max(1, math.prod(shape[1:])))
    for i in range(0, shape[0], step):
        x = torch.empty(out[i:i + step].shape, device="cuda").normal_(0.0, 64.0, generator=g).clamp_(-448, 448)
        out[i:i + step] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _scales(shape, g):
    return torch.empty(shape, device="cuda").uniform_(0.008, 0.05, generator=g)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    dt, hq, hkv, d, b = _dtype(c), c["hq"], c["hkv"], c["d"], c["block"]
    s = {"case": c, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if c["op"] == "write":
        t, nb = c["tokens"], c["pool_blocks"]
        if c["fused"]:  # rows of one fused projection
            rows = _normal((t, (hq + 2 * hkv), d), dt, g)
            s["q"], s["k"], s["v"] = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        else:
            s["q"], s["k"], s["v"] = (_normal((t, h, d), dt, g) for h in (hq, hkv, hkv))
        s["q_weight"] = s["k_weight"] = None
        if c["norm"]:
            s["q_weight"], s["k_weight"] = ((1 + 0.2 * torch.empty(d, device="cuda").normal_(generator=g)).to(dt)
                                            for _ in range(2))
        top = 131072  # positions up to the long-context range; angles in 64 bits
        inv = 500000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
        ang = torch.arange(top, dtype=torch.float64, device="cuda")[:, None] * inv[None, :]
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        start = int(torch.randint(0, top - t, (1,), device="cuda", generator=g))
        s["positions"] = (torch.arange(t, device="cuda") + start).to(torch.int32)
        slots = torch.randperm(nb * b, device="cuda", generator=g)[:t].to(torch.int32)
        if t >= b:  # a prompt fills whole blocks
            blocks = torch.randperm(nb, device="cuda", generator=g)
            i = torch.arange(t, device="cuda")
            slots = (blocks[i // b] * b + i % b).to(torch.int32)
        live = t - c.get("padding", 0)
        slots[live:] = -1
        s["slots"], s["live"] = slots, torch.arange(live, device="cuda")
        s["q_out"] = torch.empty((t, hq, d), dtype=dt, device="cuda")
        if c["kv"] == "fp8":
            s["k_pool"], s["v_pool"] = _codes((nb, b, hkv, d), g), _codes((nb, b, hkv, d), g)
            s["k_scale"], s["v_scale"] = _scales((nb, hkv), g), _scales((nb, hkv), g)
        else:
            s["k_pool"], s["v_pool"] = _normal((nb, b, hkv, d), dt, g), _normal((nb, b, hkv, d), dt, g)
    elif c["op"] == "summarize":
        nb, n = c["pool_blocks"], c["blocks"]
        ids = torch.randperm(nb, device="cuda", generator=g)[:n].to(torch.int32)
        drop = torch.randperm(n, device="cuda", generator=g)[c["live"]:]
        ids[drop] = -1
        s["ids"], s["live"] = ids, torch.nonzero(ids >= 0).reshape(-1)
        if c["kv"] == "fp8":
            s["k_pool"], s["k_scale"] = _codes((nb, b, hkv, d), g), _scales((nb, hkv), g)
        else:
            s["k_pool"] = _normal((nb, b, hkv, d), dt, g)
        s["summary"] = torch.zeros((nb, hkv, 2, d), dtype=torch.int8, device="cuda")
        s["summary_scale"] = torch.ones((nb, hkv), device="cuda")
    else:
        lens = _lens(c)
        s["tables"], n, nb = _tables(c, lens, g)
        s["lens"] = torch.from_numpy(lens).to(torch.int32).cuda()
        s["max_len"] = int(lens.max())
        s["q"] = _normal((c["seqs"], hq, d), dt, g)
        s["scale"] = d ** -0.5
        if c["op"] == "select":
            s["summary"] = torch.empty((nb, hkv, 2, d), dtype=torch.int8, device="cuda")
            s["summary_scale"] = torch.empty((nb, hkv), device="cuda")
            step = max(1, (1 << 26) // (b * hkv * d))
            for i in range(0, nb, step):  # as a prompt's blocks would have left them
                k = _normal((min(step, nb - i), b, hkv, d), dt, g)
                k += _normal((k.shape[0], 1, hkv, d), dt, g, 0.7)
                codes, sc = _bounds(k.float())
                s["summary"][i:i + step], s["summary_scale"][i:i + step] = codes, sc
            s["selected"] = torch.empty((c["seqs"], hkv, c["keep"]), dtype=torch.int32, device="cuda")
            s["counts"] = torch.empty((c["seqs"], hkv), dtype=torch.int32, device="cuda")
        else:
            keep, width = c["keep"], s["tables"].shape[1]
            # A selection as `select` leaves it: ascending, the last block always among it.
            col = torch.arange(width, device="cuda")
            order = torch.rand((c["seqs"], hkv, width), device="cuda", generator=g)
            order = torch.where(col < n[:, None, None], order, torch.full_like(order, 2.0))
            order = torch.where(col == (n - 1)[:, None, None], torch.full_like(order, -1.0), order)
            pick = torch.argsort(order, dim=2)[:, :, :keep]
            pick = torch.nn.functional.pad(pick, (0, keep - pick.shape[2]), value=width)
            count = torch.clamp(n, max=keep)[:, None, None].expand(-1, hkv, 1)
            place = torch.arange(keep, device="cuda")
            pick = torch.where(place < count, pick, torch.full_like(pick, 1 << 30))
            pick = torch.sort(pick, dim=2).values
            s["selected"] = torch.where(place < count, pick, torch.full_like(pick, -1)).to(torch.int32).contiguous()
            s["counts"] = count[:, :, 0].to(torch.int32).contiguous()
            if c["kv"] == "fp8":
                s["k_pool"], s["v_pool"] = _codes((nb, b, hkv, d), g), _codes((nb, b, hkv, d), g)
                s["k_scale"], s["v_scale"] = _scales((nb, hkv), g), _scales((nb, hkv), g)
            else:
                s["k_pool"], s["v_pool"] = _normal((nb, b, hkv, d), dt, g), _normal((nb, b, hkv, d), dt, g)
            s["out"] = torch.empty((c["seqs"], hq, d), dtype=dt, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms


def _exponent(amax):
    """The smallest e >= -126 with amax <= 127 * 2^e, as 2^e (1 where amax is 0)."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 127.0 / 128.0, x - 7, x - 6).clamp(min=-126)
    return torch.where(amax > 0, torch.exp2(e.double()), 1.0).float()


def _bounds(k):
    """k [n, B, H, D] float: codes int8 [n, H, 2, D] of the lower and upper bound of each channel, scale [n, H]."""
    lo, hi = k.amin(1), k.amax(1)
    sc = _exponent(torch.maximum(lo.abs(), hi.abs()).amax(-1))
    codes = torch.stack([torch.floor(lo / sc[..., None]), torch.ceil(hi / sc[..., None])], 2)
    return codes.to(torch.int8), sc


def _normed(x, w, eps=1e-6):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()


def _rotated(x, cos, sin, rot, interleaved):
    h = x[..., :rot]
    a, b = (h[..., 0::2], h[..., 1::2]) if interleaved else (h[..., :rot // 2], h[..., rot // 2:])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([y, z], -1).reshape(h.shape) if interleaved else torch.cat([y, z], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_write(s):
    c = s["case"]
    cs = s["cos_sin"][s["positions"].long()][:, None, :]
    cos, sin = cs[..., :c["rot"] // 2], cs[..., c["rot"] // 2:]
    q = _rotated(_normed(s["q"].float(), s["q_weight"]), cos, sin, c["rot"], c["interleaved"])
    k = _rotated(_normed(s["k"].float(), s["k_weight"]), cos, sin, c["rot"], c["interleaved"])[s["live"]]
    v = s["v"].float()[s["live"]]
    s["q_out"].copy_(q)
    slots = s["slots"].long()[s["live"]]
    row = (-1, c["hkv"], c["d"])
    if c["kv"] == "fp8":
        ks, vs = (s[n][slots // c["block"]][..., None] for n in ("k_scale", "v_scale"))
        k = (k / ks).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v / vs).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s["k_pool"].view(row).index_copy_(0, slots, k.to(s["k_pool"].dtype))
    s["v_pool"].view(row).index_copy_(0, slots, v.to(s["v_pool"].dtype))


def _plain_summarize(s):
    ids = s["ids"][s["live"]].long()
    k = s["k_pool"][ids]
    if "k_scale" in s:  # products in 64 bits: a bound is rounded outwards, and 32 bits can land on a step
        k = k.view(torch.float8_e4m3fn).double() * s["k_scale"][ids].double()[:, None, :, None]
    else:
        k = k.float()
    codes, sc = _bounds(k)
    s["summary"].index_copy_(0, ids, codes)
    s["summary_scale"].index_copy_(0, ids, sc)


def _plain_select(s):
    c, (S, width) = s["case"], s["tables"].shape
    hkv, d, keep = c["hkv"], c["d"], c["keep"]
    q = s["q"].float().view(S, hkv, -1, d)
    qs = _exponent(q.abs().amax(-1))
    qc = torch.round(q / qs[..., None])
    t = s["tables"].clamp(min=0).long()
    bounds = s["summary"][t].float().permute(0, 2, 3, 4, 1)  # [S, H, 2, D, blocks]
    whole = qc.clamp(max=0) @ bounds[:, :, 0] + qc.clamp(min=0) @ bounds[:, :, 1]  # whole numbers below 2^22
    score = (whole * qs[..., None] * s["summary_scale"][t].permute(0, 2, 1)[:, :, None]).amax(2)
    n = ((s["lens"] + c["block"] - 1) // c["block"]).long()[:, None, None]
    col = torch.arange(width, device=t.device)
    score = torch.where((col < c["first"]) | (col >= n - c["last"]), torch.full_like(score, math.inf), score)
    score = torch.where(col < n, score, torch.full_like(score, -math.inf))
    place = torch.arange(keep, device=t.device)
    pick = torch.sort(score, dim=2, descending=True, stable=True).indices[:, :, :keep]
    pick = torch.nn.functional.pad(pick, (0, keep - pick.shape[2]), value=width)
    count = n.clamp(max=keep)
    pick = torch.sort(torch.where(place < count, pick, torch.full_like(pick, 1 << 30)), dim=2).values
    s["selected"].copy_(torch.where(place < count, pick, torch.full_like(pick, -1)))
    s["counts"].copy_(count[:, :, 0].expand(-1, hkv))


def _plain_attend(s):
    c = s["case"]
    S, hkv, d, b = c["seqs"], c["hkv"], c["d"], c["block"]
    sel = s["selected"].long()
    phys = torch.gather(s["tables"].long()[:, None].expand(-1, hkv, -1), 2, sel.clamp(min=0)).clamp(min=0)
    h = torch.arange(hkv, device=sel.device)[None, :, None]
    k, v = (s[n].permute(0, 2, 1, 3)[phys, h] for n in ("k_pool", "v_pool"))  # [S, H, keep, B, D]
    if c["kv"] == "fp8":
        k, v = (x.view(torch.float8_e4m3fn).float() * s[n][phys, h][..., None, None]
                for x, n in ((k, "k_scale"), (v, "v_scale")))
    k, v = (x.reshape(S, hkv, -1, d).float() for x in (k, v))
    token = sel[..., None] * b + torch.arange(b, device=sel.device)
    live = ((sel >= 0)[..., None] & (token < s["lens"].long()[:, None, None, None])).reshape(S, hkv, 1, -1)
    score = (s["q"].float().view(S, hkv, -1, d) @ k.transpose(2, 3)) * s["scale"]
    score = torch.where(live, score, torch.full_like(score, -math.inf))
    top = score.amax(3, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(3, keepdim=True)
    # A row with no token is zero; places that hold none are left out of the sum whatever they hold.
    v = torch.where(live.transpose(2, 3), v, torch.zeros_like(v))
    s["out"].copy_(((p @ v) / torch.where(total > 0, total, torch.ones_like(total))).view(S, c["hq"], d))


def run(state):
    s = state
    c = s["case"]
    op, fp8 = c["op"], c["kv"] == "fp8"
    if own:
        import paged_kv_cache_112_gb300 as pkv

        if op == "write":
            more = dict(q_out=s["q_out"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6,
                        cos_sin=s["cos_sin"], positions=s["positions"], interleaved=c["interleaved"],
                        status=s["status"])
            if fp8:
                pkv.norm_rope_write_fp8(s["q"], s["k"], s["v"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"],
                                        s["slots"], **more)
            else:
                pkv.norm_rope_write(s["q"], s["k"], s["v"], s["k_pool"], s["v_pool"], s["slots"], **more)
        elif op == "summarize":
            if fp8:
                pkv.summarize_blocks_fp8(s["summary"], s["summary_scale"], s["k_pool"], s["k_scale"], s["ids"],
                                         status=s["status"])
            else:
                pkv.summarize_blocks(s["summary"], s["summary_scale"], s["k_pool"], s["ids"], status=s["status"])
        elif op == "select":
            pkv.select_blocks(s["selected"], s["counts"], s["q"], s["summary"], s["summary_scale"], s["tables"],
                              s["lens"], block_size=c["block"], first_blocks=c["first"], last_blocks=c["last"],
                              max_context_len=s["max_len"], status=s["status"])
        elif fp8:
            pkv.decode_sparse_fp8(s["out"], s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["tables"],
                                  s["lens"], s["selected"], s["counts"], s["scale"], max_context_len=s["max_len"],
                                  status=s["status"])
        else:
            pkv.decode_sparse(s["out"], s["q"], s["k_pool"], s["v_pool"], s["tables"], s["lens"], s["selected"],
                              s["counts"], s["scale"], max_context_len=s["max_len"], status=s["status"])
    else:
        {"write": _plain_write, "summarize": _plain_summarize, "select": _plain_select, "attend": _plain_attend}[op](s)
    if op == "write":
        # FP8 codes come back as the e4m3 values they are.
        as_values = (lambda x: x.view(torch.float8_e4m3fn)) if fp8 else (lambda x: x)
        return {"q": s["q_out"], "k_pool": as_values(s["k_pool"]), "v_pool": as_values(s["v_pool"])}
    if op == "summarize":
        # The codes are whole numbers (steps of the scale), the same to the last one in any exact arithmetic.
        return {"summary": s["summary"], "scale": s["summary_scale"]}
    if op == "select":
        return {"selected": s["selected"], "counts": s["counts"]}
    return {"out": s["out"]}


# ------------------------------------------------------------------ cost


def work(case):
    c = case
    hq, hkv, d, eb = c["hq"], c["hkv"], c["d"], 1 if c["kv"] == "fp8" else 2
    if c["op"] == "write":
        t, live = c["tokens"], c["tokens"] - c.get("padding", 0)
        # q in and out, k in, v in and both to the pools for the live rows, an angle row, position and slot a token
        return {"bytes": t * (2 * hq * d * 2 + c["rot"] * 4 + 8) + live * 2 * hkv * d * (2 + eb),
                "flops": t * (hq + hkv) * d * 7}
    if c["op"] == "summarize":
        return {"bytes": c["live"] * hkv * (c["block"] * d * eb + 2 * d + 4) + 4 * c["blocks"],
                "flops": c["live"] * hkv * c["block"] * d * 2}
    n = (_lens(c) + c["block"] - 1) // c["block"]
    if c["op"] == "select":
        # Sequences of no more than `keep` blocks need no score.
        scored = int(n[n > c["keep"]].sum())
        io = c["seqs"] * (hkv * (c["keep"] + 1) * 4 + 4 + hq * d * 2)
        return {"bytes": scored * (hkv * (2 * d + 4) + 4) + io, "flops": scored * hq * d * 4}
    lens = _lens(c)
    m = np.minimum(n, c["keep"])
    # the last, partial block is always among the selected
    tokens = int(np.where(n > 0, m * c["block"] - (n * c["block"] - lens), 0).sum())
    per = 8 if c["kv"] == "fp8" else 0
    return {"bytes": hkv * (tokens * 2 * d * eb + int(m.sum()) * (8 + per)) + c["seqs"] * hq * d * 2 * 2,
            "flops": tokens * hq * d * 4}


# ------------------------------------------------------------------ in 64 bits


def _unit(most):
    """Powers of two in 64 bits, built from their bits: the smallest 2^e with most <= 127 * 2^e."""

    def power(e):
        return ((e.long() + 1023) << 52).view(torch.float64)

    e = torch.ceil(torch.log2(most / 127))
    e = torch.where(torch.isfinite(e), e, torch.zeros_like(e))
    e = e + (127 * power(e) < most).double() - (127 * power(e - 1) >= most).double()
    return torch.where(most > 0, power(e), torch.ones_like(most))


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    hq, hkv, d, b = c["hq"], c["hkv"], c["d"], c["block"]
    G = hq // hkv
    f8 = torch.float8_e4m3fn
    if c["op"] == "write":
        pos = s["positions"].double()
        half = c["rot"] // 2
        angle = s["cos_sin"].double()[pos.long()]
        turn = torch.complex(angle[:, :half], angle[:, half:])[:, None, :]

        def head(x, w):
            x = x.double()
            if w is not None:
                x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + 1e-6) * w.double()
            y = x.clone()
            if c["interleaved"]:
                z = torch.view_as_complex(x[..., :2 * half].reshape(*x.shape[:-1], half, 2).contiguous()) * turn
                y[..., :2 * half] = torch.view_as_real(z).reshape(*x.shape[:-1], 2 * half)
            else:
                z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * turn
                y[..., :half], y[..., half:2 * half] = z.real, z.imag
            return y

        pools = {}
        for name, new, scale in (("k_pool", head(s["k"], s["k_weight"]), "k_scale"),
                                 ("v_pool", s["v"].double(), "v_scale")):
            slot = s["slots"].long()
            on = slot >= 0
            if c["kv"] == "fp8":
                pool = s[name].view(f8).double()
                new = (new[on] / s[scale].double()[slot[on] // b].unsqueeze(-1)).clamp(-448, 448)
            else:
                pool, new = s[name].double(), new[on]
            pool[slot[on] // b, slot[on] % b] = new
            pools[name] = pool
        return {"q": head(s["q"], s["q_weight"]), **pools}
    if c["op"] == "summarize":
        codes, scale = s["summary"].clone(), s["summary_scale"].double()
        on = s["ids"][s["ids"] >= 0].long()
        for part in on.split(1024):
            k = s["k_pool"][part]
            k = k.view(f8).double() * s["k_scale"].double()[part].view(-1, 1, hkv, 1) if "k_scale" in s else k.double()
            lo, hi = k.min(dim=1).values, k.max(dim=1).values
            most = torch.maximum(-lo, hi).max(dim=-1).values
            unit = _unit(most)
            codes[part, :, 0] = torch.floor(lo / unit.unsqueeze(-1)).clamp(-127, 127).to(torch.int8)
            codes[part, :, 1] = torch.ceil(hi / unit.unsqueeze(-1)).clamp(-127, 127).to(torch.int8)
            scale[part] = unit
        return {"summary": codes, "scale": scale}
    lens = s["lens"].tolist()
    if c["op"] == "select":
        sel, counts = torch.full_like(s["selected"], -1), torch.zeros_like(s["counts"])
        for i, L in enumerate(lens):
            n = -(-L // b)
            counts[i] = min(n, c["keep"])
            if n <= c["keep"]:
                sel[i, :, :n] = torch.arange(n, device="cuda", dtype=torch.int32)
                continue
            blocks = s["tables"][i, :n].long()
            q = s["q"][i].double().view(hkv, G, d)
            most = q.abs().max(dim=-1, keepdim=True).values
            unit = _unit(most)
            qq = torch.round(q / unit) * unit
            low, high = (s["summary"][blocks, :, j].double() * s["summary_scale"].double()[blocks].unsqueeze(-1)
                         for j in (0, 1))  # [n, H, D]
            score = torch.stack([torch.maximum(qq[:, j] * low, qq[:, j] * high).sum(-1) for j in range(G)]).amax(0)
            middle = score[c["first"]:n - c["last"]]  # [blocks, H]
            want = c["keep"] - c["first"] - c["last"]
            best = torch.sort(-middle, dim=0, stable=True).indices[:want] + c["first"]
            ends = torch.cat([torch.arange(c["first"]), torch.arange(n - c["last"], n)]).cuda()
            sel[i] = torch.sort(torch.cat([best, ends[:, None].expand(-1, hkv)]), dim=0).values.t().to(torch.int32)
        return {"selected": sel, "counts": counts}
    out = torch.zeros((c["seqs"], hq, d), dtype=torch.float64, device="cuda")
    pools = [s["k_pool"], s["v_pool"]]
    for i, L in enumerate(lens):
        m = min(-(-L // b), c["keep"])
        if not m:
            continue
        picked = s["selected"][i, :, :m].long()
        phys = s["tables"][i].long()[picked]
        kv = []
        for j, pool in enumerate(pools):
            rows = torch.stack([pool[phys[h], :, h] for h in range(hkv)])  # [H, m, B, D]
            if c["kv"] == "fp8":
                sc = s[("k_scale", "v_scale")[j]]
                rows = rows.view(f8).double() * torch.stack([sc[phys[h], h] for h in range(hkv)]).double()[..., None, None]
            kv.append(rows.double().reshape(hkv, m * b, d))
        at = (picked[..., None] * b + torch.arange(b, device="cuda")).reshape(hkv, 1, -1)
        logit = torch.einsum("hgd,htd->hgt", s["q"][i].double().view(hkv, G, d), kv[0]) * s["scale"]
        logit = logit.masked_fill(at >= L, -math.inf)
        out[i] = torch.einsum("hgt,htd->hgd", torch.softmax(logit, -1), kv[1]).reshape(hq, d)
    return {"out": out}
