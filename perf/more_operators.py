"""Operators for 4-bit caches, sliding windows and prompts over a paged KV cache, as measured cases.

Four operators, each in a plain form (elementary torch operations in 32 bits)
and as the calls that a user makes of the library:

  append   new rows into 4-bit pools: norms per head, position rotation, quantisation, scatter
  attend4  single-token attention over 4-bit pools
  window   single-token attention over a sliding window and a few first tokens (16-bit and 4-bit pools)
  prompt   attention of many tokens of a sequence over its paged history, causal, with or without a window

A 4-bit pool holds, per block, KV head and 16 tokens, 16 x D/2 bytes of e2m1
codes (the even channel in the low half) and then 16 x D/16 bytes of e4m3
scales, one for 16 channels of a token:
    value = code * scale * head_scale[KV head],
    scale = e4m3(max |z| / 6), code = e2m1(z / scale), z = x * (1 / head_scale)
in 32-bit arithmetic, each rounded to the nearest with ties to even.
"""
import math

import numpy as np
import torch

own = False

# (query heads, KV heads, head dim) of the repository's workloads: the
# 8B-class, the 70B-class, the prefix-sharing and the tiny layer.
H8B, H70B, HPREFIX, HTINY = (32, 8, 128), (64, 8, 128), (32, 4, 128), (4, 2, 64)


def _case(op, heads, **kw):
    c = dict(op=op, hq=heads[0], hkv=heads[1], d=heads[2], dtype="bf16", kv="16" if op in ("window", "prompt") else "4",
             block=16, head_scales=False)
    c.update(kw)
    return c


def listed():
    long_ctx = dict(seqs=8, len_lo=32768, len_hi=131072, len_seed=4)
    full_rope = dict(norm=True, rot=128, interleaved=False, fused=True)
    return [
        # One sequence generates one token into a 4-bit cache: latency alone.
        _case("append", H8B, name="append_1_token", tokens=1, pool_blocks=64, **full_rope),
        # A long prompt written at once, rows from a fused projection.
        _case("append", H8B, name="append_prompt_16384", tokens=16384, pool_blocks=1040, head_scales=True, **full_rope),
        # An odd number of tokens of a layer of small heads without norms, half of each head rotated in adjacent pairs.
        _case("append", (16, 4, 64), name="append_4097_f16", dtype="f16", tokens=4097, pool_blocks=160, block=32,
              norm=False, rot=32, interleaved=True, fused=False, padding=13),
        # One long conversation in a 4-bit cache: few rows, latency and splitting.
        _case("attend4", H8B, name="attend4_1_long", seqs=1, len_lo=100001, len_hi=100001, len_seed=4),
        # The long-context batch, whose cache is what 4 bits are for.
        _case("attend4", H8B, name="attend4_8_long", head_scales=True, **long_ctx),
        # The 70B-class batch at middling contexts, idle slots among them.
        _case("attend4", H70B, name="attend4_256_f16", dtype="f16", seqs=256, len_lo=128, len_hi=4096, len_seed=3,
              idle=3),
        # One token of one sequence of a windowed layer: latency alone.
        _case("window", H8B, name="window_1", seqs=1, len_lo=5000, len_hi=5000, len_seed=1, window=1024, sinks=4),
        # A windowed layer of the long-context batch over a 4-bit cache, an odd window.
        _case("window", HPREFIX, name="window_64_fp4", kv="4", seqs=64, len_lo=128, len_hi=32768, len_seed=2, idle=1,
              window=4095, sinks=64),
        # The 70B-class batch, the window's largest.
        _case("window", H70B, name="window_256_f16", dtype="f16", seqs=256, len_lo=512, len_hi=8192, len_seed=3, idle=3,
              window=2048, sinks=16),
        # A handful of new tokens behind a history: a short turn of a conversation.
        _case("prompt", H8B, name="prompt_turn_37", seqs=1, new_lo=37, new_hi=37, past_lo=2000, past_hi=2000, len_seed=1,
              window=0, sinks=0),
        # Ragged prompts of a windowed model, some of them with a cached prefix.
        _case("prompt", HPREFIX, name="prompt_16_window_f16", dtype="f16", seqs=16, new_lo=1, new_hi=2000, past_lo=0,
              past_hi=300, len_seed=5, window=512, sinks=4),
        # A long prompt, all of it visible: the largest.
        _case("prompt", H8B, name="prompt_8192", seqs=1, new_lo=8192, new_hi=8192, past_lo=0, past_hi=0, len_seed=1,
              window=0, sinks=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend4", "attend4", "window", "window", "prompt", "prompt"])
    heads = rng.choice([H8B, H70B, HPREFIX, (16, 2, 128), (6, 6, 128), (40, 8, 128), (9, 3, 128), HTINY, (16, 4, 64),
                        (15, 5, 64)])
    c = _case(op, heads, dtype=rng.choice(["bf16", "f16"]), block=rng.choice([16, 16, 32, 64]))
    if op == "append":
        t = _log_int(rng, 1, 16384 * H8B[0] // max(H8B[0], heads[0]))
        c.update(tokens=t, pool_blocks=t // c["block"] + rng.randint(2, 60), norm=rng.random() < 0.7,
                 rot=rng.choice([heads[2], heads[2], heads[2] // 2, 16]), interleaved=rng.random() < 0.3,
                 fused=rng.random() < 0.6, padding=rng.choice([0, 0, t // 10]), head_scales=rng.random() < 0.5)
    elif op == "prompt":
        seqs = _log_int(rng, 1, 16)
        # Sequences x query heads x new tokens x history stays below the long prompt's.
        room = 32 * 8192 * 8192 // (seqs * heads[0])
        new = _log_int(rng, 1, min(8192, int(math.sqrt(room))))
        past = rng.choice([0, _log_int(rng, 1, max(2, min(32768, room // new - new)))])
        c.update(seqs=seqs, new_lo=rng.choice([new, 1]), new_hi=new, past_lo=rng.choice([past, 0]), past_hi=past,
                 len_seed=rng.randint(0, 9999), window=0, sinks=0)
        if rng.random() < 0.5:
            c.update(window=_log_int(rng, 16, 4096), sinks=rng.choice([0, 1, 4, 130]))
    else:
        if op == "window":
            c["kv"] = rng.choice(["16", "4"])
        seqs = _log_int(rng, 1, 256)
        # The tokens x KV heads of a batch stay below the long-context batch's (16 bits: a quarter of it).
        top = (8 if c["kv"] == "4" else 2) * 64000 * 8 // (seqs * heads[1])
        hi = _log_int(rng, 64, max(65, min(131072, top)))
        c.update(seqs=seqs, len_lo=rng.choice([hi, max(1, hi // 16)]), len_hi=hi, len_seed=rng.randint(0, 9999),
                 idle=rng.choice([0, 0, (seqs + 7) // 8 if seqs > 1 else 0]),
                 head_scales=c["kv"] == "4" and rng.random() < 0.5)
        if op == "window":
            c.update(window=_log_int(rng, 16, 8192), sinks=rng.choice([0, 1, 4, 16, 100]))
    return c


# ------------------------------------------------------------------ inputs


def _lens(c):
    """Context lengths of the batch (idle slots of a captured batch hold no sequence), and a prompt's new tokens."""
    r = np.random.RandomState(c["len_seed"])
    if c["op"] == "prompt":
        new = r.randint(c["new_lo"], c["new_hi"] + 1, size=c["seqs"]).astype(np.int64)
        new[-1] = c["new_hi"]
        past = r.randint(c["past_lo"], c["past_hi"] + 1, size=c["seqs"]).astype(np.int64)
        past[-1] = c["past_hi"]
        return new + past, new
    lens = r.randint(c["len_lo"], c["len_hi"] + 1, size=c["seqs"]).astype(np.int64)
    if c.get("idle"):
        lens[r.permutation(c["seqs"] - 1)[:c["idle"]]] = 0
    lens[-1] = c["len_hi"]
    return lens, None


def _dtype(c):
    return {"bf16": torch.bfloat16, "f16": torch.float16}[c["dtype"]]


def _tables(c, lens, g):
    """Block tables of scattered physical blocks: int32 [S, widest], -1 past each sequence's end."""
    n = torch.from_numpy((lens + c["block"] - 1) // c["block"]).cuda()
    width = max(1, int(n.max()))
    total = int(n.sum())
    perm = torch.randperm(max(total, 1) + 7, device="cuda", generator=g).to(torch.int32)
    inside = torch.arange(width, device="cuda")[None, :] < n[:, None]
    order = torch.cumsum(inside.reshape(-1), 0).reshape(inside.shape) - 1
    tables = torch.where(inside, perm[order.clamp(min=0)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    return tables.contiguous(), int(perm.numel())


def _normal(shape, dt, g, scale=1.0):
    """Keys, values and queries have unit scale and a few heavy channels."""
    x = torch.empty(shape, dtype=dt, device="cuda").normal_(0.0, scale, generator=g)
    heavy = torch.ones(shape[-1], dtype=dt, device="cuda")
    heavy[:: max(1, shape[-1] // 8)] = 2.5
    return x.mul_(heavy)


def _pool4(nb, c, g, kinds=4096):
    """A 4-bit pool as prompts leave it: each tile one of `kinds` tiles of quantised rows."""
    d, tiles = c["d"], c["block"] // 16
    code, scale = _quantised(_normal((kinds, 16, d), torch.float32, g))
    kind = torch.cat([_packed(code).reshape(kinds, -1), scale.view(torch.uint8).reshape(kinds, -1)], 1)
    pick = torch.randint(0, kinds, (nb * c["hkv"] * tiles,), device="cuda", generator=g, dtype=torch.int32)
    return torch.index_select(kind, 0, pick).view(nb, c["hkv"], tiles, 9 * d)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    dt, hq, hkv, d, b = _dtype(c), c["hq"], c["hkv"], c["d"], c["block"]
    s = {"case": c, "status": torch.zeros(1, dtype=torch.int32, device="cuda"), "k_scale": None, "v_scale": None}
    if c["head_scales"]:
        s["k_scale"], s["v_scale"] = (torch.empty(hkv, device="cuda").uniform_(0.3, 3.0, generator=g) for _ in range(2))
    if c["op"] == "append":
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
        s["k_pool"], s["v_pool"] = _pool4(nb, c, g), _pool4(nb, c, g)
        s["e4m3_of"] = _e4m3_of()
        return s
    lens, new = _lens(c)
    s["tables"], nb = _tables(c, lens, g)
    s["lens"] = torch.from_numpy(lens).to(torch.int32).cuda()
    s["max_len"] = int(lens.max())
    s["scale"] = d ** -0.5
    if c["op"] == "prompt":
        start = np.concatenate([[0], np.cumsum(new)])
        s["query_start"] = torch.from_numpy(start).to(torch.int32).cuda()
        s["max_new"] = int(new.max())
        rows = int(start[-1])
        # Where each row of the batch sits in a rectangle of sequences x new tokens (the plain form's).
        s["place"] = torch.from_numpy(np.repeat(np.arange(c["seqs"]) * s["max_new"] - start[:-1], new)
                                      + np.arange(rows)).cuda()
    else:
        rows = c["seqs"]
    s["q"] = _normal((rows, hq, d), dt, g)
    if c["kv"] == "4":
        s["k_pool"], s["v_pool"] = _pool4(nb, c, g), _pool4(nb, c, g)
    else:
        s["k_pool"], s["v_pool"] = _normal((nb, b, hkv, d), dt, g), _normal((nb, b, hkv, d), dt, g)
    if c["op"] == "attend4":
        # Split-K scratch, as large as the library asks for with partitions of 1024 tokens and more.
        parts = -(-s["max_len"] // 1024)
        s["workspace"] = torch.empty(c["seqs"] * hq * parts * (d * 4 + 8) + 4096, dtype=torch.uint8, device="cuda")
    s["out"] = torch.zeros((rows, hq, d), dtype=dt, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms


def _quantised(z):
    """z [..., D] float: e2m1 codes 0..15 (int32), e4m3 scales [..., D / 16]."""
    z = z.unflatten(-1, (-1, 16))
    scale = (z.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    sc = scale.float()[..., None]
    a = torch.where(sc > 0, z.abs() / torch.where(sc > 0, sc, 1.0), 0.0).clamp(max=6.0)
    code = torch.where(a < 2, torch.round(2 * a), torch.where(a < 4, torch.round(a) + 2, torch.round(a / 2) + 4))
    return (code.to(torch.int32) + 8 * torch.signbit(z)).flatten(-2), scale


def _packed(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8)


def _values(codes):
    """Values of packed codes: [..., n] bytes -> [..., 2n] float."""
    half = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    one = torch.cat([half, -half])
    byte = torch.arange(256, device=codes.device)
    return torch.stack([one[byte & 15], one[byte >> 4]], 1)[codes.int()].flatten(-2)


def _e4m3_of():
    """The e4m3 bytes of the values of four codes (two bytes), as one 32-bit word, by the two bytes plus 32768."""
    word = torch.arange(-32768, 32768, device="cuda", dtype=torch.int16)
    return _values(word.view(torch.uint8)).to(torch.float8_e4m3fn).view(torch.int32)


def _parts(pool, d):
    """Codes [NB, H, tiles, 16, D/2] and scales [NB, H, tiles, 16, D/16] of a 4-bit pool."""
    return pool[..., :8 * d].unflatten(-1, (16, d // 2)), pool[..., 8 * d:].unflatten(-1, (16, d // 16))


def _normed(x, w, eps=1e-6):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()


def _rotated(x, cos, sin, rot, interleaved):
    h = x[..., :rot]
    a, b = (h[..., 0::2], h[..., 1::2]) if interleaved else (h[..., :rot // 2], h[..., rot // 2:])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([y, z], -1).reshape(h.shape) if interleaved else torch.cat([y, z], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _put(pool, scales, x, slots, c):
    """Rows x [T, H, D] into their slots of a 4-bit pool."""
    z = x if scales is None else x * (1.0 / scales)[:, None]
    code, sc = _quantised(z)
    codes_at, scales_at = _parts(pool, c["d"])
    h = torch.arange(c["hkv"], device=x.device)[None, :]
    blk, off = (slots // c["block"])[:, None], (slots % c["block"])[:, None]
    codes_at[blk, h, off // 16, off % 16] = _packed(code)
    scales_at[blk, h, off // 16, off % 16] = sc.view(torch.uint8)


def _plain_append(s):
    c = s["case"]
    cs = s["cos_sin"][s["positions"].long()][:, None, :]
    cos, sin = cs[..., :c["rot"] // 2], cs[..., c["rot"] // 2:]
    q = _rotated(_normed(s["q"].float(), s["q_weight"]), cos, sin, c["rot"], c["interleaved"])
    k = _rotated(_normed(s["k"].float(), s["k_weight"]), cos, sin, c["rot"], c["interleaved"])[s["live"]]
    s["q_out"].copy_(q)
    slots = s["slots"].long()[s["live"]]
    _put(s["k_pool"], s["k_scale"], k, slots, c)
    _put(s["v_pool"], s["v_scale"], s["v"].float()[s["live"]], slots, c)


def _rows_of(s, name, at):
    """Rows of K or V at positions `at` [S, n] of each sequence: [S, n, H, D] float."""
    c = s["case"]
    phys = torch.gather(s["tables"].long(), 1, (at // c["block"]).clamp(0, s["tables"].shape[1] - 1)).clamp(min=0)
    off = at % c["block"]
    if c["kv"] != "4":
        return s[name + "_pool"][phys, off].float()
    codes, scales = _parts(s[name + "_pool"], c["d"])
    h = torch.arange(c["hkv"], device=at.device)
    i = (phys[..., None], h, (off // 16)[..., None], (off % 16)[..., None])
    x = _values(codes[i]).unflatten(-1, (-1, 16)) * scales[i].view(torch.float8_e4m3fn).float()[..., None]
    x = x.flatten(-2)
    return x if s[name + "_scale"] is None else x * s[name + "_scale"][:, None]


def _plain_attention(q, k, v, live, scale):
    """q [S, H, rows, D], k and v [S, n, H, D], live [S or 1, 1, rows or 1, n]: [S, H, rows, D]."""
    score = (q @ k.permute(0, 2, 3, 1)) * scale
    score = torch.where(live, score, -math.inf)
    top = score.amax(3, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(3, keepdim=True)
    # A row with no token is zero; places that no row sees are left out whatever they hold.
    v = torch.where(live.any(2).transpose(1, 2)[..., None], v, 0.0)
    return (p @ v.transpose(1, 2)) / torch.where(total > 0, total, 1.0)


def _plain_decode(s):
    c = s["case"]
    lens = s["lens"].long()[:, None]
    if c["op"] == "window":
        first = torch.arange(c["sinks"], device=lens.device)[None, :].expand(c["seqs"], -1)
        last = lens - c["window"] + torch.arange(c["window"], device=lens.device)
        at = torch.cat([first, last], 1)
        fresh = torch.cat([first < lens, last >= c["sinks"]], 1)
    else:
        at = torch.arange(max(1, s["max_len"]), device=lens.device)[None, :].expand(c["seqs"], -1)
        fresh = at < lens
    at, live = at.clamp(min=0), fresh[:, None, None, :]
    q = s["q"].float().view(c["seqs"], c["hkv"], -1, c["d"])
    out = _plain_attention(q, _rows_of(s, "k", at), _rows_of(s, "v", at), live, s["scale"])
    s["out"].copy_(out.reshape(c["seqs"], c["hq"], c["d"]))


def _plain_prompt(s):
    c = s["case"]
    S, M, G = c["seqs"], s["max_new"], c["hq"] // c["hkv"]
    q = torch.zeros((S * M, c["hq"], c["d"]), device="cuda")
    q[s["place"]] = s["q"].float()
    q = q.view(S, M, c["hkv"], G, c["d"]).permute(0, 2, 1, 3, 4).reshape(S, c["hkv"], M * G, c["d"])
    new = (s["query_start"][1:] - s["query_start"][:-1]).long()
    p = (s["lens"].long() - new)[:, None] + torch.arange(M, device="cuda")  # positions [S, M]
    t = torch.arange(s["max_len"], device="cuda")
    live = t <= p[..., None]
    if c["window"]:
        live &= (t > p[..., None] - c["window"]) | (t < c["sinks"])
    live &= (torch.arange(M, device="cuda") < new[:, None])[..., None]
    live = live[:, :, None, :].expand(S, M, G, -1).reshape(S, 1, M * G, -1)
    at = t[None, :].expand(S, -1)
    out = _plain_attention(q, _rows_of(s, "k", at), _rows_of(s, "v", at), live, s["scale"])
    out = out.view(S, c["hkv"], M, G, c["d"]).permute(0, 2, 1, 3, 4).reshape(S * M, c["hq"], c["d"])
    s["out"].copy_(out[s["place"]])


def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if own:
        import paged_kv_cache_112_gb300 as pkv

        st = s["status"]
        if op == "append":
            pkv.norm_rope_write_fp4(s["q"], s["k"], s["v"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"],
                                    s["slots"], q_out=s["q_out"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                    eps=1e-6, cos_sin=s["cos_sin"], positions=s["positions"],
                                    interleaved=c["interleaved"], status=st)
        elif op == "attend4":
            pkv.decode_attention_fp4(s["out"], s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"],
                                     s["tables"], s["lens"], s["scale"], partition_size=1024,
                                     max_context_len=s["max_len"], workspace=s["workspace"], status=st)
        elif op == "prompt":
            pkv.prefill_attention(s["out"], s["q"], s["k_pool"], s["v_pool"], s["tables"], s["lens"], s["query_start"],
                                  s["scale"], window=c["window"], sinks=c["sinks"], max_context_len=s["max_len"],
                                  status=st)
        elif c["kv"] == "4":
            pkv.decode_window_fp4(s["out"], s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["tables"],
                                  s["lens"], s["scale"], window=c["window"], sinks=c["sinks"],
                                  max_context_len=s["max_len"], status=st)
        else:
            pkv.decode_window(s["out"], s["q"], s["k_pool"], s["v_pool"], s["tables"], s["lens"], s["scale"],
                              window=c["window"], sinks=c["sinks"], max_context_len=s["max_len"], status=st)
    else:
        {"append": _plain_append, "attend4": _plain_decode, "window": _plain_decode, "prompt": _plain_prompt}[op](s)
    if op != "append":
        return {"out": s["out"]}
    d, f8 = c["d"], torch.float8_e4m3fn

    def values(pool):  # codes as the values they are, four at a time
        words = pool[..., :8 * d].view(torch.int16).int().add_(32768)
        return torch.index_select(s["e4m3_of"], 0, words.view(-1)).view(f8)

    return {"q": s["q_out"], "k": values(s["k_pool"]), "k_scale": s["k_pool"][..., 8 * d:].view(f8),
            "v": values(s["v_pool"]), "v_scale": s["v_pool"][..., 8 * d:].view(f8)}


# ------------------------------------------------------------------ cost


def _visible(c):
    """Per sequence: visible tokens (decode), or visible (query, token) pairs and the tokens that some query sees."""
    lens, new = _lens(c)
    if c["op"] != "prompt":
        seen = lens if c["op"] == "attend4" else np.minimum(lens, c["window"] + np.minimum(
            c["sinks"], np.maximum(lens - c["window"], 0)))
        return int(seen.sum()), int(seen.sum())
    pairs = tokens = 0
    for L, n in zip(lens, new):
        p = np.arange(L - n, L)
        w = c["window"] or int(L)
        low = np.maximum(p - w + 1, 0)
        pairs += int((p + 1 - low + np.minimum(low, c["sinks"])).sum())
        tokens += int(L - low[0] + min(low[0], c["sinks"]))
    return pairs, tokens


def work(case):
    c = case
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    row = 2 * (d * 9 // 16 if c["kv"] == "4" else 2 * d)  # K and V of a token and KV head
    if c["op"] == "append":
        t, live = c["tokens"], c["tokens"] - c.get("padding", 0)
        # q in and out, k and v in and to the pools for the live rows, an angle row, position and slot a token
        return {"bytes": t * (2 * hq * d * 2 + c["rot"] * 4 + 8) + live * hkv * (4 * d + row),
                "flops": t * (hq + hkv) * d * 7}
    pairs, tokens = _visible(c)
    rows = int(_lens(c)[1].sum()) if c["op"] == "prompt" else c["seqs"]
    return {"bytes": tokens * (hkv * row + 4.0 / c["block"]) + rows * hq * d * 4, "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ in 64 bits

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_E4M3 = tuple(m * 2.0 ** -9 for m in range(8)) + tuple((1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)
                                                       if e < 8 or m < 7)


def _nearest(x, grid):
    """|x| to the nearest value of an ascending grid (ties to the even index, the largest beyond it), with x's sign."""
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    middle = (grid[1:] + grid[:-1]) / 2
    a = x.abs()
    i = torch.bucketize(a, middle)  # a tie: the lower index
    i = i + ((i < len(middle)) & (a == middle[i.clamp(max=len(middle) - 1)]) & (i % 2 == 1)).long()
    return torch.copysign(grid[i], x)


def _pool_values(pool, d, head_scale):
    """[NB, H, B, D] in 64 bits."""
    nb, hkv, tiles, _ = pool.shape
    e2m1 = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float64, device=pool.device)
    byte = pool[..., :8 * d].reshape(nb, hkv, tiles * 16, d // 2).long()
    x = torch.stack([e2m1[byte % 16], e2m1[torch.div(byte, 16, rounding_mode="floor")]], -1).view(nb, hkv, -1, d)
    e4m3 = torch.tensor(_E4M3 + (math.nan,), dtype=torch.float64, device=pool.device)
    sc = e4m3[pool[..., 8 * d:].reshape(nb, hkv, tiles * 16, d // 16).long()]
    x = x * sc.repeat_interleave(16, -1)
    return x if head_scale is None else x * head_scale.double().view(1, -1, 1, 1)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    hq, hkv, d, b = c["hq"], c["hkv"], c["d"], c["block"]
    if c["op"] == "append":
        half = c["rot"] // 2
        angle = s["cos_sin"].double()[s["positions"].long()]
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

        out = {"q": head(s["q"], s["q_weight"])}
        slot = s["slots"].long()
        on = slot >= 0
        slot = slot[on]
        for n, new in (("k", head(s["k"], s["k_weight"])), ("v", s["v"].double())):
            pool = s[n + "_pool"]
            nb, _, tiles, _ = pool.shape
            e2m1 = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float64, device="cuda")
            e4m3 = torch.tensor(_E4M3 + (math.nan,), dtype=torch.float64, device="cuda")
            byte = pool[..., :8 * d].long()
            code = torch.stack([e2m1[byte & 15], e2m1[byte >> 4]], -1).view(nb, hkv, b, d)
            scale = e4m3[pool[..., 8 * d:].long()].view(nb, hkv, b, d // 16)
            z = new[on] if s[n + "_scale"] is None else new[on] / s[n + "_scale"].double()[:, None]
            z = z.view(*z.shape[:-1], -1, 16)
            sc = _nearest(z.abs().max(-1).values / 6, _E4M3)
            got = torch.where(sc[..., None] > 0, _nearest(z / sc.clamp(min=2.0 ** -10)[..., None], _E2M1), 0.0)
            at = (slot // b, slice(None), slot % b)
            code[at] = got.flatten(-2)
            scale[at] = sc
            out[n], out[n + "_scale"] = code.reshape(-1), scale.view(nb, hkv, tiles, d)
        return out
    lens, new = _lens(c)
    if c["kv"] == "4":
        k_of, v_of = ((lambda blocks, p=s[n + "_pool"], sc=s[n + "_scale"]: _pool_values(p[blocks], d, sc).transpose(0, 1)
                       .reshape(hkv, -1, d)) for n in ("k", "v"))
    else:
        k_of, v_of = ((lambda blocks, p=s[n + "_pool"]: p[blocks].double().permute(2, 0, 1, 3).reshape(hkv, -1, d))
                      for n in ("k", "v"))
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for i, L in enumerate(int(x) for x in lens):
        n = int(new[i]) if new is not None else 1
        rows, row = slice(row, row + n), row + n
        if L == 0:
            continue
        blocks = s["tables"][i, :-(-L // b)].long()
        k, v = k_of(blocks)[:, :L], v_of(blocks)[:, :L]
        for part in torch.arange(L - n, L, device="cuda").split(1024):
            q = s["q"][rows][part - (L - n)].double().view(len(part), hkv, -1, d)
            logit = torch.einsum("mhgd,htd->hgmt", q, k) * s["scale"]
            t = torch.arange(L, device="cuda")
            hidden = t[None, :] > part[:, None]
            if c.get("window"):
                hidden |= (t[None, :] <= part[:, None] - c["window"]) & (t >= c["sinks"])[None, :]
            weight = torch.softmax(logit.masked_fill(hidden, -math.inf), -1)
            out[rows][part - (L - n)] = torch.einsum("hgmt,htd->mhgd", weight, v).reshape(len(part), hq, d)
    return {"out": out}
