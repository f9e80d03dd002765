"""Cases of two operators of serving around the per-head windowed cache: rotary positions applied on the way into the
cache (a token or a chunk of them turned and stored in one call), and decode attention of sequences that share long
prefixes, each prefix stored and read once for all of them.

``run`` computes a case either in plain torch operations (``own`` false) or through the framework's public entry
points (``own`` true); both work on the same state, and ``exact`` says what the definition gives in 64 bits.

Notation: B sequences, H KV heads of windows w_h, Hq = G H query heads, D head_dim.  Head h keeps its newest tokens
in a ring of C_h = ceil(w_h / block_size) * block_size slots, position p in slot p mod C_h; blocks are numbered
(sequence, head, block) and a block holds block_size K rows, then block_size V rows.  An 8-bit cache stores e4m3 codes
and, for each 16 consecutive slots and K or V, the scale 2^e with the smallest e >= -120 such that
max |finite value| <= 448 * 2^e.

append: row i < n_s of sequence s is token pos_s + i.  Its query and key turn by the angle of position pos_s + i +
(tokens of a prefix kept elsewhere); the turned key and the value go to slot (pos_s + i) mod C_h of every head (the
last C_h rows where there are more).  In an 8-bit cache every group of 16 slots that a row goes to is stored anew, once: the
slots whose tokens are in the window of the new length keep their value or get their row, the others become zero.

shared: sequence s has L_s tokens of its own behind a prefix f = prefix_of[s] of P_f tokens (or behind none, f < 0).
Its one query, of the newest token, attends to its own newest min(w_h, L_s) tokens and to the prefix's tokens at
positions [max(0, P_f + L_s - w_h), P_f), w_h being the own cache's window in the first and the prefix cache's in the second.
"""
import math

import numpy as np
import torch

own = False

LEVELS = (1024, 4096, 16384, 65536)
POLICY = (4096, 4096, 16384, 16384, 65536, 65536, 65536, 65536)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
GROUP = 16        # slots that share a scale
E_MIN = -120      # smallest scale exponent


def _text(windows):
    return " ".join(str(w) for w in windows)


def listed():
    return [
        # the newest token of one sequence: query and key turned, key and value stored; latency alone
        {"name": "append one token", "op": "append", "type": "bf16", "B": 1, "n": 1, "G": 4, "D": 128, "bs": 16,
         "windows": _text(LEVELS + LEVELS), "rot": 128, "layout": "half", "scaling": "none", "fused": True, "keys": False,
         "ahead": 0, "pos_lo": 164864, "pos_hi": 164864},
        # a token each for 64 ragged sequences behind a prefix kept elsewhere, 8-bit cache: every new row has its group scaled anew
        {"name": "append tokens 8-bit", "op": "append", "type": "e4m3", "B": 64, "n": 1, "G": 4, "D": 128, "bs": 16,
         "windows": _text((1024,) * 4 + (4096,) * 4), "rot": 128, "layout": "half", "scaling": "none", "fused": True,
         "keys": False, "ahead": 32768, "pos_lo": 0, "pos_hi": 6000},
        # chunks of four prompts from a fused query-key-value projection, far positions scaled by parts
        {"name": "append chunk", "op": "append", "type": "bf16", "B": 4, "n": 2048, "G": 4, "D": 128, "bs": 16,
         "windows": _text(POLICY), "rot": 128, "layout": "half", "scaling": "by_parts", "fused": True, "keys": False,
         "ahead": 0, "pos_lo": 100000, "pos_hi": 114688},
        # the same into an 8-bit cache, with the turned keys wanted for the chunk's own attention, neighbouring pairs
        {"name": "append chunk 8-bit", "op": "append", "type": "e4m3", "B": 4, "n": 2048, "G": 4, "D": 128, "bs": 16,
         "windows": _text((1024, 4096, 4096, 4096, 16384, 16384, 16384, 16384)), "rot": 128, "layout": "interleaved",
         "scaling": "linear", "fused": True, "keys": True, "ahead": 0, "pos_lo": 10000, "pos_hi": 20000},
        # fp32, part of the head turned, odd blocks and ragged odd chunks longer than the shortest window
        {"name": "append part of the head", "op": "append", "type": "f32", "B": 3, "n": 129, "G": 2, "D": 64, "bs": 5,
         "windows": "23 40 1000 300", "rot": 20, "layout": "half", "scaling": "ntk", "fused": False, "keys": True,
         "ahead": 77, "pos_lo": 0, "pos_hi": 5000},
        # a few sequences that just began behind a short common instruction: the smallest step with a prefix
        {"name": "shared short", "op": "shared", "pool": "bf16", "pre": "bf16", "B": 4, "P": 1, "G": 4, "D": 64, "bs": 16,
         "windows": "512 512 1024 1024", "own": "128 128 256 256", "pre_lo": 900, "pre_hi": 900, "len_lo": 1, "len_hi": 60,
         "alone": 0, "append": True, "cap": 0.0, "bias": False},
        # 16 conversations behind one 32K document, windows of the example policy: bound by reading the document once
        {"name": "shared document", "op": "shared", "pool": "bf16", "pre": "bf16", "B": 16, "P": 1, "G": 4, "D": 128, "bs": 16,
         "windows": _text(POLICY), "own": _text((2048,) * 8), "pre_lo": 32768, "pre_hi": 32768, "len_lo": 1, "len_hi": 2000,
         "alone": 0, "append": True, "cap": 0.0, "bias": False},
        # 128 short answers behind one 60000-token context, groups of 8: 1024 query rows for each key, bound by the products
        {"name": "shared large batch", "op": "shared", "pool": "bf16", "pre": "bf16", "B": 128, "P": 1, "G": 8, "D": 128,
         "bs": 16, "windows": _text(POLICY), "own": _text((512,) * 8), "pre_lo": 60000, "pre_hi": 60000, "len_lo": 1,
         "len_hi": 300, "alone": 0, "append": True, "cap": 0.0, "bias": False},
        # several prefixes of odd lengths, some sequences empty or behind none, narrow heads in groups of 16, larger blocks, no append
        {"name": "shared several", "op": "shared", "pool": "bf16", "pre": "bf16", "B": 41, "P": 5, "G": 16, "D": 64, "bs": 64,
         "windows": "1000 4096 16384 16384", "own": "1000 1500 1500 1500", "pre_lo": 501, "pre_hi": 12001, "len_lo": 0,
         "len_hi": 1501, "alone": 3, "append": False, "cap": 0.0, "bias": False},
        # 8-bit caches on both sides, 32 sequences behind two 32K prefixes
        {"name": "shared 8-bit", "op": "shared", "pool": "e4m3", "pre": "e4m3", "B": 32, "P": 2, "G": 4, "D": 128, "bs": 16,
         "windows": _text(POLICY), "own": _text((2048,) * 8), "pre_lo": 32768, "pre_hi": 32768, "len_lo": 1, "len_hi": 2000,
         "alone": 0, "append": True, "cap": 0.0, "bias": False},
        # capped scores lowered with distance, 24 sequences behind one 16K prefix
        {"name": "shared capped biased", "op": "shared", "pool": "bf16", "pre": "bf16", "B": 24, "P": 1, "G": 8, "D": 128,
         "bs": 32, "windows": "4096 8192 16384 16384", "own": "1024 1024 1024 1024", "pre_lo": 16001, "pre_hi": 16001,
         "len_lo": 0, "len_hi": 1000, "alone": 1, "append": True, "cap": 50.0, "bias": True},
        # fp32 caches with odd blocks: the check of a model in full precision
        {"name": "shared fp32", "op": "shared", "pool": "f32", "pre": "f32", "B": 6, "P": 2, "G": 2, "D": 64, "bs": 24,
         "windows": "300 2000 3000 3001", "own": "300 500 500 500", "pre_lo": 1001, "pre_hi": 2999, "len_lo": 0,
         "len_hi": 499, "alone": 1, "append": True, "cap": 0.0, "bias": False},
    ]


def _between(rng, lo, hi):
    """A whole number from [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("append", "shared"))
    D = rng.choice((64, 128))
    H = rng.choice((1, 2, 3, 4, 8))
    if op == "append":
        kind = rng.choice(("bf16", "bf16", "e4m3", "f32"))
        bs = rng.choice((16, 32, 64, 128) if kind == "e4m3" else (16, 32, 64, 5, 24))
        n = rng.choice((1, _between(rng, 1, 2048)))
        pos = _between(rng, 1, 160000)
        return {"op": "append", "type": kind, "B": _between(rng, 1, max(1, min(64, 8192 // n))), "n": n,
                "G": _between(rng, 1, 8 if H < 8 else 4), "D": D, "bs": bs, "windows": _text(_between(rng, 1, 16384) for _ in range(H)),
                "rot": rng.choice((D, D, 2 * rng.randint(1, D // 2))), "layout": rng.choice(("half", "interleaved")),
                "scaling": rng.choice(("none", "linear", "ntk", "by_parts")), "fused": rng.random() < 0.5,
                "keys": rng.random() < 0.3, "ahead": rng.choice((0, 0, _between(rng, 1, 100000))), "pos_lo": rng.choice((0, pos // 2, pos)),
                "pos_hi": pos}
    pool, pre = rng.choice((("bf16", "bf16"), ("bf16", "bf16"), ("e4m3", "e4m3"), ("bf16", "e4m3"), ("e4m3", "bf16"), ("f32", "f32")))
    small = pool == "f32"
    bs = rng.choice((16, 24, 5) if small else (16, 16, 32, 64, 128))
    B = _between(rng, 1, 24 if small else 128)
    P = _between(rng, 1, min(B, 8))
    hi = _between(rng, 1, 4000 if small else 30000)
    length = _between(rng, 1, 2000)
    scored = rng.random() < 0.3
    return {"op": "shared", "pool": pool, "pre": pre, "B": B, "P": P, "G": _between(rng, 1, 4 if B > 48 else 16), "D": D, "bs": bs,
            "windows": _text(_between(rng, 1, 65536) for _ in range(H)), "own": _text(_between(rng, 1, 2048) for _ in range(H)),
            "pre_lo": rng.choice((0, hi // 2, hi)), "pre_hi": hi, "len_lo": rng.choice((0, length // 2)), "len_hi": length,
            "alone": rng.choice((0, 0, min(B, 2))), "append": rng.random() < 0.7,
            "cap": rng.choice((20.0, 50.0, 0.0)) if scored else 0.0, "bias": scored and rng.random() < 0.6}


# ---- the cache's geometry -----------------------------------------------------------------------------------------
def _ints(text):
    return [int(w) for w in text.split()]


def _rings(windows, bs):
    """(window, ring capacity, first block within a sequence) of each head, and the blocks of a sequence."""
    at, rings = 0, []
    for w in _ints(windows):
        n = -(-w // bs)
        rings.append((w, n * bs, at))
        at += n
    return rings, at


def _whole(lo, hi, seed, n):
    return np.random.default_rng(seed).integers(lo, hi, size=n, endpoint=True).astype(np.int64)


def _slopes(heads):
    """The usual geometric slopes of a distance bias: 2^(-8 (i + 1) / heads)."""
    return [2.0 ** (-8.0 * (i + 1) / heads) for i in range(heads)]


def _freqs(case):
    """Radians per position of each rotated pair, and the factor on the result, in 64 bits."""
    rot, base, factor, first = case["rot"], 10000.0, 8.0, 16384
    i = np.arange(rot // 2, dtype=np.float64)
    if case["scaling"] == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "by_parts":
        turns = first * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return f * keep + f / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0
    return f, 1.0


# ---- inputs -------------------------------------------------------------------------------------------------------
def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _randn(gen, shape, scale=1.0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=gen.device).mul_(scale).to(dtype)


def _i32(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _power(e):
    """2^e as fp32, exactly, for whole -126 <= e <= 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(amax):
    """The smallest e >= E_MIN with amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    m, ex = torch.frexp(amax)
    e = ex - 9 + (m > 0.875).to(ex.dtype)
    return torch.where(amax > 0, e.clamp(min=E_MIN), torch.full_like(e, E_MIN))


def _encode(x):
    """Codes and scales of groups x [..., 16, D] of finite fp32 values."""
    e = _exponent(x.abs().amax((-1, -2)))
    return (x * _power(-e)[..., None, None]).to(torch.float8_e4m3fn), _power(e)


def _cache(gen, kind, windows, bs, seqs, D):
    """Blocks and scales of a cache in the middle of serving: every slot holds a row."""
    _, per_seq = _rings(windows, bs)
    blocks = _randn(gen, (seqs * per_seq, 2, bs, D), 1.0, torch.float32 if kind == "f32" else torch.bfloat16)
    blocks[:, 0, :, : D // 16] *= 4  # a few strong channels, as keys have
    if kind != "e4m3":
        return blocks, None
    codes, scales = _encode(blocks.view(seqs * per_seq, 2, bs // GROUP, GROUP, D).float())
    return codes.view(seqs * per_seq, 2, bs, D), scales.transpose(1, 2).contiguous()


def _pool(kind, windows, bs, seqs, D, G, blocks, scales):
    import head_budgeted_kv_gb300 as hw
    H = len(_ints(windows))
    pool = hw.Pool(1, H, D, bs, [_ints(windows)], seqs, DTYPES[kind], q_heads=G * H)
    pool.blocks().copy_(blocks)
    if scales is not None:
        pool.scales().copy_(scales)
    return pool


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    s = {"case": case}
    B, G, D, bs = (case[k] for k in ("B", "G", "D", "bs"))
    H = len(_ints(case["windows"]))
    if case["op"] == "append":
        kind, n = case["type"], case["n"]
        io = torch.float32 if kind == "f32" else torch.bfloat16
        if case["fused"]:  # query, key and value heads of one projection's output
            qkv = _randn(gen, (B, n, (G + 2) * H, D), 1.0, io)
            s["q"], s["k"], s["v"] = qkv.split((G * H, H, H), 2)
        else:
            s["q"] = _randn(gen, (B, n, G * H, D), 1.0, io)
            s["k"], s["v"] = (_randn(gen, (B, n, H, D), 1.0, io) for _ in range(2))
        s["q_out"] = torch.zeros((B, n, G * H, D), dtype=io, device=dev)
        s["k_out"] = torch.zeros((B, n, H, D), dtype=io, device=dev) if case["keys"] else None
        pos = _whole(case["pos_lo"], case["pos_hi"], seed, B)
        s["pos"], s["n"] = _i32(pos, dev), _i32(_whole((n + 1) // 2, n, seed + 1, B), dev)
        s["turn_pos"] = _i32(pos + case["ahead"], dev) if case["ahead"] else None
        f, s["factor"] = _freqs(case)
        s["freq"] = torch.tensor(f, dtype=torch.float64, device=dev)
        s["blocks"], s["scales"] = _cache(gen, kind, case["windows"], bs, B, D)
        if own:
            import head_budgeted_kv_gb300 as hw
            s["table"] = hw.rope_table(D, rot_dim=case["rot"], base=10000.0, layout=case["layout"], scaling=case["scaling"],
                                       factor=8.0, original_len=16384)
            s["pool"] = _pool(kind, case["windows"], bs, B, D, G, s.pop("blocks"), s["scales"])
        return s
    io = torch.float32 if case["pool"] == "f32" else torch.bfloat16
    s["q"] = _randn(gen, (B, G * H, D), 2.0, io)
    s["k"], s["v"] = (_randn(gen, (B, H, D), 1.0, io) for _ in range(2))
    s["out"] = torch.zeros_like(s["q"])
    s["slopes"] = torch.tensor(_slopes(G * H), dtype=torch.float32, device=dev) if case["bias"] else None
    s["scale"] = 1.0 / math.sqrt(D)
    s["lens"] = _i32(_whole(case["len_lo"], case["len_hi"], seed, B), dev)
    s["pre_lens"] = _i32(_whole(case["pre_lo"], case["pre_hi"], seed + 1, case["P"]), dev)
    of = _whole(0, case["P"] - 1, seed + 2, B)
    of[np.random.default_rng(seed + 3).permutation(B)[: case["alone"]]] = -1
    s["prefix_of"] = _i32(of, dev)
    s["blocks"], s["scales"] = _cache(gen, case["pool"], case["own"], bs, B, D)
    s["pre_blocks"], s["pre_scales"] = _cache(gen, case["pre"], case["windows"], bs, case["P"], D)
    if own:
        s["pool"] = _pool(case["pool"], case["own"], bs, B, D, G, s.pop("blocks"), s["scales"])
        s["prefix"] = _pool(case["pre"], case["windows"], bs, case["P"], D, G, s.pop("pre_blocks"), s["pre_scales"])
    return s


# ---- the plain forms ----------------------------------------------------------------------------------------------
def _turned(x, angle, factor, rot, halves):
    """x [B, n, heads, D] with the pairs of its first rot dims turned, in fp32; angle [B, n, pairs] in 64 bits."""
    cos, sin = ((t * factor).float()[:, :, None] for t in (angle.cos(), angle.sin()))
    y = x.float().clone()
    first, second = (slice(0, rot // 2), slice(rot // 2, rot)) if halves else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., first].float(), x[..., second].float()
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_append(s):
    case = s["case"]
    rings, per_seq = _rings(case["windows"], case["bs"])
    B, n, D, bs = case["B"], case["n"], case["D"], case["bs"]
    dev = s["pos"].device
    i = torch.arange(n, device=dev)[None]
    pos, rows = s["pos"].long()[:, None], s["n"].long()[:, None]
    at = (s["pos"] if s["turn_pos"] is None else s["turn_pos"]).double()[:, None] + i
    angle = at[..., None] * s["freq"]                                 # 64 bits: far positions
    halves = case["layout"] == "half"
    q, k = (_turned(s[x], angle, s["factor"], case["rot"], halves) for x in ("q", "k"))
    mine = (i < rows)[..., None, None]
    got = {"q": s["q_out"]}
    s["q_out"].copy_(torch.where(mine, q.to(s["q_out"].dtype), s["q_out"]))
    if case["keys"]:
        s["k_out"].copy_(torch.where(mine, k.to(s["k_out"].dtype), s["k_out"]))
        got["k"] = s["k_out"]
    for h, (w, C, first) in enumerate(rings):
        new = torch.stack((k[:, :, h], s["v"][:, :, h].float()), 2)   # [B, n, 2, D]
        if s["scales"] is None:
            b, j = torch.nonzero((i < rows) & (i >= rows - C), as_tuple=True)
            slot = (pos[b, 0] + j) % C
            s["blocks"][b * per_seq + first + slot // bs, :, slot % bs] = new[b, j].to(s["blocks"].dtype)
            continue
        # groups of 16 positions, as many as a chunk can touch, the newest of each ring place
        end = pos + rows
        last = (end - 1) // GROUP
        m = pos // GROUP + torch.arange((n + 2 * GROUP - 2) // GROUP, device=dev)[None]
        b, j = torch.nonzero((m <= last) & (m > last - C // GROUP) & (rows > 0), as_tuple=True)
        m = m[b, j][:, None]
        t = torch.arange(GROUP, device=dev)[None]
        p = m * GROUP + t                                             # [groups, 16]
        p = torch.where(p < end[b], p, p - C)                         # the newest position of each slot
        live = (p >= 0) & (p >= end[b] - w)
        g = m[:, 0] * GROUP % C
        blk, sub = b * per_seq + first + g // bs, g % bs // GROUP
        old = s["blocks"].view(-1, 2, bs // GROUP, GROUP, D)[blk, :, sub].float() * s["scales"][blk, sub][..., None, None]
        fresh = new[b[:, None], (p - pos[b]).clamp(0, n - 1)].transpose(1, 2)
        x = torch.where((p >= pos[b])[:, None, :, None], fresh, old)
        codes, sc = _encode(torch.where(live[:, None, :, None], x, torch.zeros_like(x)))
        s["blocks"].view(torch.uint8).view(-1, 2, bs // GROUP, GROUP, D)[blk, :, sub] = codes.view(torch.uint8)
        s["scales"][blk, sub] = sc
    got["blocks"] = s["blocks"]
    if s["scales"] is not None:
        got["scales"] = s["scales"]
    return got


def _plain_store(s):
    """The new row of every (sequence, head) into its slot of the sequences' own cache."""
    case = s["case"]
    rings, per_seq = _rings(case["own"], case["bs"])
    B, D, bs, dev = case["B"], case["D"], case["bs"], s["lens"].device
    w, C, first = (torch.tensor(v, device=dev)[None] for v in zip(*rings))
    pos = s["lens"].long()[:, None]
    t = pos % C                                                       # [B, H]
    blk = torch.arange(B, device=dev)[:, None] * per_seq + first + t // bs
    new = torch.stack((s["k"], s["v"]), 2)                            # [B, H, 2, D]
    if s["scales"] is None:
        s["blocks"][blk, :, t % bs] = new
        return
    g, r = t % bs // GROUP, t % GROUP
    age = (r[..., None] - torch.arange(GROUP, device=dev)) % C[..., None]
    live = (age > 0) & (age < w[..., None]) & (age <= pos[..., None])
    groups = s["blocks"].view(-1, 2, bs // GROUP, GROUP, D)
    x = groups[blk, :, g].float() * s["scales"][blk, g][..., None, None]
    x = torch.where(live[:, :, None, :, None], x, torch.zeros_like(x))
    x = torch.where((age == 0)[:, :, None, :, None], new.float()[..., None, :], x)
    codes, sc = _encode(x)
    groups.view(torch.uint8)[blk, :, g] = codes.view(torch.uint8)
    s["scales"][blk, g] = sc


def _plain_rows(blocks, scales, per_seq, first, n):
    """K and V of all slots of one head of a cache as fp32 [sequences, C, D]."""
    bs, D = blocks.shape[2:]
    x = blocks.view(-1, per_seq, 2, bs, D)[:, first:first + n].float()
    if scales is not None:
        sc = scales.view(-1, per_seq, bs // GROUP, 2)[:, first:first + n].transpose(2, 3)
        x = (x.view(-1, n, 2, bs // GROUP, GROUP, D) * sc[..., None, None]).view(-1, n, 2, bs, D)
    return x[:, :, 0].reshape(-1, n * bs, D), x[:, :, 1].reshape(-1, n * bs, D)


def _scored(x, cap, slopes, distance):
    if cap > 0:
        x = cap * torch.tanh(x / cap)
    return x if slopes is None else x - slopes * distance


def _plain_shared(s):
    case = s["case"]
    B, P, G, D, bs = (case[k] for k in ("B", "P", "G", "D", "bs"))
    (mine, per_own), (pre, per_pre) = _rings(case["own"], bs), _rings(case["windows"], bs)
    if case["append"]:
        _plain_store(s)
    lens = s["lens"].long()[:, None] + (1 if case["append"] else 0)   # [B, 1]
    q = s["q"].float().view(B, len(mine), G, D)
    dev = lens.device
    members = [torch.nonzero(s["prefix_of"] == f)[:, 0] for f in range(-1, P)]
    for h, ((w, C, at), (pw, pC, pat)) in enumerate(zip(mine, pre)):
        k, v = _plain_rows(s["blocks"], s["scales"], per_own, at, C // bs)
        pk, pv = _plain_rows(s["pre_blocks"], s["pre_scales"], per_pre, pat, pC // bs)
        age = (lens - 1 - torch.arange(C, device=dev)) % C            # distance from the query's token
        seen = (age < w) & (age < lens)
        v = torch.where(seen[..., None], v, torch.zeros_like(v))
        slopes = None if s["slopes"] is None else s["slopes"][h * G:(h + 1) * G].view(1, G, 1)
        for f, idx in enumerate(members, -1):
            if not len(idx):
                continue
            qf = q[idx, h]                                            # [m, G, D]
            x = _scored((qf @ k[idx].transpose(1, 2)) * s["scale"], case["cap"], slopes, age[idx][:, None].float())
            x = torch.where(seen[idx][:, None], x, torch.full_like(x, -math.inf))
            if f >= 0:  # the prefix's keys, one product for all of its sequences
                N = s["pre_lens"][f].long()
                t = torch.arange(pC, device=dev)
                p = N - 1 - (N - 1 - t) % pC                          # the newest position of each slot
                d = N + lens[idx] - 1 - p                             # [m, pC]
                visible = ((p >= 0) & (d < pw))[:, None]
                y = _scored((qf.reshape(-1, D) @ pk[f].T).view(-1, G, pC) * s["scale"], case["cap"], slopes, d[:, None].float())
                x = torch.cat((x, torch.where(visible, y, torch.full_like(y, -math.inf))), 2)
            top = x.amax(-1, keepdim=True)
            e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
            total = e.sum(-1, keepdim=True)
            o = e[..., :C] @ v[idx]
            if f >= 0:
                o = o + (e[..., C:].reshape(-1, pC) @ pv[f]).view(-1, G, D)
            s["out"][idx, h * G:(h + 1) * G] = (o / torch.where(total > 0, total, torch.ones_like(total))).to(s["out"].dtype)
    return _with_cache(case, s["out"], s["blocks"], s["scales"])


def _with_cache(case, out, blocks, scales):
    if not case["append"]:
        return {"out": out}
    return {"out": out, "blocks": blocks} if scales is None else {"out": out, "blocks": blocks, "scales": scales}


def run(s):
    case = s["case"]
    if not own:
        return _plain_append(s) if case["op"] == "append" else _plain_shared(s)
    pool = s["pool"]
    if case["op"] == "append":
        q, k = pool.rope_append(0, s["table"], s["q"], s["k"], s["v"], s["pos"], n=s["n"], q_out=s["q_out"], k_out=s["k_out"],
                                turn_pos=s["turn_pos"])
        got = {"q": q, "k": k, "blocks": pool.blocks()} if case["keys"] else {"q": q, "blocks": pool.blocks()}
        if s["scales"] is not None:
            got["scales"] = pool.scales()
        return got
    score = {"softcap": case["cap"], "slopes": s["slopes"]} if case["cap"] > 0 or case["bias"] else {}
    new = {"k_new": s["k"], "v_new": s["v"]} if case["append"] else {}
    out = pool.shared_decode(0, s["prefix"], s["q"], s["scale"], s["lens"], s["prefix_of"], s["pre_lens"], out=s["out"], **new, **score)
    return _with_cache(case, out, pool.blocks(), pool.scales() if case["pool"] == "e4m3" else None)


# ---- what a pass cannot do without --------------------------------------------------------------------------------
_BYTES = {"e4m3": 1, "bf16": 2, "f32": 4}


def work(case):
    G, D = case["G"], case["D"]
    wins = np.array(_ints(case["windows"]), dtype=np.float64)
    H = len(wins)
    if case["op"] == "append":
        size, kind = (4 if case["type"] == "f32" else 2), case["type"]
        n = 0.75 * case["n"] if case["n"] > 1 else 1.0  # rows a sequence has: half of n to all of it
        rows = case["B"] * n
        stored = case["B"] * float(np.minimum(wins, n).sum())  # rows that stay
        read = rows * (G * H + (H if case["keys"] else 0)) * D * size + stored * 2 * D * size - (stored * D * size if case["keys"] else 0)
        wrote = rows * (G * H + (H if case["keys"] else 0)) * D * size + stored * (2 * D * _BYTES[kind] + (8 / GROUP if kind == "e4m3" else 0))
        return {"bytes": read + wrote, "flops": 3 * rows * (G + 1) * H * D}
    B, P = case["B"], case["P"]
    mine = np.array(_ints(case["own"]), dtype=np.float64)
    io = 4 if case["pool"] == "f32" else 2
    per = {k: 2 * D * _BYTES[case[k]] + (8 / GROUP if case[k] == "e4m3" else 0) for k in ("pool", "pre")}
    lens = np.linspace(case["len_lo"], case["len_hi"], 65)[:, None] + (1 if case["append"] else 0)
    plen = np.linspace(case["pre_lo"], case["pre_hi"], 65)[:, None]
    own_tokens = B * float(np.minimum(mine, lens).sum(1).mean())
    visible = np.clip(np.minimum(plen[:, :, None], wins - lens.reshape(1, -1, 1)), 0, None)  # a prefix's keys that a row sees
    pairs = (B - case["alone"]) * float(visible.sum(2).mean())
    # a prefix is read as far as its sequence with the shortest own part looks
    used = min(P, B - case["alone"])
    read = used * float(np.clip(np.minimum(plen, wins - lens.min()), 0, None).sum(1).mean())
    fresh = B * H * 2 * D * (io + _BYTES[case["pool"]]) if case["append"] else 0
    return {"bytes": own_tokens * per["pool"] + read * per["pre"] + fresh + 2 * B * G * H * D * io,
            "flops": 4.0 * G * D * (own_tokens + pairs)}


# ---- the definitions in 64 bits, apart from the plain forms --------------------------------------------------------
def _nearest_e4m3(y):
    """The e4m3 value nearest to each |y| <= 448 (ties to even): steps of 2^-9 below 2^-6, of an eighth of the power of two above."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(y / step) * step


def _group64(x):
    """Code values and scales of groups [..., 16, D] in 64 bits."""
    top = x.abs().amax((-1, -2))
    e = torch.ceil(torch.log2((top / 448.0).clamp(min=2.0 ** E_MIN)))
    e = torch.where(448.0 * torch.exp2(e - 1) >= top, e - 1, e).clamp(min=E_MIN)  # a logarithm may round up at a power of two
    e = torch.where(448.0 * torch.exp2(e) < top, e + 1, e)
    return _nearest_e4m3(x / torch.exp2(e)[..., None, None]), torch.exp2(e)


def _turn64(x, positions, s, case):
    """Rows x [n, heads, D] turned as complex numbers at positions [n]."""
    half = case["rot"] // 2
    lo = torch.arange(half) if case["layout"] == "half" else torch.arange(0, case["rot"], 2)
    hi = lo + (half if case["layout"] == "half" else 1)
    angle = torch.outer(positions.double(), s["freq"])
    z = torch.complex(x[..., lo].double(), x[..., hi].double()) * torch.polar(torch.full_like(angle, s["factor"]), angle)[:, None]
    y = x.double().clone()
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _store64(blocks, scales, b0, ring, bs, pos, rows):
    """Stores rows [2][n, D] (64-bit K and V) of positions pos .. of one (sequence, head) in the cache's 64-bit copy."""
    w, C = ring
    n, D, dev = rows[0].shape[0], rows[0].shape[1], blocks.device
    end = pos + n
    new = torch.arange(max(pos, end - C), end, device=dev)
    if not len(new):
        return
    slot = new % C
    if scales is None:
        for i in range(2):
            blocks[b0 + slot // bs, i, slot % bs] = rows[i][new - pos]
        return
    nb = C // bs
    hit = torch.zeros(C, dtype=torch.bool, device=dev)
    hit[slot] = True
    hit = hit.view(nb, bs // GROUP, GROUP).any(-1)                      # groups stored anew
    kept = torch.arange(min(pos, max(0, end - w)), pos, device=dev) % C  # slots that keep their value
    fresh = torch.arange(max(pos, end - w), end, device=dev)
    for i in range(2):
        was = (blocks[b0:b0 + nb, i].view(nb, bs // GROUP, GROUP, D) * scales[b0:b0 + nb, :, i][..., None, None]).view(C, D)
        x = torch.zeros_like(was)
        x[kept] = was[kept]
        x[fresh % C] = rows[i][fresh - pos]
        val, sc = _group64(x.view(nb, bs // GROUP, GROUP, D))
        old = blocks[b0:b0 + nb, i].view(nb, bs // GROUP, GROUP, D)
        blocks[b0:b0 + nb, i] = torch.where(hit[..., None, None], val, old).view(nb, bs, D)
        scales[b0:b0 + nb, :, i] = torch.where(hit, sc, scales[b0:b0 + nb, :, i])


def _exact_append(case, s):
    rings, per_seq = _rings(case["windows"], case["bs"])
    blocks = s["blocks"].double()
    scales = None if s["scales"] is None else s["scales"].double()
    got = {"q": s["q_out"].double()}
    if case["keys"]:
        got["k"] = s["k_out"].double()
    for b, (pos, n) in enumerate(zip(s["pos"].tolist(), s["n"].tolist())):
        at = pos + case["ahead"] + torch.arange(n, device=blocks.device)
        got["q"][b, :n] = _turn64(s["q"][b, :n], at, s, case)
        k = _turn64(s["k"][b, :n], at, s, case)
        if case["keys"]:
            got["k"][b, :n] = k
        for h, (w, C, first) in enumerate(rings):
            _store64(blocks, scales, b * per_seq + first, (w, C), case["bs"], pos, (k[:, h], s["v"][b, :n, h].double()))
    got["blocks"] = blocks
    if scales is not None:
        got["scales"] = scales
    return got


def _newest64(blocks, scales, b0, C, bs, first, end):
    """K and V at positions first .. end - 1 of one (sequence, head), 64 bits."""
    slot = torch.arange(first, end, device=blocks.device) % C
    kv = [blocks[b0 + slot // bs, i, slot % bs] for i in range(2)]
    if scales is not None:
        kv = [x * scales[b0 + slot // bs, slot % bs // GROUP, i][:, None] for i, x in enumerate(kv)]
    return kv


def _exact_shared(case, s):
    B, P, G, D, bs, cap = (case[k] for k in ("B", "P", "G", "D", "bs", "cap"))
    (mine, per_own), (pre, per_pre) = _rings(case["own"], bs), _rings(case["windows"], bs)
    blocks, pre_blocks = s["blocks"].double(), s["pre_blocks"].double()
    scales, pre_scales = (None if t is None else t.double() for t in (s["scales"], s["pre_scales"]))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=blocks.device)
    of, lens = s["prefix_of"].tolist(), s["lens"].tolist()
    for h, ((w, C, at), (pw, pC, pat)) in enumerate(zip(mine, pre)):
        slopes = None if s["slopes"] is None else s["slopes"][h * G:(h + 1) * G].double()[:, None]
        shared = [None] * P
        for f, N in enumerate(s["pre_lens"].tolist()):
            shared[f] = (max(0, N - pw), N, _newest64(pre_blocks, pre_scales, f * per_pre + pat, pC, bs, max(0, N - pw), N))
        for b in range(B):
            b0, L = b * per_own + at, lens[b]
            if case["append"]:
                _store64(blocks, scales, b0, (w, C), bs, L, (s["k"][b, h].double()[None], s["v"][b, h].double()[None]))
                L += 1
            first = max(0, L - w)
            k, v = _newest64(blocks, scales, b0, C, bs, first, L)
            d = L - 1 - torch.arange(first, L, device=blocks.device)
            if of[b] >= 0:
                lo, N, (pk, pv) = shared[of[b]]
                since = max(lo, N + L - pw)                               # the oldest token that the window reaches
                if since < N:
                    k, v = torch.cat((pk[since - lo:], k)), torch.cat((pv[since - lo:], v))
                    d = torch.cat((N + L - 1 - torch.arange(since, N, device=d.device), d))
            if not len(d):
                continue
            x = s["q"][b, h * G:(h + 1) * G].double() @ k.T * s["scale"]
            if cap > 0:
                x = cap * torch.tanh(x / cap)
            if slopes is not None:
                x = x - slopes * d
            out[b, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v
    return _with_cache(case, out, blocks, scales)


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return _exact_append(case, s) if case["op"] == "append" else _exact_shared(case, s)
