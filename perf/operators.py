"""Cases of the operators around the per-head windowed cache: the 8-bit pool (prompt storage, append and decode
attention), rotary positions, and attention with capped or distance-biased scores.

``run`` computes a case either in plain torch operations (``own`` false) or through the framework's public entry
points (``own`` true); both work on the same state, and ``exact`` says what the definition gives in 64 bits.

Notation: B sequences, H KV heads of windows w_h, Hq = G H query heads, D head_dim.  Head h keeps its newest tokens
in a ring of C_h = ceil(w_h / block_size) * block_size slots, position p in slot p mod C_h; blocks are numbered
(sequence, head, block) and a block holds block_size K rows, then block_size V rows.  An 8-bit pool stores e4m3 codes
and, for each 16 consecutive slots and K or V, the scale 2^e with the smallest e >= -120 such that
max |finite value| <= 448 * 2^e; storing a token scales its whole group anew from the stored values of the slots that
are still in the window, and writes zeros to the others.
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


def listed():
    return [
        # a short prompt of one sequence stored in a small 8-bit pool: windows that are no multiple of a block
        {"name": "store short prompt", "op": "store", "B": 1, "D": 64, "bs": 16, "windows": "33 128", "len_lo": 77,
         "len_hi": 77},
        # one layer of a four-sequence prefill of up to 32K tokens stored with the example policy's windows
        {"name": "store policy layer", "op": "store", "B": 4, "D": 128, "bs": 16, "windows": _text(POLICY),
         "len_lo": 30000, "len_hi": 32768},
        # one decode step of one layer at batch 1 and 161K context: the smallest step that serving meets
        {"name": "decode8 batch 1", "op": "decode", "pool": "e4m3", "B": 1, "G": 4, "D": 128, "bs": 16,
         "windows": _text(LEVELS + LEVELS), "len_lo": 164864, "len_hi": 164864, "append": True, "cap": 0.0, "bias": False},
        # one decode step of one layer, four sequences at 112K with the example policy
        {"name": "decode8 policy layer", "op": "decode", "pool": "e4m3", "B": 4, "G": 4, "D": 128, "bs": 16,
         "windows": _text(POLICY), "len_lo": 114688, "len_hi": 114688, "append": True, "cap": 0.0, "bias": False},
        # 64 ragged sequences, some of them empty, narrow heads in groups of 16, larger blocks, no append
        {"name": "decode8 ragged", "op": "decode", "pool": "e4m3", "B": 64, "G": 16, "D": 64, "bs": 64,
         "windows": "1000 4096 16384 16384", "len_lo": 0, "len_hi": 20000, "append": False, "cap": 0.0, "bias": False},
        # the query and key of one new token, batch 1: latency alone
        {"name": "rope one token", "op": "rope", "type": "bf16", "B": 1, "n": 1, "H": 8, "G": 4, "D": 128, "rot": 128,
         "layout": "half", "scaling": "none", "fused": False, "pos_lo": 164864, "pos_hi": 164864},
        # a prefill chunk inside a fused query-key-value projection, far positions scaled by parts
        {"name": "rope chunk", "op": "rope", "type": "bf16", "B": 4, "n": 2048, "H": 8, "G": 4, "D": 128, "rot": 128,
         "layout": "half", "scaling": "by_parts", "fused": True, "pos_lo": 100000, "pos_hi": 114688},
        # fp32, pairs of neighbours, only part of the head rotated, ragged odd chunk
        {"name": "rope part of the head", "op": "rope", "type": "f32", "B": 3, "n": 129, "H": 4, "G": 2, "D": 64, "rot": 24,
         "layout": "interleaved", "scaling": "linear", "fused": False, "pos_lo": 0, "pos_hi": 5000},
        # capped scores, decode of eight sequences at 32K
        {"name": "capped decode", "op": "decode", "pool": "bf16", "B": 8, "G": 4, "D": 128, "bs": 16,
         "windows": _text(LEVELS + LEVELS), "len_lo": 32768, "len_hi": 32768, "append": True, "cap": 50.0, "bias": False},
        # capped scores with a distance bias over an 8-bit pool, a few short ragged sequences
        {"name": "capped biased decode8", "op": "decode", "pool": "e4m3", "B": 5, "G": 8, "D": 128, "bs": 32,
         "windows": "100 1000 777 2048", "len_lo": 1, "len_hi": 3001, "append": True, "cap": 30.0, "bias": True},
        # a prefill chunk of 1024 tokens with capped scores at a 40000-token context
        {"name": "capped prefill", "op": "prefill", "B": 1, "n": 1024, "G": 4, "D": 128, "bs": 16,
         "windows": _text(LEVELS + LEVELS), "len_lo": 40000, "len_hi": 40000, "cap": 50.0, "bias": False},
        # short ragged chunks with a distance bias
        {"name": "biased prefill", "op": "prefill", "B": 3, "n": 200, "G": 2, "D": 64, "bs": 16,
         "windows": "64 500 1024 300", "len_lo": 0, "len_hi": 900, "cap": 0.0, "bias": True},
    ]


def _text(windows):
    return " ".join(str(w) for w in windows)


def _between(rng, lo, hi):
    """A whole number from [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("store", "decode", "decode", "rope", "scored", "prefill"))
    D = rng.choice((64, 128))
    bs = rng.choice((16, 16, 32, 64, 128))
    H = rng.choice((1, 2, 4, 8))
    if op == "rope":
        rot = rng.choice((D, D, 2 * rng.randint(1, D // 2)))
        n = rng.choice((1, _between(rng, 1, 2048)))
        pos = _between(rng, 1, 160000)
        return {"op": "rope", "type": rng.choice(("bf16", "bf16", "f32")), "B": _between(rng, 1, max(1, min(64, 8192 // n))),
                "n": n, "H": H, "G": _between(rng, 1, 4), "D": D, "rot": rot, "layout": rng.choice(("half", "interleaved")),
                "scaling": rng.choice(("none", "linear", "ntk", "by_parts")), "fused": rng.random() < 0.5,
                "pos_lo": pos // 2, "pos_hi": pos}
    windows = _text(_between(rng, 1, 16384) for _ in range(H))
    B = _between(rng, 1, 16)
    hi = _between(rng, 1, 30000)
    lo = rng.choice((0, hi // 2, hi))
    if op == "store":
        return {"op": "store", "B": min(B, 6), "D": D, "bs": bs, "windows": windows, "len_lo": lo, "len_hi": hi}
    if op == "prefill":
        return {"op": "prefill", "B": min(B, 3), "n": _between(rng, 1, 700), "G": _between(rng, 1, 4), "D": D, "bs": bs,
                "windows": windows, "len_lo": lo, "len_hi": hi, "cap": rng.choice((0.0, 30.0, 50.0)), "bias": rng.random() < 0.5}
    scored = op == "scored"
    return {"op": "decode", "pool": rng.choice(("e4m3", "bf16", "f32")) if scored else "e4m3", "B": B,
            "G": _between(rng, 1, 16), "D": D, "bs": bs, "windows": windows, "len_lo": lo, "len_hi": hi,
            "append": rng.random() < 0.7, "cap": rng.choice((20.0, 50.0)) if scored else 0.0,
            "bias": scored and rng.random() < 0.6}


# ---- the cache's geometry -----------------------------------------------------------------------------------------
def _windows(case):
    return [int(w) for w in case["windows"].split()]


def _rings(case):
    """(window, ring capacity, first block within a sequence) of each head, and the blocks of a sequence."""
    bs, at, rings = case["bs"], 0, []
    for w in _windows(case):
        n = -(-w // bs)
        rings.append((w, n * bs, at))
        at += n
    return rings, at


def _lens(case, seed, n, lo="len_lo", hi="len_hi"):
    rng = np.random.default_rng(seed)
    return rng.integers(case[lo], case[hi], size=n, endpoint=True).astype(np.int64)


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


def _power(e):
    """2^e as fp32, exactly, for whole -126 <= e <= 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(amax):
    """The smallest e >= E_MIN with amax <= 448 * 2^e (448 = 0.875 * 2^9)."""
    m, ex = torch.frexp(amax)
    e = ex - 9 + (m > 0.875).to(ex.dtype)
    return torch.where(amax > 0, e.clamp(min=E_MIN), torch.full_like(e, E_MIN))


def _encode(x):
    """Codes and scales of groups x [..., 16, D] in fp32; what is not finite becomes NaN and does not count."""
    fine = torch.isfinite(x)
    e = _exponent(torch.where(fine, x, torch.zeros_like(x)).abs().amax((-1, -2)))
    y = torch.where(fine, x * _power(-e)[..., None, None], torch.full_like(x, math.nan))
    return y.to(torch.float8_e4m3fn), _power(e)


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "rope":
        B, n, H, G, D = (case[k] for k in ("B", "n", "H", "G", "D"))
        dt = DTYPES[case["type"]]
        if case["fused"]:  # query, key and value heads of one projection's output
            qkv = _randn(gen, (B, n, (G + 2) * H, D), 1.0, dt)
            s["q"], s["k"] = qkv[:, :, :G * H], qkv[:, :, G * H:(G + 1) * H]
        else:
            s["q"], s["k"] = _randn(gen, (B, n, G * H, D), 1.0, dt), _randn(gen, (B, n, H, D), 1.0, dt)
        s["q_out"] = torch.zeros((B, n, G * H, D), dtype=dt, device=dev)
        s["k_out"] = torch.zeros((B, n, H, D), dtype=dt, device=dev)
        pos = _lens(case, seed, B, "pos_lo", "pos_hi")
        rows = np.random.default_rng(seed + 1).integers((n + 1) // 2, n, size=B, endpoint=True)
        s["pos"] = torch.tensor(pos, dtype=torch.int32, device=dev)
        s["n"] = torch.tensor(rows, dtype=torch.int32, device=dev)
        f, s["factor"] = _freqs(case)
        s["freq"] = torch.tensor(f, dtype=torch.float64, device=dev)
        if own:
            import head_budgeted_kv_gb300 as hw
            s["table"] = hw.rope_table(D, rot_dim=case["rot"], base=10000.0, layout=case["layout"], scaling=case["scaling"],
                                       factor=8.0, original_len=16384)
            s["pool"] = hw.Pool(1, H, D, 16, [[16] * H], B, dt, q_heads=G * H)
        return s
    B, D, bs = case["B"], case["D"], case["bs"]
    rings, per_seq = _rings(case)
    H = len(rings)
    lens = _lens(case, seed, B)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    if case["op"] == "store":
        n = max(1, int(lens.max()))
        s["k"], s["v"] = (_randn(gen, (B, H, n, D)) for _ in range(2))
        s["k"][..., : D // 16] *= 4  # a few strong channels, as keys have
        s["blocks"] = torch.zeros((B * per_seq, 2, bs, D), dtype=torch.float8_e4m3fn, device=dev)
        s["scales"] = torch.zeros((B * per_seq, bs // GROUP, 2), device=dev)
        pool_type = "e4m3"
    else:
        pool_type = case.get("pool", "bf16")
        io = torch.float32 if pool_type == "f32" else torch.bfloat16
        Hq = case["G"] * H
        rows = (B, case["n"]) if case["op"] == "prefill" else (B,)
        s["q"] = _randn(gen, rows + (Hq, D), 2.0, io)
        s["k"], s["v"] = (_randn(gen, rows + (H, D), 1.0, io) for _ in range(2))
        s["out"] = torch.zeros_like(s["q"])
        s["slopes"] = torch.tensor(_slopes(Hq), dtype=torch.float32, device=dev) if case["bias"] else None
        s["scale"] = 1.0 / math.sqrt(D)
        if case["op"] == "prefill":
            n = np.random.default_rng(seed + 1).integers((case["n"] + 1) // 2, case["n"], size=B, endpoint=True)
            s["n"] = torch.tensor(n, dtype=torch.int32, device=dev)
        # a pool in the middle of serving: every slot holds a row, of this sequence or of an earlier one
        blocks = _randn(gen, (B * per_seq, 2, bs, D), 1.0, io)
        blocks[:, 0, :, : D // 16] *= 4
        s["blocks"], s["scales"] = blocks, None
        if pool_type == "e4m3":
            codes, scales = _encode(blocks.view(B * per_seq, 2, bs // GROUP, GROUP, D).float())
            s["blocks"] = codes.view(B * per_seq, 2, bs, D)
            s["scales"] = scales.transpose(1, 2).contiguous()
    if own:
        import head_budgeted_kv_gb300 as hw
        pool = s["pool"] = hw.Pool(1, H, D, bs, [_windows(case)], B, DTYPES[pool_type], q_heads=case.get("G", 1) * H)
        pool.blocks().copy_(s.pop("blocks"))
        if s["scales"] is not None:
            pool.scales().copy_(s["scales"])
    return s


# ---- the plain forms ----------------------------------------------------------------------------------------------
def _plain_store(s):
    case, (rings, per_seq) = s["case"], _rings(s["case"])
    B, D, bs = case["B"], case["D"], case["bs"]
    lens = s["lens"].long()[:, None]
    blocks = s["blocks"].view(B, per_seq, 2, bs // GROUP, GROUP, D)
    scales = s["scales"].view(B, per_seq, bs // GROUP, 2)
    for h, (w, C, at) in enumerate(rings):
        slot = torch.arange(C, device=lens.device)[None]
        p = lens - 1 - (lens - 1 - slot) % C                          # newest position of each slot
        live = (p >= 0) & (p >= lens - w)                             # [B, C]
        rows = p.clamp(min=0)[..., None].expand(-1, -1, D)
        x = torch.stack([t[:, h].gather(1, rows).float() for t in (s["k"], s["v"])], 1)
        x = torch.where(live[:, None, :, None], x, torch.zeros_like(x))
        codes, sc = _encode(x.view(B, 2, C // GROUP, GROUP, D))       # [B, 2, groups, 16, D]
        n = C // bs
        touched = live.view(B, n, bs // GROUP, GROUP).any(-1)
        codes = codes.view(B, 2, n, bs // GROUP, GROUP, D).transpose(1, 2)
        sc = sc.view(B, 2, n, bs // GROUP).permute(0, 2, 3, 1)
        old, old_sc = blocks[:, at:at + n], scales[:, at:at + n]
        blocks[:, at:at + n] = torch.where(touched[:, :, None, :, None, None], codes.view(torch.uint8),
                                           old.view(torch.uint8)).view(torch.float8_e4m3fn)
        scales[:, at:at + n] = torch.where(touched[..., None], sc, old_sc)
    return {"blocks": s["blocks"], "scales": s["scales"]}


def _plain_append(s):
    """The new row of every (sequence, head) into its slot, all heads at once."""
    case, (rings, per_seq) = s["case"], _rings(s["case"])
    B, D, bs, dev = case["B"], case["D"], case["bs"], s["lens"].device
    w, C, at = (torch.tensor(v, device=dev)[None] for v in zip(*rings))
    pos = s["lens"].long()[:, None]                                   # [B, 1], the new token's position
    t = pos % C                                                       # [B, H]
    blk = torch.arange(B, device=dev)[:, None] * per_seq + at + t // bs
    new = torch.stack((s["k"], s["v"]), 2)                            # [B, H, 2, D]
    if s["scales"] is None:
        s["blocks"][blk, :, t % bs] = new
        return
    g, r = t % bs // GROUP, t % GROUP
    age = (r[..., None] - torch.arange(GROUP, device=dev)) % C[..., None]
    live = (age > 0) & (age < w[..., None]) & (age <= pos[..., None])
    groups = s["blocks"].view(-1, 2, bs // GROUP, GROUP, D)
    x = groups[blk, :, g].float() * s["scales"][blk, g][..., None, None]  # [B, H, 2, 16, D]
    x = torch.where(live[:, :, None, :, None], x, torch.zeros_like(x))
    x = torch.where((age == 0)[:, :, None, :, None], new.float()[..., None, :], x)
    codes, sc = _encode(x)
    groups.view(torch.uint8)[blk, :, g] = codes.view(torch.uint8)
    s["scales"][blk, g] = sc


def _plain_rows(s, at, n):
    """K and V of all slots of one head as fp32 [B, C, D]."""
    case, per_seq = s["case"], _rings(s["case"])[1]
    B, D, bs = case["B"], case["D"], case["bs"]
    x = s["blocks"].view(B, per_seq, 2, bs, D)[:, at:at + n].float()
    if s["scales"] is not None:
        sc = s["scales"].view(B, per_seq, bs // GROUP, 2)[:, at:at + n].transpose(2, 3)
        x = (x.view(B, n, 2, bs // GROUP, GROUP, D) * sc[..., None, None]).view(B, n, 2, bs, D)
    return x[:, :, 0].reshape(B, n * bs, D), x[:, :, 1].reshape(B, n * bs, D)


def _softmax_rows(scores, seen, v):
    """softmax(scores) v over the seen keys; a row that sees none gives zeros."""
    scores = torch.where(seen, scores, torch.full_like(scores, -math.inf))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total > 0, total, torch.ones_like(total))


def _scored(x, s, h, distance):
    """Raw scaled scores x [B, G, ...] capped, then lowered by slope times distance [B, 1, ...]."""
    cap, G = s["case"]["cap"], s["case"]["G"]
    if cap > 0:
        x = cap * torch.tanh(x / cap)
    if s["slopes"] is not None:
        x = x - s["slopes"][h * G:(h + 1) * G].view((1, G) + (1,) * (x.dim() - 2)) * distance
    return x


def _plain_decode(s):
    case, (rings, _) = s["case"], _rings(s["case"])
    B, G, D, bs = case["B"], case["G"], case["D"], case["bs"]
    if case["append"]:
        _plain_append(s)
    lens = s["lens"].long()[:, None] + (1 if case["append"] else 0)
    q = s["q"].float().view(B, len(rings), G, D)
    for h, (w, C, at) in enumerate(rings):
        k, v = _plain_rows(s, at, C // bs)
        age = (lens - 1 - torch.arange(C, device=lens.device)) % C    # distance from the newest position
        seen = (age < w) & (age < lens)
        x = _scored((q[:, h] @ k.transpose(1, 2)) * s["scale"], s, h, age[:, None].float())
        v = torch.where(seen[..., None], v, torch.zeros_like(v))
        s["out"][:, h * G:(h + 1) * G] = _softmax_rows(x, seen[:, None], v).to(s["out"].dtype)
    if not case["append"]:
        return {"out": s["out"]}
    return _with_cache(s["out"], s["blocks"], s["scales"])


def _with_cache(out, blocks, scales):
    return {"out": out, "blocks": blocks} if scales is None else {"out": out, "blocks": blocks, "scales": scales}


def _plain_prefill(s):
    case, (rings, per_seq) = s["case"], _rings(s["case"])
    B, G, D, bs, n = case["B"], case["G"], case["D"], case["bs"], case["n"]
    dev = s["q"].device
    pos, rows = s["lens"].long()[:, None], s["n"].long()[:, None]
    i = torch.arange(n, device=dev)[None]
    q = s["q"].float().view(B, n, len(rings), G, D)
    qp = pos + i                                                      # [B, n]
    mine = (i < rows)[:, None, :, None]
    for h, (w, C, at) in enumerate(rings):
        k, v = _plain_rows(s, at, C // bs)
        age = (pos - 1 - torch.arange(C, device=dev)) % C
        kp = torch.cat((torch.where((age < w) & (age < pos), pos - 1 - age, torch.full_like(age, -1)),
                        torch.where(i < rows, qp, torch.full_like(qp, -1))), 1)
        k = torch.cat((k, s["k"][:, :, h].float()), 1)
        v = torch.cat((v, s["v"][:, :, h].float()), 1)
        v = torch.where((kp >= 0)[..., None], v, torch.zeros_like(v))
        distance = qp[:, None, :, None] - kp[:, None, None]           # [B, 1, n, keys]
        seen = (kp >= 0)[:, None, None] & (distance >= 0) & (distance < w)
        x = (q[:, :, h].transpose(1, 2) @ k[:, None].transpose(2, 3)) * s["scale"]
        o = _softmax_rows(_scored(x, s, h, distance.float()), seen, v[:, None]).to(s["out"].dtype)
        old = s["out"].view(B, n, len(rings), G, D)[:, :, h]
        old.copy_(torch.where(mine, o, old.transpose(1, 2)).transpose(1, 2))
        # the chunk's last min(C, rows) tokens into their slots
        b, j = torch.nonzero((i < rows) & (i >= rows - C), as_tuple=True)
        slot = (pos[b, 0] + j) % C
        blk = b * per_seq + at + slot // bs
        s["blocks"][blk, 0, slot % bs] = s["k"][b, j, h]
        s["blocks"][blk, 1, slot % bs] = s["v"][b, j, h]
    return {"out": s["out"], "blocks": s["blocks"]}


def _plain_rope(s):
    case = s["case"]
    n, D, rot = case["n"], case["D"], case["rot"]
    i = torch.arange(n, device=s["pos"].device)[None]
    angle = (s["pos"].double()[:, None] + i)[..., None] * s["freq"]   # [B, n, pairs], 64 bits: far positions
    cos, sin = ((t * s["factor"]).float()[:, :, None] for t in (angle.cos(), angle.sin()))
    mine = (i < s["n"][:, None])[..., None, None]
    halves = case["layout"] == "half"
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        y = x.float().clone()
        a = x[..., : rot // 2].float() if halves else x[..., 0:rot:2].float()
        b = x[..., rot // 2: rot].float() if halves else x[..., 1:rot:2].float()
        lo, hi = a * cos - b * sin, b * cos + a * sin
        if halves:
            y[..., : rot // 2], y[..., rot // 2: rot] = lo, hi
        else:
            y[..., 0:rot:2], y[..., 1:rot:2] = lo, hi
        out.copy_(torch.where(mine, y.to(out.dtype), out))
    return {"q": s["q_out"], "k": s["k_out"]}


def run(s):
    case = s["case"]
    if not own:
        return {"store": _plain_store, "decode": _plain_decode, "prefill": _plain_prefill, "rope": _plain_rope}[case["op"]](s)
    pool = s["pool"]
    if case["op"] == "rope":
        pool.rope(s["table"], s["q"], s["k"], s["pos"], n=s["n"], q_out=s["q_out"], k_out=s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if case["op"] == "store":
        pool.materialize(0, s["k"], s["v"], s["lens"])
        return {"blocks": pool.blocks(), "scales": pool.scales()}
    score = {"softcap": case["cap"], "slopes": s["slopes"]} if case["cap"] > 0 or case["bias"] else {}
    if case["op"] == "prefill":
        out = pool.prefill(0, s["q"], s["scale"], s["k"], s["v"], s["lens"], s["n"], out=s["out"], **score)
        return {"out": out, "blocks": pool.blocks()}
    if not case["append"]:
        return {"out": pool.decode(0, s["q"], s["scale"], s["lens"], out=s["out"], **score)}
    out = pool.append_decode(0, s["q"], s["scale"], s["k"], s["v"], s["lens"], out=s["out"], **score)
    return _with_cache(out, pool.blocks(), pool.scales() if case["pool"] == "e4m3" else None)


# ---- what a pass cannot do without --------------------------------------------------------------------------------
def work(case):
    if case["op"] == "rope":
        size = 4 if case["type"] == "f32" else 2
        values = case["B"] * case["n"] * (case["G"] + 1) * case["H"] * case["D"]
        values = values * 0.75 if case["n"] > 1 else values  # rows a sequence has: half of n to all of it
        return {"bytes": 2 * size * values, "flops": 3 * values}
    wins = np.array(_windows(case), dtype=np.float64)
    B, D, H = case["B"], case["D"], len(wins)
    lens = np.linspace(case["len_lo"], case["len_hi"], 65)[:, None]  # the mean over the range of lengths
    if case["op"] == "store":
        tokens = B * float(np.minimum(wins, lens).sum(1).mean())
        return {"bytes": tokens * (2 * D * 3 + 8 / GROUP), "flops": 4 * tokens * D}
    G = case["G"]
    kind = case.get("pool", "bf16")
    size, io = {"e4m3": 1, "bf16": 2, "f32": 4}[kind], 4 if kind == "f32" else 2
    row = 2 * D * size + (8 / GROUP if kind == "e4m3" else 0)
    if case["op"] == "prefill":
        n = 0.75 * case["n"]  # rows a sequence has: half of n to all of it
        i = np.linspace(0, n, 65)[None, :, None]
        pairs = B * n * float(np.minimum(wins, lens[:, :, None] + i + 1).sum(2).mean())
        read = B * float(np.minimum(wins, lens).sum(1).mean()) * row
        fresh = B * n * H * 2 * D * 2
        return {"bytes": read + 2 * fresh + 2 * B * n * G * H * D * 2, "flops": 4.0 * G * D * pairs}
    tokens = B * float(np.minimum(wins, lens + (1 if case["append"] else 0)).sum(1).mean())
    fresh = B * H * 2 * D * (io + size) if case["append"] else 0
    return {"bytes": tokens * row + fresh + 2 * B * G * H * D * io, "flops": 4.0 * tokens * G * D}


# ---- the definitions in 64 bits, apart from the plain forms --------------------------------------------------------
def _nearest_e4m3(y):
    """The e4m3 value nearest to each |y| <= 448 (ties to even): steps of 2^-9 below 2^-6, of an eighth of the power of two above."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(y / step) * step


def _group64(x):
    """Code values and scale of one group in 64 bits."""
    top = x.abs().amax((-1, -2))
    e = torch.ceil(torch.log2((top / 448.0).clamp(min=2.0 ** E_MIN)))
    e = torch.where(448.0 * torch.exp2(e - 1) >= top, e - 1, e).clamp(min=E_MIN)  # a logarithm may round up at a power of two
    e = torch.where(448.0 * torch.exp2(e) < top, e + 1, e)
    return _nearest_e4m3(x / torch.exp2(e)[..., None, None]), torch.exp2(e)


def _exact_attention(q, k, v, scale, cap, slopes, distance, seen):
    """q [G, n, D], k and v [keys, D], distance and seen [n, keys]; all 64-bit."""
    x = torch.einsum("gnd,kd->gnk", q, k) * scale
    if cap > 0:
        x = cap * torch.tanh(x / cap)
    if slopes is not None:
        x = x - slopes[:, None, None] * distance
    x = x.masked_fill(~seen, -math.inf)
    x = torch.softmax(x, -1).nan_to_num(0.0)
    return torch.einsum("gnk,kd->gnd", x, v)


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "rope":
        return _exact_rope(case, s)
    rings, per_seq = _rings(case)
    B, D, bs = case["B"], case["D"], case["bs"]
    lens = [int(x) for x in s["lens"].tolist()]
    dev = s["lens"].device
    if case["op"] == "store":
        codes, scales = s["blocks"].double(), s["scales"].double()
        for b in range(B):
            for h, (w, C, at) in enumerate(rings):
                first = max(0, lens[b] - w)
                p = torch.arange(first, lens[b], device=dev)
                if not len(p):
                    continue
                ring = torch.zeros((2, C, D), dtype=torch.float64, device=dev)
                ring[0, p % C], ring[1, p % C] = s["k"][b, h, first:lens[b]].double(), s["v"][b, h, first:lens[b]].double()
                hit = torch.zeros(C, dtype=torch.bool, device=dev)
                hit[p % C] = True
                val, sc = _group64(ring.view(2, C // GROUP, GROUP, D))
                b0, n = b * per_seq + at, C // bs
                hit = hit.view(n, bs // GROUP, GROUP).any(-1)
                new = val.view(2, n, bs // GROUP, GROUP, D).transpose(0, 1)
                old = codes[b0:b0 + n].view(n, 2, bs // GROUP, GROUP, D)
                codes[b0:b0 + n] = torch.where(hit[:, None, :, None, None], new, old).reshape(n, 2, bs, D)
                scales[b0:b0 + n] = torch.where(hit[..., None], sc.view(2, n, bs // GROUP).permute(1, 2, 0), scales[b0:b0 + n])
        return {"blocks": codes, "scales": scales}
    G, cap = case["G"], case["cap"]
    pre = case["op"] == "prefill"
    add = case.get("append", False)
    blocks = s["blocks"].double()
    scales = None if s["scales"] is None else s["scales"].double()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    rows = s["n"].tolist() if pre else [1] * B
    for b in range(B):
        for h, (w, C, at) in enumerate(rings):
            b0, n, L = b * per_seq + at, C // bs, lens[b]
            slopes = None if s["slopes"] is None else s["slopes"][h * G:(h + 1) * G].double()
            if pre:
                new = [t[b, :rows[b], h].double() for t in (s["k"], s["v"])]
            elif add:
                new = [t[b, h].double()[None] for t in (s["k"], s["v"])]
            if add and scales is not None:  # the group of the new token, scaled anew
                t = L % C
                g0 = t // GROUP * GROUP
                blk, sub = b0 + t // bs, t % bs // GROUP
                for kv in range(2):
                    x = blocks[blk, kv, g0 % bs:g0 % bs + GROUP] * scales[blk, sub, kv]
                    for j in range(GROUP):
                        p = L - (t - g0 - j) % C  # the position that slot holds
                        if p < 0 or p <= L - w:
                            x[j] = 0
                    x[t - g0] = new[kv][0]
                    val, sc = _group64(x)
                    blocks[blk, kv, g0 % bs:g0 % bs + GROUP], scales[blk, sub, kv] = val, sc
            elif add:
                blocks[b0 + L % C // bs, 0, L % C % bs], blocks[b0 + L % C // bs, 1, L % C % bs] = new[0][0], new[1][0]
            now = L + 1 if add else L
            p = torch.arange(max(0, now - w), now, device=dev)
            slot = p % C
            kv = [blocks[b0 + slot // bs, i, slot % bs] for i in range(2)]
            if scales is not None:
                kv = [x * scales[b0 + slot // bs, slot % bs // GROUP, i][:, None] for i, x in enumerate(kv)]
            if pre:
                kv = [torch.cat(x) for x in zip(kv, new)]
                qp = L + torch.arange(rows[b], device=dev)
                p = torch.cat((p, qp))
                q = s["q"][b, :rows[b], h * G:(h + 1) * G].double().transpose(0, 1)
            else:
                qp = torch.tensor([now - 1], device=dev)
                q = s["q"][b, h * G:(h + 1) * G].double()[:, None]
            if len(p):
                d = qp[:, None] - p[None]
                o = _exact_attention(q, *kv, s["scale"], cap, slopes, d.double(), (d >= 0) & (d < w))
                if pre:
                    out[b, :rows[b], h * G:(h + 1) * G] = o.transpose(0, 1)
                else:
                    out[b, h * G:(h + 1) * G] = o[:, 0]
            if pre:
                p = L + torch.arange(max(0, rows[b] - C), rows[b], device=dev)
                slot = p % C
                for i in range(2):
                    blocks[b0 + slot // bs, i, slot % bs] = new[i][p - L]
    if pre:
        return {"out": out, "blocks": blocks}
    return _with_cache(out, blocks, scales) if add else {"out": out}


def _exact_rope(case, s):
    """Each pair as a complex number turned by its angle, in 64 bits."""
    rot, half = case["rot"], case["rot"] // 2
    lo = torch.arange(half) if case["layout"] == "half" else torch.arange(0, rot, 2)
    hi = lo + (half if case["layout"] == "half" else 1)
    got = {}
    for name in ("q", "k"):
        x = s[name].double()
        y = torch.zeros_like(s[name + "_out"]).double()
        for b, (p, n) in enumerate(zip(s["pos"].tolist(), s["n"].tolist())):
            angle = torch.outer(torch.arange(p, p + n, device=x.device, dtype=torch.float64), s["freq"])
            turned = torch.complex(x[b, :n][..., lo], x[b, :n][..., hi]) * torch.polar(torch.full_like(angle, s["factor"]), angle)[:, None]
            y[b, :n] = x[b, :n]
            y[b, :n, :, lo], y[b, :n, :, hi] = turned.real, turned.imag
        got[name] = y
    return got
