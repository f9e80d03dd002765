"""Capped and distance-biased scores on the GPU, decode and chunked prefill, against 64 bits.

Tolerance, per element, with A = sum_p softmax_p |v_p| and T the largest |score| of the row:
* the score's own error: 2^-20 T from the cap (header) and 2^-22 T from the fp32 products, the log2
  units and the bias, against a dot product whose 128 terms each round by 2^-24 of |q||k| (2^-17 of
  sum |q_d k_d| scale, bounded by S below); the exponential 2^-22: each weight is off by
  e = 2^-19 T + 2^-17 S + 2^-22 relatively, and the sum it is normalised by as well: 2 e A;
* tensor-core paths round the weights to bf16 (2^-8 A more, 8-bit pools to fp16, 2^-11 A; the sum is
  taken of the unrounded weights); bf16 outputs round by 2^-8 of the value;
* fp32 pools take tanhf (2 units) instead: e = 2^-21 T + 2^-17 S + 2^-22, outputs 2^-23."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import head_budgeted_kv_gb300 as hw
from reference_ops import Ring8, attention

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hw.binding.load()
    yield
    torch.cuda.synchronize()


def np64(t):
    return t.float().cpu().double().numpy()


def tolerance(kind, q, k, v, scale, distance, cap, slope):
    ref, mass, top = attention(q, k, v, scale, distance, cap, slope)
    size = float((np.abs(k) @ np.abs(q)).max(initial=0.0)) * abs(scale)
    e = 2.0 ** (-21 if kind == "f32" else -19) * top + 2.0 ** -17 * size + 2.0 ** -22
    tol = 2 * e * mass + {"f32": 0.0, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -10}[kind] * mass
    return ref, tol + (2.0 ** -23 if kind == "f32" else 2.0 ** -8) * np.abs(ref) + 1e-30


def histories(gen, B, H, L, D, dtype):
    return (torch.randn((B, H, L, D), generator=gen, device="cuda").to(dtype) for _ in range(2))


SCORES = {"cap": (15.0, False), "bias": (0.0, True), "both": (8.0, True), "tiny cap": (1e-3, False), "large cap": (1e5, False),
          "low": (60.0, False), "half": (25.0, False)}


@pytest.mark.parametrize("score", sorted(SCORES))
@pytest.mark.parametrize("kind,D,G,bs,windows,lens", [
    ("bf16", 128, 4, 16, [64, 200, 1], [300, 20]),
    ("bf16", 64, 16, 32, [100, 40], [333, 0]),
    ("bf16", 128, 9, 16, [700], [1000]),
    ("bf16", 128, 3, 5, [23, 60], [100, 9]),        # CUDA-core kernel
    ("f32", 128, 4, 16, [64, 200], [300, 20]),
    ("f32", 64, 3, 16, [33], [100, 7]),
    ("f32", 64, 10, 16, [130, 20], [400, 3]),       # CUDA-core kernel, two slices of heads
    ("e4m3", 128, 4, 16, [64, 200, 33], [300, 20]),
    ("e4m3", 64, 16, 48, [100, 40], [333, 0]),
    ("e4m3", 128, 1, 16, [2000], [2500]),
])
def test_decode(kind, D, G, bs, windows, lens, score):
    cap, biased = SCORES[score]
    B, H = len(lens), len(windows)
    gen = torch.Generator(device="cuda").manual_seed(len(windows) * 100 + G)
    pool = hw.Pool(1, H, D, bs, [windows], B, TYPES[kind], q_heads=G * H)
    io = pool.io_dtype
    k, v = histories(gen, B, H, max(lens) + 1, D, io)
    pos = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pool.materialize(0, k, v, pos)
    q = (torch.randn((B, G * H, D), generator=gen, device="cuda") * 3).to(io)
    slopes = torch.tensor([0.0 if g == 1 else 2.0 ** (-8.0 * (g + 1) / (G * H)) for g in range(G * H)], device="cuda")
    kw = dict(softcap=cap, slopes=slopes if biased else None)
    at = torch.arange(B, device="cuda")
    kn, vn = k[at, :, pos.long()].contiguous(), v[at, :, pos.long()].contiguous()
    scale = D ** -0.5
    before = pool.decode(0, q, scale, pos, **kw)
    after = pool.append_decode(0, q, scale, kn, vn, pos, **kw)
    qq, kk, vv = np64(q), np64(k), np64(v)
    for s in range(B):
        for h in range(H):
            ring = Ring8(windows[h], bs, D) if kind == "e4m3" else None
            if ring:
                ring.materialize(kk[s, h], vv[s, h], lens[s])
            for out, n in ((before, lens[s]), (after, lens[s] + 1)):
                if ring and n > lens[s]:
                    ring.append(kk[s, h, n - 1], vv[s, h, n - 1], n - 1)
                p, rk, rv = ring.resident(n) if ring else (np.arange(max(0, n - windows[h]), n), None, None)
                rk, rv = (rk, rv) if ring else (kk[s, h, p], vv[s, h, p])
                got = np64(out)[s]
                for g in range(h * G, (h + 1) * G):
                    slope = float(slopes[g]) if biased else 0.0
                    ref, tol = tolerance(kind, qq[s, g], rk, rv, scale, n - 1 - p, cap, slope)
                    assert (np.abs(got[g] - ref) <= tol).all(), (s, g, n, float((np.abs(got[g] - ref) / tol).max()))
    # a prepared launch with early reads gives the same bits
    out = torch.empty_like(q)
    launch = pool.decode_launch(0, q, scale, pos + 1, out, early_reads=True, **kw)
    launch()
    again = pool.decode(0, q, scale, pos + 1, **kw)
    assert torch.equal(out, again)
    assert pool.check_device_errors() == 0


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
def test_neither_cap_nor_slopes_is_the_plain_call(kind):
    gen = torch.Generator(device="cuda").manual_seed(4)
    pool = hw.Pool(1, 2, 64, 16, [[64, 200]], 2, TYPES[kind], q_heads=8)
    k, v = histories(gen, 2, 2, 300, 64, pool.io_dtype)
    lens = torch.tensor([300, 41], dtype=torch.int32, device="cuda")
    pool.materialize(0, k, v, lens)
    q = torch.randn((2, 8, 64), generator=gen, device="cuda").to(pool.io_dtype)
    out = torch.empty_like(q)
    hw.hwkv_decode_attn_score(pool.handle, 0, q, hw.binding.score(0.125), lens, out, pool.workspace)
    assert torch.equal(out, pool.decode(0, q, 0.125, lens))
    # zero slopes take the scored kernels: the same scores up to their rounding
    zero = pool.decode(0, q, 0.125, lens, slopes=torch.zeros(8, device="cuda"))
    assert (zero.float() - out.float()).abs().max() <= 2.0 ** -7 * out.float().abs().max()


def test_long_groups_merge_alike():
    """A biased group split over many CTAs, and few, against the same formula."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    pool = hw.Pool(1, 1, 128, 16, [[8000]], 1, torch.bfloat16, q_heads=4)
    k, v = histories(gen, 1, 1, 9000, 128, torch.bfloat16)
    lens = torch.tensor([9000], dtype=torch.int32, device="cuda")
    pool.materialize(0, k, v, lens)
    q = torch.randn((1, 4, 128), generator=gen, device="cuda").bfloat16()
    slopes = torch.tensor([1e-4, 1e-3, 0.0, 1.0], device="cuda")
    p = np.arange(1000, 9000)
    for workers in (0, 1, 40, 280):
        pool.set_decode_config(workers=workers)
        got = np64(pool.decode(0, q, 0.09, lens, softcap=20.0, slopes=slopes))
        for g in range(4):
            ref, tol = tolerance("bf16", np64(q)[0, g], np64(k)[0, 0, p], np64(v)[0, 0, p], 0.09, 8999 - p, 20.0,
                                 float(slopes[g]))
            assert (np.abs(got[0, g] - ref) <= tol).all(), (workers, g)


@pytest.mark.parametrize("score", ["cap", "bias", "both", "low", "half", "tiny cap", "large cap"])
@pytest.mark.parametrize("D,G,bs,windows,pos,n,max_stages", [
    (128, 4, 16, [64, 200], [0, 150], [130, 7], 0),
    (64, 2, 16, [40, 500, 16], [333, 20], [50, 100], 0),
    (128, 16, 32, [100], [300], [33], 0),
    (64, 1, 64, [129, 700], [1000, 64], [300, 1], 0),
    (128, 3, 48, [333], [90], [200], 0),
    (128, 4, 16, [3000], [4000], [40], 8),          # a split key stream
    (64, 8, 16, [24], [24], [0], 0),                # an empty chunk
])
def test_prefill(D, G, bs, windows, pos, n, max_stages, score):
    cap, biased = SCORES[score]
    B, H, n_max = len(pos), len(windows), max(max(n), 1)
    gen = torch.Generator(device="cuda").manual_seed(sum(pos) + G)
    pool = hw.Pool(1, H, D, bs, [windows], B, torch.bfloat16, q_heads=G * H)
    pool.set_prefill_config(max_stages)
    L = max(p + c for p, c in zip(pos, n)) + n_max
    k, v = histories(gen, B, H, L, D, torch.bfloat16)
    tpos = torch.tensor(pos, dtype=torch.int32, device="cuda")
    tn = torch.tensor(n, dtype=torch.int32, device="cuda")
    pool.materialize(0, k, v, tpos)
    q = (torch.randn((B, n_max, G * H, D), generator=gen, device="cuda") * 3).bfloat16()
    kn, vn = (torch.stack([t[s, :, pos[s]:pos[s] + n_max].transpose(0, 1) for s in range(B)]).contiguous() for t in (k, v))
    slopes = torch.tensor([2.0 ** (-8.0 * (g + 1) / (G * H)) for g in range(G * H)], device="cuda")
    out = torch.full_like(q, 7.0)
    scale = D ** -0.5
    pool.prefill(0, q, scale, kn, vn, tpos, tn, out=out, softcap=cap, slopes=slopes if biased else None)
    assert pool.check_device_errors() == 0
    qq, kk, vv, got = np64(q), np64(k), np64(v), np64(out)
    for s in range(B):
        assert (got[s, n[s]:] == 7.0).all()
        for i in {0, 1, n[s] // 3, n[s] // 2, n[s] - 2, n[s] - 1} & set(range(n[s])):
            for h, w in enumerate(windows):
                at = pos[s] + i
                p = np.arange(max(0, at + 1 - w), at + 1)
                for g in range(h * G, (h + 1) * G):
                    ref, tol = tolerance("bf16", qq[s, i, g], kk[s, h, p], vv[s, h, p], scale, at - p, cap,
                                         float(slopes[g]) if biased else 0.0)
                    assert (np.abs(got[s, i, g] - ref) <= tol).all(), (s, i, g, float((np.abs(got[s, i, g] - ref) / tol).max()))
    # the chunk is appended: decoding the last token of each sequence gives the chunk's last row
    if min(n) > 0:
        last = torch.stack([q[s, n[s] - 1] for s in range(B)])
        dec = np64(pool.decode(0, last, scale, tpos + tn, softcap=cap, slopes=slopes if biased else None))
        for s in range(B):
            np.testing.assert_allclose(dec[s], got[s, n[s] - 1], atol=2.0 ** -5, rtol=2.0 ** -6)


@pytest.mark.parametrize("cap", [0.0, 6.0, 40.0])
@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
def test_negative_scales_and_slopes(kind, cap):
    """A negative scale turns the scores around, a negative slope favours the farthest keys; the decode of
    every pool type, and the chunked prefill of bf16 pools."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    windows, L = [70, 333], 400
    pool = hw.Pool(1, 2, 64, 16, [windows], 1, TYPES[kind], q_heads=8)
    k, v = histories(gen, 1, 2, L, 64, pool.io_dtype)
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    q = (torch.randn((1, 8, 64), generator=gen, device="cuda") * 2).to(pool.io_dtype)
    slopes = torch.tensor([(-0.5) ** g for g in range(8)], device="cuda")
    for scale in (-0.125, 0.125):
        pool.materialize(0, k, v, lens)
        outs = [pool.decode(0, q, scale, lens, softcap=cap, slopes=slopes)]
        if kind == "bf16":
            n = 37
            pool.materialize(0, k, v, lens - n)
            kn, vn = (t[:, :, L - n:].transpose(1, 2).contiguous() for t in (k, v))
            chunk = q[:, None].expand(1, n, 8, 64).contiguous()
            outs.append(pool.prefill(0, chunk, scale, kn, vn, lens - n, lens * 0 + n, softcap=cap, slopes=slopes)[:, n - 1])
        for h, w in enumerate(windows):
            p = np.arange(L - w, L)
            rk, rv = np64(k)[0, h, p], np64(v)[0, h, p]
            if kind == "e4m3":
                ring = Ring8(w, 16, 64)
                ring.materialize(np64(k)[0, h], np64(v)[0, h], L)
                p, rk, rv = ring.resident(L)
            for g in range(4 * h, 4 * h + 4):
                ref, tol = tolerance(kind, np64(q)[0, g], rk, rv, scale, L - 1 - p, cap, float(slopes[g]))
                for i, out in enumerate(outs):
                    got = np64(out)[0, g]
                    assert (np.abs(got - ref) <= tol).all(), (scale, g, i, float((np.abs(got - ref) / tol).max()))
    assert pool.check_device_errors() == 0


@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
def test_first_call_of_a_process_captured(kind):
    """A step captured before any of its kernels ran in the process."""
    code = f"""
import torch, head_budgeted_kv_gb300 as hw
from head_budgeted_kv_gb300.graph import DecodeStepGraph
pool = hw.Pool(2, 2, 64, 16, [[64, 30], [200, 16]], 1, {TYPES[kind]}, q_heads=8)
pos = torch.tensor([0], dtype=torch.int32, device="cuda")
kw = dict(softcap=10.0, slopes=torch.ones(8, device="cuda"))
step = DecodeStepGraph(pool, 0.2, 8, pos, rope=hw.rope_table(64), **kw)
q, k, v = (torch.randn(s, device="cuda").to(pool.io_dtype) for s in (step.q.shape, step.k_new.shape, step.v_new.shape))
step.q.copy_(q), step.k_new.copy_(k), step.v_new.copy_(v)
step.replay()
for l in range(2):
    qr, kr = pool.rope(hw.rope_table(64), q[l], k[l], pos)
    assert torch.equal(pool.append_decode(l, qr, 0.2, kr, v[l], pos, **kw), step.out[l])
assert pool.check_device_errors() == 0 and step.out.abs().sum() > 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_captured_step(kind):
    from head_budgeted_kv_gb300.graph import DecodeStepGraph
    slopes = torch.tensor([2.0 ** -(i + 1) for i in range(8)], device="cuda")
    results = []
    for graph in (False, True):
        gen = torch.Generator(device="cuda").manual_seed(8)

        def randn(*shape):
            return torch.randn(shape, generator=gen, device="cuda").bfloat16()

        pool = hw.Pool(2, 2, 64, 16, [[64, 30], [200, 16]], 1, TYPES[kind], q_heads=8)
        pos = torch.tensor([70], dtype=torch.int32, device="cuda")
        for l in range(2):
            pool.materialize(l, randn(1, 2, 70, 64), randn(1, 2, 70, 64), pos)
        # the scored kernels load on their first call: make it before a capture
        pool.decode(0, randn(1, 8, 64), 0.2, pos, softcap=10.0, slopes=slopes)
        step = DecodeStepGraph(pool, 0.2, 8, pos, softcap=10.0, slopes=slopes, rope=hw.rope_table(64)) if graph else None
        outs = []
        for _ in range(4):
            q, k, v = randn(2, 1, 8, 64), randn(2, 1, 2, 64), randn(2, 1, 2, 64)
            if graph:
                step.q.copy_(q), step.k_new.copy_(k), step.v_new.copy_(v)
                step.replay()
                outs.append(step.out.clone())
            else:
                one = []
                for l in range(2):
                    qr, kr = pool.rope(hw.rope_table(64), q[l], k[l], pos)
                    one.append(pool.append_decode(l, qr, 0.2, kr, v[l], pos, softcap=10.0, slopes=slopes))
                outs.append(torch.stack(one))
                pos = pos + 1
        results.append(torch.stack(outs))
    assert torch.equal(results[0], results[1])


@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("max_stages", [0, 4])
def test_captured_prefill(softcap, max_stages):
    """Chunks captured one after another, turned and attended, replayed on new inputs and positions, give the
    bits of eager calls and the same rings (max_stages 4: split streams, merged in the finish launch)."""
    gen = torch.Generator(device="cuda").manual_seed(12)
    table = hw.rope_table(64)

    def make():
        pool = hw.Pool(2, 2, 64, 16, [[64, 700], [30, 2000]], 2, torch.bfloat16, q_heads=8)
        pool.set_prefill_config(max_stages)
        return pool

    shape_q, shape_k = (2, 90, 8, 64), (2, 90, 2, 64)
    static = [torch.zeros(s, device="cuda").bfloat16() for s in (shape_q, shape_k, shape_k)]
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    n = torch.tensor([90, 41], dtype=torch.int32, device="cuda")
    outs = [torch.zeros(shape_q, device="cuda").bfloat16() for _ in range(2)]
    captured, eager = make(), make()

    def chunk(pool, q, k, v, p, into=None):
        res = []
        for l in range(2):
            qr, kr = pool.rope(table, q, k, p, n, q_out=turned[0], k_out=turned[1])
            res.append(pool.prefill(l, qr, 0.2, kr, v, p, n, out=into[l] if into else torch.zeros_like(q),
                                    softcap=softcap))
        return res

    turned = [torch.zeros(s, device="cuda").bfloat16() for s in (shape_q, shape_k)]
    chunk(captured, *static, pos, outs)  # sizes the workspace; position 0 is stored again below
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chunk(captured, *static, pos, outs)
    at = torch.zeros(2, dtype=torch.int32, device="cuda")
    for _ in range(12):
        new = [torch.randn(s.shape, generator=gen, device="cuda").bfloat16() for s in static]
        for t, x in zip(static, new):
            t.copy_(x)
        pos.copy_(at)
        graph.replay()
        got = [o.clone() for o in outs]
        want = chunk(eager, *new, at)
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1, :41], b[1, :41])
        at = at + n
    # every slot that holds a position of the sequences
    assert captured.check_device_errors() == 0 and eager.check_device_errors() == 0
    last = torch.randn((2, 8, 64), generator=gen, device="cuda").bfloat16()
    for l in range(2):
        assert torch.equal(captured.decode(l, last, 0.2, at), eager.decode(l, last, 0.2, at))


def test_refusals():
    pool = hw.Pool(1, 2, 64, 16, [[64, 200]], 1, torch.bfloat16, q_heads=4)
    q = torch.zeros((1, 4, 64), device="cuda").bfloat16()
    lens = torch.tensor([5], dtype=torch.int32, device="cuda")
    ok = torch.zeros(4, device="cuda")
    for bad in (ok[:3], ok.double(), torch.zeros(8, device="cuda")[::2], ok.cpu()):
        with pytest.raises(ValueError):
            pool.decode(0, q, 0.1, lens, slopes=bad)
    for scale, cap in ((0.1, -1.0), (0.1, float("nan")), (0.1, float("inf")), (float("nan"), 5.0), (1e30, 1e-30), (1.0, 3e38)):
        with pytest.raises(hw.HwkvError) as e:
            pool.decode(0, q, scale, lens, softcap=cap)
        assert e.value.status == hw.binding.HWKV_ERR_INVALID_ARG
    chunk = torch.zeros((1, 1, 4, 64), device="cuda").bfloat16()
    with pytest.raises(hw.HwkvError):
        pool.prefill(0, chunk, 0.1, chunk[:, :, :2].contiguous(), chunk[:, :, :2].contiguous(), lens, lens, softcap=-1.0)
