"""The operators around the cache at the ends of what their inputs may be: V scales far apart, the
largest values, slots outside the window, positions before the first, far angles, steep slopes.

Attention tolerance of 8-bit pools, per element, with A = sum_p w_p |v_p| and w the softmax weights: the
output's rounding to bf16 (2^-8 |ref|); each weight's rounding to fp16 (2^-11) and the error of its
score and exponential (2^-12, see test_gpu_q8.py), both counted twice for the sum they are
normalised by.  A product w_p v_scale_p below fp16's normal range is off by an absolute amount
instead: the kernel holds it times 2^11 / ref with ref between half of the head's largest such product
and that product (a lagging reference makes what it holds larger), steps below 2^-14 are 2^-24, so half of
one is 2^-25 and the output is off by at most 2^-36 max(w_p v_scale_p) sum_p |c_p|."""
import weakref
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import head_budgeted_kv_gb300 as hw
from reference_ops import Ring8, attention
from test_gpu_q8 import Case, np64

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hw.binding.load()
    yield
    torch.cuda.synchronize()


def check_head(got, q, ring, n, scale, slope=0.0, cap=0.0, what=""):
    """One query head of an 8-bit pool against 64 bits."""
    p, k, v = ring.resident(n)
    ref, mass, top = attention(q, k, v, scale, n - 1 - p, cap, slope)
    s = k @ q * scale
    if cap > 0:
        s = cap * np.tanh(s / cap)
    s = s - slope * (n - 1 - p)
    w = np.exp(s - s.max())
    w /= w.sum()
    floor = 2.0 ** -36 * float((w * np.repeat(ring.scales[1], 16)[p % ring.C]).max())
    floor = floor * np.abs(ring.codes[1][p % ring.C]).sum(0)
    e = 2.0 ** -11 + 2.0 ** -12 + (2.0 ** -19 * top if cap > 0 or slope else 0.0)
    tol = 2.0 ** -8 * np.abs(ref) + 2 * e * mass + floor
    # what lies half a step or more past bf16's largest number, (2 - 2^-7) 2^127, rounds to infinity
    over = np.abs(ref) >= 2.0 ** 128 - 2.0 ** 119
    with np.errstate(invalid="ignore"):
        off = np.where(over, 0.0, np.abs(got - ref))
    assert (got[over] == np.sign(ref[over]) * np.inf).all(), f"{what}: {got[over]} past the largest number"
    worst = off / np.maximum(tol, 1e-300)
    assert (off <= tol).all(), f"{what}: off by {off.max():.3e} of {np.abs(ref).max():.3e}, {worst.max():.3g} times the tolerance"


def keys_for(scores, D):
    """Rows whose product with a query of 8 in dim 0 is `scores`, as far as e4m3 holds them."""
    k = torch.zeros((1, 1, len(scores), D), device="cuda")
    k[0, 0, :, 0] = torch.tensor(scores, device="cuda") / 8.0
    return k.bfloat16()


# ---- 8-bit pools: the largest values ------------------------------------------------------------------
# 3.3895e38, bf16's largest number, is 255 * 2^120, which e4m3 rounds to 256 * 2^120 = 2^128: such a row
# on its own gives infinity, the nearest thing bf16 has.  3.2e38 is stored as 240 * 2^120.
@pytest.mark.parametrize("workers", [0, 4])
@pytest.mark.parametrize("big", [3.3895e38, 3.2e38])
@pytest.mark.parametrize("D,group", [(128, 4), (64, 16)])
def test_the_largest_values_come_out(D, group, big, workers):
    """V rows at the end of bf16's range: a lone token, and one among many others of less weight, whatever the
    order in which the maximum meets them."""
    c = Case([200], 2, group, D, 16, 9, None, workers)
    v = torch.zeros((2, 1, 200, D), device="cuda")
    v[0, 0, 0] = big
    v[1, 0, 30, ::2], v[1, 0, 30, 1::2] = big, -big
    v[1, 0, 160] = 1.5e38
    # the maximum rises by less than the reference's slack towards the large rows
    scores = [0.0 if i < 16 else 1.0 if i < 100 else 2.0 for i in range(200)]
    scores[30], scores[160] = 2.5, 0.0
    k = torch.cat((keys_for([0.0] * 200, D), keys_for([x * 0.8 for x in scores], D)))
    c.materialize([1, 200], k, v.bfloat16())
    q = torch.zeros((2, group, D), device="cuda").bfloat16()
    q[..., 0] = 8.0
    out = np64(c.pool.decode(0, q, 1.0, c.i32([1, 200])))
    for s, n in enumerate((1, 200)):
        for g in range(group):
            check_head(out[s, g], np64(q)[s, g], c.rings[s][0], n, 1.0, what=f"seq {s} head {g}")
    c.close()


@pytest.mark.parametrize("x", [3.3895e38, 3.2e38, 2.0 ** 116, 2.0 ** -110, 2.0 ** -129])
def test_one_token_gives_its_value(x):
    """Largest to smallest magnitudes, appended in the launch that attends to them."""
    c = Case([5], 1, 4, 64, 16, 1)
    kn, vn = torch.zeros((2, 1, 1, 64), device="cuda").bfloat16().unbind(0)
    vn = vn + torch.tensor(x, device="cuda").bfloat16()
    out = c.pool.append_decode(0, c.randn(1, 4, 64), 0.1, kn, vn, c.i32([0]))
    c.ref_append(kn, vn, [0])
    want = c.rings[0][0].resident(1)[2][0]
    if x == 3.3895e38:
        assert (want == 2.0 ** 128).all() and (np64(out) == np.inf).all()
        return
    # below 2^-126 bf16's step is 2^-133: half of one
    assert (np.abs(np64(out)[0] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -134).all()
    c.close()


# ---- 8-bit pools: V scales far apart ------------------------------------------------------------------
@pytest.mark.parametrize("where", [0, 2, 5], ids=["first", "middle", "last"])
@pytest.mark.parametrize("power", [20, 24, 30, 37, 60, 110])
@pytest.mark.parametrize("D,group", [(128, 2), (64, 16)])
def test_value_group_without_weight_leaves_the_others_alone(D, group, power, where):
    """One group of V is 2^power times the others and has no weight; the others' weights are 2^-11.5 of the
    largest one's, or all alike."""
    for lead in (8.0, 0.0):
        c = Case([96], 1, group, D, 16, 3)
        scores = [0.0] * 96
        scores[16 * where:16 * where + 16] = [-120.0] * 16
        scores[16 * ((where + 1) % 6)] = lead
        v = c.randn(1, 1, 96, D).float()
        v[0, 0, 16 * where:16 * where + 16] *= 2.0 ** power
        c.materialize([96], keys_for(scores, D), v.bfloat16())
        q = torch.zeros((1, group, D), device="cuda").bfloat16()
        q[..., 0] = 8.0
        out = np64(c.pool.decode(0, q, 1.0, c.i32([96])))
        for g in range(group):
            check_head(out[0, g], np64(q)[0, g], c.rings[0][0], 96, 1.0, what=f"lead {lead} head {g}")
        c.close()


@pytest.mark.parametrize("workers", [0, 1, 5])
@pytest.mark.parametrize("power", [30, 40, 100])
@pytest.mark.parametrize("fused", [False, True], ids=["decode", "fused"])
def test_values_that_slopes_suppress(power, fused, workers):
    """Steep slopes leave an old group of far larger V no weight in some heads, and all of it in others (negative
    slopes), also when the merges of many CTAs join them."""
    c = Case([700, 40], 2, 4, 128, 16, 5, 2, workers)
    n = 800
    k, v = c.randn(2, 2, n, 128), c.randn(2, 2, n, 128).float()
    v[0, :, 200:340] *= 2.0 ** power
    v[1, :, 100:480] *= 2.0 ** -power
    c.materialize([n, n - 300], k, v.bfloat16())
    slopes = torch.tensor([1.0, 0.25, 0.0, -0.5, 4.0, 0.125, 1e-3, -2.0], device="cuda")
    q = c.randn(2, 8, 128)
    if fused:
        kn, vn = c.randn(2, 2, 128), c.randn(2, 2, 128)
        out = c.pool.append_decode(0, q, c.scale, kn, vn, c.i32([n, n - 300]), slopes=slopes)
        c.ref_append(kn, vn, [n, n - 300])
        lens = [n + 1, n - 299]
    else:
        lens = [n, n - 300]
        out = c.pool.decode(0, q, c.scale, c.i32(lens), slopes=slopes)
    for s in range(2):
        for g in range(8):
            check_head(np64(out)[s, g], np64(q)[s, g], c.rings[s][g // 4], lens[s], c.scale, float(slopes[g]), what=f"seq {s} head {g}")
    c.close()


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("workers", [0, 3])
def test_value_scales_over_their_whole_range(seed, workers):
    """Each group of V at a power of its own between 2^-110 and 2^110, appended rows among them."""
    rng = np.random.default_rng(seed)
    D, group = [(128, 4), (64, 1), (128, 16), (64, 8)][seed]
    c = Case([300, 37], 1, group, D, 16, seed, seed, workers)
    k, v = c.randn(1, 2, 350, D), c.randn(1, 2, 350, D).float()
    for g in range(0, 350, 16):
        v[:, :, g:g + 16] *= 2.0 ** float(rng.integers(-110, 110))
    c.materialize([350], k, v.bfloat16())
    pos = 350
    for i in range(3):
        q = c.randn(1, 2 * group, D, scale=4.0)
        kn, vn = c.randn(1, 2, D), (c.randn(1, 2, D).float() * 2.0 ** float(rng.integers(-110, 110))).bfloat16()
        out = c.pool.append_decode(0, q, c.scale, kn, vn, c.i32([pos]))
        c.ref_append(kn, vn, [pos])
        pos += 1
        for g in range(2 * group):
            check_head(np64(out)[0, g], np64(q)[0, g], c.rings[0][g // group], pos, c.scale, what=f"step {i} head {g}")
    c.close()


@pytest.mark.parametrize("size", [1e3, 1e6, 1e9, 1e12])
def test_huge_scores(size):
    """Scores so large that one key takes all the weight: its V comes out, whatever the scales about it."""
    c = Case([96], 1, 2, 64, 16, 7)
    k = keys_for([float(8 * (i % 48)) / 64 for i in range(95)] + [0.0], 64)
    k[0, 0, 50, 0] = 14.0  # the others stay below 1: a gap of more than 100 sizes
    v = c.randn(1, 1, 96, 64).float()
    for g in range(6):
        v[0, 0, 16 * g:16 * g + 16] *= 2.0 ** (7 * (g - 3))
    c.materialize([96], k, v.bfloat16())
    q = torch.zeros((1, 2, 64), device="cuda").bfloat16()
    q[..., 0] = 8.0
    for scale in (size, -size):
        q[0, 1, 0] = 8.0 if scale > 0 else -8.0
        q[0, 0, 0] = q[0, 1, 0]
        out = np64(c.pool.decode(0, q, scale, c.i32([96])))
        want = c.rings[0][0].resident(96)[2][50]
        assert (np.abs(out[0] - want) <= 2.0 ** -8 * np.abs(want)).all()
    c.close()


def test_far_smaller_rows_than_a_huge_scale():
    """8-bit pools with a bias: rows and queries so small that a scale of 2^126 still gives no score."""
    c = Case([48], 1, 2, 64, 16, 21)
    k = (c.randn(1, 1, 48, 64).float() * 2.0 ** -125).bfloat16()
    c.materialize([48], k, c.randn(1, 1, 48, 64))
    q = (c.randn(1, 2, 64).float() * 2.0 ** -110).bfloat16()
    out = c.pool.decode(0, q, 2.0 ** 126, c.i32([48]), slopes=torch.zeros(2, device="cuda"))
    for g in range(2):
        check_head(np64(out)[0, g], np64(q)[0, g], c.rings[0][0], 48, 2.0 ** 126, what=f"head {g}")
    c.close()


# ---- 8-bit pools: what lies outside the window --------------------------------------------------------
@pytest.mark.parametrize("cap,biased", [(20.0, False), (6.0, False), (6.0, True), (0.0, True), (0.0, False)])
@pytest.mark.parametrize("D,group", [(128, 4), (64, 16), (64, 1)])
def test_slots_outside_the_window_do_not_change_a_bit(D, group, cap, biased):
    """Expired rows as large as codes go and along the query, past the cap where those in the window stay below
    it, or zeros, in the slots around the window."""
    outs = []
    for fill in (0.0, 448.0):
        c = Case([40, 70, 9], 2, group, D, 16, 15)
        lens = [100, 230]
        c.materialize(lens)
        q = c.randn(2, 3 * group, D)
        codes = c.pool.blocks().float()
        for s in range(2):
            for h in range(3):
                ring, ids = c.rings[s][h], c.pool.block_table(s, 0, h)
                inside = {p % ring.C for p in range(max(0, lens[s] - ring.w), lens[s])}
                for t in set(range(ring.C)) - inside:
                    codes[int(ids[t // 16]), :, t % 16] = fill * torch.sign(q[s, h * group].float())
        c.pool.blocks().copy_(codes.to(torch.float8_e4m3fn))
        slopes = torch.linspace(0.01, 0.3, 3 * group, device="cuda") if biased else None
        outs.append([c.pool.decode(0, q, c.scale, c.i32(lens), softcap=cap, slopes=slopes),
                     c.pool.append_decode(0, q, c.scale, c.randn(2, 3, D), c.randn(2, 3, D), c.i32(lens), softcap=cap, slopes=slopes)])
        c.close()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


# ---- positions before the first -----------------------------------------------------------------------
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("kind,bs,group", [("bf16", 16, 4), ("f32", 16, 4), ("e4m3", 16, 4), ("bf16", 5, 2), ("f32", 16, 6)])
@pytest.mark.parametrize("first", [-1, -3])
def test_fused_step_flags_negative_positions(kind, bs, group, softcap, first):
    """As the append on its own: flagged, nothing stored, a zero output; the other sequences go on."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    pool = hw.Pool(1, 2, 64, bs, [[64, 30]], 2, TYPES[kind], q_heads=2 * group)
    k = torch.randn((2, 2, 80, 64), generator=gen, device="cuda").to(pool.io_dtype)
    pool.materialize(0, k, k, torch.tensor([80, 80], dtype=torch.int32, device="cuda"))
    q, kn = torch.randn((2, 2 * group, 64), generator=gen, device="cuda").to(pool.io_dtype), k[:, :, 5].contiguous()
    separate = pool.buffer.clone()
    pos = torch.tensor([first, 80], dtype=torch.int32, device="cuda")
    out = pool.append_decode(0, q, 0.125, kn, kn, pos, softcap=softcap)
    assert pool.check_device_errors() == hw.binding.HWKV_DEVERR_NEG_LENGTH
    assert (out[0] == 0).all() and out[1].abs().sum() > 0
    fused = pool.buffer.clone()
    pool.buffer.copy_(separate)
    pool.append(0, kn, kn, pos)
    assert pool.check_device_errors() == hw.binding.HWKV_DEVERR_NEG_LENGTH
    assert torch.equal(pool.buffer, fused) and not torch.equal(fused, separate)
    want = pool.decode(0, q, 0.125, pos + 1, softcap=softcap)
    assert torch.equal(want, out)
    pool.check_device_errors()
    # position 0 is a first token, not an error
    pool.append_decode(0, q, 0.125, kn, kn, pos * 0, softcap=softcap)
    assert pool.check_device_errors() == 0


# ---- rotary positions: far angles ---------------------------------------------------------------------
@pytest.mark.parametrize("pos", [1, 164864, 2 ** 24 - 2, 2 ** 30 + 12345, 2 ** 31 - 9])
@pytest.mark.parametrize("top", [1.0, 6.0, 1e6, 1e9])
def test_far_angles_are_exact(pos, top):
    """The angle of position times frequency is good to 2^-23 rad whatever their sizes: cos and sin of it, two
    units of fp32 (2^-23) from the function, are within 2^-22 of the exact product's."""
    getcontext().prec = 80
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534")
    rng = np.random.default_rng(pos % 1000)
    pool = hw.Pool(1, 1, 64, 16, [[16]], 1, torch.float32, q_heads=1)
    table = hw.rope_table(64)
    freqs = [float(f) for f in top * rng.uniform(-1.0, 1.0, 32)]
    freqs[0], freqs[1] = top, -top
    for i, f in enumerate(freqs):
        table.freq[i] = f
    x = torch.zeros((1, 8, 1, 64), device="cuda")
    x[..., :32] = 1.0  # the output is (cos, sin)
    got = pool.rope(table, None, x, torch.tensor([pos], dtype=torch.int32, device="cuda"))[1].cpu().double().numpy()
    for i in range(8):
        t = np.array([float((Decimal(pos + i) * Decimal(f)) % (2 * pi)) for f in freqs])
        assert np.abs(got[0, i, 0, :32] - np.cos(t)).max() <= 2.0 ** -22
        assert np.abs(got[0, i, 0, 32:] - np.sin(t)).max() <= 2.0 ** -22


# ---- steep slopes and small scales --------------------------------------------------------------------
@pytest.mark.parametrize("scale,slope", [(1e-6, 1e32), (1e-6, -1e32), (1e-11, 1e29), (0.125, 1e33), (1e-11, 3.0), (-0.125, 1e30)])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_steep_slopes_leave_one_key(scale, slope, softcap):
    """A slope whose product with every distance is finite: the newest (or farthest) visible key alone counts,
    in the chunk and in the decode step."""
    D, w, n, n0 = 64, 150, 40, 333
    pool = hw.Pool(1, 1, D, 16, [[w]], 1, torch.bfloat16, q_heads=2)
    gen = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((1, 1, n0 + n, D), generator=gen, device="cuda").bfloat16() for _ in range(2))
    pos = torch.tensor([n0], dtype=torch.int32, device="cuda")
    pool.materialize(0, k, v, pos)
    q = torch.randn((1, n, 2, D), generator=gen, device="cuda").bfloat16()
    kn, vn = (t[:, :, n0:].transpose(1, 2).contiguous() for t in (k, v))
    slopes = torch.tensor([slope, slope / 4], device="cuda")
    out = np64(pool.prefill(0, q, scale, kn, vn, pos, pos * 0 + n, softcap=softcap, slopes=slopes))[0]
    last = np64(pool.decode(0, q[:, -1].contiguous(), scale, pos + n, softcap=softcap, slopes=slopes))[0]
    for i in range(n):
        at = n0 + i
        p = np.arange(at + 1 - w, at + 1)
        for g in range(2):
            ref, mass, _ = attention(np64(q)[0, i, g], np64(k)[0, 0, p], np64(v)[0, 0, p], scale, at - p, softcap, float(slopes[g]))
            # with the steep slopes one weight is 1 and the others 0; with those of 3 and 3/4 the scores stay below
            # 700 log2 units, 8 roundings of which are 2^-11 of a weight (and of the sum); weights round to bf16
            tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -10) * mass
            assert (np.abs(out[i, g] - ref) <= tol).all(), (i, g)
            if i == n - 1:
                assert (np.abs(last[g] - ref) <= tol).all(), g
    assert pool.check_device_errors() == 0


# ---- captured graphs beside later calls that need more room ------------------------------------------
@pytest.mark.parametrize("kind", ["bf16", "f32", "e4m3"])
def test_captured_decode_outlives_a_larger_configuration(kind):
    """A graph captured before the grid (and with it the arrival counters) grew counts in what it was captured
    with, and gives the same bits."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    pool = hw.Pool(1, 2, 64, 16, [[3000, 64]], 2, TYPES[kind], q_heads=8)
    pool.set_decode_config(workers=20)
    k = torch.randn((2, 2, 3100, 64), generator=gen, device="cuda").to(pool.io_dtype)
    lens = torch.tensor([3100, 700], dtype=torch.int32, device="cuda")
    pool.materialize(0, k, k, lens)
    q = torch.randn((2, 8, 64), generator=gen, device="cuda").to(pool.io_dtype)
    out = torch.empty_like(q)
    want = pool.decode(0, q, 0.125, lens).clone()
    pool.decode(0, q, 0.125, lens, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pool.decode(0, q, 0.125, lens, out=out)
    keep = pool.workspace  # the captured launch's
    pool.set_decode_config(workers=3000)
    wide = pool.decode(0, q, 0.125, lens)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
        assert torch.equal(pool.decode(0, q, 0.125, lens), wide)
    assert keep is not None and pool.check_device_errors() == 0
    pool.close()


def test_captured_calls_keep_their_workspaces():
    """A pool's workspaces that captured launches use stay when later calls need larger ones; others go."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    pool = hw.Pool(1, 2, 64, 16, [[3000, 64]], 1, torch.bfloat16, q_heads=4)
    k = torch.randn((1, 2, 3100, 64), generator=gen, device="cuda").bfloat16()
    lens = torch.tensor([3100], dtype=torch.int32, device="cuda")
    pool.materialize(0, k, k, lens)
    q = torch.randn((1, 4, 64), generator=gen, device="cuda").bfloat16()
    out = torch.empty_like(q)
    want = pool.decode(0, q, 0.125, lens).clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pool.decode(0, q, 0.125, lens, out=out)
    used = weakref.ref(pool.workspace)
    pool.decode(0, q.repeat(1, 8, 1), 0.125, lens)  # a larger group
    assert pool.workspace is not used() and used() is not None
    graph.replay()
    assert torch.equal(out, want)

    # chunks: the workspace of splits grows with the chunk
    pool.set_prefill_config(4)
    chunk = torch.randn((1, 300, 4, 64), generator=gen, device="cuda").bfloat16()
    kn = torch.randn((1, 300, 2, 64), generator=gen, device="cuda").bfloat16()

    def call(n, into=None):
        return pool.prefill(0, chunk[:, :n].contiguous(), 0.125, kn[:, :n].contiguous(), kn[:, :n].contiguous(), lens, lens * 0 + n,
                            out=into)

    call(20)
    plain = weakref.ref(pool.prefill_workspace)
    call(60)
    assert pool.prefill_workspace.numel() > 0 and plain() is None  # no capture used it
    args = [t[:, :60].contiguous() for t in (chunk, kn, kn)]
    n60, into = lens * 0 + 60, torch.zeros((1, 60, 4, 64), device="cuda").bfloat16()
    pool.materialize(0, k, k, lens)  # the ring as it was before the chunks
    want = pool.prefill(0, args[0], 0.125, args[1], args[2], lens, n60).clone()
    torch.cuda.synchronize()
    graph2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph2):
        pool.prefill(0, args[0], 0.125, args[1], args[2], lens, n60, out=into)
    used = weakref.ref(pool.prefill_workspace)
    call(300)
    assert pool.prefill_workspace is not used() and used() is not None
    pool.materialize(0, k, k, lens)
    graph2.replay()
    assert torch.equal(into, want)
    assert pool.check_device_errors() == 0
