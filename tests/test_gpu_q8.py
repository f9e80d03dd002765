"""8-bit pools (HWKV_E4M3) on the GPU: codes and scales bit for bit against the 64-bit reference,
attention within what its roundings allow.

Attention tolerance, per element, with A = sum_p softmax_p |v_p|: the output's rounding to bf16
(2^-8 |ref|); the weights' rounding to fp16 (2^-11 A); and the fp32 scores: a score of log2 size s
carries a few roundings of 2^-24 s and the exponential 2^-22, so each weight is off by at most
2^-11 for |s| up to 2^9 (scores here stay below 2^8; 8 roundings) in all 2^-12 A more.  Weights are
normalised by their own sum, whose error is bounded the same way: both terms count twice.
A fp16 weight below its normal range is off by an absolute amount instead: the kernel's weights are
2^11 p / p_ref (v_scale / v_scale_max) with p_ref between p_max / 2^4 and p_max, steps below 2^-14
are 2^-24, half of one is 2^-25, so a weight times its V code c is off by at most
2^-36 |c| v_scale_max in the output (p_ref over the sum is at most 1): 2^-36 v_scale_max sum |c| in
all.  It matters where the large weights meet zeros."""
import numpy as np
import pytest
import torch

import head_budgeted_kv_gb300 as hw
from reference_ops import Ring8, attention

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hw.binding.load()
    yield
    torch.cuda.synchronize()


def np64(t):
    return t.float().cpu().double().numpy()


class Case:
    """A one-layer 8-bit pool beside its reference rings."""

    def __init__(self, windows, batch, group=4, D=128, bs=16, seed=0, table_seed=None, workers=0):
        self.windows, self.B, self.G, self.D, self.bs = windows, batch, group, D, bs
        self.H, self.dev = len(windows), torch.device("cuda")
        self.gen = torch.Generator(device=self.dev).manual_seed(seed)
        self.pool = hw.Pool(1, self.H, D, bs, [windows], batch, E4M3, q_heads=group * self.H)
        if workers:
            self.pool.set_decode_config(workers=workers)
        if table_seed is not None:
            n = self.pool.geometry()[1]
            self.pool.set_block_table(np.random.default_rng(table_seed).permutation(n).astype(np.int32))
        self.rings = [[Ring8(w, bs, D) for w in windows] for _ in range(batch)]
        self.scale = D ** -0.5

    def randn(self, *shape, scale=1.0):
        return (torch.randn(shape, generator=self.gen, device=self.dev) * scale).bfloat16()

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device=self.dev)

    def materialize(self, lens, k=None, v=None):
        n = max(1, max(lens))
        k = self.randn(self.B, self.H, n, self.D) if k is None else k
        v = self.randn(self.B, self.H, n, self.D) if v is None else v
        self.pool.materialize(0, k, v, self.i32(lens))
        kk, vv = np64(k), np64(v)
        for s in range(self.B):
            for h in range(self.H):
                self.rings[s][h].materialize(kk[s, h], vv[s, h], lens[s])

    def ref_append(self, k, v, pos):
        kk, vv = np64(k), np64(v)
        for s in range(self.B):
            for h in range(self.H):
                self.rings[s][h].append(kk[s, h], vv[s, h], pos[s])

    def check_pool(self, what=""):
        blocks, scales = np64(self.pool.blocks()), self.pool.scales().cpu().double().numpy()
        for s in range(self.B):
            for h in range(self.H):
                ring, ids = self.rings[s][h], self.pool.block_table(s, 0, h)
                got = blocks[ids].transpose(1, 0, 2, 3).reshape(2, ring.C, self.D)
                np.testing.assert_array_equal(got, ring.codes, err_msg=f"{what} codes of seq {s} head {h}")
                got = scales[ids].transpose(2, 0, 1).reshape(2, -1)
                np.testing.assert_array_equal(got, ring.scales, err_msg=f"{what} scales of seq {s} head {h}")

    def check_out(self, q, out, lens, what=""):
        qq, got = np64(q), np64(out)
        for s in range(self.B):
            for h in range(self.H):
                ring = self.rings[s][h]
                p, k, v = ring.resident(lens[s])
                used = np.repeat(ring.scales[1], 16)[p % ring.C]
                floor = 2.0 ** -36 * np.nansum(np.abs(ring.codes[1][p % ring.C]), 0) * used.max(initial=0.0)
                for g in range(h * self.G, (h + 1) * self.G):
                    ref, mass, top = attention(qq[s, g], k, v, self.scale, lens[s] - 1 - p)
                    assert not top > 128, "outside the tolerance's range"
                    tol = 2.0 ** -8 * np.abs(ref) + 2 * (2.0 ** -11 + 2.0 ** -12) * mass + floor
                    bad = ~(np.abs(got[s, g] - ref) <= tol)
                    bad &= ~(np.isnan(ref) & np.isnan(got[s, g]))
                    assert not bad.any(), (f"{what} seq {s} query head {g}: off by "
                                           f"{np.abs(got[s, g] - ref).max():.3e} of {np.abs(ref).max():.3e}")

    def step(self, pos, fused=True, what="", kscale=1.0, vscale=1.0, check=True, k=None, v=None):
        q = self.randn(self.B, self.G * self.H, self.D, scale=1.5)
        k = self.randn(self.B, self.H, self.D, scale=kscale) if k is None else k
        v = self.randn(self.B, self.H, self.D, scale=vscale) if v is None else v
        lens = [p + 1 for p in pos]
        if fused:
            out = self.pool.append_decode(0, q, self.scale, k, v, self.i32(pos))
        else:
            self.pool.append(0, k, v, self.i32(pos))
            out = self.pool.decode(0, q, self.scale, self.i32(lens))
        self.ref_append(k, v, pos)
        if check:
            self.check_pool(what)
            self.check_out(q, out, lens, what)
        return q, out

    def close(self):
        assert self.pool.check_device_errors() == 0
        self.pool.close()


GEOMETRIES = {
    "plain": dict(windows=[64, 200], batch=2, lens=[300, 90]),
    "w1": dict(windows=[1, 1, 2], batch=2, lens=[50, 3]),
    "c_gt_w": dict(windows=[40, 24, 33], batch=3, lens=[300, 47, 0]),
    "under_a_group": dict(windows=[3, 15, 17], batch=2, lens=[2, 100]),
    "empty": dict(windows=[64, 100], batch=3, lens=[0, 0, 1]),
    "d64": dict(windows=[64, 500, 33], batch=2, D=64, lens=[700, 20]),
    "bs32": dict(windows=[100, 70], batch=2, bs=32, lens=[130, 64]),
    "bs48_d64": dict(windows=[100, 49], batch=2, bs=48, D=64, lens=[170, 48]),
    "bs128": dict(windows=[300, 129], batch=2, bs=128, lens=[1000, 200]),
    "g1": dict(windows=[200], batch=2, group=1, lens=[333, 17]),
    "g3_d64": dict(windows=[200, 64], batch=1, group=3, D=64, lens=[333]),
    "g8": dict(windows=[128, 700], batch=2, group=8, lens=[900, 5]),
    "g9": dict(windows=[128, 40], batch=1, group=9, lens=[200]),
    "g16": dict(windows=[256, 48], batch=2, group=16, lens=[600, 31]),
    "g16_d64": dict(windows=[256, 48], batch=2, group=16, D=64, lens=[600, 31]),
}


@pytest.mark.parametrize("fused", [False, True], ids=["append", "fused"])
@pytest.mark.parametrize("name", sorted(GEOMETRIES))
def test_store_append_decode(name, fused):
    spec = dict(GEOMETRIES[name])
    lens = spec.pop("lens")
    c = Case(seed=1, table_seed=5, **spec)
    c.materialize(lens)
    c.check_pool(f"{name} stored")
    q = c.randn(c.B, c.G * c.H, c.D)
    c.check_out(q, c.pool.decode(0, q, c.scale, c.i32(lens)), lens, f"{name} prompt")
    pos = list(lens)
    for i in range(4):
        # rows of growing and shrinking size, so that groups are scaled up and down
        c.step(pos, fused, f"{name} step {i}", kscale=(1.0, 9.0, 0.05, 2.0)[i], vscale=(1.0, 0.01, 40.0, 1.0)[i])
        pos = [p + 1 for p in pos]
    c.close()


@pytest.mark.parametrize("seed", range(12))
def test_random_geometries(seed):
    rng = np.random.default_rng(100 + seed)
    H = int(rng.integers(1, 5))
    c = Case([int(x) for x in rng.integers(1, 400, H)], int(rng.integers(1, 5)), int(rng.integers(1, 17)),
             int(rng.choice([64, 128])), int(rng.choice([16, 32, 64, 80])), seed, seed + 1, int(rng.choice([0, 1, 2, 7, 40])))
    lens = [int(x) for x in rng.integers(0, 600, c.B)]
    c.materialize(lens)
    c.check_pool()
    for i in range(3):
        c.step(lens, bool(i % 2), f"step {i}")
        lens = [p + 1 for p in lens]
    c.close()


@pytest.mark.parametrize("workers", [0, 1, 3, 33, 200])
@pytest.mark.parametrize("D,group", [(128, 4), (64, 16)])
def test_long_ring_through_every_merge(workers, D, group):
    """One long group split over many CTAs: direct, flat and two-level merges."""
    c = Case([6000, 16], 1, group, D, 16, 3, None, workers)
    c.materialize([7001])
    c.step([7001], True, f"workers {workers}")
    c.close()


def test_ring_goes_round_and_sequences_start_over():
    """Appends through two laps of the rings, then the sequence is replaced by a shorter one: rows
    of the earlier one never show, and leave the scales of the groups that are stored anew."""
    c = Case([20, 33], 2, 4, 64, 16, 7)
    c.materialize([5, 0])
    pos = [5, 0]
    for i in range(75):
        c.step(pos, i % 2 == 0, f"lap step {i}", vscale=3.0 ** (i % 5 - 2), check=i % 9 == 0 or i > 70)
        pos = [p + 1 for p in pos]
    pos = [0, 3]
    for i in range(18):
        c.step(pos, i % 2 == 0, f"new sequence step {i}", kscale=0.01, check=i % 4 == 0)
        pos = [p + 1 for p in pos]
    c.close()


def test_values_at_the_edges_of_the_types():
    """Zeros, bf16 subnormals, the largest bf16, exact powers of two around the scale's border."""
    c = Case([48], 1, 1, 64, 16, 0)
    rows = torch.zeros((1, 1, 48, 64), device=c.dev)
    rows[0, 0, 16:32] = torch.linspace(-1, 1, 64, device=c.dev) * 2.0 ** -130
    rows[0, 0, 20, 3] = 2.0 ** -133
    rows[0, 0, 32, 0], rows[0, 0, 33, 1] = 448.0, -449.0     # bf16 rounds 449 to 448
    rows[0, 0, 34, 2], rows[0, 0, 35, 5] = 2.0 ** -9, 3 * 2.0 ** -10
    big = rows.clone()
    big[0, 0, 3, 7], big[0, 0, 4, 8], big[0, 0, 32, 0] = 3.3895e38, -1.5, 450.0
    c.materialize([48], rows.bfloat16(), big.bfloat16())
    c.check_pool("edges")
    for x in (0.0, 2.0 ** -133, 3.3895e38, 448.0, 452.0):
        row = torch.zeros((1, 1, 64), device=c.dev)
        row[0, 0, 5] = x
        c.pool.append(0, row.bfloat16(), -row.bfloat16(), c.i32([48]))
        c.ref_append(row.bfloat16(), -row.bfloat16(), [48])
        c.check_pool(f"append {x}")
    c.close()


@pytest.mark.parametrize("fused", [False, True], ids=["append", "fused"])
def test_non_finite_rows_stay_in_their_window(fused):
    """A NaN or infinite row makes the results that see it NaN, and no other one, neither while the
    ring still holds it outside the window (C > w) nor afterwards."""
    c = Case([5, 40], 1, 4, 128, 16, 11)
    c.materialize([100])
    for i in range(60):
        k, v = c.randn(1, 2, 128), c.randn(1, 2, 128)
        if i == 0:
            v[0, :, 9], k[0, 1, 3] = float("nan"), float("inf")
        if i == 1:
            v[0, 0, 4] = float("-inf")
        q, out = c.step([100 + i], fused, f"step {i}", k=k, v=v, check=False)
        c.check_pool(f"step {i}")
        got = np64(out)[0]
        assert np.isnan(got[:4]).any() == (i <= 5), i
        assert np.isnan(got[4:]).any() == (i < 40), i
        if i >= 40:
            c.check_out(q, out, [101 + i], f"step {i}")
    c.close()


def test_slots_outside_the_window_may_hold_anything():
    """Codes and scales of slots past the length or out of the window are arbitrary bits."""
    c = Case([40, 33], 2, 4, 128, 16, 13)
    c.pool.buffer.fill_(0x7F)  # NaN codes, NaN scales
    lens = [21, 100]
    c.materialize(lens)
    q = c.randn(2, 8, 128)
    c.check_out(q, c.pool.decode(0, q, c.scale, c.i32(lens)), lens)
    zero = c.pool.decode(0, q, c.scale, c.i32([0, 0]))
    assert (zero == 0).all()
    c.close()


def test_queries_of_very_different_sizes():
    """A query head is scaled by a power of two inside the kernel; a zero head gives the mean."""
    c = Case([64, 30], 1, 4, 64, 16, 17)
    c.materialize([80])
    q = c.randn(1, 8, 64)
    q[0, 1] *= 1e-30
    q[0, 2] = 0
    q[0, 3, 1:] *= 1e-6
    q[0, 5] *= 20
    out = c.pool.decode(0, q, c.scale, c.i32([80]))
    c.check_out(q, out, [80])
    c.close()


def test_value_scales_far_apart():
    """Groups whose V scales differ by many powers of two, in either order."""
    c = Case([96], 1, 2, 128, 16, 19)
    k, v = c.randn(1, 1, 96, 128), c.randn(1, 1, 96, 128)
    for g, e in enumerate((-20, 3, 30, -60, 12, 30)):
        v[0, 0, 16 * g:16 * (g + 1)] *= 2.0 ** e
    c.materialize([96], k, v)
    q = c.randn(1, 2, 128)
    c.check_out(q, c.pool.decode(0, q, c.scale, c.i32([96])), [96])
    c.check_out(q, c.pool.decode(0, q, c.scale, c.i32([64])), [64])  # only earlier groups are seen
    c.close()


def test_fused_step_is_append_then_decode_and_repeats_bit_for_bit():
    outs, pools = [], []
    for fused in (True, True, False):
        c = Case([300, 2000, 50], 3, 4, 128, 16, 23)
        c.materialize([2500, 40, 700])
        _, out = c.step([2500, 40, 700], fused)
        outs.append(out)
        pools.append(c.pool.buffer.clone())
        c.close()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert torch.equal(pools[0], pools[1]) and torch.equal(pools[0], pools[2])


def test_other_entry_points_take_8_bit_pools():
    """The call without a workspace, prepared launches with early reads, a side stream, and a
    captured step: the same bits as the plain call."""
    c = Case([300, 64], 2, 4, 128, 16, 29)
    c.materialize([500, 10])
    lens = c.i32([500, 10])
    q = c.randn(2, 8, 128)
    want = c.pool.decode(0, q, c.scale, lens)
    out = torch.empty_like(q)
    hw.binding.hwkv_decode_attn_noalloc(c.pool.handle, 0, q, c.scale, lens, out)
    assert torch.equal(out, want)
    out.zero_()
    launch = c.pool.decode_launch(0, q, c.scale, lens, out, early_reads=True)
    launch()
    assert torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.pool.decode(0, q, c.scale, lens)
    side.synchronize()
    assert torch.equal(got, want)
    c.close()


def test_captured_steps_match_eager_steps():
    from head_budgeted_kv_gb300.graph import DecodeStepGraph
    results = []
    for graph in (False, True):
        gen = torch.Generator(device="cuda").manual_seed(5)

        def randn(*shape):
            return torch.randn(shape, generator=gen, device="cuda").bfloat16()

        pool = hw.Pool(2, 2, 128, 16, [[64, 30], [200, 16]], 2, E4M3, q_heads=8)
        pos = torch.tensor([70, 3], dtype=torch.int32, device="cuda")
        for l in range(2):
            pool.materialize(l, randn(2, 2, 70, 128), randn(2, 2, 70, 128), pos)
        step = DecodeStepGraph(pool, 128 ** -0.5, 8, pos) if graph else None
        outs = []
        for _ in range(4):
            q, k, v = randn(2, 2, 8, 128), randn(2, 2, 2, 128), randn(2, 2, 2, 128)
            if graph:
                step.q.copy_(q), step.k_new.copy_(k), step.v_new.copy_(v)
                step.replay()
                outs.append(step.out.clone())
            else:
                outs.append(torch.stack([pool.append_decode(l, q[l], 128 ** -0.5, k[l], v[l], pos) for l in range(2)]))
                pos = pos + 1
        results.append((torch.stack(outs), pool.buffer.clone()))
        assert pool.check_device_errors() == 0
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])


def test_bad_lengths_are_flagged_and_skipped():
    c = Case([64, 20], 2, 4, 128, 16, 31)
    before = c.pool.buffer.clone()
    k = c.randn(2, 2, 8, 128)
    c.pool.materialize(0, k, k, c.i32([-1, 9]))
    assert c.pool.check_device_errors() == hw.binding.HWKV_DEVERR_NEG_LENGTH | hw.binding.HWKV_DEVERR_SRC_RANGE
    c.pool.append(0, k[:, :, 0].contiguous(), k[:, :, 0].contiguous(), c.i32([-3, -1]))
    assert c.pool.check_device_errors() == hw.binding.HWKV_DEVERR_NEG_LENGTH
    assert torch.equal(c.pool.buffer, before)
    c.close()


def test_footprint_and_views():
    c = Case([33, 128], 3, 4, 64, 16, 37)
    assert c.pool.nbytes == c.pool.buffer.numel() == 3 * 11 * 2 * 16 * 64 + (3 * 11 * 8 + 15) // 16 * 16
    assert c.pool.blocks().shape == (33, 2, 16, 64) and c.pool.scales().shape == (33, 1, 2)
    assert (c.pool.buffer == 0).all()
    # a saved pool is restored through its views
    c.materialize([200, 5, 64])
    codes, scales = c.pool.blocks().clone(), c.pool.scales().clone()
    d = Case([33, 128], 3, 4, 64, 16, 37)
    d.pool.blocks().copy_(codes)
    d.pool.scales().copy_(scales)
    q, lens = c.randn(3, 8, 64), c.i32([200, 5, 64])
    assert torch.equal(c.pool.decode(0, q, c.scale, lens), d.pool.decode(0, q, c.scale, lens))
    c.close(), d.close()


@pytest.mark.parametrize("scale", [-0.2, 0.0])
def test_negative_and_zero_scale(scale):
    """A negative scale attends to the least alike keys; a zero one gives the mean of the values."""
    c = Case([64, 30], 1, 4, 64, 16, 41)
    c.scale = scale
    c.materialize([80])
    q = c.randn(1, 8, 64)
    c.check_out(q, c.pool.decode(0, q, scale, c.i32([80])), [80])
    c.close()


def test_more_sequences_than_lengths_staged():
    """Past 256 sequences the lengths are read from global memory; some prompts are empty."""
    lens = [(i * 37) % 90 for i in range(300)]
    c = Case([20, 48], 300, 2, 64, 16, 43)
    c.materialize(lens)
    c.check_pool()
    c.step(lens, True, check=False)
    c.check_pool("appended")
    q = c.randn(300, 4, 64)
    now = [x + 1 for x in lens]
    c.check_out(q, c.pool.decode(0, q, c.scale, c.i32(now)), now)
    c.close()


def test_source_by_strides():
    """The prompt's K and V may be slices of larger tensors."""
    a, b = Case([40, 20], 2, 4, 64, 16, 47), Case([40, 20], 2, 4, 64, 16, 47)
    big = a.randn(2, 5, 90, 64)
    k, v = big[:, 0:2], big[:, 2:4]
    a.pool.materialize(0, k, v, a.i32([90, 33]))
    b.pool.materialize(0, k.contiguous(), v.contiguous(), b.i32([90, 33]))
    assert torch.equal(a.pool.buffer, b.pool.buffer) and a.pool.buffer.any()
    a.close(), b.close()


def test_refusals():
    c = Case([64, 30], 1, 4, 64, 16, 53)
    q, k, lens = c.randn(1, 8, 64), c.randn(1, 2, 64), c.i32([5])
    for call in (lambda: c.pool.decode(0, q.float(), 0.1, lens), lambda: c.pool.append(0, k.float(), k, lens),
                 lambda: c.pool.append_decode(0, q, 0.1, k, k.half(), lens),
                 lambda: c.pool.materialize(0, k[:, :, None].float(), k[:, :, None].float(), lens),
                 lambda: c.pool.decode(0, q, 0.1, lens, out=torch.empty_like(q, dtype=torch.float32))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: c.pool.set_decode_config(kernel=hw.HWKV_KERNEL_SIMT),
                 lambda: c.pool.prefill(0, q[:, None].contiguous(), 0.1, k[:, None].contiguous(), k[:, None].contiguous(),
                                        lens, lens)):
        with pytest.raises(hw.HwkvError) as e:
            call()
        assert e.value.status == hw.binding.HWKV_ERR_UNSUPPORTED
    plain = hw.Pool(1, 1, 64, 16, [[16]], 1, torch.bfloat16)
    with pytest.raises(ValueError):
        plain.scales()
    assert plain.io_dtype == torch.bfloat16 and c.pool.io_dtype == torch.bfloat16
    c.close()


def test_serving_run_with_every_operator():
    """A prompt stored in 8 bits, then steps of rotary positions, the append and capped, biased
    attention, against the reference of all three."""
    from reference_ops import rope, rope_frequencies
    c = Case([48, 200], 2, 4, 64, 16, 59, table_seed=3)
    table = hw.rope_table(64, base=500000.0, scaling="by_parts", factor=4.0, original_len=128)
    freqs, magnitude = rope_frequencies(64, 500000.0, "by_parts", 4.0, 128)
    slopes = torch.tensor([2.0 ** -(g + 1) for g in range(8)], device=c.dev)
    lens = [150, 7]
    k = c.randn(2, 150, 2, 64)
    _, kr = c.pool.rope(table, None, k, c.i32([0, 0]), c.i32(lens))
    v = c.randn(2, 2, 150, 64)
    c.materialize(lens, kr.transpose(1, 2).contiguous(), v)
    c.check_pool("prompt")
    for _ in range(5):
        q, k, v = c.randn(2, 8, 64), c.randn(2, 2, 64), c.randn(2, 2, 64)
        pos = c.i32(lens)
        qr, kr = c.pool.rope(table, q, k, pos)
        for x, y in ((q, qr), (k, kr)):
            for s in range(2):
                ref = rope(np64(x)[s], lens[s], freqs, "half", magnitude)
                size = np.abs(np64(x)[s]).max() * 2 ** 0.5 * magnitude
                assert (np.abs(np64(y)[s] - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * size).all()
        out = c.pool.append_decode(0, qr, c.scale, kr, v, pos, softcap=20.0, slopes=slopes)
        c.ref_append(kr, v, lens)
        lens = [n + 1 for n in lens]
        c.check_pool("step")
        for s in range(2):
            for h in range(2):
                p, rk, rv = c.rings[s][h].resident(lens[s])
                for g in range(4 * h, 4 * h + 4):
                    ref, mass, top = attention(np64(qr)[s, g], rk, rv, c.scale, lens[s] - 1 - p, 20.0, float(slopes[g]))
                    # the capped score is off by 2^-20 of itself (header): 2^-19 top more on each weight
                    tol = 2.0 ** -8 * np.abs(ref) + 2 * (2.0 ** -11 + 2.0 ** -12 + 2.0 ** -19 * top) * mass
                    assert (np.abs(np64(out)[s, g] - ref) <= tol + 2.0 ** -36 * np.abs(rv).sum(0)).all()
    c.close()
