"""Decode behind shared prefixes at the ends of what its inputs may be, against the 64-bit definition.

Tolerance, per element, with softmax weights p_i, values v_i and A = sum p_i |v_i|.  A score carries head_dim + 4 roundings or
truncations of 2^-23 of |scale| sum |q k_i|; a cap 2^-20 of the cap; a bias eight fp32 roundings (2^-24) of
|s_i| + |slope| (distance + 64), the keys of a stage of 64 sharing an offset: the slope in log2 units and over the scale (3), the offset (2),
the key's own term (1), the maximum (1), the difference with it (1).  The exponential is off by 2^-21.  Together delta_i.

A key whose score is further from the best than both of theirs and 104 (2^-150, below all fp32 numbers) has no weight.  Among the
others, when one is left its weight is 1 whatever its delta; else their deltas are at most 2^-4, and as exp(x) - 1 <= 1.07 x for
x <= 2^-3 they put 1.07 sum p_i |v_i| (delta_i + sum p_j delta_j) into the result.  Weights of bf16 pools are rounded to bf16
(2^-8 A), those of 8-bit pools are closer (see test_gpu_shared.py for their floor), the joins put 2^-20 A and the
output rounds by 2^-8 of the value (fp32: 2^-24)."""
import numpy as np
import pytest
import torch

import head_budgeted_kv_gb300 as hw
from test_gpu_shared import BF16, E4M3, F32, PAIR_IDS, PAIRS, Case, i32, np64

pytestmark = pytest.mark.gpu
NO_WEIGHT = 104.0


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hw.binding.load()
    yield
    torch.cuda.synchronize()


class Ranged(Case):
    def keys_of(self, s, h):
        """(K, V, distances, floor) of what the heads of KV head h of sequence s attend to."""
        n, f = self.own.lens[s], self.of[s]
        p, k, v, floor = self.own.newest(s, h, 0)
        d = n - 1 - p
        if f >= 0:
            N = self.pre.lens[f]
            pp, pk, pv, _ = self.pre.newest(f, h, N + n - self.pre.windows[h])
            k, v, d = np.concatenate((pk, k)), np.concatenate((pv, v)), np.concatenate((N + n - 1 - pp, d))
        return k, v, d, floor

    def check(self, out, seqs=None, what=""):
        """Returns how many heads had more than one key of weight."""
        got, q, mixed = np64(out), np64(self.q), 0
        half = self.io == BF16
        for s in range(self.B) if seqs is None else seqs:
            for h in range(self.H):
                k, v, d, floor = self.keys_of(s, h)
                for g in range(h * self.G, (h + 1) * self.G):
                    if len(k) == 0:
                        assert (got[s, g] == 0).all(), (what, s, g)
                        continue
                    x = k @ q[s, g] * self.scale
                    delta = np.abs(k) @ np.abs(q[s, g]) * abs(self.scale) * (self.D + 4) * 2.0 ** -23 + 2.0 ** -21
                    if self.cap > 0:
                        x = self.cap * np.tanh(x / self.cap)
                        delta += self.cap * 2.0 ** -20
                    if self.slopes is not None:
                        slope = float(self.slopes[g])
                        delta += 8 * 2.0 ** -24 * (np.abs(x) + abs(slope) * (d + 64.0))
                        x = x - slope * d
                    best = int(x.argmax())
                    some = x + delta >= x[best] - delta[best] - NO_WEIGHT
                    w = np.where(some, np.exp(np.minimum(x - x[best], 0.0)), 0.0)
                    w /= w.sum()
                    if some.sum() == 1:
                        delta = np.zeros_like(delta)
                    else:
                        mixed += 1
                        assert delta[some].max() <= 2.0 ** -4, (what, s, g, delta[some].max())
                    ref, A = w @ v, w @ np.abs(v)
                    tol = 1.07 * ((w * (delta + (w * delta).sum())) @ np.abs(v)) + 2.0 ** -20 * A + floor
                    tol += 2.0 ** -8 * (A + np.abs(ref)) if half else 2.0 ** -24 * np.abs(ref)
                    err = np.abs(got[s, g] - ref)
                    assert (err <= tol).all(), f"{what} seq {s} head {g}: {err.max():.3e}, {(err / tol).max():.2f} of what is allowed"
        return mixed


def ranged(types, G=4, D=64, seed=7, **kw):
    return Ranged([64, 40, 300], [700, 90, 500], [0, 5, 30, 63, 200], [500, 100, 30], [0, 1, 0, 0, 2], G, D, 16, types, seed=seed, **kw)


def refill(side, k, v):
    """Other keys and values in a side's pool, and in what is known of it."""
    side.k, side.v = k, v
    side.pool.materialize(0, k, v, i32(side.lens))
    side.kk, side.vv = np64(k), np64(v)
    if side.rings:
        for s, n in enumerate(side.lens):
            for h in range(len(side.windows)):
                side.rings[s][h].materialize(side.kk[s, h], side.vv[s, h], n)


def every_other(heads, steep):
    """Slopes of both signs, whole and a quarter, side by side."""
    return torch.tensor([steep * (1.0, -1.0, 0.25, -0.25)[i % 4] for i in range(heads)], device="cuda")


@pytest.mark.parametrize("types", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("scale,steep", [(0.125, 1.1e5), (0.125, 1e6), (-0.125, 1e9), (1e-6, 1e32), (0.125, 3e35)])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_steep_slopes_leave_one_key(types, cap, scale, steep):
    """The newest key of all, or the farthest that is seen, in whichever of the two pools it lies."""
    c = ranged(types, cap=cap)
    c.scale, c.slopes = scale, every_other(4 * 3, steep)
    assert c.check(c.call()) == 0
    c.step()


@pytest.mark.parametrize("types", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("steep", [1e4, 1e6])
def test_scores_as_large_as_steep_slopes(types, steep):
    """Scores of whole multiples of what a slope takes per position: the farther key wins where its score is that much larger.
    (|a - 0.937 b| is at least 0.063 for whole |a| < 8 and any whole b but a = b = 0: one key always takes all.)"""
    c = Ranged([64, 40], [60, 90], [3, 20, 30], [50, 31], [0, 1, 0], 4, 64, 16, types, seed=3)
    gen = np.random.default_rng(5)
    for side in (c.own, c.pre):
        k = torch.zeros_like(side.k)
        k[..., 0] = torch.tensor(gen.integers(0, 8, k.shape[:-1]), device="cuda").to(k.dtype)
        refill(side, k, side.v)
    c.q.zero_()
    c.q[..., 0] = 8.0
    c.scale, c.slopes = steep / 8, every_other(8, 0.937 * steep)
    assert c.check(c.call()) == 0


@pytest.mark.parametrize("types", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("G,D,N", [(4, 128, 256), (1, 64, 700), (16, 64, 300)])
def test_the_largest_values_do_not_overflow(types, G, D, N):
    """Sums are held relative to the largest weight: a value of 2^125 under a weight e^5 times those before it, at places of every
    stage and chain, gives its share of the result, not infinity."""
    places = list(range(5, N, 61))
    c = Ranged([16], [N], [0] * 20, [N] * len(places), [i % len(places) for i in range(20)], G, D, 16, types, seed=1)
    k, v = torch.zeros_like(c.pre.k), c.pre.v.clone()
    for f, p in enumerate(places):
        k[f, :, p, 0] = 5.0
        v[f, :, p] = 2.0 ** 125 * torch.where(v[f, :, p] < 0, -1.0, 1.0).to(v.dtype)
    refill(c.pre, k, v)
    c.q.zero_()
    c.q[..., 0] = 8.0
    c.scale = 0.125
    c.check(c.call())


def alternating(heads):
    """Slopes of both signs that halve from head to head."""
    return torch.tensor([(-0.5) ** i for i in range(heads)], device="cuda")


@pytest.mark.parametrize("types", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("scale,cap,biased", [(-0.125, 0.0, False), (0.0, 0.0, False), (-0.125, 20.0, False), (0.0, 20.0, False),
                                              (4.0, 3.0, False), (2.0, 30.0, True), (0.125, 500.0, False), (-0.125, 0.0, True),
                                              (0.0, 0.0, True), (1e-14, 0.0, True), (0.125, 0.0, True), (-0.125, 6.0, True),
                                              (1e-14, 6.0, True)])
def test_scales_caps_and_slopes(types, scale, cap, biased):
    """Negative, zero and tiny scales, scores far past the cap and far below it, slopes of both signs."""
    for G, D in ((4, 64), (7, 128)):
        c = ranged(types, G, D, cap=cap)
        c.scale, c.slopes = scale, alternating(3 * G) if biased else None
        c.step(append=False)
        c.step()


class Counted:
    """Queries of zero: every visible key has the same weight.  With values of 1 in one place of a row, of zero in the others, a result
    times the number of visible keys counts the keys whose values lie in that place."""

    def __init__(self, types, own, pre, lens, pre_lens, of, G, D, bs, seed):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.H, self.G, self.D = len(lens), len(own), G, D
        self.own_w, self.pre_w, self.lens, self.pre_lens, self.of = own, pre, lens, pre_lens, of
        self.own = hw.Pool(1, self.H, D, bs, [own], self.B, types[0], q_heads=G * self.H)
        self.pre = hw.Pool(1, self.H, D, bs, [pre], len(pre_lens), types[1], q_heads=G * self.H)
        for pool in (self.own, self.pre):
            pool.set_block_table(np.random.default_rng(seed).permutation(pool.geometry()[1]).astype(np.int32))
        self.q = torch.zeros((self.B, G * self.H, D), dtype=self.own.io_dtype, device="cuda")
        self.keys = [torch.randn((p.num_seqs, self.H, max(1, max(ls)), D), generator=self.gen, device="cuda").to(p.io_dtype)
                     for p, ls in ((self.own, lens), (self.pre, pre_lens))]

    def check(self, own_place, pre_place):
        """own_place, pre_place: the places of the values of position p of head h (-1: none), from [n] to [n]."""
        D = self.D
        places = []
        for pool, keys, lens, place in ((self.own, self.keys[0], self.lens, own_place), (self.pre, self.keys[1], self.pre_lens, pre_place)):
            at = np.stack([place(h, np.arange(keys.shape[2])) for h in range(self.H)])
            t = torch.tensor(at, device="cuda")
            rows = (torch.arange(D, device="cuda") == t[..., None]).to(keys.dtype)  # [H, n, D]
            pool.materialize(0, keys, rows.expand(keys.shape).contiguous(), i32(lens))
            # how many of the first p positions have their values in each place
            some = at[..., None] == np.arange(D)
            places.append(np.concatenate((np.zeros((self.H, 1, D), np.int64), np.cumsum(some, 1)), 1))
        out = self.own.shared_decode(0, self.pre, self.q, 0.125, i32(self.lens), i32(self.of), i32(self.pre_lens))
        assert self.own.check_device_errors() == 0
        got = np64(out).reshape(self.B, self.H, self.G, D)
        half = 2.0 ** -8 if self.own.io_dtype == BF16 else 2.0 ** -22
        for s, (n, f) in enumerate(zip(self.lens, self.of)):
            for h in range(self.H):
                total, count = min(n, self.own_w[h]), places[0][h][n] - places[0][h][max(0, n - self.own_w[h])]
                if f >= 0:
                    N = self.pre_lens[f]
                    first = min(N, max(0, N + n - self.pre_w[h]))
                    total, count = total + N - first, count + places[1][h][N] - places[1][h][first]
                want = count / max(total, 1)
                assert (np.abs(got[s, h] - want) <= half * want + 2.0 ** -22).all(), (s, h, n, f, np.abs(got[s, h] * total - count).max())
        return out

    def check_all(self, rounds):
        """Tile by tile, then around the ends of windows, rings, tiles, stages and wherever chance has it."""
        D = self.D
        whole = self.check(lambda h, p: (p + h) % D, lambda h, p: (p // 16 + h) % D)
        rng = np.random.default_rng(len(self.lens))
        for r in range(rounds):
            def place(h, p):
                N, w = max(self.pre_lens), self.pre_w[h]
                C = -(-w // self.pre.block_size) * self.pre.block_size
                some = [x + d for n in rng.choice(self.lens, 8) for x in (N + n - w, N - w) for d in (-1, 0)]
                some += [x + d for x in range(C, N + 1, C) for d in (-1, 0)][:8] + [0, N - 1, N - 2]
                some += [64 * int(i) + d for i in rng.integers(0, max(1, N // 64) + 1, D) for d in (-1, 0)]
                at = np.full(len(p), -1)
                some = [x for x in dict.fromkeys(some) if 0 <= x < len(p)][:D]
                at[some] = np.arange(len(some))
                return at
            self.check(lambda h, p: np.full(len(p), -1), place)
        return whole


@pytest.mark.parametrize("types", [(BF16, BF16), (E4M3, E4M3), (BF16, E4M3)], ids=["bf16", "e4m3", "bf16-e4m3"])
@pytest.mark.parametrize("G,D,B", [(8, 128, 40), (4, 64, 70)])
def test_every_key_of_a_long_prefix_counts_once(types, G, D, B):
    """One prefix, a pair of query tiles and a single one per head (B sequences, 32 or 64 to a pair), 2 x 4256 stages: more than 32 to
    a CTA, whose stage slots go round many times, and segments that begin and end within a head."""
    lens = [(37 * i) % 200 for i in range(B)]
    c = Counted(types, [200] * 8, [40000, 39999, 33333, 20000, 48000, 45001, 64, 47003], lens, [47003], [0] * B, G, D, 16, 5)
    c.check_all(4)


@pytest.mark.parametrize("types", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("D", [64, 128])
def test_every_key_of_many_prefixes_counts_once(types, D):
    """200 prefixes of 1 to 400 tokens and four heads: several segments to a CTA, of one query tile and of two, of one stage and of
    more, one prefix with 40 sequences (groups of 16: eight to a tile), some with none."""
    rng = np.random.default_rng(D)
    pre_lens = rng.integers(1, 400, 200).tolist()
    pre_lens[3], pre_lens[7] = 0, 64
    of = [5] * 40 + [int(f) if f != 11 else -1 for f in rng.integers(0, 190, 220)]
    of = [of[i] for i in rng.permutation(260)]
    c = Counted(types, [32, 48, 16, 64], [400, 300, 100, 64], rng.integers(0, 60, 260).tolist(), pre_lens, of, 16, D, 32, 6)
    first = c.check_all(4)
    for _ in range(3):
        assert torch.equal(c.check(lambda h, p: (p + h) % D, lambda h, p: (p // 16 + h) % D), first)


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16)], ids=["f32", "bf16"])
def test_every_key_counts_once_on_cuda_cores(types):
    rng = np.random.default_rng(2)
    lens, of = rng.integers(0, 90, 30).tolist(), rng.integers(-1, 3, 30).tolist()
    Counted(types, [90, 7, 40], [3000, 5000, 777], lens, [5000, 1203, 77], of, 3, 64, 24, 7).check_all(4)


@pytest.mark.parametrize("dtype,bs", [(F32, 16), (BF16, 24)], ids=["f32", "bf16"])
def test_prefixes_that_nobody_is_behind_split_no_coarser(dtype, bs):
    """What the CUDA cores take at a time goes by the prefixes that sequences can be behind: the partials' room is that of as many."""
    own = hw.Pool(1, 2, 64, bs, [[64, 64]], 8, dtype, q_heads=8)
    pres = [hw.Pool(1, 2, 64, bs, [[3000, 900]], n, dtype, q_heads=8) for n in (8, 64, 500)]
    need = [hw.binding.hwkv_decode_shared_workspace_bytes(own.handle, p.handle, 8) for p in pres]
    assert need[0] == need[1] == need[2]


@pytest.mark.parametrize("types", PAIRS[:4], ids=PAIR_IDS[:4])
@pytest.mark.parametrize("G,D", [(16, 64), (4, 128)])
def test_many_segments_against_the_definition(types, G, D):
    """As above with random keys, and the same bits from call to call."""
    rng = np.random.default_rng(G)
    of = [2] * (3 * (128 // G) + 1) + rng.integers(-1, 60, 150).tolist()
    c = Ranged([32, 48, 16, 64], [400, 300, 100, 64], rng.integers(0, 60, len(of)).tolist(), rng.integers(1, 400, 60).tolist(),
               [int(f) for f in rng.permutation(of)], G, D, 32, types, seed=G)
    first = c.call().clone()
    c.check(first, seqs=list(range(0, len(of), 9)))
    for _ in range(3):
        assert torch.equal(c.call(), first)
    c.scale, c.slopes, c.cap = 0.2, alternating(4 * G), 5.0
    c.check(c.call(), seqs=list(range(1, len(of), 17)))


@pytest.mark.parametrize("types", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("size", [1e3, 5e5])
@pytest.mark.parametrize("biased", [False, True])
def test_huge_scores(types, size, biased):
    """Scores (up to 5.6e7) so large that one key takes all the weight, in the prefix or among the own ones: its value comes out."""
    places = [23, 70, 140, 250, 299]
    for own_wins in (False, True):
        c = Ranged([40], [300], [20] * 10, [300] * len(places), [i % len(places) for i in range(10)], 4, 64, 16, types, seed=1)
        for side in (c.own, c.pre):
            k = torch.zeros_like(side.k)
            k[..., 0] = (torch.arange(k.shape[2], device="cuda") * 7 % 48 / 64).to(k.dtype)
            for i in range(len(side.lens)):
                k[i, :, 11 if side is c.own else places[i], 0] = 14.0 if (side is c.own) == own_wins else 0.0
            refill(side, k, side.v)
        c.q.zero_()
        c.slopes = torch.tensor([0.5, 0.25, -0.25, 0.0], device="cuda") if biased else None
        for c.scale in (size, -size):
            c.q[..., 0] = 8.0 if c.scale > 0 else -8.0
            assert c.check(c.call()) == 0, c.scale


@pytest.mark.parametrize("types", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("slope", [2e4, -2e4, 8e4])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_slopes_over_long_distances(types, cap, slope):
    """What the distance takes passes 2^31 log2 units within the window: the newest key, or the farthest, takes all the weight."""
    c = Ranged([40], [160000], [20, 0, 39], [150000, 149000], [0, 0, 1], 4, 64, 16, types, seed=1, cap=cap)
    c.slopes = torch.tensor([slope, slope / 2, slope, slope / 4], device="cuda")
    assert c.check(c.call()) == 0
