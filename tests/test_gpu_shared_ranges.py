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
