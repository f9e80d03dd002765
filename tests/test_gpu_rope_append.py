"""Rotary positions on the way into the pool: queries and keys against the 64-bit formula, rings against
the slots' definition, 8-bit groups against the codes of the turned values.

Tolerance of a turned element: as in test_gpu_rope.py, 2^-20 of r = magnitude * sqrt(a^2 + b^2), then the output's
rounding (bf16 2^-8 of the value).  An 8-bit code is off by half a step of the turned fp32 value: 2^-4 of the value, or 2^-10 of the
scale below 2^-6 of it, beside the 2^-20 r.  Values that do not turn are compared bit for bit."""
import numpy as np
import pytest
import torch

import head_budgeted_kv_gb300 as hw
from reference_ops import GROUP, encode_group, rope, rope_frequencies

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
TYPES = [torch.bfloat16, torch.float32, E4M3]
IDS = ["bf16", "f32", "e4m3"]


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hw.binding.load()
    yield
    torch.cuda.synchronize()


def np64(t):
    return t.float().cpu().double().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """A pool in the middle of serving, and what it held."""

    def __init__(self, windows, B, G=2, D=64, bs=16, dtype=torch.bfloat16, seed=0, layers=1):
        self.windows, self.B, self.G, self.D, self.bs, self.dtype, self.H = windows, B, G, D, bs, dtype, len(windows)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.pool = hw.Pool(layers, self.H, D, bs, [windows] * layers, B, dtype, q_heads=G * self.H)
        n = self.pool.geometry()[1]
        self.pool.set_block_table(np.random.default_rng(seed).permutation(n).astype(np.int32))
        raw = torch.randn(self.pool.blocks().shape, generator=self.gen, device="cuda")
        if dtype == E4M3:
            self.pool.blocks().copy_((raw * 100).to(E4M3))
            self.pool.scales().copy_(torch.exp2(torch.randint(-8, -5, self.pool.scales().shape, generator=self.gen, device="cuda")))
        else:
            self.pool.blocks().copy_(raw.to(dtype))
        self.keep()

    def keep(self):
        self.was = self.pool.blocks().clone()
        self.was_scales = self.pool.scales().clone() if self.dtype == E4M3 else None

    def randn(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda").to(self.pool.io_dtype)

    def ring(self, blocks, s, h, layer=0):
        """[2, C, D] of one head, in the slots' order."""
        return blocks[self.pool.block_table(s, layer, h)].transpose(1, 0, 2, 3).reshape(2, -1, self.D)

    def check(self, k, v, turned, radius, pos, n, layer=0):
        """The layer after rows `turned` (64-bit keys, or None: k as it is) and v went to positions pos .., and the rest as before."""
        got, was, vv, kk = (np64(t) for t in (self.pool.blocks(), self.was, v, k))
        if self.dtype == E4M3:
            got_s, was_s = (t.cpu().double().numpy() for t in (self.pool.scales(), self.was_scales))
        exact = turned is None
        kt = kk if exact else turned
        seen = np.zeros(len(got), dtype=bool)
        for s in range(self.B):
            end = pos[s] + n[s]
            for h, w in enumerate(self.windows):
                ids = self.pool.block_table(s, layer, h)
                seen[ids] = True
                new, old = self.ring(got, s, h, layer), self.ring(was, s, h, layer)
                C = new.shape[1]
                rows = np.arange(max(0, n[s] - C), n[s])
                slot = (pos[s] + rows) % C
                if self.dtype != E4M3:
                    want = old.copy()
                    want[1, slot] = vv[s, rows, h]
                    np.testing.assert_array_equal(new[1], want[1], err_msg=f"V of {s}, {h}")
                    other = np.setdiff1d(np.arange(C), slot)
                    np.testing.assert_array_equal(new[0, other], old[0, other], err_msg=f"other K of {s}, {h}")
                    ref = kt[s, rows, h]
                    tol = 0.0 if exact else 2.0 ** -20 * radius[s, rows, h] + (2.0 ** -8 * np.abs(ref) if self.dtype == torch.bfloat16 else 0.0)
                    assert (np.abs(new[0, slot] - ref) <= tol).all(), f"K of {s}, {h}"
                    continue
                sc = got_s[ids].transpose(2, 0, 1).reshape(2, -1)
                osc = was_s[ids].transpose(2, 0, 1).reshape(2, -1)
                hit = np.zeros(C, dtype=bool)
                hit[slot] = True
                for g in range(C // GROUP):
                    at = slice(g * GROUP, (g + 1) * GROUP)
                    if not hit[at].any():
                        np.testing.assert_array_equal(new[:, at], old[:, at])
                        np.testing.assert_array_equal(sc[:, g], osc[:, g])
                        continue
                    for kv, src in enumerate((kt, vv)):
                        x, r = np.zeros((2, GROUP, self.D))
                        for j in range(GROUP):
                            p = end - 1 - (end - 1 - (g * GROUP + j)) % C
                            if p < 0 or p < end - w:
                                continue
                            if p >= pos[s]:
                                x[j] = src[s, p - pos[s], h]
                                r[j] = 0.0 if exact or kv else radius[s, p - pos[s], h]
                            else:
                                x[j] = old[kv, g * GROUP + j] * osc[kv, g]
                        codes, scale = encode_group(x)
                        assert sc[kv, g] == scale, (s, h, g, kv)
                        if exact or kv:
                            np.testing.assert_array_equal(new[kv, at], codes, err_msg=f"{s}, {h}, {g}, {kv}")
                        else:
                            # a kept value's code is the nearest one, or one of the two nearest to a turned value
                            assert (np.abs(new[kv, at] * scale - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale) + 2.0 ** -20 * r).all(), (s, h, g)
                            assert ((new[kv, at] == codes) | (r > 0)).all()
        if self.pool.layers == 1:
            assert seen.all()
        else:  # the other layers
            keep = ~seen
            np.testing.assert_array_equal(got[keep], was[keep])
            if self.dtype == E4M3:
                np.testing.assert_array_equal(got_s[keep], was_s[keep])


def turned64(x, at, n, freqs, layout, magnitude):
    """(turned rows, radius of each element's pair), 64 bits; rows past n are not filled."""
    y, r = x.copy(), np.zeros_like(x)
    f = len(freqs)
    a, b = (np.arange(f), np.arange(f) + f) if layout == "half" else (2 * np.arange(f), 2 * np.arange(f) + 1)
    for s in range(x.shape[0]):
        for i in range(n[s]):
            y[s, i] = rope(x[s, i], at[s] + i, freqs, layout, magnitude)
        r[s][..., a] = r[s][..., b] = magnitude * np.hypot(x[s][..., a], x[s][..., b])
    return y, r


def check_rows(got, old, ref, radius, n, io):
    """Rows below n near ref, the others as they were."""
    got, old = np64(got), np64(old)
    for s in range(got.shape[0]):
        tol = 2.0 ** -20 * radius[s, :n[s]] + (2.0 ** -8 * np.abs(ref[s, :n[s]]) if io == torch.bfloat16 else 0.0)
        assert (np.abs(got[s, :n[s]] - ref[s, :n[s]]) <= tol).all(), s
        np.testing.assert_array_equal(got[s, n[s]:], old[s, n[s]:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("windows,B,n,G,D,bs,rot,pos", [
    ([64], 1, 1, 1, 64, 16, 64, [0]),                          # the first token
    ([33, 128, 1], 3, 1, 4, 128, 16, 128, [40, 127, 100000]),  # one token each, windows that fill no block
    ([64, 16], 2, 16, 2, 64, 16, 64, [16, 0]),                 # whole groups
    ([100, 20], 2, 37, 2, 64, 32, 20, [5, 95]),                # ragged, pairs that no vector holds whole
    ([16, 17, 48], 2, 53, 1, 128, 16, 64, [3, 14]),            # chunks longer than rings: laps within a chunk
    ([40, 33, 47], 3, 44, 2, 64, 16, 30, [7, 20, 1000]),       # a chunk that ends in the group it began in
    ([16], 2, 20, 1, 64, 16, 2, [13, 0]),                      # one group, rows of two laps in the window
    ([1, 2], 2, 5, 3, 64, 16, 62, [30, 0]),
    ([700, 300], 4, 300, 2, 64, 64, 64, [0, 500, 699, 12345]),  # several rows of a CTA
])
def test_against_the_formula(windows, B, n, G, D, bs, rot, pos, dtype, layout):
    c = Case(windows, B, G, D, bs, dtype, seed=n + rot)
    rng = np.random.default_rng(rot)
    rows = rng.integers(0, n, B, endpoint=True)
    rows[0] = n
    ahead = [0, 50000][n % 2]
    scaling = ("none", "linear", "ntk", "by_parts")[(n + rot // 2) % 4]
    table = hw.rope_table(D, rot, 10000.0, layout, scaling, 4.0, 4096)
    freqs, magnitude = rope_frequencies(rot, 10000.0, scaling, 4.0, 4096)
    qkv = c.randn(B, n, (G + 2) * c.H, D)   # slices of one projection
    q, k, v = qkv.split((G * c.H, c.H, c.H), 2)
    q_out, k_out = torch.full_like(c.randn(B, n, G * c.H, D), 3.0), torch.full_like(c.randn(B, n, c.H, D), -5.0)
    oq, ok = q_out.clone(), k_out.clone()
    turn = i32([p + ahead for p in pos]) if ahead else None
    keys = n % 3 != 2
    got = c.pool.rope_append(0, table, q, k, v, i32(pos), i32(rows), q_out, k_out if keys else None, turn)
    assert got[0] is q_out and got[1] is (k_out if keys else None)
    at = [p + ahead for p in pos]
    yq, rq = turned64(np64(q), at, rows, freqs, layout, magnitude)
    yk, rk = turned64(np64(k), at, rows, freqs, layout, magnitude)
    check_rows(q_out, oq, yq, rq, rows, c.pool.io_dtype)
    check_rows(k_out, ok, yk if keys else np64(ok), rk, rows if keys else [0] * B, c.pool.io_dtype)
    c.check(k, v, yk, rk, pos, rows)
    assert c.pool.check_device_errors() == 0


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("windows,n,pos,bs", [([40, 100], 33, [9, 200], 16), ([17], 70, [0, 16], 32), ([300, 20], 1, [299, 19], 16)])
def test_without_turning_rows_are_stored_as_they_are(windows, n, pos, bs, dtype):
    c = Case(windows, 2, 1, 128, bs, dtype, seed=n)
    k, v = c.randn(2, n, c.H, 128), c.randn(2, n, c.H, 128)
    c.pool.rope_append(0, None, None, k, v, i32(pos))
    c.check(k, v, None, None, pos, [n, n])
    # queries go with them unturned
    q = c.randn(2, n, 2 * c.H, 128)
    q_out, _ = c.pool.rope_append(0, None, q, k, v, i32(pos))
    assert torch.equal(q_out, q)
    assert c.pool.check_device_errors() == 0


@pytest.mark.parametrize("dtype,bs", [(torch.bfloat16, 16), (torch.float32, 16), (torch.bfloat16, 5), (torch.float32, 24)])
def test_equals_rope_and_appends_in_turn(dtype, bs):
    """bf16 and fp32: the same bits as the separate calls, odd blocks too."""
    a, b = (Case([23, 64, 9], 3, 2, 64, bs, dtype, seed=5, layers=2) for _ in range(2))
    q, k, v = a.randn(3, 30, 6, 64), a.randn(3, 30, 3, 64), a.randn(3, 30, 3, 64)
    table = hw.rope_table(64, 40, layout="interleaved")
    pos, n = [0, 17, 90], [30, 11, 0]
    qa, ka = a.pool.rope_append(1, table, q, k, v, i32(pos), i32(n), k_out=torch.zeros_like(k))
    qb, kb = b.pool.rope(table, q, k, i32(pos), i32(n))
    assert torch.equal(qa, qb) and torch.equal(ka, kb)
    for i in range(30):
        live = [s for s in range(3) if i < n[s]]
        blocks = b.pool.blocks().clone()
        b.pool.append(1, kb[:, i].contiguous(), v[:, i].contiguous(), i32([p + i for p in pos]))
        for s in range(3):  # append takes every sequence: give back the rows that a finished one lost
            if s not in live:
                for h in range(3):
                    ids = torch.tensor(b.pool.block_table(s, 1, h), device="cuda").long()
                    b.pool.blocks()[ids] = blocks[ids]
    assert torch.equal(a.pool.blocks(), b.pool.blocks())


def test_8_bit_token_without_turning_equals_append():
    a, b = (Case([40, 100, 16], 4, 1, 128, 16, E4M3, seed=3) for _ in range(2))
    for pos in ([0, 39, 40, 1000], [1, 40, 41, 1001], [15, 47, 48, 1015]):
        k, v = a.randn(4, 3, 128), a.randn(4, 3, 128)
        a.pool.rope_append(0, None, None, k, v, i32(pos))
        b.pool.append(0, k, v, i32(pos))
        assert torch.equal(a.pool.blocks().view(torch.uint8), b.pool.blocks().view(torch.uint8))
        assert torch.equal(a.pool.scales(), b.pool.scales())


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("layout,rot", [("half", 64), ("interleaved", 64), ("half", 20)])
def test_in_place(dtype, layout, rot):
    c, d = (Case([30, 90], 2, 3, 64, 16, dtype, seed=rot) for _ in range(2))
    q, k, v = c.randn(2, 41, 6, 64), c.randn(2, 41, 2, 64), c.randn(2, 41, 2, 64)
    table = hw.rope_table(64, rot, layout=layout)
    pos, n = i32([3, 77]), i32([41, 20])
    keys = dtype != E4M3
    want_q, want_k = c.pool.rope_append(0, table, q, k, v, pos, n, k_out=k.clone() if keys else None)
    qi, ki = q.clone(), k.clone()
    d.pool.rope_append(0, table, qi, ki, v, pos, n, q_out=qi, k_out=ki if keys else None)
    for s, m in enumerate([41, 20]):
        assert torch.equal(qi[s, :m], want_q[s, :m]) and torch.equal(qi[s, m:], q[s, m:])
    assert torch.equal(ki, want_k if keys else k)
    assert torch.equal(c.pool.blocks().view(torch.uint8), d.pool.blocks().view(torch.uint8))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_bad_positions_are_flagged_and_skipped(dtype):
    c = Case([40, 33], 6, 1, 64, 16, dtype, seed=1)
    q, k, v = c.randn(6, 9, 2, 64), c.randn(6, 9, 2, 64), c.randn(6, 9, 2, 64)
    q_out = torch.full_like(q, 7.0)
    pos, n = [-1, 2 ** 31 - 9, 5, 5, 0, 2 ** 31 - 10], [3, 9, 10, -1, 4, 9]
    # positions past the last one, more rows than n_max, a negative count; the last sequence's end at 2^31 - 1
    c.pool.rope_append(0, None, q, k, v, i32(pos), i32(n), q_out)
    assert c.pool.check_device_errors() == hw.binding.HWKV_DEVERR_NEG_LENGTH
    c.check(k, v, None, None, [0, 0, 0, 0, 0, 2 ** 31 - 10], [0, 0, 0, 0, 4, 9])
    assert (q_out[:4] == 7).all() and torch.equal(q_out[4, :4], q[4, :4]) and (q_out[4, 4:] == 7).all()
    c.keep()
    c.pool.rope_append(0, hw.rope_table(64), q, k, v, i32([0] * 6), i32([1] * 6), q_out, turn_pos=i32([0, 0, -3, 2 ** 31 - 1, 0, 0]))
    assert c.pool.check_device_errors() == hw.binding.HWKV_DEVERR_NEG_LENGTH
    for s in (2, 3):
        for h in range(2):
            ids = torch.tensor(c.pool.block_table(s, 0, h), device="cuda").long()
            assert torch.equal(c.pool.blocks()[ids].view(torch.uint8), c.was[ids].view(torch.uint8))


def test_values_that_are_not_finite():
    """They pass through bf16 pools and are stored as NaN in 8-bit ones, without changing the others' codes."""
    for dtype in (torch.bfloat16, E4M3):
        c, d = (Case([64], 1, 1, 64, 16, dtype, seed=8) for _ in range(2))
        k, v = c.randn(1, 20, 1, 64), c.randn(1, 20, 1, 64)
        c.pool.rope_append(0, None, None, k, v, i32([5]))
        kk, vv = k.clone(), v.clone()
        kk[0, 3, 0, 7], vv[0, 12, 0, 60] = float("inf"), float("nan")
        for t, a in ((k, kk), (v, vv)):  # none of them is its group's largest
            a[0, 3, 0, 8] = t[0, 3, 0, 8]
        d.pool.rope_append(0, None, None, kk, vv, i32([5]))
        x, y = c.ring(np64(c.pool.blocks()), 0, 0), d.ring(np64(d.pool.blocks()), 0, 0)
        assert np.isnan(y[1, 17, 60]) and (np.isnan(y[0, 8, 7]) if dtype == E4M3 else np.isinf(y[0, 8, 7]))
        x[1, 17, 60] = x[0, 8, 7] = y[1, 17, 60] = y[0, 8, 7] = 0
        np.testing.assert_array_equal(x, y)


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_new_outputs_belong_to_the_stream_of_the_call(raw):
    """Zeros past n are filled on the stream that turns the rows, not on a current stream that is behind."""
    c = Case([40, 100], 2, 1, 128, 16, torch.bfloat16, seed=2)
    q, k, v = c.randn(2, 33, 4, 128), c.randn(2, 33, 2, 128), c.randn(2, 33, 2, 128)
    table, pos, n = hw.rope_table(128), i32([9, 200]), i32([33, 12])
    want, _ = c.pool.rope_append(0, table, q, k, v, pos, n)
    want = want.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(50_000_000)  # tens of milliseconds
    got, _ = c.pool.rope_append(0, table, q, k, v, pos, n, stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and not got[1, 12:].any()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_captured_chunks_move_on(dtype):
    """A captured call replays at the positions of the moment, as eager calls do; another stream than the current one."""
    c, d = (Case([50, 120], 2, 2, 64, 16, dtype, seed=2) for _ in range(2))
    table = hw.rope_table(64)
    q, k, v = c.randn(2, 7, 4, 64), c.randn(2, 7, 2, 64), c.randn(2, 7, 2, 64)
    pos, n = i32([0, 30]), i32([7, 4])
    q_out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.pool.rope_append(0, table, q, k, v, pos, n, q_out)
        c.pool.advance_positions(pos, delta=5)
    want = i32([0, 30])
    for _ in range(30):
        graph.replay()
        torch.cuda.synchronize()
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        got, _ = d.pool.rope_append(0, table, q, k, v, want, n, stream=other)
        other.synchronize()
        for s, m in enumerate([7, 4]):
            assert torch.equal(got[s, :m], q_out[s, :m])
        want += 5
    assert torch.equal(c.pool.blocks().view(torch.uint8), d.pool.blocks().view(torch.uint8))
    assert c.pool.check_device_errors() == 0


def test_refusals():
    c = Case([32, 32], 2, 2, 64, 16)
    B = hw.binding
    q, k, v = c.randn(2, 3, 4, 64), c.randn(2, 3, 2, 64), c.randn(2, 3, 2, 64)
    pos, table = i32([0, 0]), hw.rope_table(64)

    def refused(error, status=None, **kw):
        args = dict(layer=0, table=table, q=q, k=k, v=v, pos=pos) | kw
        with pytest.raises(error) as e:
            c.pool.rope_append(**args)
        if status is not None:
            assert e.value.status == status

    refused(B.HwkvError, B.HWKV_ERR_INVALID_ARG, layer=1)
    refused(B.HwkvError, B.HWKV_ERR_INVALID_ARG, table=hw.rope_table(128, 128))  # wider than the head
    refused(ValueError, pos=pos.long())
    refused(ValueError, pos=pos[:1])
    refused(ValueError, pos=pos.cpu())
    refused(ValueError, n=pos.long())
    refused(ValueError, turn_pos=pos[:1])
    refused(ValueError, k=k.float())
    refused(ValueError, v=c.randn(2, 3, 3, 64))
    refused(ValueError, v=c.randn(2, 2, 2, 64))
    refused(ValueError, q=c.randn(2, 2, 4, 64))
    refused(ValueError, q=c.randn(2, 3, 3, 64))
    refused(ValueError, q=None, q_out=q)
    refused(ValueError, k=k.transpose(2, 3).contiguous().transpose(2, 3))
    refused(ValueError, q_out=torch.zeros_like(q).float())
    refused(ValueError, k_out=torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16))  # on the host
    refused(B.HwkvError, B.HWKV_ERR_INVALID_ARG, q_out=torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16, device="cuda").expand(2, 3, 4, 64))
    refused(B.HwkvError, B.HWKV_ERR_INVALID_ARG, k_out=v)
    wide = torch.zeros(2, 3, 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")[..., :128].view(2, 3, 2, 64)
    refused(B.HwkvError, B.HWKV_ERR_ALIGNMENT, v=wide)
    flat = torch.zeros(2 * 3 * 2 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 3, 2, 64)
    refused(B.HwkvError, B.HWKV_ERR_ALIGNMENT, k=flat)
    assert torch.equal(c.pool.blocks(), c.was)  # nothing was launched
    e = Case([32, 32], 2, 2, 64, 16, E4M3)
    with pytest.raises(B.HwkvError) as err:
        e.pool.rope_append(0, table, q, k, v, pos, k_out=k)
    assert err.value.status == B.HWKV_ERR_UNSUPPORTED
