"""Decode behind shared prefixes against the 64-bit definition.

Tolerance, per element, with softmax weights p_i, values v_i and A = sum p_i |v_i|.  A score s_i = scale <q, k_i> carries
head_dim + 4 roundings or truncations of 2^-23 of scale sum |q k_i|; a cap 2^-20 of the cap (header), a bias 4 fp32
roundings of |s_i| + slope * distance, the exponential 2^-21: delta_i in all, so the weights put
sum p_i |v_i| (delta_i + sum p_j delta_j) into the result.  Weights rounded to bf16 put 2^-8 A there (fp32 pools round none;
fp16 ones of 8-bit pools are closer, but for those below fp16's range: 2^-36 v_scale_max sum |code|, see test_gpu_q8.py), the
partials' joins 2^-20 A, and the output rounds by 2^-8 of the value (fp32: 2^-24)."""
import numpy as np
import pytest
import torch

import head_budgeted_kv_gb300 as hw
from reference_ops import Ring8

pytestmark = pytest.mark.gpu
E4M3, BF16, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32


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


class Side:
    """A pool filled from histories, and what its rings hold as values."""

    def __init__(self, gen, windows, seqs, D, bs, dtype, lens, q_heads, seed, spare=4, kscale=1.0):
        self.windows, self.D, self.dtype, self.lens = windows, D, dtype, list(lens)
        H = len(windows)
        self.pool = hw.Pool(1, H, D, bs, [windows], seqs, dtype, q_heads=q_heads)
        self.pool.set_block_table(np.random.default_rng(seed).permutation(self.pool.geometry()[1]).astype(np.int32))
        n = max(1, max(lens)) + spare
        self.k, self.v = ((torch.randn((seqs, H, n, D), generator=gen, device="cuda") * s).to(self.pool.io_dtype) for s in (kscale, 1.0))
        raw = torch.randn(self.pool.blocks().shape, generator=gen, device="cuda")  # slots that hold another sequence's rows
        self.pool.blocks().copy_(raw.to(dtype))
        if dtype == E4M3:
            self.pool.scales().fill_(0.25)
        self.pool.materialize(0, self.k, self.v, i32(lens))
        self.kk, self.vv = np64(self.k), np64(self.v)
        self.rings = None
        if dtype == E4M3:
            self.rings = [[Ring8(w, bs, D) for w in windows] for _ in range(seqs)]
            for s in range(seqs):
                for h in range(H):
                    self.rings[s][h].materialize(self.kk[s, h], self.vv[s, h], lens[s])

    def append(self, k, v):
        """Reference of appending k, v [B, H, D] at the present lengths."""
        kk, vv = np64(k), np64(v)
        for s, p in enumerate(self.lens):
            self.kk[s, :, p], self.vv[s, :, p] = kk[s], vv[s]
            if self.rings:
                for h in range(len(self.windows)):
                    self.rings[s][h].append(kk[s, h], vv[s, h], p)
            self.lens[s] = p + 1

    def newest(self, s, h, since):
        """(positions, K, V, sum of |codes| scaled as the floor has it) from `since` on, within the window."""
        n, w = self.lens[s], self.windows[h]
        p = np.arange(max(0, n - w, since), n)
        if self.rings is None:
            return p, self.kk[s, h, p], self.vv[s, h, p], 0.0
        r = self.rings[s][h]
        k, v = r.values(0)[p % r.C], r.values(1)[p % r.C]
        floor = 2.0 ** -36 * np.abs(r.codes[1][p % r.C]).sum(0) * np.repeat(r.scales[1], 16)[p % r.C].max(initial=0.0)
        return p, k, v, floor


class Case:
    def __init__(self, own, pre, lens, pre_lens, of, G=4, D=128, bs=16, types=(BF16, BF16), pre_bs=None, cap=0.0, bias=False,
                 seed=0, kscale=1.0):
        gen = self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.H, self.G, self.D, self.cap, self.of = len(lens), len(own), G, D, cap, list(of)
        self.own = Side(gen, own, self.B, D, bs, types[0], lens, G * self.H, seed, kscale=kscale)
        self.pre = Side(gen, pre, len(pre_lens), D, pre_bs or bs, types[1], pre_lens, G * self.H, seed + 1, kscale=kscale)
        self.io = self.own.pool.io_dtype
        self.scale = D ** -0.5
        self.slopes = torch.tensor([2.0 ** (-8.0 * (i + 1) / (G * self.H)) for i in range(G * self.H)], device="cuda") if bias else None
        self.q = (torch.randn((self.B, G * self.H, D), generator=gen, device="cuda") * 2).to(self.io)

    def new_rows(self):
        return ((torch.randn((self.B, self.H, self.D), generator=self.gen, device="cuda")).to(self.io) for _ in range(2))

    def call(self, **kw):
        lens = kw.pop("lens", None)
        return self.own.pool.shared_decode(0, self.pre.pool, self.q, self.scale, i32(self.own.lens) if lens is None else lens,
                                           i32(self.of), i32(self.pre.lens), softcap=self.cap, slopes=self.slopes, **kw)

    def step(self, append=True, **kw):
        if append:
            k, v = self.new_rows()
            out = self.call(k_new=k, v_new=v, **kw)
            self.own.append(k, v)
        else:
            out = self.call(**kw)
        self.check(out)
        return out

    def check(self, out, seqs=None, what=""):
        got, q = np64(out), np64(self.q)
        half = self.io == BF16
        for s in range(self.B) if seqs is None else seqs:
            for h in range(self.H):
                n = self.own.lens[s]
                p, k, v, floor = self.own.newest(s, h, 0)
                d = n - 1 - p
                f = self.of[s]
                if f >= 0:
                    N = self.pre.lens[f]
                    pp, pk, pv, _ = self.pre.newest(f, h, N + n - self.pre.windows[h])
                    k, v, d = np.concatenate((pk, k)), np.concatenate((pv, v)), np.concatenate((N + n - 1 - pp, d))
                rows = slice(h * self.G, (h + 1) * self.G)
                if len(k) == 0:
                    assert (got[s, rows] == 0).all(), (what, s, h)
                    continue
                x = q[s, rows] @ k.T * self.scale
                delta = np.abs(q[s, rows]) @ np.abs(k).T * self.scale * (self.D + 4) * 2.0 ** -23 + 2.0 ** -21
                if self.cap > 0:
                    x = self.cap * np.tanh(x / self.cap)
                    delta += self.cap * 2.0 ** -20
                if self.slopes is not None:
                    slope = np64(self.slopes)[rows, None] * d
                    delta += 4 * 2.0 ** -24 * (np.abs(x) + slope)
                    x = x - slope
                w = np.exp(x - x.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                ref, A = w @ v, w @ np.abs(v)
                tol = (w * (delta + (w * delta).sum(1, keepdims=True))) @ np.abs(v) + 2.0 ** -20 * A + floor
                tol += 2.0 ** -8 * (A + np.abs(ref)) if half else 2.0 ** -24 * np.abs(ref)
                err = np.abs(got[s, rows] - ref)
                assert (err <= tol).all(), f"{what} seq {s} head {h}: {err.max():.3e}, {(err / tol).max():.2f} of what is allowed"


PAIRS = [(BF16, BF16), (E4M3, E4M3), (BF16, E4M3), (E4M3, BF16), (F32, F32)]
PAIR_IDS = ["bf16", "e4m3", "bf16-e4m3", "e4m3-bf16", "f32"]


@pytest.mark.parametrize("types", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("own,pre,lens,pre_lens,of,G,D,bs", [
    # the first token behind a prefix of one token
    ([16], [16], [0], [1], [0], 1, 64, 16),
    # one prefix, windows beyond it, ragged own parts
    ([64, 33], [1024, 500], [0, 1, 40, 15], [333], [0, 0, 0, 0], 4, 128, 16),
    # two prefixes (one empty), sequences without one, in no order; windows that leave nothing of the prefix to some rows
    ([100, 256], [100, 300], [0, 99, 150, 200, 7, 0], [0, 400], [1, -1, 1, 0, -5, 1], 2, 64, 32),
    # prefixes longer than their rings, windows that no block divides, a group of 16
    ([17, 40, 128], [77, 1000, 130], [3, 16, 30, 90, 120], [1203, 64, 129], [2, 0, 1, 0, 2], 16, 64, 16),
    # a window of one token: own alone, and the prefix's last where there is none
    ([1, 16], [1, 2], [0, 3], [50], [0, 0], 3, 128, 16),
    # long prefixes, few rows
    ([300], [5000], [10, 299], [7001, 4990], [1, 0], 8, 128, 64),
    # more rows than one tile, more than two (40 x 8 = 320)
    ([48, 64], [300, 1100], [(7 * i) % 60 for i in range(40)], [900], [0] * 40, 8, 64, 16),
    # groups that divide no tile
    ([48], [400], [(5 * i) % 45 for i in range(50)], [350, 20], [i % 3 - 1 for i in range(50)], 7, 128, 16),
])
def test_against_the_definition(own, pre, lens, pre_lens, of, G, D, bs, types):
    c = Case(own, pre, lens, pre_lens, of, G, D, bs, types, seed=len(lens) + D)
    c.step(append=False)
    c.step()
    c.step()
    assert c.own.pool.check_device_errors() == 0 and c.pre.pool.check_device_errors() == 0


@pytest.mark.parametrize("types", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("cap,bias", [(20.0, False), (0.0, True), (30.0, True)])
def test_scores(types, cap, bias):
    c = Case([64, 40], [700, 90], [0, 5, 30, 63], [500, 100], [0, 1, 0, 0], 4, 64, 16, types, cap=cap, bias=bias, seed=7, kscale=3.0)
    c.step(append=False)
    c.step()


@pytest.mark.parametrize("types,bs,pre_bs", [((F32, F32), 5, 24), ((F32, F32), 24, 16), ((BF16, BF16), 5, 7), ((BF16, BF16), 16, 64), ((BF16, BF16), 24, 16),
                                             ((BF16, BF16), 64, 48), ((E4M3, E4M3), 32, 128), ((BF16, E4M3), 5, 16), ((E4M3, BF16), 16, 5)])
def test_blocks_of_other_sizes(types, bs, pre_bs):
    c = Case([50, 300], [60, 777], [0, 20, 51], [70, 1000], [1, 1, 0], 6, 64, bs, types, pre_bs=pre_bs, seed=bs)
    c.step()
    c.step(append=False)


def test_equals_decode_of_whole_contexts():
    """Behind a prefix or with the whole context in its own pool, a sequence attends to the same tokens."""
    c = Case([1024, 256], [1024, 256], [5, 60, 200], [900], [0, 0, 0], 4, 128, seed=3)
    whole = hw.Pool(1, 2, 128, 16, [[1024, 256]], 3, BF16, q_heads=8)
    k = torch.cat((c.pre.k[:1, :, :900].expand(3, -1, -1, -1), c.own.k), 2)
    v = torch.cat((c.pre.v[:1, :, :900].expand(3, -1, -1, -1), c.own.v), 2)
    lens = i32([905, 960, 1100])
    whole.materialize(0, k, v, lens)
    a, b = np64(c.step(append=False)), np64(whole.decode(0, c.q, c.scale, lens))
    assert np.abs(a - b).max() <= 2.0 ** -6 * np.abs(b).max()  # each within 2^-7 of the definition's largest


@pytest.mark.parametrize("types", PAIRS[:2], ids=PAIR_IDS[:2])
def test_many_prefixes(types):
    """As many as there may be, most without a sequence."""
    rng = np.random.default_rng(0)
    of = [767, 0, 500, 499, 500, 767, 767, -1, 31]
    c = Case([20], [40], rng.integers(0, 30, 9).tolist(), rng.integers(0, 90, 768).tolist(), of, 2, 128, 16, types, seed=1)
    c.step()


def test_nothing_to_attend_to():
    c = Case([16, 32], [16, 8], [0, 0, 20, 40], [0, 30], [0, -1, 1, 1], 4, 64, seed=2)
    out = c.step(append=False)
    assert (out[0] == 0).all() and (out[1] == 0).all() and (out[2] != 0).any()


def test_bad_prefixes_and_lengths_are_flagged():
    B = hw.binding
    c = Case([32], [64], [4, 5, 6], [20, 30], [0, 1, 0], 4, 64, seed=2)
    want = c.step(append=False).clone()
    of, pre_lens = c.of, c.pre.lens
    c.of = [0, 2, 0]  # one the pool does not hold: as none
    out = c.call()
    assert c.own.pool.check_device_errors() == B.HWKV_DEVERR_BAD_PREFIX
    c.of = [0, -1, 0]
    c.check(out)
    c.of, c.pre.lens = of, [20, -7]
    out = c.call()
    assert c.own.pool.check_device_errors() == B.HWKV_DEVERR_NEG_LENGTH
    c.pre.lens = [20, 0]
    c.check(out)
    c.pre.lens = pre_lens
    out = c.call(lens=i32([4, -1, 6]))
    assert c.own.pool.check_device_errors() == B.HWKV_DEVERR_NEG_LENGTH
    assert torch.equal(out[[0, 2]], want[[0, 2]])


@pytest.mark.parametrize("types", [(BF16, BF16), (E4M3, E4M3), (F32, F32)], ids=["bf16", "e4m3", "f32"])
def test_captured_steps_move_on(types):
    """A captured step (turn and store at positions of both pools, attend) replays at the lengths of the moment, and so do
    eager calls on another stream."""
    lens, pre_lens, of = [0, 3, 20, 9], [300, 45], [0, 1, 0, -1]
    c, d = (Case([64, 40], [400, 100], lens, pre_lens, of, 4, 64, 16, types, seed=9) for _ in range(2))
    table = hw.rope_table(64)
    q0 = c.q.clone()
    k, v = c.new_rows()
    pos, t_of, t_pre = i32(lens), i32(of), i32(pre_lens)
    turn = i32([pre_lens[f] + n if f >= 0 else n for f, n in zip(of, lens)])
    q_out, out = torch.zeros_like(q0), torch.zeros_like(q0)

    def step(case, pos, turn, q_out, out, stream=None):
        p = case.own.pool
        p.rope_append(0, table, q0, k, v, pos, q_out=q_out, turn_pos=turn, stream=stream)
        p.advance_positions(pos, stream=stream)
        p.advance_positions(turn, stream=stream)
        p.shared_decode(0, case.pre.pool, q_out, case.scale, pos, t_of, t_pre, out=out, stream=stream)

    warm = torch.zeros_like(out)
    c.own.pool.shared_decode(0, c.pre.pool, q0, c.scale, pos, t_of, t_pre, out=warm)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(c, pos, turn, q_out, out)
    pos2, turn2 = pos.clone(), turn.clone()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    out2, q2 = torch.zeros_like(q0), torch.zeros_like(q0)
    for _ in range(70):  # past the own windows
        graph.replay()
        step(d, pos2, turn2, q2, out2, other)
        torch.cuda.synchronize()
        assert torch.equal(out, out2) and torch.equal(q_out, q2)
    assert torch.equal(c.own.pool.blocks().view(torch.uint8), d.own.pool.blocks().view(torch.uint8))
    assert c.own.pool.check_device_errors() == 0 and d.own.pool.check_device_errors() == 0


@pytest.mark.parametrize("rope", [False, True], ids=["plain", "rope"])
@pytest.mark.parametrize("types", [(BF16, BF16), (E4M3, E4M3), (F32, F32)], ids=["bf16", "e4m3", "f32"])
def test_step_graph_behind_prefixes(types, rope):
    """DecodeStepGraph over two layers equals the calls one by one, token after token, past the own windows."""
    from head_budgeted_kv_gb300.graph import DecodeStepGraph
    own, pre, lens, pre_lens, of = [[24, 40], [16, 8]], [[200, 90], [64, 300]], [0, 5, 30], [150, 33], [1, -1, 0]
    gen = torch.Generator(device="cuda").manual_seed(1)

    def pools():
        a, b = hw.Pool(2, 2, 64, 16, own, 3, types[0], q_heads=8), hw.Pool(2, 2, 64, 16, pre, 2, types[1], q_heads=8)
        g = torch.Generator(device="cuda").manual_seed(2)
        for p, n, ls in ((a, 40, lens), (b, 160, pre_lens)):
            for layer in range(2):
                k, v = (torch.randn((p.num_seqs, 2, n, 64), generator=g, device="cuda").to(p.io_dtype) for _ in range(2))
                p.materialize(layer, k, v, i32(ls))
        return a, b

    (a, pa), (b, pb) = pools(), pools()
    table = hw.rope_table(64) if rope else None
    step = DecodeStepGraph(a, 0.125, 8, lens, rope=table, prefix=pa, prefix_of=of, prefix_lens=pre_lens)
    assert step.turn_pos.tolist() == [33, 5, 180]
    for i in range(50):
        q, k, v = (torch.randn(t.shape, generator=gen, device="cuda").to(a.io_dtype) for t in (step.q, step.k_new, step.v_new))
        step.q.copy_(q), step.k_new.copy_(k), step.v_new.copy_(v)
        step.replay()
        pos, turn = i32([n + i for n in lens]), i32([n + i for n in (33, 5, 180)])
        for layer in range(2):
            if rope:
                qq, _ = b.rope_append(layer, table, q[layer], k[layer], v[layer], pos, turn_pos=turn)
                out = b.shared_decode(layer, pb, qq, 0.125, pos + 1, i32(of), i32(pre_lens))
            else:
                out = b.shared_decode(layer, pb, q[layer], 0.125, pos, i32(of), i32(pre_lens), k_new=k[layer].contiguous(),
                                      v_new=v[layer].contiguous())
            assert torch.equal(out, step.out[layer]), (i, layer)
    assert torch.equal(a.blocks().view(torch.uint8), b.blocks().view(torch.uint8))
    assert a.check_device_errors() == 0


def test_output_in_place_of_the_queries():
    for types in ((BF16, BF16), (F32, F32)):
        c = Case([64], [900], [3, 60, 17], [800], [0, 0, -1], 4, 128, types=types, seed=4)
        want = c.call().clone()
        q = c.q.clone()
        got = c.own.pool.shared_decode(0, c.pre.pool, q, c.scale, i32(c.own.lens), i32(c.of), i32(c.pre.lens), out=q)
        assert got is q and torch.equal(q, want)


def test_two_pools_share_a_prefix_on_two_streams():
    a = Case([64], [900], [3, 60, 17], [800], [0, 0, 0], 4, 128, seed=4)
    b = Case([64], [900], [3, 60, 17], [800], [0, 0, 0], 4, 128, seed=4)
    b.pre = a.pre
    want_a, want_b = a.call().clone(), b.call().clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(20):
        got.append((a.call(stream=streams[0]), b.call(stream=streams[1])))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, want_a) and torch.equal(y, want_b)


def test_what_a_call_allocates_belongs_to_its_stream():
    """Memory that the current stream freed and still reads is not the workspace or output of a call on another stream."""
    c = Case([64], [900], [3, 60, 17], [800], [0, 0, -1], 4, 128, seed=4)
    need = hw.binding.hwkv_decode_shared_workspace_bytes(c.own.pool.handle, c.pre.pool.handle, c.q.shape[1])
    lens, of, pre_lens = i32(c.own.lens), i32(c.of), i32(c.pre.lens)
    held = [torch.ones(need, dtype=torch.uint8, device="cuda"), torch.ones_like(c.q)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()  # no other free block fits as well
    torch.cuda._sleep(50_000_000)  # tens of milliseconds
    read = [t.clone() for t in held]
    t = held = None
    got = c.own.pool.shared_decode(0, c.pre.pool, c.q, c.scale, lens, of, pre_lens, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(bool((t == 1).all()) for t in read)
    assert torch.equal(got, c.call())


def test_the_workspace_grows_and_other_pools_take_turns():
    """One own pool behind small and large prefix pools, other groups of heads, other decode settings."""
    c = Case([64, 64], [300, 300], [3, 60, 17], [200], [0, 0, 0], 2, 64, seed=4)
    c.step(append=False)
    e = Case([64, 64], [9000, 300], [3, 60, 17], [8000, 100], [0, 1, 0], 8, 64, seed=6)
    e.own = c.own
    e.step(append=False)
    e.own.pool.set_decode_config(workers=7)
    e.step()
    c.q = c.q[:, : 2 * 2].contiguous()
    c.step(append=False)
    c.own.pool.set_decode_config(kernel=hw.HWKV_KERNEL_SIMT)
    c.step()


def test_results_do_not_change_from_call_to_call():
    c = Case([300, 64], [3000, 5000], [(13 * i) % 290 for i in range(24)], [4000, 2500], [i % 2 for i in range(24)], 4, 128, seed=8)
    first = c.call().clone()
    c.check(first, seqs=[0, 1, 23])
    for _ in range(10):
        assert torch.equal(c.call(), first)


@pytest.mark.parametrize("types,bs", [((F32, F32), 5), ((F32, F32), 16), ((BF16, BF16), 24)])
def test_cuda_core_results_do_not_change_and_see_the_row_just_appended(types, bs):
    """The own parts run beside the prefixes' kernel: their new rows are stored before either."""
    c = Case([300, 40], [3000, 300], [(7 * i) % 290 for i in range(24)], [2500, 100], [i % 2 for i in range(24)], 8, 128, bs, types, seed=9)
    k, v = c.new_rows()
    lens, of, pre_lens = i32(c.own.lens), i32(c.of), i32(c.pre.lens)
    outs = []
    for i in range(20):
        if i % 2:  # other rows in their place
            c.own.pool.append(0, torch.zeros_like(k), torch.zeros_like(v), lens)
        outs.append(c.own.pool.shared_decode(0, c.pre.pool, c.q, c.scale, lens, of, pre_lens, k_new=k, v_new=v))
    c.own.append(k, v)
    c.check(outs[0], seqs=[0, 1, 23])
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_refusals():
    B = hw.binding
    c = Case([32], [64], [4, 5], [20], [0, 0], 4, 64, seed=2)
    pool, pre, q = c.own.pool, c.pre.pool, c.q
    lens, of, pl = i32([4, 5]), i32([0, 0]), i32([20])
    k, v = c.new_rows()

    def refused(error, status=None, prefix=pre, q=q, lens=lens, of=of, pl=pl, **kw):
        with pytest.raises(error) as e:
            pool.shared_decode(kw.pop("layer", 0), prefix, q, 0.125, lens, of, pl, **kw)
        if status is not None:
            assert e.value.status == status

    refused(B.HwkvError, B.HWKV_ERR_INVALID_ARG, layer=1)
    refused(B.HwkvError, B.HWKV_ERR_INVALID_ARG, prefix=pool, pl=i32([20, 20]))
    for other in (hw.Pool(1, 2, 64, 16, [[64, 64]], 1, BF16), hw.Pool(1, 1, 128, 16, [[64]], 1, BF16), hw.Pool(1, 1, 64, 16, [[64]], 1, F32),
                  hw.Pool(2, 1, 64, 16, [[64], [64]], 1, BF16)):
        refused(B.HwkvError, B.HWKV_ERR_INVALID_ARG, prefix=other)
    many = hw.Pool(1, 1, 64, 16, [[16]], 769, BF16)
    refused(B.HwkvError, B.HWKV_ERR_UNSUPPORTED, prefix=many, pl=i32([1] * 769))
    refused(B.HwkvError, B.HWKV_ERR_UNSUPPORTED, q=torch.zeros(2, 17, 64, dtype=BF16, device="cuda"))
    refused(B.HwkvError, B.HWKV_ERR_INVALID_ARG, softcap=-1.0)
    refused(ValueError, lens=lens.long())
    refused(ValueError, of=of[:1])
    refused(ValueError, pl=pl.cpu())
    refused(ValueError, k_new=k)
    refused(ValueError, k_new=k, v_new=v.float())
    refused(ValueError, q=q.float())
    refused(ValueError, q=q.transpose(1, 2).contiguous().transpose(1, 2))
    refused(ValueError, out=torch.zeros(2, 4, 64, dtype=F32, device="cuda"))
    refused(ValueError, slopes=torch.ones(3, device="cuda"))
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(B.HwkvError) as e:
        B.hwkv_decode_attn_shared(pool.handle, pre.handle, 0, q, B.score(0.125), lens, of, pl, torch.empty_like(q), small)
    assert e.value.status == B.HWKV_ERR_WORKSPACE_TOO_SMALL
    need = B.hwkv_decode_shared_workspace_bytes(pool.handle, pre.handle, 4)
    odd = torch.empty(need + 8, dtype=torch.uint8, device="cuda")[8:]
    with pytest.raises(B.HwkvError) as e:
        B.hwkv_decode_attn_shared(pool.handle, pre.handle, 0, q, B.score(0.125), lens, of, pl, torch.empty_like(q), odd)
    assert e.value.status == B.HWKV_ERR_ALIGNMENT
    assert pool.check_device_errors() == 0
