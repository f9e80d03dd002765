"""Rotary positions on the GPU against the 64-bit formula, at near and far positions.

Tolerance, per element of a pair (a, b) with r = magnitude * sqrt(a^2 + b^2): the angle is within
2^-23 rad (header), sincospif within 2 units of fp32 (2^-22 of at most 1), cos * magnitude, the two
products and the sum each round once in fp32 (4 * 2^-24): 2^-23 + 2^-22 + 2^-22 < 2^-20 of r in all;
then bf16 outputs round by 2^-8 of the value, fp32 outputs by 2^-24 (inside the 2^-20)."""
import numpy as np
import pytest
import torch

import head_budgeted_kv_gb300 as hw
from reference_ops import rope, rope_frequencies

pytestmark = pytest.mark.gpu
PI = np.longdouble("3.14159265358979323846264338327950288")


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hw.binding.load()
    yield
    torch.cuda.synchronize()


def make_pool(B, H, D, dtype):
    return hw.Pool(1, H, D, 16, [[16] * H], B, dtype, q_heads=H)


def check(x, got, pos, n, freqs, layout, magnitude, old, what):
    """Rows below n turned, the others as they were."""
    x, got, old = (t.float().cpu().double().numpy() for t in (x, got, old))
    bf16 = what.startswith("bf16")
    rot = 2 * len(freqs)
    first = (np.arange(rot) % len(freqs)) if layout == "half" else np.arange(rot) // 2
    for s in range(x.shape[0]):
        np.testing.assert_array_equal(got[s, n[s]:], old[s, n[s]:])
        for i in range(n[s]):
            ref = rope(x[s, i], pos[s] + i, freqs, layout, magnitude)
            a, b = (np.arange(len(freqs)), np.arange(len(freqs)) + len(freqs)) if layout == "half" else \
                (2 * np.arange(len(freqs)), 2 * np.arange(len(freqs)) + 1)
            r = magnitude * np.hypot(x[s, i][..., a], x[s, i][..., b])[..., first]
            tol = 2.0 ** -20 * r + (2.0 ** -8 * np.abs(ref[..., :rot]) if bf16 else 0.0)
            assert (np.abs(got[s, i][..., :rot] - ref[..., :rot]) <= tol).all(), (what, s, i)
            np.testing.assert_array_equal(got[s, i][..., rot:], x[s, i][..., rot:])


@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in_place"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.float8_e4m3fn], ids=["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("B,n,H,G,D,rot", [
    (1, 1, 8, 4, 128, 128),    # one token
    (3, 5, 2, 3, 64, 64),      # ragged rows
    (2, 7, 1, 1, 128, 64),     # half of the head
    (2, 3, 3, 2, 64, 20),      # pairs that no vector holds whole
    (1, 4, 2, 1, 128, 2),      # one pair
    (2, 2, 2, 2, 64, 62),
    (4, 300, 1, 2, 64, 32),    # several rows of a CTA
])
def test_against_the_formula(B, n, H, G, D, rot, dtype, layout, in_place):
    gen = torch.Generator(device="cuda").manual_seed(B * n + rot)
    pool = make_pool(B, H, D, dtype)
    io = pool.io_dtype
    rng = np.random.default_rng(rot)
    pos = rng.integers(0, 200000, B)
    rows = rng.integers(0, n, B, endpoint=True)
    rows[0] = n
    scaling = ("none", "linear", "ntk", "by_parts")[(n + rot // 2) % 4]
    table = hw.rope_table(D, rot, 10000.0, layout, scaling, 4.0, 4096)
    freqs, magnitude = rope_frequencies(rot, 10000.0, scaling, 4.0, 4096)
    q = torch.randn((B, n, G * H, D), generator=gen, device="cuda").to(io)
    k = torch.randn((B, n, H, D), generator=gen, device="cuda").to(io)
    tpos = torch.tensor(pos, dtype=torch.int32, device="cuda")
    tn = torch.tensor(rows, dtype=torch.int32, device="cuda")
    qi, ki = q.clone(), k.clone()
    if in_place:
        qo, ko, old_q, old_k = qi, ki, q, k
    else:
        qo, ko = torch.full_like(q, 3.0), torch.full_like(k, -5.0)
        old_q, old_k = qo.clone(), ko.clone()
    pool.rope(table, qi, ki, tpos, tn, qo, ko)
    kind = "f32" if io == torch.float32 else "bf16"
    check(q, qo, pos, rows, freqs, layout, magnitude, old_q, f"{kind} q")
    check(k, ko, pos, rows, freqs, layout, magnitude, old_k, f"{kind} k")
    assert pool.check_device_errors() == 0


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,n,H,G,D,rot", [(2, 4200, 2, 4, 64, 64), (1, 700, 3, 1, 128, 20), (3, 171, 8, 4, 128, 128),
                                           (1, 9001, 1, 1, 64, 34), (2, 1111, 5, 3, 64, 32)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_long_chunks_are_their_rows(B, n, H, G, D, rot, dtype, layout):
    """However a call shares its rows out, a row's bits are those of a short call."""
    pool = make_pool(B, H, D, dtype)
    table = hw.rope_table(D, rot, 10000.0, layout)
    gen = torch.Generator(device="cuda").manual_seed(n)
    q = torch.randn((B, n, G * H, D), generator=gen, device="cuda").to(dtype)
    k = torch.randn((B, n, H, D), generator=gen, device="cuda").to(dtype)
    pos = torch.arange(B, dtype=torch.int32, device="cuda") * 1000 + 7
    whole = pool.rope(table, q, k, pos)
    part = [(pool.rope(table, q[:, i:i + 160], k[:, i:i + 160], pos + i)) for i in range(0, n, 160)]
    assert torch.equal(whole[0], torch.cat([p[0] for p in part], 1))
    assert torch.equal(whole[1], torch.cat([p[1] for p in part], 1))
    qi, ki = q.clone(), k.clone()
    pool.rope(table, qi, ki, pos, q_out=qi, k_out=ki)
    assert torch.equal(qi, whole[0]) and torch.equal(ki, whole[1])
    assert pool.check_device_errors() == 0


@pytest.mark.parametrize("pos", [0, 1, 65535, 164864, 2 ** 24 - 2, 2 ** 31 - 9])
def test_far_positions(pos):
    """The angle keeps its accuracy; beyond 2^24 the frequency's own 64-bit rounding shows (2^-52 of
    the angle's whole size, at most 2^-21 rad)."""
    pool = make_pool(1, 1, 64, torch.float32)
    table = hw.rope_table(64)
    freqs, _ = rope_frequencies(64)
    x = torch.zeros((1, 8, 1, 64), device="cuda")
    x[..., :32] = 1.0  # the output is (cos, sin)
    got = pool.rope(table, None, x, torch.tensor([pos], dtype=torch.int32, device="cuda"))[1].cpu().double().numpy()
    for i in range(8):
        # the product of a 31-bit position and a 53-bit frequency in extended precision
        t = np.array([float(np.mod(np.longdouble(pos + i) * np.longdouble(f), 2 * PI)) for f in freqs])
        tol = 2.0 ** -20 + (2.0 ** -20 if pos >= 2 ** 24 - 2 else 0.0)
        assert np.abs(got[0, i, 0, :32] - np.cos(t)).max() <= tol
        assert np.abs(got[0, i, 0, 32:] - np.sin(t)).max() <= tol


@pytest.mark.parametrize("in_place", [False, True])
def test_slices_of_a_fused_projection(in_place):
    B, n, H, G, D = 2, 9, 2, 3, 128
    pool = make_pool(B, H, D, torch.bfloat16)
    table = hw.rope_table(D)
    qkv = torch.randn((B, n, (G + 2) * H, D), device="cuda").bfloat16()
    was = qkv.clone()
    pos = torch.tensor([5, 1000], dtype=torch.int32, device="cuda")
    q, k = qkv[:, :, :G * H], qkv[:, :, G * H:(G + 1) * H]
    want = pool.rope(table, q.contiguous(), k.contiguous(), pos)
    got = pool.rope(table, q, k, pos, q_out=q if in_place else None, k_out=k if in_place else None)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(qkv[:, :, (G + 1) * H:], was[:, :, (G + 1) * H:])
    if not in_place:
        assert torch.equal(qkv, was)
    # rows before sequences, as a time-major program keeps them
    tm = was.transpose(0, 1).contiguous().transpose(0, 1)
    got = pool.rope(table, tm[:, :, :G * H], None, pos, q_out=torch.empty_like(tm)[:, :, :G * H])
    assert torch.equal(got[0], want[0]) and got[1] is None


def test_single_rows_and_scores_depend_on_distance_alone():
    """[B][heads][D] rows; q . k after turning depends on the distance of their positions."""
    pool = make_pool(1, 1, 64, torch.float32)
    table = hw.rope_table(64, layout="interleaved")
    q, k = torch.randn((2, 1, 1, 64), device="cuda").unbind(0)

    def turned(x, p, query):
        pos = torch.tensor([p], dtype=torch.int32, device="cuda")
        got = pool.rope(table, x if query else None, None if query else x, pos)
        return got[0 if query else 1].double()

    near = (turned(q, 100, True) * turned(k, 93, False)).sum().item()
    far = (turned(q, 160100, True) * turned(k, 160093, False)).sum().item()
    # each of 128 turned elements is off by 2^-20 of its pair's size
    assert abs(near - far) <= 2 * 2.0 ** -20 * 2 * float(q.norm() * k.norm())


def test_refusals_and_flags():
    B, H, D = 2, 2, 64
    pool = make_pool(B, H, D, torch.bfloat16)
    table = hw.rope_table(D)
    q = torch.randn((B, 3, 4, D), device="cuda").bfloat16()
    k = torch.randn((B, 3, H, D), device="cuda").bfloat16()
    pos = torch.tensor([0, 7], dtype=torch.int32, device="cuda")
    for bad in (lambda: pool.rope(table, q.float(), k, pos), lambda: pool.rope(table, q, k[:, :, :1], pos),
                lambda: pool.rope(table, q, k[:, :2], pos), lambda: pool.rope(table, q, k, pos.long()),
                lambda: pool.rope(table, q.transpose(1, 2), None, pos), lambda: pool.rope(table, q[:1], None, pos),
                lambda: pool.rope(table, q, k, pos, q_out=k), lambda: pool.rope(table, q, k, pos.cpu()),
                lambda: pool.rope(table, q, k, pos[:1]), lambda: pool.rope(table, q, k, pos, pos[:1]),
                lambda: pool.rope(table, q, k, torch.arange(4, dtype=torch.int32, device="cuda")[::2]),
                lambda: pool.rope(table, q, None, pos, q_out=torch.empty(q.shape, dtype=q.dtype))):
        with pytest.raises(ValueError):
            bad()

    def status(call):
        with pytest.raises(hw.HwkvError) as e:
            call()
        return e.value.status

    wide = hw.rope_table(128)
    assert status(lambda: pool.rope(wide, q, k, pos)) == hw.binding.HWKV_ERR_INVALID_ARG
    assert status(lambda: pool.rope(table, None, None, pos)) == hw.binding.HWKV_ERR_INVALID_ARG
    one = torch.zeros((1, 1, 4, D), device="cuda").bfloat16().expand(B, 3, 4, D)
    assert status(lambda: pool.rope(table, q, None, pos, q_out=one)) == hw.binding.HWKV_ERR_INVALID_ARG
    assert status(lambda: pool.rope(table, q, q[:, :, :H], pos, q_out=q, k_out=q[:, :, :H])) == hw.binding.HWKV_ERR_INVALID_ARG
    kk = torch.zeros((B, 3, H, D), device="cuda").bfloat16()
    assert status(lambda: pool.rope(table, kk, k, pos, q_out=k, k_out=kk)) == hw.binding.HWKV_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        pool.rope(table, q.cpu(), None, pos)
    odd = torch.empty(B * 3 * 4 * D + 1, device="cuda").bfloat16()[1:].view(B, 3, 4, D)
    assert status(lambda: pool.rope(table, odd, None, pos)) == hw.binding.HWKV_ERR_ALIGNMENT
    broken = hw.rope_table(D)
    broken.freq[3] = float("nan")
    assert status(lambda: pool.rope(broken, q, k, pos)) == hw.binding.HWKV_ERR_INVALID_ARG
    # an expanded input is read as it is
    got, _ = pool.rope(table, one, None, pos)
    assert torch.equal(got, torch.zeros_like(got))
    assert pool.check_device_errors() == 0
    out = torch.full_like(q, 2.0)
    pool.rope(table, q, None, torch.tensor([-1, 7], dtype=torch.int32, device="cuda"),
              torch.tensor([1, 4], dtype=torch.int32, device="cuda"), q_out=out)
    assert pool.check_device_errors() == hw.binding.HWKV_DEVERR_NEG_LENGTH
    assert (out == 2.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("fused", [True, False])
def test_captured_step_turns_appends_and_attends(dtype, fused):
    """A captured step with rotary positions gives the bits of the separate calls."""
    from head_budgeted_kv_gb300.graph import DecodeStepGraph
    table = hw.rope_table(64, base=500000.0, scaling="by_parts", factor=4.0, original_len=64)
    results = []
    for graph in (False, True):
        gen = torch.Generator(device="cuda").manual_seed(3)

        def randn(*shape):
            return torch.randn(shape, generator=gen, device="cuda").bfloat16()

        pool = hw.Pool(2, 2, 64, 16, [[64, 30], [200, 16]], 2, dtype, q_heads=8)
        pos = torch.tensor([70, 0], dtype=torch.int32, device="cuda")
        for l in range(2):
            pool.materialize(l, randn(2, 2, 70, 64), randn(2, 2, 70, 64), pos)
        step = DecodeStepGraph(pool, 0.125, 8, pos, fused=fused, rope=table) if graph else None
        outs = []
        for _ in range(5):
            q, k, v = randn(2, 2, 8, 64), randn(2, 2, 2, 64), randn(2, 2, 2, 64)
            if graph:
                step.q.copy_(q), step.k_new.copy_(k), step.v_new.copy_(v)
                step.replay()
                outs.append(step.out.clone())
            else:
                one = []
                for l in range(2):
                    qr, kr = pool.rope(table, q[l], k[l], pos)
                    one.append(pool.append_decode(l, qr, 0.125, kr, v[l], pos))
                outs.append(torch.stack(one))
                pos = pos + 1
        assert pool.check_device_errors() == 0
        results.append((torch.stack(outs), pool.buffer.clone()))
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
