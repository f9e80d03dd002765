"""Host side of the operators around the cache, without a GPU: footprints, refusals, and the
64-bit reference the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

from head_budgeted_kv_gb300 import _build, binding
from reference_ops import Ring8, encode_group, nearest_e4m3


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load()


def _pool_bytes(*args):
    return binding.hwkv_pool_bytes(*args)


@pytest.mark.parametrize("D,bs,B", [(64, 16, 1), (128, 16, 3), (128, 64, 2), (64, 48, 5)])
def test_8_bit_footprint(lib, D, bs, B):
    windows = [[33, 128, 1], [700, 16, 17]]
    blocks = B * sum(-(-w // bs) for row in windows for w in row)
    want = blocks * 2 * bs * D + (blocks * (bs // 16) * 8 + 15) // 16 * 16
    for dtype in (torch.float8_e4m3fn, "e4m3", binding.HWKV_E4M3):
        assert _pool_bytes(2, 3, D, bs, windows, B, dtype) == want


@pytest.mark.parametrize("bs", [1, 5, 8, 24])
def test_8_bit_pools_need_whole_groups(lib, bs):
    with pytest.raises(binding.HwkvError) as e:
        _pool_bytes(1, 1, 64, bs, [[64]], 1, torch.float8_e4m3fn)
    assert e.value.status == binding.HWKV_ERR_UNSUPPORTED


def test_seqcalib_budgets_8_bit_pools(lib):
    cand = np.array([[[64], [1024]]], dtype=np.int32)
    budget = _pool_bytes(1, 1, 128, 16, [[1024]], 1, "e4m3")
    w, choice, nbytes = binding.hwkv_seqcalib(cand, np.array([[2.0, 1.0]]), budget, 128, 16, 1, "e4m3")
    assert choice.tolist() == [1] and nbytes == budget
    w, choice, nbytes = binding.hwkv_seqcalib(cand, np.array([[2.0, 1.0]]), budget - 1, 128, 16, 1, "e4m3")
    assert choice.tolist() == [0]


def test_seqcalib_of_8_bit_layers_predicts_the_pool(lib):
    """Scales of odd block counts: layers chosen together cost what one pool of them takes."""
    windows = [[16], [33], [1], [80]]
    cand = np.array([[w] for w in windows], dtype=np.int32)
    want = _pool_bytes(4, 1, 64, 16, windows, 1, "e4m3")
    w, _, nbytes = binding.hwkv_seqcalib(cand, np.ones((4, 1)), want, 64, 16, 1, "e4m3")
    assert nbytes == want and w.tolist() == windows
    assert binding.hwkv_seqcalib(cand, np.ones((4, 1)), want + 15, 64, 16, 1, "e4m3")[2] == want
    with pytest.raises(binding.HwkvError) as e:
        binding.hwkv_seqcalib(cand, np.ones((4, 1)), want - 1, 64, 16, 1, "e4m3")
    assert e.value.status == binding.HWKV_ERR_BUDGET


def test_seqcalib_refuses_a_negative_count_of_layers(lib):
    """A status, as from every entry point: sizing its tables from the count would throw across the C boundary."""
    cand = np.ones((1, 1, 1), dtype=np.int32)
    out = np.zeros(1, dtype=np.int32)
    fn = binding.DISTORTION_FN(lambda *a: 0.0)
    p = cand.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    for layers in (-1, -(2 ** 31)):
        rc = lib.hwkv_seqcalib(layers, 1, 64, 16, 1, binding.HWKV_BF16, 1, p, fn, None, 1 << 20,
                               out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), None, None)
        assert rc == binding.HWKV_ERR_INVALID_ARG


def test_reference_codes_are_torchs_codes():
    """The reference's rounding to e4m3 is the nearest one with ties to even, as torch's cast has it."""
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(20000, generator=gen) * torch.exp2(torch.randint(-14, 9, (20000,), generator=gen))
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    every = every[torch.isfinite(every)].sort().values
    x = torch.cat((x.clamp(-448, 448), every, (every[1:] + every[:-1]) / 2))
    want = x.to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(nearest_e4m3(x.double().numpy()), want)


def test_reference_group_scale():
    for top, e in ((448.0, 0), (448.0001, 1), (449.0, 1), (896.0, 1), (224.0, -1), (224.5, 0), (1.0, -8), (0.0, -120),
                   (2.0 ** -133, -120), (3.3895e38, 120)):
        rows = np.zeros((16, 64))
        rows[3, 5] = -top
        assert encode_group(rows)[1] == 2.0 ** e, top


def test_reference_ring_keeps_the_window():
    """A ring filled by appends holds what a stored prompt holds, up to a second rounding of subnormal codes."""
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((2, 90, 64))
    a, b = Ring8(40, 16, 64), Ring8(40, 16, 64)
    a.materialize(k, v, 90)
    for p in range(90):
        b.append(k[p], v[p], p)
    for x, y, src in zip(a.resident(90)[1:], b.resident(90)[1:], (k, v)):
        assert np.abs(x - y).max() <= 2.0 ** -9 * a.scales.max()
        assert (np.abs(x - src[50:]) <= 2.0 ** -4 * np.abs(src[50:]) + 2.0 ** -10 * a.scales.max()).all()


# ---- rotary tables and refusals --------------------------------------------------------------------
from reference_ops import rope_frequencies  # noqa: E402

SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}


@pytest.mark.parametrize("scaling", sorted(SCALINGS))
@pytest.mark.parametrize("rot", [2, 24, 64, 128])
def test_rope_table_follows_its_formulas(lib, scaling, rot):
    import head_budgeted_kv_gb300 as hw
    t = hw.rope_table(128, rot_dim=rot, base=500000.0, scaling=scaling, factor=8.0, original_len=8192)
    f, m = rope_frequencies(rot, 500000.0, scaling, 8.0, 8192)
    assert t.rot_dim == rot and t.layout == 0
    np.testing.assert_allclose(list(t.freq)[:rot // 2], f, rtol=1e-13)
    assert abs(t.magnitude - m) < 1e-14


@pytest.mark.parametrize("args", [
    (0, 0, 1e4, 0, 1.0, 0.0, 32.0, 1.0), (3, 0, 1e4, 0, 1.0, 0.0, 32.0, 1.0), (130, 0, 1e4, 0, 1.0, 0.0, 32.0, 1.0),
    (64, 2, 1e4, 0, 1.0, 0.0, 32.0, 1.0), (64, 0, 0.0, 0, 1.0, 0.0, 32.0, 1.0), (64, 0, float("inf"), 0, 1.0, 0.0, 32.0, 1.0),
    (64, 0, 1e4, 4, 1.0, 0.0, 32.0, 1.0), (64, 0, 1e4, 1, 0.5, 0.0, 32.0, 1.0), (64, 0, 1e4, 2, float("nan"), 0.0, 32.0, 1.0),
    (64, 0, 1e4, 3, 8.0, 0.0, 32.0, 1.0), (64, 0, 1e4, 3, 8.0, 8192.0, 1.0, 1.0),
])
def test_bad_rope_tables_are_refused(lib, args):
    out = binding.RopeTable()
    assert lib.hwkv_rope_table(*args, ctypes.byref(out)) == binding.HWKV_ERR_INVALID_ARG
    assert lib.hwkv_rope_table(64, 0, 1e4, 0, 1.0, 0.0, 32.0, 1.0, None) == binding.HWKV_ERR_INVALID_ARG


def test_rope_needs_a_pool(lib):
    t = binding.hwkv_rope_table(64)
    assert lib.hwkv_rope(None, t, None, 4, None, 1, None, None, None, None, None) == binding.HWKV_ERR_INVALID_ARG


def test_scored_calls_check_their_arguments(lib):
    s = binding.Score(1.0, 0.0, None)
    assert lib.hwkv_decode_attn_score(None, 0, None, 4, s, None, None, None, None, None, 0, 0, None) == binding.HWKV_ERR_INVALID_ARG
    assert lib.hwkv_prefill_attn_score(None, 0, None, 4, s, None, None, 1, None, None, None, None, 0, None) == binding.HWKV_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        binding.score(1.0, 0.0, torch.zeros(4), torch.zeros(1, 5, 64))
    with pytest.raises(ValueError):
        binding.score(1.0, 0.0, torch.zeros(4).double())


def test_tanh_form():
    """The polynomial and the exponential form the kernels use for tanh, in fp32 steps: below 2^-20
    relative error over the range."""
    c = [np.float32(v) for v in (0.9999994039535522, -0.3332904279232025, 0.13281433284282684, -0.05160565674304962,
                                 0.016743095591664314, -0.0030670526903122663)]
    u = np.concatenate([np.linspace(-12, 12, 400001), np.geomspace(1e-20, 1.0, 20000)]).astype(np.float32)
    t = (u * u).astype(np.float32)
    p = np.full_like(t, c[5])
    for v in c[4::-1]:
        p = (p * t + v).astype(np.float32)
    p = (u * p).astype(np.float32)
    r = (np.float32(1) - np.float32(2) / (np.float32(1) + np.exp2(u * np.float32(2.8853900817779268)).astype(np.float32)))
    got = np.where(np.abs(u) <= 1, p, r).astype(np.float64)
    want = np.tanh(u.astype(np.float64))
    fine = want != 0
    assert (np.abs(got - want)[fine] <= 2.0 ** -20 * np.abs(want)[fine]).all()
    # the shorter polynomial below half of the cap
    c = [np.float32(v) for v in (0.999999463558197, -0.33326318860054016, 0.13190296292304993, -0.04440220072865486)]
    low = (np.abs(u) <= 0.5) & fine
    p = np.full_like(t, c[3])
    for v in c[2::-1]:
        p = (p * t + v).astype(np.float32)
    got = (u * p).astype(np.float32).astype(np.float64)
    assert (np.abs(got - want)[low] <= 2.0 ** -20 * np.abs(want)[low]).all()
