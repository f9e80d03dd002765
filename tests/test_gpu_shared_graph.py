"""DecodeStepGraph behind shared prefixes: what it takes, and how it counts."""
import pytest
import torch

import head_budgeted_kv_gb300 as hw
from head_budgeted_kv_gb300.graph import DecodeStepGraph
from test_gpu_shared import i32

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    hw.binding.load()
    yield
    torch.cuda.synchronize()


def pools(dtype=BF16):
    """Two layers of two heads: 3 sequences of 0, 5 and 30 tokens, 2 prefixes of 150 and 33."""
    a, b = hw.Pool(2, 2, 64, 16, [[24, 40], [16, 8]], 3, dtype, q_heads=8), hw.Pool(2, 2, 64, 16, [[200, 90], [64, 300]], 2, dtype, q_heads=8)
    g = torch.Generator(device="cuda").manual_seed(2)
    for p, n, lens in ((a, 40, [0, 5, 30]), (b, 160, [150, 33])):
        for layer in range(2):
            k, v = (torch.randn((p.num_seqs, 2, n, 64), generator=g, device="cuda").to(p.io_dtype) for _ in range(2))
            p.materialize(layer, k, v, i32(lens))
    return a, b


def inputs(step, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    for t in (step.q, step.k_new, step.v_new):
        t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))


def test_a_negative_prefix_length_is_none():
    """For the positions that queries and keys turn by as for the attention."""
    table = hw.rope_table(64)
    results = []
    for lens in ([150, -7], [150, 0]):
        own, pre = pools()
        step = DecodeStepGraph(own, 0.125, 8, [0, 5, 30], rope=table, prefix=pre, prefix_of=[1, -1, 0], prefix_lens=lens)
        assert step.turn_pos.tolist() == [0, 5, 180]
        for i in range(3):
            inputs(step, i)
            step.replay()
        torch.cuda.synchronize()
        results.append((step.out.clone(), own.blocks().clone()))
        assert own.check_device_errors() == (hw.binding.HWKV_DEVERR_NEG_LENGTH if lens[1] < 0 else 0)
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])


@pytest.mark.parametrize("rope", [False, True], ids=["plain", "rope"])
@pytest.mark.parametrize("dtype", [BF16, torch.float8_e4m3fn, torch.float32], ids=["bf16", "e4m3", "f32"])
def test_an_append_apart_gives_the_same(dtype, rope):
    """fused=False appends in a launch of its own (with a rope the two are the same step), bit for bit as the fused step."""
    results, launches = [], []
    for fused in (True, False):
        own, pre = pools(dtype)
        before = hw.hwkv_kernel_launches()
        step = DecodeStepGraph(own, 0.125, 8, [0, 5, 30], fused=fused, rope=hw.rope_table(64) if rope else None, prefix=pre,
                               prefix_of=[1, -1, 0], prefix_lens=[150, 33])
        launches.append(hw.hwkv_kernel_launches() - before)
        outs = []
        for i in range(20):  # past the own windows
            inputs(step, i)
            step.replay()
            outs.append(step.out.clone())
        assert step.pos.tolist() == [20, 25, 50] and own.check_device_errors() == 0
        results.append((torch.stack(outs), own.buffer.clone()))
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])
    # an append for each layer and the lengths once
    assert launches[1] - launches[0] == (0 if rope else 3)
