"""What DecodeStepGraph refuses behind shared prefixes, without a GPU."""
import types

import pytest
import torch

from head_budgeted_kv_gb300.graph import DecodeStepGraph


def pool(seqs):
    return types.SimpleNamespace(buffer=torch.empty(0), layers=1, num_seqs=seqs, kv_heads=1, head_dim=64, io_dtype=torch.bfloat16, q_heads=4)


@pytest.mark.parametrize("given", [dict(prefix=pool(1)), dict(prefix=pool(1), prefix_of=[0, 0]), dict(prefix=pool(1), prefix_lens=[3]),
                                   dict(prefix_of=[0, 0]), dict(prefix_lens=[3]), dict(prefix_of=[0, 0], prefix_lens=[3])])
def test_prefixes_and_what_lies_behind_them_go_together(given):
    with pytest.raises(ValueError, match="go together"):
        DecodeStepGraph(pool(2), 0.125, 4, [0, 0], **given)


@pytest.mark.parametrize("of,lens", [([0], [3]), ([0, 0, 0], [3]), ([[0, 0]], [3]), ([0, 0], [])])
def test_one_prefix_a_sequence_and_one_length_a_prefix(of, lens):
    with pytest.raises(ValueError, match="must hold"):
        DecodeStepGraph(pool(2), 0.125, 4, [0, 0], prefix=pool(1), prefix_of=of, prefix_lens=lens)
