"""Refusals of the calls that store turned rows and attend behind prefixes, without a GPU."""
import ctypes

import pytest

from head_budgeted_kv_gb300 import _build, binding


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load()


def test_rope_append_needs_a_pool(lib):
    t = binding.hwkv_rope_table(64)
    rows = binding.Rows(None, 0, 0)
    assert lib.hwkv_rope_append(None, 0, t, None, 0, ctypes.byref(rows), ctypes.byref(rows), 1, None, None, None, None, None,
                                None) == binding.HWKV_ERR_INVALID_ARG
    assert "pool" in binding.last_error()


def test_shared_decode_needs_its_pools(lib):
    s = binding.Score(1.0, 0.0, None)
    assert lib.hwkv_decode_attn_shared(None, None, 0, None, 4, s, None, None, None, None, None, None, None, 0,
                                       None) == binding.HWKV_ERR_INVALID_ARG
    out = ctypes.c_uint64(7)
    assert lib.hwkv_decode_shared_workspace_bytes(None, None, 4, ctypes.byref(out)) == binding.HWKV_ERR_INVALID_ARG
    assert out.value == 7
