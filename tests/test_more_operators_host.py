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
