"""Counts that a 32-bit host array cannot hold are refused, not wrapped (CPU only: the checks come before
the library)."""
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc
from kv_cache_quantization_witcert_gb300 import _lib


@pytest.fixture
def cache(monkeypatch):
    c = object.__new__(wc.Cache)
    c.cfg = _lib.witcert_config(1, 8, 2, 128, 2, 64, 0, _lib.BF16, 0, 1, 0, 0, 0, 0, 0)
    c.dtype = torch.bfloat16
    c.v_witness = False
    c._h = None

    def nothing():
        raise AssertionError("the library was called")

    monkeypatch.setattr(wc, "load", nothing)
    return c


BAD = [2 ** 32, 2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1, 10 ** 30]


@pytest.mark.parametrize("bad", BAD)
def test_counts_beyond_32_bits(cache, bad):
    kv = torch.zeros((0, 2, 128), dtype=torch.bfloat16)
    rope = wc.Rope(128)
    for call in (lambda: cache.witcert_truncate(0, [bad, 3], stream=None),
                 lambda: cache.read(0, [1, bad]),
                 lambda: cache.read(0, [1, 1], [bad, 0]),
                 lambda: cache.attend(0, kv, [bad, 0]),
                 lambda: cache.witcert_attend_workspace(0, [0, bad]),
                 lambda: cache.witcert_write_ragged(0, kv, kv, [bad, 0]),
                 lambda: cache.witcert_write_rope_ragged(0, kv, kv, [0, bad], rope)):
        with pytest.raises(ValueError, match="32"):
            call()


def test_counts_within_32_bits(cache):
    counts, arr = cache._counts("n_tok", [2 ** 31 - 1, -2 ** 31])
    assert counts == [2 ** 31 - 1, -2 ** 31] and list(arr) == counts
