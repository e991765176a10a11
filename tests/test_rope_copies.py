"""Copies of a rotation's plan hold their own memory (CPU only)."""
import copy
import ctypes
import gc
import pickle

import pytest

import kv_cache_quantization_witcert_gb300 as wc
from kv_cache_quantization_witcert_gb300 import _lib

PLANS = [dict(), dict(rotary_dim=48, base=1e6, interleaved=True, scaling="by_parts", factor=8.0),
         dict(rotary_dim=8, freq=[1.0, -2.0, 3.0, 4.0], scale=0.5)]


@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("clone", [copy.copy, copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r)),
                                   lambda r: copy.deepcopy({"layers": [r]})["layers"][0]])
def test_copies_are_plans_of_their_own(plan, clone):
    rope = wc.Rope(**plan)
    want = bytes(rope._cfg)
    other = clone(rope)
    assert other._ref == ctypes.addressof(other._cfg)
    assert (other.freq, other.scale, other.rotary_dim, other.interleaved) == (rope.freq, rope.scale, rope.rotary_dim, rope.interleaved)
    del rope
    gc.collect()
    assert ctypes.string_at(ctypes.addressof(other._cfg), ctypes.sizeof(_lib.witcert_rope_config)) == want
    assert other._ref == ctypes.addressof(other._cfg)
