"""A rotation's scale that fp32 cannot hold is refused (CPU only: before any CUDA call)."""
import ctypes

import pytest

import kv_cache_quantization_witcert_gb300 as wc
from kv_cache_quantization_witcert_gb300 import _lib


@pytest.mark.parametrize("scale,status", [(1e39, _lib.EINVAL), (-1e300, _lib.EINVAL), (3.4e38, _lib.OK), (1e-300, _lib.OK)])
def test_scales(scale, status):
    from kv_cache_quantization_witcert_gb300 import build
    try:
        build.build()
    except RuntimeError as e:  # no toolkit on this machine
        pytest.skip(str(e))
    rope = wc.Rope(128, scale=scale)
    t = _lib.witcert_rope_tensor(16, 16, 2, 256, 128, 256, 128)
    # no tokens: an accepted call has nothing to launch
    assert wc.load().witcert_rope(rope._ref, _lib.BF16, 128, 0, None, ctypes.addressof(t), None, 0, None) == status
