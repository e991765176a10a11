"""Host memory that runs out at a C entry is a status code, not a C++ exception that ends the process
(CPU only: the host's tables are made before any CUDA call).  In a process of its own, with a limit on
its address space."""
import os
import subprocess
import sys

import pytest

from kv_cache_quantization_witcert_gb300 import build

CODE = """
import ctypes, resource, sys
sys.path.insert(0, {root!r})
lib = ctypes.CDLL({lib!r})
lib.witcert_last_error.restype = ctypes.c_char_p
class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("n_layers", "n_q_heads", "n_kv_heads", "head_dim", "batch", "max_tokens", "scheme",
                "kv_dtype")] + [("seed", ctypes.c_uint64)] + [(n, ctypes.c_int) for n in ("total_steps", "n_splits",
                "max_repair_blocks", "pos_offset", "v_witness", "max_pages")]
held = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (held + (1 << 30),) * 2)
out = ctypes.c_void_p(1)
cfg = Config(65535, 1, 1, 128, 2 ** 31 - 1, 16, 1, 1, 0, 1, 0, 0, 0, 0, 0)
print(lib.witcert_create(ctypes.byref(cfg), ctypes.byref(out)), out.value, lib.witcert_last_error().decode())
"""


def test_create_without_host_memory():
    try:
        lib = build.build()
    except RuntimeError as e:  # no toolkit on this machine
        pytest.skip(str(e))
    r = subprocess.run([sys.executable, "-c", CODE.format(root=os.path.dirname(build.PKG), lib=lib)], capture_output=True,
                       text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split(None, 2) == ["-2", "None", "host allocation failed\n"]


@pytest.mark.parametrize("change", [dict(n_layers=64, batch=64, n_kv_heads=65535, n_q_heads=65535, max_tokens=2 ** 31 - 16),
                                    dict(batch=1 << 14, n_kv_heads=1 << 12, n_q_heads=1 << 12, n_splits=2 ** 31 - 1),
                                    dict(n_layers=65535, n_kv_heads=65535, n_q_heads=65535, max_pages=2 ** 31 - 1)])
def test_sizes_beyond_64_bits(change):
    """Refused before anything is allocated, not wrapped to a small allocation."""
    import ctypes

    from kv_cache_quantization_witcert_gb300 import _lib, load
    try:
        build.build()
    except RuntimeError as e:  # no toolkit on this machine
        pytest.skip(str(e))
    cfg = _lib.witcert_config(1, 1, 1, 128, 1, 16, 1, _lib.BF16, 0, 1, 0, 0, 0, 0, 0)
    for name, value in change.items():
        setattr(cfg, name, value)
    out = ctypes.c_void_p(1)
    assert load().witcert_create(ctypes.byref(cfg), ctypes.byref(out)) == _lib.ENOMEM
    assert out.value is None and b"addressed" in load().witcert_last_error()
