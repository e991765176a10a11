"""Rotary plans and the refusals of the rotation, rotated-append, read and truncate entry points
(CPU only: every check comes before any CUDA call)."""
import ctypes
import math

import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc
from kv_cache_quantization_witcert_gb300 import _lib

B, HQ, HKV = 2, 8, 2


@pytest.fixture(scope="module")
def lib():
    from kv_cache_quantization_witcert_gb300 import build
    try:
        build.build()
    except RuntimeError as e:  # no toolkit on this machine
        pytest.skip(str(e))
    return wc.load()


@pytest.fixture
def cache():
    c = object.__new__(wc.Cache)          # no witcert_create: every call below must fail first
    c.cfg = _lib.witcert_config(1, HQ, HKV, 128, B, 64, 0, _lib.BF16, 0, 1, 0, 0, 0, 0, 0)
    c.dtype = torch.bfloat16
    c.v_witness = False
    c._h = None
    return c


def test_plain_linear_and_by_parts_frequencies():
    r = wc.Rope(64, base=1e4)
    assert r.scale == 1.0 and len(r.freq) == 32
    assert r.freq[5] == pytest.approx(1e4 ** (-10 / 64), rel=1e-15)
    assert wc.Rope(64, base=1e4, scaling="linear", factor=4.0).freq[5] == pytest.approx(r.freq[5] / 4, rel=1e-15)
    y = wc.Rope(128, base=1e4, scaling="by_parts", factor=8.0, original_tokens=4096)
    plain = wc.Rope(128, base=1e4).freq
    turns = [4096 * f / (2 * math.pi) for f in plain]
    for f, p, t in zip(y.freq, plain, turns):
        if t >= 32:
            assert f == p
        elif t <= 1:
            assert f == pytest.approx(p / 8, rel=1e-15)
        else:
            assert p / 8 < f < p
    assert y.scale == pytest.approx(0.1 * math.log(8.0) + 1)
    own = wc.Rope(8, freq=[1.0, 2.0, 3.0, 4.0], scale=0.5)
    assert own.freq == (1.0, 2.0, 3.0, 4.0) and own.scale == 0.5


def test_bad_plans_are_refused():
    for dim in (0, 4, 12, 264):
        with pytest.raises(ValueError, match="rotary_dim"):
            wc.Rope(dim)
    with pytest.raises(ValueError, match="scaling"):
        wc.Rope(64, scaling="other")
    with pytest.raises(ValueError, match="base"):
        wc.Rope(64, base=-1.0)
    with pytest.raises(ValueError, match="factor"):
        wc.Rope(64, scaling="linear", factor=0.0)
    with pytest.raises(ValueError, match="one entry per pair"):
        wc.Rope(16, freq=[1.0])
    with pytest.raises(ValueError, match="finite"):
        wc.Rope(8, freq=[1.0, 2.0, math.nan, 4.0])
    with pytest.raises(ValueError, match="by_parts"):
        wc.Rope(64, scaling="by_parts", factor=2.0, fast=1.0, slow=1.0)


def test_rope_refuses_what_it_cannot_address():
    rope = wc.Rope(128)
    pos = torch.arange(3)
    q = torch.zeros((3, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="Rope"):
        wc.witcert_rope(None, pos, q)
    with pytest.raises(ValueError, match="channels of a head"):
        wc.witcert_rope(rope, pos, q[..., :64])
    with pytest.raises(ValueError, match="bfloat16 or"):
        wc.witcert_rope(rope, pos, q.half())
    with pytest.raises(ValueError, match="int64"):
        wc.witcert_rope(rope, pos.int(), q)
    with pytest.raises(ValueError, match="positions must have shape"):
        wc.witcert_rope(rope, torch.arange(4), q)
    with pytest.raises(ValueError, match="CUDA"):
        wc.witcert_rope(rope, pos, q)
    with pytest.raises(ValueError, match="n_tok, heads, head_dim"):
        wc.witcert_rope(rope, pos, q[0])


def test_rope_tensors_are_checked():
    q = torch.zeros((3, 4, 128), dtype=torch.bfloat16)
    check = lambda x, y: wc._rope_tensor("k", x, y, 3, q)
    with pytest.raises(ValueError, match="k must have shape"):
        check(q[:2], q[:2])
    with pytest.raises(ValueError, match="k_out must have shape"):
        check(q, q[:, :2])
    with pytest.raises(ValueError, match="k must be torch.bfloat16"):
        check(q.float(), q)
    with pytest.raises(ValueError, match="adjacent channels"):
        check(q.transpose(1, 2).contiguous().transpose(1, 2), q)
    with pytest.raises(ValueError, match="k must be a CUDA"):
        check(q, q)


def test_cache_calls_check_their_tensors(cache):
    rope = wc.Rope(128)
    kv = torch.zeros((B, 3, HKV, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="rope must be a Rope"):
        cache.witcert_write_rope(0, kv, kv, None)
    with pytest.raises(ValueError, match="channels of a head"):
        cache.witcert_write_rope(0, kv, kv, wc.Rope(256))
    with pytest.raises(ValueError, match="shape"):
        cache.witcert_write_rope(0, kv, kv[:, :2].contiguous(), rope)
    with pytest.raises(ValueError, match="CUDA"):
        cache.witcert_write_rope(0, kv, kv, rope)
    packed = torch.zeros((5, HKV, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="per sequence"):
        cache.witcert_write_rope_ragged(0, packed, packed, [5], rope)
    with pytest.raises(ValueError, match="CUDA"):
        cache.witcert_write_rope_ragged(0, packed, packed, [2, 3], rope)
    with pytest.raises(ValueError, match="lengths needs one count per sequence"):
        cache.witcert_truncate(0, [1])
    with pytest.raises(ValueError, match="K must have shape"):
        cache.witcert_read(0, None, [1, 1], packed, packed)
    with pytest.raises(ValueError, match="t0 needs one count"):
        cache.witcert_read(0, [0], [2, 3], packed, packed)


def test_library_refuses_bad_arguments(lib):
    fake, cfg = ctypes.c_void_p(16), wc.Rope(128)._cfg
    t = _lib.witcert_rope_tensor(16, 16, 2, 256, 128, 256, 128)
    ref, rt = ctypes.addressof(cfg), ctypes.addressof(t)

    def rope(c=ref, dt=_lib.BF16, dim=128, n=1, pos=fake, q=rt, k=None):
        return lib.witcert_rope(c, dt, dim, n, pos, q, k, 0, None)

    assert rope(c=None) == _lib.EINVAL
    assert rope(dt=7) == _lib.EINVAL
    assert rope(dim=127) == _lib.EINVAL and rope(dim=258) == _lib.EINVAL and rope(dim=64) == _lib.EINVAL
    assert rope(n=-1) == _lib.EINVAL
    assert rope(pos=None) == _lib.EINVAL and b"positions" in lib.witcert_last_error()
    assert rope(q=None) == _lib.EINVAL
    headless = _lib.witcert_rope_tensor(16, 16, 0, 0, 0, 0, 0)
    assert rope(k=ctypes.addressof(headless)) == _lib.EINVAL and b"n_heads" in lib.witcert_last_error()
    nothing = _lib.witcert_rope_tensor(None, 16, 2, 256, 128, 256, 128)
    assert rope(q=ctypes.addressof(nothing)) == _lib.EINVAL
    shared = _lib.witcert_rope_tensor(16, 16, 2, 256, 128, 0, 128)
    assert rope(n=2, q=ctypes.addressof(shared)) == _lib.EINVAL and b"stride 0" in lib.witcert_last_error()
    odd = _lib.witcert_rope_tensor(17, 16, 2, 256, 128, 256, 128)
    assert rope(q=ctypes.addressof(odd)) == _lib.EINVAL and b"aligned" in lib.witcert_last_error()
    assert rope(n=0) == _lib.OK                                  # nothing to do, no GPU needed
    for dim, freq, scale in ((12, 1.0, 1.0), (136, 1.0, 1.0), (128, math.inf, 1.0), (128, 1.0, math.nan)):
        bad = _lib.witcert_rope_config(dim, 0, scale, (ctypes.c_double * 128)(*([freq] * 128)))
        assert rope(c=ctypes.addressof(bad)) == _lib.EINVAL
    counts = (ctypes.c_int32 * 1)(1)
    assert lib.witcert_write_rope(None, 0, fake, fake, None, None, 1, ref, None) == _lib.EINVAL
    assert lib.witcert_write_rope_ragged(None, 0, fake, fake, None, None, counts, ref, None) == _lib.EINVAL
    assert lib.witcert_truncate(None, 0, counts, None) == _lib.EINVAL
    assert lib.witcert_read(None, 0, None, counts, fake, fake, None) == _lib.EINVAL
