"""Forks, beam selections and paths refuse bad arguments before any CUDA call (CPU only)."""
import ctypes

import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc
from kv_cache_quantization_witcert_gb300 import _lib, build


@pytest.fixture(scope="module")
def lib():
    try:
        build.build()
    except RuntimeError as e:  # no toolkit on this machine
        pytest.skip(str(e))
    return wc.load()


GOOD = dict(dtype=_lib.BF16, n_requests=2, n_beams=4, vocab=1000, n_out=4, eos=7, logits=4096, request_stride=4000,
            beam_stride=1000, scores=4096, finished=4096, out_scores=8192, rows=8192, tokens=8192, out_finished=8192)


@pytest.mark.parametrize("change, text", [
    (dict(dtype=7), b"dtype"), (dict(n_requests=-1), b"n_requests"), (dict(n_beams=0), b"n_beams"), (dict(n_beams=129), b"n_beams"),
    (dict(vocab=0), b"vocab"), (dict(vocab=2 ** 25 + 1), b"vocab"), (dict(n_out=0), b"n_out"), (dict(n_out=257), b"n_out"),
    (dict(eos=1000), b"eos"), (dict(eos=-2), b"eos"), (dict(eos=-1), b"eos"), (dict(n_requests=2 ** 30), b"rows"),
    (dict(logits=4097), b"aligned"), (dict(logits=None), b"NULL"), (dict(scores=None), b"NULL"), (dict(out_scores=None), b"NULL"),
    (dict(rows=None), b"NULL"), (dict(tokens=None), b"NULL"), (dict(n_out=8, out_scores=4096), b"n_out = n_beams"),
    (dict(n_out=8, out_finished=4096), b"n_out = n_beams"), (dict(n_requests=2 ** 24, vocab=2 ** 25), b"logits"), ({}, b"workspace")])
def test_steps(lib, change, text):
    step = _lib.witcert_beam_step(**{**GOOD, **change})
    assert lib.witcert_beam_select(ctypes.addressof(step), None, 1 << 40, None) == _lib.EINVAL
    assert text in lib.witcert_last_error()


def test_workspace(lib):
    step, n = _lib.witcert_beam_step(**GOOD), ctypes.c_size_t()
    assert lib.witcert_beam_workspace(ctypes.addressof(step), ctypes.byref(n)) == _lib.OK and n.value >= 8 * 4
    assert lib.witcert_beam_workspace(ctypes.addressof(step), None) == _lib.EINVAL
    assert lib.witcert_beam_workspace(None, ctypes.byref(n)) == _lib.EINVAL
    assert lib.witcert_beam_select(ctypes.addressof(step), 16, n.value - 1, None) == _lib.EINVAL
    assert lib.witcert_beam_select(ctypes.addressof(step), 24, n.value + 64, None) == _lib.EINVAL
    step.n_requests = 0
    assert lib.witcert_beam_select(ctypes.addressof(step), None, 0, None) == _lib.OK


def test_paths(lib):
    p = 4096
    for args in ((None, p, 2, 2, 2, None, -1, p), (p, None, 2, 2, 2, None, -1, p), (p, p, 2, 2, 2, None, -1, None),
                 (p, p, -1, 2, 2, None, -1, p), (p, p, 2, -1, 2, None, -1, p), (p, p, 2, 2, 0, None, -1, p),
                 (p, p, 2, 2, 129, None, -1, p), (p, p, 2, 2 ** 30, 4, None, -1, p)):
        assert lib.witcert_beam_paths(*args, None) == _lib.EINVAL, args
    assert lib.witcert_beam_paths(None, None, 0, 2, 2, None, -1, None, None) == _lib.OK


def test_fork(lib):
    parents = (ctypes.c_int32 * 1)(0)
    assert lib.witcert_fork(None, parents, None, None) == _lib.EINVAL
    assert lib.witcert_fork(1 << 20, None, None, None) == _lib.EINVAL        # the cache is not looked at first
    c = object.__new__(wc.Cache)
    c.cfg = _lib.witcert_config(1, 4, 2, 128, 3, 64, 0, _lib.BF16, 0, 1, 0, 0, 0, 0, 0)
    c._h = None
    with pytest.raises(ValueError, match="per sequence"):
        c.witcert_fork([0, 0])
    with pytest.raises(ValueError, match="lengths"):
        c.witcert_fork([0, 0, 0], [1, 2])
    with pytest.raises(ValueError, match="32 bits"):
        c.witcert_fork([0, 0, 2 ** 31])


def test_binding():
    x, s = torch.zeros(2, 4, 10, dtype=torch.bfloat16), torch.zeros(2, 4)
    for bad, text in (((x[0], s), "requests"), ((x.half(), s), "bfloat16"), ((x.transpose(1, 2).contiguous().transpose(1, 2), s), "adjacent"),
                      ((x, s.double()), "scores"), ((x, s[:1]), "scores"), ((x, s), "CUDA"), ((None, s), "logits")):
        with pytest.raises(ValueError, match=text):
            wc.witcert_beam_select(*bad)
    with pytest.raises(ValueError, match="finished"):
        wc.witcert_beam_select(x, s, finished=torch.zeros(2, 4), eos=1)
    r = torch.zeros(5, 2, 4, dtype=torch.int32)
    for bad, text in (((r[0], r[0]), "rows"), ((r, r[:4]), "tokens"), ((r.long(), r), "rows"), ((r, r), "CUDA"),
                      ((r, r, torch.zeros(3, dtype=torch.int32)), "length")):
        with pytest.raises(ValueError, match=text):
            wc.witcert_beam_paths(*bad)


def test_search_needs_whole_requests():
    c = object.__new__(wc.Cache)
    c.cfg = _lib.witcert_config(1, 4, 2, 128, 6, 64, 0, _lib.BF16, 0, 1, 0, 0, 0, 0, 0)
    c._h = None
    for beams, steps in ((4, 8), (0, 8), (-1, 8), (3, 0)):
        with pytest.raises(ValueError):
            wc.BeamSearch(c, beams, steps)
