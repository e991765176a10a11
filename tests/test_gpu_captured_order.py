"""Calls that are only captured do not stand for launches: what overlaps what outside a capture goes by what was
launched, and within one by what was captured there."""
import ctypes

import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc
from kv_cache_quantization_witcert_gb300 import _lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wc.load()


def rows(n, heads=2):
    return torch.randn(n, heads, 128, device="cuda").bfloat16()


class Edge(ctypes.Structure):
    _fields_ = [("from_port", ctypes.c_ubyte), ("to_port", ctypes.c_ubyte), ("type", ctypes.c_ubyte), ("reserved", ctypes.c_ubyte * 5)]


def edges(work):
    """Captures work() and launches nothing: of each node but the first, whether it waits for the end of the node before
    (0) or may start before that (1)."""
    cu, ptr = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p
    side, graph = torch.cuda.Stream(), ptr()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        assert cu.cuStreamBeginCapture_v2(ptr(side.cuda_stream), 2) == 0
        work()
        assert cu.cuStreamEndCapture(ptr(side.cuda_stream), ctypes.byref(graph)) == 0
    n = ctypes.c_size_t(0)
    assert cu.cuGraphGetEdges_v2(graph, None, None, None, ctypes.byref(n)) == 0 and n.value > 0
    a, b, e = (ptr * n.value)(), (ptr * n.value)(), (Edge * n.value)()
    assert cu.cuGraphGetEdges_v2(graph, a, b, e, ctypes.byref(n)) == 0
    after = {a[k]: (b[k], e[k].type) for k in range(n.value)}
    at, kinds = (set(after) - {x for x, _ in after.values()}).pop(), []
    while at in after:
        at, kind = after[at]
        kinds.append(kind)
    assert len(kinds) == n.value                            # one chain
    assert cu.cuGraphDestroy(graph) == 0
    return kinds


def first_edge(work):
    return edges(work)[0]


def test_what_follows_a_fork():
    """What follows a fork starts after its end, also where other calls have been captured in between."""
    c = wc.Cache(1, 4, 2, 2, 64, "int8_rtn")
    k = rows(40).view(2, 20, 2, 128)
    one = rows(2).view(2, 1, 2, 128)
    q, out, x = rows(2, 4), torch.empty(2, 4, 128, device="cuda"), torch.empty(64, device="cuda")
    c.witcert_write(0, k, k)

    def decode():
        x.fill_(1.0)
        c.witcert_decode(0, q, 1e-2, out)

    decode()
    assert first_edge(decode) == 1                          # the usual chain
    c.witcert_fork([1, 0])
    assert first_edge(decode) == 0
    assert first_edge(decode) == 0                          # the first one was not launched
    decode()
    assert first_edge(decode) == 1
    c.witcert_reset_sequence(1)                             # lengths that the decode reads at once
    assert first_edge(decode) == 0
    assert first_edge(decode) == 0
    c.witcert_write_ragged(0, one[0], one[0], [0, 1])
    assert first_edge(decode) == 1


def test_an_export_of_nothing_launches_nothing():
    """What it follows still is the last launch: the resets' lengths, that a decode reads at once."""
    c = wc.Cache(1, 4, 2, 2, 64, "int8_rtn")
    k, x = rows(40).view(2, 20, 2, 128), torch.empty(64, device="cuda")
    q, out, dst = rows(2, 4), torch.empty(2, 4, 128, device="cuda"), torch.empty(64, dtype=torch.uint8, device="cuda")

    def decode():
        x.fill_(1.0)
        c.witcert_decode(0, q, 1e-2, out)

    c.witcert_write(0, k, k)
    c.witcert_export(0, _lib.X_K_CODES, torch.empty(2 * 20 * 2 * 128, dtype=torch.uint8, device="cuda"))
    assert first_edge(decode) == 1
    for i in range(2):
        c.witcert_reset_sequence(i)
    c.witcert_export(0, _lib.X_K_CODES, dst)
    assert first_edge(decode) == 0
    torch.cuda.synchronize()


def test_calls_outside_a_capture_in_its_middle():
    """What a capture goes on with behind a launched call starts after what it has captured so far."""
    c = wc.Cache(2, 4, 2, 2, 64, "int8_rtn")
    k, one, q, out = rows(40).view(2, 20, 2, 128), rows(2).view(2, 1, 2, 128), rows(2, 4), torch.empty(2, 4, 128, device="cuda")
    other = torch.cuda.Stream()
    for layer in range(2):
        c.witcert_write(layer, k, k)
    torch.cuda.synchronize()

    def work(between):
        c.witcert_write(0, one, one)
        if between:
            with torch.cuda.stream(other):
                c.witcert_decode(1, q, 1e-2, out)
        c.witcert_decode(0, q, 1e-2, out)

    assert first_edge(lambda: work(False)) == 1             # a decode behind an append
    assert first_edge(lambda: work(True)) == 0
    torch.cuda.synchronize()


def test_launches_between_captures():
    """Forks, appends and decodes with captured decodes among them, against the same calls without."""
    torch.manual_seed(2)
    k, new = rows(4 * 1000).view(4, 1000, 2, 128), [rows(4).view(4, 1, 2, 128) for _ in range(6)]
    q, outs = rows(4, 4), []
    for captures in (False, True):
        c = wc.Cache(2, 4, 2, 4, 1100, "int8_dither", seed=3, max_pages=300)
        out = torch.empty(4, 4, 128, device="cuda")
        got = []
        for layer in range(2):
            c.witcert_write(layer, k, k)
        for step, x in enumerate(new):
            c.witcert_fork([(i + step) % 4 for i in (1, 1, 3, 2)])
            for layer in range(2):
                if captures:
                    edges(lambda: [c.witcert_decode(layer, q, 1e-2, out) for _ in range(2)])
                c.witcert_write(layer, x, x)
                if captures:
                    edges(lambda: [c.witcert_decode(layer, q, 1e-2, out) for _ in range(2)])
                got.append(c.decode(layer, q, 1e-2, meters=False)[0])
        outs.append(got)
    assert all(torch.equal(a, b) for a, b in zip(*outs))
