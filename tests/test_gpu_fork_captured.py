"""A decode captured while the sequences' lengths differed follows them: a fork that makes them equal, and what is
appended and cut behind it, reach its replays."""
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wc.load()


def rows(n, heads=2):
    return torch.randn(n, heads, 128, device="cuda").bfloat16()


@pytest.mark.parametrize("noalloc", [False, True])
@pytest.mark.parametrize("pages", [0, 48])
def test_replays_see_the_present_lengths(pages, noalloc):
    """A decode captured while the lengths differed, replayed after forks that make them equal and what follows.
    Replays cut the sequences into other splits than a fresh decode: sums in another order, 2^-13."""
    torch.manual_seed(1)
    c = wc.Cache(2, 4, 2, 3, 200, "fp8_e4m3", max_pages=pages)
    for layer in range(2):
        k = rows(100 + 37 + 64)
        c.witcert_write_ragged(layer, k, k.flip(0), [100, 37, 64])
    q = rows(3, 4)
    out, meter = torch.empty(3, 4, 128, device="cuda"), torch.empty(3, 4, device="cuda")
    call = c.witcert_decode_noalloc if noalloc else c.witcert_decode
    call(1, q, 1e-2, out, meter)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(1, q, 1e-2, out, meter)

    def same():
        q.copy_(rows(3, 4))
        g.replay()
        got, got_a = out.clone(), meter.clone()
        want, m = c.decode(1, q, 1e-2)
        assert (got - want).abs().max() <= 2.0 ** -13 * max(1.0, want.abs().max().item())
        assert ((got_a - m["meter_a"]).abs() <= 2e-4 * m["meter_a"] + 2.0 ** -99).all()

    def append(n):
        for layer in range(2):
            k = rows(sum(n))
            c.witcert_write_ragged(layer, k, k.flip(0), n)

    same()
    c.witcert_fork([1, 1, 1])                               # 37 each
    same()
    append([5, 5, 5])
    same()
    c.witcert_truncate(-1, [30, 30, 30])
    same()
    c.witcert_fork([0, 1, 0], [20, 20, 20])
    same()
    append([9, 0, 1])
    same()
    c.witcert_reset_sequence(1)
    append([0, 29, 8])
    same()
    c.witcert_fork([2, 2, 2], [29, 29, 29])
    append([1, 1, 1])
    same()
