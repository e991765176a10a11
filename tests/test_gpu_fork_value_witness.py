"""Value witnesses of forked sequences: those of the tokens held, and none of an old occupant behind them."""
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc
from kv_cache_quantization_witcert_gb300 import _lib

from test_gpu_histories import SCHEMES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wc.load()


@pytest.mark.parametrize("pages", [0, 64])
@pytest.mark.parametrize("scheme", SCHEMES)
def test_shorter_parents_and_cuts(scheme, pages):
    c = wc.Cache(2, 4, 2, 5, 100, scheme, seed=5, v_witness=True, max_pages=pages)
    n = [90, 20, 35, 50, 61]
    for layer in range(2):
        k, v = (torch.randn(sum(n), 2, 128, device="cuda").bfloat16() for _ in range(2))
        c.witcert_write_ragged(layer, k, v, n, *((k / 2, v / 2) if scheme == "blackbox" else ()))
    look = lambda layer: c.export(layer, _lib.X_V_WITNESS)

    def compare(before, parents, lens):
        for layer in range(2):
            got = look(layer)
            assert got.shape[1] == max(lens)
            for i, (p, m) in enumerate(zip(parents, lens)):
                assert torch.equal(got[i, :m], before[layer][p, :m])
                assert not got[i, m:].any()

    before = [look(layer) for layer in range(2)]
    assert all((x[i, :m] > 0).any() for x in before for i, m in enumerate(n))
    parents = [0, 1, 1, 2, -1]                              # a shorter parent, a longer one's start, an empty one
    cut = [90, 20, 16, 32, 0]
    c.witcert_fork(parents, cut)
    compare(before, parents, cut)
    c.witcert_fork([0, 0, 2, 3, 4], [48, 90, 16, 32, 0])    # cut where it is, and a fork of the whole
    compare([x[[0, 1, 1, 2, 0]] for x in before], [0, 0, 2, 3, 4], [48, 90, 16, 32, 0])
    before = [look(layer) for layer in range(2)]
    c.witcert_truncate(-1, [32, 80, 0, 32, 0])
    compare(before, range(5), [32, 80, 0, 32, 0])
