"""Rows of a block past its sequence's length, whatever they hold, leave no trace in a decode.

Such rows are tokens that witcert_truncate dropped, the rows of a sequence that was reset, or a page's
rows from its sequence before.  A cache whose block holds them decodes to the same bits, out and every
meter, as one that never held them: the same blocks, splits and order of sums.  The rows here have
values that are not numbers, or so far off that the value witness is +inf in fp16 (0 x inf is a NaN).
"""
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc

pytestmark = pytest.mark.gpu

SCHEMES = ["int8_dither", "fp8_e4m3", "kivi2", "int8_rtn", "blackbox"]
HQ, HKV = 6, 2


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wc.load()


def rows(seed, dtype, *shape):
    g = torch.Generator().manual_seed(seed)
    return tuple(torch.randn(*shape, HKV, 128, generator=g).to("cuda", dtype) for _ in range(2))


def append(cache, scheme, K, V, n, V_hat=None):
    hat = (K, V if V_hat is None else V_hat) if scheme == "blackbox" else ()
    cache.witcert_write_ragged(0, K, V, n, *hat)


def same(a, b, scheme):
    q = torch.randn(a.cfg.batch, HQ, 128, generator=torch.Generator().manual_seed(9)).to("cuda", a.dtype)
    (oa, ma), (ob, mb) = a.decode(0, q, 1e-2), b.decode(0, q, 1e-2)
    assert oa.isfinite().all() and torch.equal(oa, ob)
    for name in ma:
        if name.endswith("_b") and scheme != "int8_dither":
            assert ma[name].isnan().all() and mb[name].isnan().all()
        else:
            assert not ma[name].isnan().any(), name
            assert torch.equal(ma[name], mb[name]), name
    plain, _ = a.decode(0, q, 1e-2, meters=False)
    assert torch.equal(plain, oa)


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf", "1e30"])
def test_truncated_tokens(scheme, dtype, bad):
    lens, extra = [37, 1, 64 + 13], [5, 3, 1]              # the dropped tokens lie in the last block
    mk = lambda: wc.Cache(1, HQ, HKV, 3, 96, scheme, dtype=dtype, seed=3, v_witness=True)
    a, b = mk(), mk()
    K, V = rows(1, dtype, sum(lens))
    for c in (a, b):
        append(c, scheme, K, V, lens)
    K2, V2 = rows(2, dtype, sum(extra))
    K2[:], V2[:, :, 3:] = float(bad), float(bad)
    append(a, scheme, K2, V2, extra)
    a.witcert_truncate(0, lens)
    same(a, b, scheme)


def test_a_tensor_function_that_is_far_off():
    """Finite values 1e5 away from the exact ones: the witness alone is out of fp16's range."""
    mk = lambda: wc.Cache(1, HQ, HKV, 1, 64, "blackbox", seed=3, v_witness=True)
    a, b = mk(), mk()
    K, V = rows(1, torch.bfloat16, 20)
    for c in (a, b):
        append(c, "blackbox", K, V, [20], V * 0.875)
    append(a, "blackbox", K[:4], V[:4], [4], V[:4] + 1e5)
    a.witcert_truncate(0, [20])
    same(a, b, "blackbox")


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("pages", [0, 6])
def test_rows_of_a_sequence_before(scheme, pages):
    """A slot, or a page, whose sequence held such values serves another, shorter one."""
    mk = lambda: wc.Cache(1, HQ, HKV, 2, 48, scheme, seed=3, v_witness=True, max_pages=pages)
    a, b = mk(), mk()
    K, V = rows(4, torch.bfloat16, 48)
    bad = V.clone()
    bad[:, 1, ::5] = float("nan")
    append(a, scheme, K, bad, [48, 0])
    a.witcert_reset_sequence(0)
    b.witcert_reset_sequence(0)                            # both keep their lengths on the device
    K, V = rows(5, torch.bfloat16, 26)
    for c in (a, b):
        append(c, scheme, K, V, [21, 5])
    same(a, b, scheme)
