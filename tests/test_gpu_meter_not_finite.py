"""Meters of tokens whose error is beyond every number: a bound is +inf (1 where it is capped), never 0.

A witness above fp16's range is +inf, and a NaN input has a NaN witness.  The sums that the meters are
formed from are then inf or NaN, the NaN also from 0 x inf where a token's weight underflows."""
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc
from kv_cache_quantization_witcert_gb300 import _lib

pytestmark = pytest.mark.gpu

SCHEMES = ["int8_dither", "fp8_e4m3", "kivi2", "int8_rtn", "blackbox"]
HQ, HKV = 4, 2


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wc.load()


def cache(scheme, n, seed=1, **kw):
    g = torch.Generator().manual_seed(seed)
    K, V = (torch.randn(1, n, HKV, 128, generator=g).bfloat16().cuda() for _ in range(2))
    return wc.Cache(1, HQ, HKV, 1, n, scheme, seed=2, v_witness=True, **kw), K, V


def write(c, K, V, K_hat=None, V_hat=None):
    if c.scheme == "blackbox":
        c.witcert_write_hat(0, K, V, K if K_hat is None else K_hat, V if V_hat is None else V_hat)
    else:
        c.witcert_write(0, K, V)


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("n", [5, 16, 700])                 # one block, and splits
def test_value_witness_out_of_range(scheme, n):
    c, K, V = cache(scheme, n)
    bad = V.clone()
    bad[:, n // 2, 1] = 1e30                               # KV head 1: query heads 2 and 3
    write(c, K, bad, V_hat=V)
    wv = c.export(0, _lib.X_V_WITNESS)[0]
    assert wv[n // 2, 1].isinf() and wv[:, 0].isfinite().all()
    _, m = c.decode(0, torch.randn(1, HQ, 128, generator=torch.Generator().manual_seed(3)).bfloat16().cuda(), 1e-2)
    assert m["meter_v"][0, :2].isfinite().all() and (m["meter_v"][0, 2:] == float("inf")).all()


def test_weight_that_underflows_against_an_infinite_witness():
    c, K, V = cache("fp8_e4m3", 40)
    q = torch.full((1, HQ, 128), 4.0).bfloat16().cuda()
    K = torch.full_like(K, 4.0)
    K[:, 7] = -400.0                                       # logit -18102 against 181: its weight is 0
    V[:, 7] = 1e30
    write(c, K, V)
    out, m = c.decode(0, q, 1e-2)
    assert out.isfinite().all() and (m["meter_v"] == float("inf")).all()


@pytest.mark.parametrize("scheme", ["fp8_e4m3", "int8_rtn", "blackbox"])
@pytest.mark.parametrize("n", [16, 700])
def test_key_witness_out_of_range(scheme, n):
    """Tier A's bound of a key that is far off: raw +inf, meter 1, and the gate repairs its block first."""
    c, K, V = cache(scheme, n, max_repair_blocks=8)
    bad = K.clone()
    bad[:, 3] = 1e30 if scheme != "int8_rtn" else 1e9
    write(c, bad, V, K_hat=K)
    q = torch.zeros(1, HQ, 128).bfloat16().cuda()
    q[..., 5] = 1e-30                                      # logits of a few units, bounds beyond all
    q[..., 70] = 1.0
    assert c.export(0, _lib.X_WITNESS)[0, 3].isinf().any()
    _, m = c.decode(0, q, 1e-2)
    assert (m["raw_a"] == float("inf")).all() and (m["meter_a"] == 1).all()
    risk = c.export(0, _lib.X_BLOCK_RISK)[0]
    assert not (risk[:, 0] < 3e38).any()                   # inf (a NaN counts as that too)
    c.witcert_gate(0, 1e6)
    assert c.witcert_gate_stats()["blocks_paged_in"] == HKV
    assert (c.export(0, _lib.X_SLOTS)[0, :, 0] >= 0).all()


def test_an_empty_cache_has_meters_of_zero():
    c, _, _ = cache("fp8_e4m3", 16)
    _, m = c.decode(0, torch.ones(1, HQ, 128).bfloat16().cuda(), 1e-2)
    for name in ("meter_a", "raw_a", "meter_v"):
        assert (m[name] == 0).all()
