"""An error that a call has reported does not come back from the next one, nor from torch."""
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc
from kv_cache_quantization_witcert_gb300 import _lib

pytestmark = pytest.mark.gpu


def test_calls_after_a_cache_that_does_not_fit():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    x = torch.randn(3, 2, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    pos, rope = torch.arange(3, device="cuda"), wc.Rope(128)
    c = wc.Cache(1, 2, 2, 1, 16, "int8_dither")
    c.witcert_write(0, x[None], x[None])
    calls = [lambda: wc.witcert_rope(rope, pos, x), lambda: c.read(0, [3])[0], lambda: c.attend(0, x, [3]),
             lambda: c.export(0, _lib.X_K_CODES), lambda: wc.witcert_dither(1, 0, 0, 0, 4, 0),
             lambda: wc.witcert_gate_select(torch.ones(1, 2, 4, device="cuda"), 2, 0.5), lambda: x.float() + 1]
    want = [f() for f in calls]
    for f, w in zip(calls, want):
        with pytest.raises(wc.WitcertError) as e:
            wc.Cache(1, 64, 64, 1, 1 << 30, "fp8_e4m3")    # 20 TB
        assert e.value.status == _lib.ENOMEM
        assert torch.equal(f(), w)
    torch.cuda.synchronize()


def test_calls_after_polling_a_gate():
    """witcert_gate_stats asks for the gate's event until it is there: "not ready" is no error of later calls."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator().manual_seed(2)
    K = torch.randn(1, 64, 2, 128, generator=g).bfloat16().cuda()
    q = torch.randn(1, 4, 128, generator=g).bfloat16().cuda()
    pos, rope = torch.arange(64, device="cuda"), wc.Rope(128)
    c = wc.Cache(1, 4, 2, 1, 64, "fp8_e4m3", max_repair_blocks=16)
    c.witcert_write(0, K, K)
    c.decode(0, q, 1e-2)
    for f in (lambda: wc.witcert_rope(rope, pos, K[0]), lambda: c.read(0, [64]), lambda: c.attend(0, q, [1]),
              lambda: K.float() + 1):
        torch.cuda._sleep(100_000_000)                     # 50 ms that the gate waits for
        c.witcert_gate(0, 0.0)
        c.witcert_gate_stats()
        f()
        c.decode(0, q, 1e-2)
    with pytest.raises(wc.WitcertError) as e:              # a deadline that runs out
        torch.cuda._sleep(400_000_000)
        c.witcert_gate(0, 0.0)
        c.witcert_gate_stats(1)
    assert e.value.status == _lib.ETIMEDOUT
    wc.witcert_rope(rope, pos, K[0])
    torch.cuda.synchronize()
