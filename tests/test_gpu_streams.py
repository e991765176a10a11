"""Calls on a stream that is not the current one leave the current stream's memory alone.

A tensor is copied behind a pause on the current stream and freed: its block may be handed out again,
but only to work that follows the copy.  Calls with stream= run at once; had they taken their outputs or
workspace from the current stream's free blocks, the copy would find them there."""
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc
from kv_cache_quantization_witcert_gb300 import _lib

pytestmark = pytest.mark.gpu

HQ, HKV, N = 8, 2, 400


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wc.load()


@pytest.fixture(scope="module")
def setup():
    g = torch.Generator().manual_seed(1)
    c = wc.Cache(1, HQ, HKV, 2, N, "int8_dither", seed=4)
    K, V = (torch.randn(2, N, HKV, 128, generator=g).bfloat16().cuda() for _ in range(2))
    c.witcert_write(0, K, V)
    q = torch.randn(2 * 300, HQ, 128, generator=g).bfloat16().cuda()
    more = dict(pos=torch.arange(600, device="cuda"), rope=wc.Rope(128), risk=torch.ones(2, HQ, 640, device="cuda"),
                parts=c.decode_partial(0, q[:2], 1e-2, N)[:, :, None].expand(2, HQ, 3, -1).contiguous())
    return c, q, more


CALLS = {
    "rope": lambda c, q, m, **kw: wc.witcert_rope(m["rope"], m["pos"], q, q[:, :HKV], **kw),
    "attend_images": lambda c, q, m, **kw: c.attend(0, q, [300, 300], **kw),
    "attend_few": lambda c, q, m, **kw: c.attend(0, q[:60], [30, 30], **kw),
    "attend_tiny": lambda c, q, m, **kw: c.attend(0, q[:8], [4, 4], **kw),
    "read": lambda c, q, m, **kw: c.read(0, [N, N], **kw),
    "decode": lambda c, q, m, **kw: c.decode(0, q[:2], 1e-2, **kw)[0],
    "decode_partial": lambda c, q, m, **kw: c.decode_partial(0, q[:2], 1e-2, N, **kw),
    "export": lambda c, q, m, **kw: c.export(0, _lib.X_K_CODES, **kw),
    "merge": lambda c, q, m, **kw: wc.witcert_merge_partials(m["parts"], "int8_dither", **kw)[0],
    "gate_select": lambda c, q, m, **kw: wc.witcert_gate_select(m["risk"], HKV, 0.5, **kw),
    "dither": lambda c, q, m, **kw: wc.witcert_dither(7, 0, 1, 0, 999, 0, **kw),
}


def flat(x):
    return list(x) if isinstance(x, tuple) else [x]


@pytest.mark.parametrize("name", list(CALLS))
def test_freed_blocks_of_the_current_stream(setup, name):
    call = CALLS[name]
    want = flat(call(*setup))                              # and the kernels are loaded
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    flat(call(*setup, stream=side))
    torch.cuda.synchronize()
    # blocks of every size an output or a workspace may have
    sizes = {t.numel() * t.element_size() for t in want}
    if name.startswith("attend"):
        sizes.add(setup[0].witcert_attend_workspace(0, {"images": [300, 300], "few": [30, 30], "tiny": [4, 4]}[name[7:]]))
    sizes = [s for s in sizes for _ in range(3)]
    torch.cuda.empty_cache()
    kept = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in sizes]
    held = [torch.full((s,), 7, dtype=torch.uint8, device="cuda") for s in sizes]
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)                         # about 0.2 s
    for k, h in zip(kept, held):
        k.copy_(h)
    del h, held
    got = flat(call(*setup, stream=side))
    torch.cuda.synchronize()
    for k in kept:
        assert (k == 7).all()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
