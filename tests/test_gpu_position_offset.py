"""A cache whose first token stands at pos_offset: the dithered store's values.

The dither is counted by the token's global position, so the value is s (code - xi(pos_offset + t)).
Reads and every way of the chunk attention (the dither formed where it is used, formed once for several
sequences, operand images) are held against the float64 store, with test_gpu_attend's bound."""
import numpy as np
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc
from oracle.philox import dither
from oracle.quant import write_int8_dither

import test_gpu_attend as base

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wc.load()


class Store:
    """One sequence's keys and values [1, n, Hkv, 128] through the oracle's quantizer at its positions."""

    def __init__(self, K, V, seed, offset):
        self.kv = []
        for tensor, x in enumerate((K, V)):
            pos = np.arange(offset, offset + x.shape[1])
            self.kv.append(np.stack([write_int8_dither(x[0, :, h], dither(seed, 0, h, pos, tensor))[2]
                                     for h in range(x.shape[2])], 1))

    def group_view(self, layer, i, h):
        return self.kv[0][:, h], self.kv[1][:, h]


class Pair(base.Pair):
    def __init__(self, hq, hkv, lens, offset, seed=21, **kw):
        super().__init__("int8_dither", hq, hkv, lens, seed=seed, pos_offset=offset, **kw)
        g = torch.Generator().manual_seed(seed)            # the inputs that the base class drew
        K = torch.randn(sum(lens), hkv, 128, generator=g)
        K[..., 10:12] *= 6
        K, V = K.bfloat16().float().numpy(), torch.randn(sum(lens), hkv, 128, generator=g).bfloat16().float().numpy()
        at = np.cumsum([0] + lens)
        self.refs = [Store(K[None, a:b], V[None, a:b], seed, offset) for a, b in zip(at, at[1:])]


OFFSETS = [16, 1000, 5, 3 << 20]


@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_reads(offset, dtype):
    n, hkv, seed = 70, 2, 33
    g = torch.Generator().manual_seed(offset)
    K, V = (torch.randn(1, n, hkv, 128, generator=g).to(dtype) for _ in range(2))
    c = wc.Cache(1, hkv, hkv, 1, 80, "int8_dither", dtype=dtype, seed=seed, pos_offset=offset)
    c.witcert_write(0, K.cuda(), V.cuda())
    ref = Store(K.float().numpy(), V.float().numpy(), seed, offset)
    half = torch.finfo(dtype).eps / 2
    for t0, m in ((0, n), (17, 30), (n - 1, 1)):
        for got, want in zip(c.read(0, [m], [t0]), ref.kv):
            want = want[t0:t0 + m]
            # fp32 roundings of code - xi and of its product with s (|x| <= 6 here), then half a step
            err = np.abs(got.double().cpu().numpy() - want)
            assert np.all(err <= half * np.abs(want) * (1 + 2.0 ** -20) + 3 * 2.0 ** -24 * 6)


@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("pages", [0, 80])
@pytest.mark.parametrize("lens,n", [([300], [4]),                      # up to 32 rows, its own dither
                                    ([300], [30]),                     # up to 128 rows
                                    ([300, 290, 17], [4, 3, 2]),       # a dither shared by the sequences
                                    ([300, 290, 180], [30, 40, 20]),
                                    ([300], [200]),                    # images, their own dither
                                    ([300, 290], [200, 99])])          # images, shared
def test_chunk_attention(offset, pages, lens, n):
    Pair(8, 2, lens, offset, max_pages=pages).check(n)
