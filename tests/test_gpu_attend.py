"""Chunk attention over the compressed cache against float64.

The reference is softmax(q k^T / sqrt d) v in float64 over the oracle's reconstructed keys and
values, row by row.  Error bound of a row, from the roundings the entry point documents:
  * decoded keys rounded to fp16 (2^-11 relative, |k| here far below 65504; black-box keys are exact
    in bf16): a logit moves by at most d = 2^-11 sum_c |q_c k_c| / sqrt(128), queries are exact;
  * weights rounded to fp16 (2^-11) or, black box, bf16 (2^-8): with the logits' shift every weight,
    and the sum that divides, is within a factor exp(d) (1 + u) of exact;
  * values rounded to fp16 (2^-11); fp32 sums of at most 4096 terms (2^-24 x 4096 = 2^-12, never
    reached: sums of that length round to about 2^-20), taken as 2^-14;
  * the output's half step, 2^-8.
so |o - o64| <= (exp(2 d) (1 + u)^2 - 1 + 2^-11 + 2^-14) sum_t p_t |v_t| + 2^-8 |o|.
The 2-norm over all outputs is held tighter: independent roundings of 2^-8 / sqrt 3 (output) and, in
bf16, the same again (weights), with the rest below half of one: 4e-3 in all.
"""
import math

import numpy as np
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc
from oracle import OracleCache

from gpu_helpers import tensor_function

pytestmark = pytest.mark.gpu

SCHEMES = ["int8_dither", "fp8_e4m3", "kivi2", "int8_rtn", "blackbox"]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wc.load()


class Pair:
    """A GPU cache of ragged sequences and one oracle cache per sequence."""

    def __init__(self, scheme, hq, hkv, lens, seed=1, max_pages=0, **kw):
        self.scheme, self.hq, self.hkv, self.lens = scheme, hq, hkv, list(lens)
        B = len(lens)
        self.gpu = wc.Cache(1, hq, hkv, B, max(max(lens), 1) + 8, scheme, seed=seed, max_pages=max_pages, **kw)
        self.refs = [OracleCache(1, hq, hkv, 1, scheme, seed, 1) for _ in lens]
        g = torch.Generator().manual_seed(seed)
        K = torch.randn(sum(lens), hkv, 128, generator=g)
        K[..., 10:12] *= 6
        K, V = K.bfloat16(), torch.randn(sum(lens), hkv, 128, generator=g).bfloat16()
        hat = ()
        if scheme == "blackbox":
            hat = tuple(torch.from_numpy(tensor_function(x.float().numpy(), seed + i)).bfloat16() for i, x in enumerate((K, V)))
        self.gpu.witcert_write_ragged(0, K.cuda(), V.cuda(), self.lens, *(h.cuda() for h in hat))
        row = 0
        for i, n in enumerate(lens):
            if n:
                part = [x[row:row + n].float().numpy()[None] for x in (K, V) + hat]
                self.refs[i].write(0, *part)
            row += n

    def queries(self, n, seed=5, scale=1.5):
        g = torch.Generator().manual_seed(seed)
        return (scale * torch.randn(sum(n), self.hq, 128, generator=g)).bfloat16()

    def reference(self, q, n):
        """(o64, bound) [sum n, Hq, 128]."""
        q = q.double().numpy()
        o, bound = np.zeros(q.shape), np.zeros(q.shape)
        grp, u = self.hq // self.hkv, 2.0 ** -8 if self.scheme == "blackbox" else 2.0 ** -11
        row = 0
        for i, m in enumerate(n):
            s = self.lens[i]
            for h in range(self.hkv if m else 0):
                k, v = self.refs[i].group_view(0, i=0, h=h)[:2]
                k, v = np.asarray(k, np.float64)[:s], np.asarray(v, np.float64)[:s]
                seen = np.arange(s)[None] <= np.arange(s - m, s)[:, None]
                for j in range(h * grp, (h + 1) * grp):
                    x = q[row:row + m, j]
                    lg = np.where(seen, x @ k.T / math.sqrt(128), -np.inf)
                    p = np.exp(lg - lg.max(1, keepdims=True))
                    p /= p.sum(1, keepdims=True)
                    d = 0.0
                    if self.scheme != "blackbox":
                        d = (2.0 ** -11 * np.where(seen, np.abs(x) @ np.abs(k).T, 0) / math.sqrt(128)).max(1, keepdims=True)
                    o[row:row + m, j] = p @ v
                    rel = np.exp(2 * d) * (1 + u) ** 2 - 1 + 2.0 ** -11 + 2.0 ** -14
                    bound[row:row + m, j] = rel * (p @ np.abs(v)) + 2.0 ** -8 * np.abs(p @ v) + 1e-12
            row += m
        return o, bound

    def check(self, n, seed=5, scale=1.5):
        q = self.queries(n, seed, scale)
        got = self.gpu.attend(0, q.cuda(), n)
        assert got.dtype == torch.bfloat16 and got.shape == q.shape
        g = got.double().cpu().numpy()
        o, bound = self.reference(q, n)
        assert self.gpu.witcert_stats()["device_errors"] == 0
        assert np.isfinite(g).all()
        err = np.abs(g - o)
        assert np.all(err <= bound), (float((err / bound).max()), np.argwhere(err > bound)[:4])
        if o.size:
            assert np.linalg.norm(g - o) <= 4e-3 * np.linalg.norm(o)
        return got


@pytest.mark.parametrize("scheme", SCHEMES)
def test_small_tiles(scheme):
    """One token; a few; the edges of a 16-token block, a 128-token tile, 128 and 256 query rows."""
    for lens, n, hq, hkv in (([1], [1], 1, 1), ([5], [5], 2, 1), ([17], [3], 4, 2), ([127], [2], 7, 1),
                             ([128], [128], 1, 1), ([129], [128], 2, 2), ([130], [33], 8, 2), ([256], [256], 1, 1),
                             ([257], [129], 2, 1), ([300], [300], 7, 1)):
        Pair(scheme, hq, hkv, lens, seed=sum(lens)).check(n)


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("pages", [0, 120])
def test_ragged_batches(scheme, pages):
    p = Pair(scheme, 8, 2, [1, 300, 64, 0, 517, 130], max_pages=pages)
    for n in ([1, 4, 1, 0, 4, 3], [0, 300, 64, 0, 100, 0], [1, 0, 33, 0, 517, 32], [0, 0, 0, 0, 1, 0]):
        p.check(n)


@pytest.mark.parametrize("scheme", ["int8_dither", "blackbox"])
@pytest.mark.parametrize("hq,hkv", [(28, 4), (32, 4), (5, 5)])
def test_longer_contexts_are_split(scheme, hq, hkv):
    Pair(scheme, hq, hkv, [2000, 1111], seed=3).check([5, 2])
    Pair(scheme, hq, hkv, [1500], seed=4).check([70])


def test_more_sequences_than_a_launch_takes():
    lens = [1 + (37 * i) % 90 for i in range(150)]
    Pair("fp8_e4m3", 2, 1, lens).check([min(x, 1 + i % 40 * (i % 3)) for i, x in enumerate(lens)])


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed):
    """Lengths, chunk sizes, heads and stores at random: every kernel, cut and merge there is."""
    rng = np.random.default_rng(seed)
    B = int(rng.integers(1, 7))
    hkv, grp = int(rng.integers(1, 4)), int(rng.integers(1, 9))
    lens = [int(np.exp(rng.uniform(0, np.log(900)))) for _ in range(B)]
    # decodes, drafts, chunks and whole prompts side by side
    n = [min(s, int(rng.choice([0, 1, 1 + rng.integers(8), 1 + rng.integers(150), s]))) for s in lens]
    if not any(n):
        n[0] = 1
    scheme = SCHEMES[seed % 5]
    pages = int(rng.integers(2)) * (sum((s + 15) // 16 for s in lens) + 3)
    Pair(scheme, hkv * grp, hkv, lens, seed=seed, max_pages=pages, pos_offset=int(rng.integers(2)) * 16 if scheme != "int8_dither" else 0).check(n, seed)


@pytest.mark.parametrize("scale", [1e-3, 30.0])
def test_flat_and_sharp_weights(scale):
    """Nearly equal weights, and one key that takes all (rescaling, weights that vanish)."""
    Pair("fp8_e4m3", 4, 1, [700], seed=8).check([9], scale=scale)
    Pair("blackbox", 4, 1, [700], seed=8).check([200], scale=scale)


def test_rows_equal_the_single_token_decode():
    """Each row is what the decode gives when the sequence ends there (2e-3 of max |V|, the decode's
    own tolerance, plus this path's bound)."""
    p = Pair("int8_dither", 4, 2, [90], seed=6)
    n = 6
    q = p.queries([n])
    got = p.gpu.attend(0, q.cuda(), [n]).double().cpu().numpy()
    _, bound = p.reference(q, [n])
    vmax = np.abs(p.refs[0].v[0]).max()
    for j in range(n - 1, -1, -1):
        p.gpu.witcert_truncate(0, [90 - n + 1 + j])
        out, _ = p.gpu.decode(0, q[j:j + 1].cuda(), 1e-2, meters=False)
        assert np.all(np.abs(out.double().cpu().numpy()[0] - got[j]) <= bound[j] + 2e-3 * vmax)


def test_repaired_blocks_are_exact():
    p = Pair("fp8_e4m3", 4, 2, [200], seed=9, max_repair_blocks=64)
    q1 = p.queries([1])
    p.gpu.decode(0, q1.cuda(), 1e-2)
    p.gpu.witcert_gate(0, 0.0)
    assert p.gpu.witcert_gate_stats()["blocks_paged_in"] > 0
    slots = p.gpu.export(0, 8).cpu().numpy()              # [B, Hkv, nblk], -1 = not repaired
    p.refs[0].repaired[0] = (slots >= 0)
    p.check([40])


def test_hidden_keys_that_are_not_numbers():
    """A NaN key changes no row that does not see it."""
    K = torch.randn(1, 50, 1, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    q = torch.randn(10, 2, 128, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    outs = []
    for bad in (False, True):
        c = wc.Cache(1, 2, 1, 1, 64, "fp8_e4m3")
        K2 = K.clone()
        if bad:
            K2[:, 45] = float("nan")
        c.witcert_write(0, K2, K)
        outs.append(c.attend(0, q, [10]))
    assert torch.equal(outs[0][:5], outs[1][:5])          # positions 40 .. 44
    assert outs[1][5:].isnan().all()


def test_queries_of_any_magnitude():
    """Rows are scaled by powers of two: times 2^k in q and 2^-k in the keys changes nothing."""
    outs = []
    for k in (0, 60):
        c = wc.Cache(1, 2, 1, 1, 64, "blackbox")
        d = wc.Cache(1, 2, 1, 1, 64, "fp8_e4m3")
        K = torch.randn(1, 40, 1, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
        q = torch.randn(3, 2, 128, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
        c.witcert_write_hat(0, K, K, K * 2.0 ** -k, K)
        outs.append(c.attend(0, q * 2.0 ** k, [3]))
        d.witcert_write(0, K, K)
        tiny = d.attend(0, q * 2.0 ** -60, [3])           # all logits vanish: the mean of the visible values
        V = d.read(0, [40])[1].double()
        for j in range(3):
            want = V[:38 + j].mean(0)
            assert (tiny[j].double() - want).abs().max() <= 2.0 ** -8 * want.abs().max() + 2.0 ** -10
    assert torch.equal(outs[0], outs[1])


def test_attend_on_another_stream_and_twice():
    p = Pair("kivi2", 8, 2, [333, 40], seed=12)
    n = [33, 7]
    q = p.queries(n).cuda()
    first = p.gpu.attend(0, q, n)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = p.gpu.attend(0, q, n)
    side.synchronize()
    assert torch.equal(first, again)


def test_misaligned_buffers_are_refused():
    c = wc.Cache(1, 2, 1, 1, 64, "fp8_e4m3")
    flat = torch.zeros(64 * 128 + 64, dtype=torch.bfloat16, device="cuda")
    off = lambda n, rows, heads: flat[n:n + rows * heads * 128].view(rows, heads, 128)
    with pytest.raises(wc.WitcertError, match="aligned"):
        c.witcert_write(0, off(1, 5, 1)[None].view(1, 5, 1, 128), off(0, 5, 1).view(1, 5, 1, 128))
    assert c.witcert_length(0) == 0
    c.witcert_write(0, off(4, 5, 1).view(1, 5, 1, 128), off(0, 5, 1).view(1, 5, 1, 128))
    with pytest.raises(wc.WitcertError, match="aligned"):
        c.attend(0, off(8, 5, 2), [5])
    with pytest.raises(wc.WitcertError, match="aligned"):
        c.witcert_read(0, None, [5], off(0, 5, 1), off(4, 5, 1))
    assert c.attend(0, off(16, 5, 2), [5]).shape == (5, 2, 128)


def test_calls_can_be_captured():
    """A captured step (rotation and chunk attention) replays on new queries."""
    p = Pair("int8_dither", 8, 2, [400, 90], seed=13)
    n = [4, 3]
    rope, pos = wc.Rope(128), torch.arange(7, device="cuda")
    q = p.queries(n).cuda()
    out = torch.empty_like(q)
    ws = torch.empty(p.gpu.witcert_attend_workspace(0, n), dtype=torch.uint8, device="cuda")

    def step():
        p.gpu.witcert_attend(0, wc.witcert_rope(rope, pos, q), n, out, ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    q.copy_(p.queries(n, seed=99))
    g.replay()
    torch.cuda.synchronize()
    got = out.clone()
    step()
    assert torch.equal(got, out)


def test_refusals():
    c = wc.Cache(1, 4, 2, 2, 64, "fp8_e4m3")
    K = torch.zeros(2, 5, 2, 128, dtype=torch.bfloat16, device="cuda")
    c.witcert_write(0, K, K)
    q = torch.zeros(6, 4, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(wc.WitcertError, match="do not fit"):
        c.attend(0, q, [6, 0])
    with pytest.raises(wc.WitcertError, match="out of range"):
        c.attend(1, q, [3, 3])
    with pytest.raises(ValueError, match="shape"):
        c.attend(0, q, [3, 2])
    with pytest.raises(wc.WitcertError, match="workspace needs"):
        c.witcert_attend(0, q, [3, 3], torch.empty_like(q), torch.empty(64, dtype=torch.uint8, device="cuda"))
    f = wc.Cache(1, 4, 2, 2, 64, "fp8_e4m3", dtype=torch.float32)
    with pytest.raises(wc.WitcertError, match="bf16"):
        f.attend(0, q, [0, 0])
    assert c.attend(0, q[:0], [0, 0]).shape == (0, 4, 128)
