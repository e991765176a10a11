"""Sequences that take each other's state, against caches that are written at once.

Random histories (test_gpu_histories) with forks among them: any map of the sequences in place, cut to
any lengths, over shared and copied pages.  Reads and chunk attention must be those of a cache written
with the tokens held, to the bit.  Then the page pool's accounting, long cycles, and refusals."""
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc
from kv_cache_quantization_witcert_gb300 import _lib

from test_gpu_histories import SCHEMES, History

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wc.load()


class ForkHistory(History):
    def fork(self):
        r, B = self.r, self.B
        kind = r.choice(["any", "any", "swap", "prompt", "cycle", "empty", "cut"])
        parents = list(range(B))
        if kind == "any":
            parents = [r.randrange(B) for _ in range(B)]
        elif kind == "swap":
            r.shuffle(parents)
        elif kind == "prompt":
            parents = [r.randrange(B)] * B
        elif kind == "cycle":
            parents = parents[1:] + parents[:1]
        elif kind == "empty":
            parents = [r.choice([p, p, -1]) for p in parents]
        lengths = None
        if kind == "cut" or r.random() < 0.4:
            lengths = []
            for p in parents:
                now = [self.lens(x)[p] if p >= 0 else 0 for x in range(self.L)]
                t = max(0, r.choice([min(now), max(now), max(now) + 5]) - r.choice([0, 0, 1, 2, 17, 40]))
                if self.scheme == "kivi2" and any(t < m and t % 16 and t // 16 < m // 16 for m in now):
                    t = t // 16 * 16
                lengths.append(t)
        self.cache.witcert_fork(parents, lengths)
        for layer in self.held:
            old = list(layer)
            for i, p in enumerate(parents):
                src = old[p] if p >= 0 else [a[:0] for a in old[i]]
                layer[i] = [a[:lengths[i]] for a in src] if lengths else list(src)


@pytest.mark.parametrize("seed", range(60))
def test_random_histories(seed):
    h = ForkHistory(seed)
    for _ in range(40):
        layer = h.r.randrange(h.L)
        what = h.r.choice(["append"] * 5 + ["fork"] * 5 + ["truncate", "truncate all", "reset", "dropped", "compare"])
        if what == "append":
            h.append(layer)
        elif what == "fork":
            h.fork()
        elif what == "truncate":
            h.truncate(layer)
        elif what == "truncate all":
            h.truncate(-1)
        elif what == "reset" and h.r.random() < 0.4:
            h.reset()
        elif what == "dropped":
            h.dropped(layer)
        else:
            h.compare(layer)
    for layer in range(h.L):
        h.compare(layer)
    assert h.cache.witcert_stats()["device_errors"] == 0


def rows(n, heads=2, dtype=torch.bfloat16):
    return torch.randn(n, heads, 128, device="cuda").to(dtype)


def write(c, layer, n, k=None, v=None):
    k, v = rows(sum(n)) if k is None else k, rows(sum(n)) if v is None else v
    c.witcert_write_ragged(layer, k, v, n, *((k, v) if c.cfg.scheme == _lib.BLACKBOX else ()))
    return k, v


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scheme", SCHEMES)
def test_everything_a_sequence_has(scheme, dtype):
    """Codes, scales, witnesses and the unfinished block's exact keys, of fp32 caches too."""
    torch.manual_seed(3)
    c = wc.Cache(2, 4, 2, 4, 100, scheme, dtype=dtype, seed=5, v_witness=True)
    hat = scheme == "blackbox"
    for layer in range(2):
        k, v = rows(4 * 39, dtype=dtype).view(4, 39, 2, 128), rows(4 * 39, dtype=dtype).view(4, 39, 2, 128)
        (c.witcert_write_hat(layer, k, v, k / 2, v / 2) if hat else c.witcert_write(layer, k, v))
    kinds = [_lib.X_K_CODES, _lib.X_V_CODES, _lib.X_WITNESS, _lib.X_V_WITNESS]
    kinds += {"int8_dither": [_lib.X_K_SCALES, _lib.X_V_SCALES], "int8_rtn": [_lib.X_K_SCALES, _lib.X_V_SCALES],
              "kivi2": [_lib.X_V_SCALES, _lib.X_V_ZEROS, _lib.X_KIVI_K_SCALE, _lib.X_KIVI_K_ZERO]}.get(scheme, [])
    look = lambda: [c.export(layer, kind) for layer in range(2) for kind in kinds] + \
        [x.view(4, 39, 2, 128) for layer in range(2) for x in c.read(layer, [39] * 4)]
    before = look()
    parents = [2, 0, 1, 0]
    c.witcert_fork(parents)
    for a, b in zip(before, look()):
        assert torch.equal(a[parents].view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("scheme", SCHEMES)
def test_pages_are_shared_until_written(scheme):
    c = wc.Cache(2, 4, 2, 4, 160, scheme, seed=1, max_pages=12)
    used = lambda: c.witcert_stats()["pages_used"]
    k, v = zip(*(write(c, layer, [67, 0, 0, 0]) for layer in range(2)))
    assert used() == 5
    c.witcert_fork([0, 0, 0, 0])
    assert used() == 5 and [c.witcert_seq_length(1, i) for i in range(4)] == [67] * 4
    new = [rows(3), rows(3)]
    write(c, 0, [0, 1, 1, 1], new[0], new[0])
    assert used() == 8                                         # three copies of the last block; sequence 0 keeps it
    write(c, 1, [0, 1, 1, 1], new[1], new[1])
    assert used() == 8
    # 12 pages: the pool has four left, and a whole new block for each of the four and one more fails
    before = [[x.clone() for x in c.read(layer, [67, 68, 68, 68])] for layer in range(2)]
    with pytest.raises(wc.WitcertError) as e:
        write(c, 0, [30, 13, 13, 13])                          # 0: blocks 5 and 6; the others one each
    assert e.value.status == _lib.ENOMEM and used() == 8
    for layer in range(2):
        assert all(torch.equal(a, b) for a, b in zip(before[layer], c.read(layer, [67, 68, 68, 68])))
    c.witcert_fork([0, -1, -1, 0], [64, 0, 0, 66] if scheme != "kivi2" else [64, 0, 0, 64])
    assert used() == (5 if scheme != "kivi2" else 4)
    c.witcert_reset_sequence(3)
    assert used() == 4
    c.witcert_fork([-1] * 4)
    assert used() == 0 and [c.witcert_length(layer) for layer in range(2)] == [0, 0]
    write(c, 0, [100, 0, 80, 0])                               # every page can be taken again
    assert used() == 12


def test_exhausted_pool_keeps_the_sharing():
    """An append that needs copies of shared blocks and fails leaves them shared and whole."""
    c = wc.Cache(1, 4, 2, 3, 64, "fp8_e4m3", max_pages=3)
    write(c, 0, [20, 0, 0])
    c.witcert_fork([0, 0, 0])
    want = [x.clone() for x in c.read(0, [20] * 3)]
    with pytest.raises(wc.WitcertError) as e:
        write(c, 0, [1, 1, 1])                                 # two copies; the pool has one page
    assert e.value.status == _lib.ENOMEM and c.witcert_stats()["pages_used"] == 2
    assert all(torch.equal(a, b) for a, b in zip(want, c.read(0, [20] * 3)))
    write(c, 0, [0, 1, 0])                                     # one copy fits
    assert c.witcert_stats()["pages_used"] == 3
    got = c.read(0, [20] * 3, [0] * 3)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_cut_pages_go_back():
    c = wc.Cache(1, 4, 2, 2, 100, "int8_rtn", max_pages=14)
    k, v = write(c, 0, [100, 90])
    c.witcert_truncate(0, [40, 90])
    assert c.witcert_stats()["pages_used"] == 13
    c.witcert_fork([0, 1], [40, 90])                           # nothing to cut but the pages behind
    assert c.witcert_stats()["pages_used"] == 9
    c.witcert_fork([0, 1], [40, 17])
    assert c.witcert_stats()["pages_used"] == 5
    want = wc.Cache(1, 4, 2, 2, 100, "int8_rtn")
    write(want, 0, [40, 17], torch.cat([k[:40], k[100:117]]), torch.cat([v[:40], v[100:117]]))
    assert all(torch.equal(a, b) for a, b in zip(c.read(0, [40, 17]), want.read(0, [40, 17])))


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("ragged", [False, True])
def test_more_moves_than_a_launch_holds(paged, ragged):
    """A cycle of 700 sequences, then a fan out of one of them with chains behind it."""
    B, g = 700, torch.Generator().manual_seed(2)
    c = wc.Cache(1, 2, 1, B, 32, "int8_rtn", max_pages=2 * B if paged else 0)
    n = [17 + i % 3 if ragged else 18 for i in range(B)]
    k, v = rows(sum(n), 1), rows(sum(n), 1)
    c.witcert_write_ragged(0, k, v, n)
    held = list(zip(*(x.split(n) for x in c.read(0, n))))
    perm = torch.randperm(B, generator=g).tolist()
    cycle = [0] * B
    for a, b in zip(perm, perm[1:] + perm[:1]):
        cycle[a] = b
    chains = [max(0, i - 1) if i % 5 else 3 for i in range(B)]
    for parents in (cycle, chains, [(i + 1) % B for i in range(B)]):
        c.witcert_fork(parents)
        held = [held[p] for p in parents]
        n = [n[p] for p in parents]
        assert [c.witcert_seq_length(0, i) for i in range(B)] == n
        got = c.read(0, n)
        assert torch.equal(got[0], torch.cat([a for a, _ in held])) and torch.equal(got[1], torch.cat([b for _, b in held]))


def test_other_sequences_and_rows_behind_stay():
    """A fork touches nothing but the blocks it fills: sequences that stay, and rows past the longer of the two."""
    c = wc.Cache(1, 2, 1, 3, 64, "fp8_e4m3")
    c.witcert_write(0, *(rows(3 * 60, 1).view(3, 60, 1, 128) for _ in range(2)))
    before = c.export(0, _lib.X_K_CODES)
    c.witcert_fork([0, 0, 2], [60, 20, 60])
    after = c.export(0, _lib.X_K_CODES)
    assert torch.equal(before[[0, 2]], after[[0, 2]])
    assert torch.equal(after[1, :20], before[0, :20]) and torch.equal(after[1, 32:], before[1, 32:])


def test_on_a_stream():
    """A fork on another stream follows that stream's writes and precedes its decodes."""
    s = torch.cuda.Stream()
    c = wc.Cache(2, 4, 2, 4, 4096, "int8_dither", seed=3)
    q = torch.randn(4, 4, 128, device="cuda").bfloat16()
    k, v = (rows(4 * 4000).view(4, 4000, 2, 128) for _ in range(2))
    torch.cuda.synchronize()
    outs = []
    with torch.cuda.stream(s):
        for layer in range(2):
            c.witcert_write(layer, k, v)
        for parents in ([1, 0, 3, 2], [1, 0, 3, 2], [0, 0, 0, 0]):
            c.witcert_fork(parents)
            outs.append(c.decode(1, q, 1e-2, meters=False)[0])
    s.synchronize()
    want = wc.Cache(2, 4, 2, 4, 4096, "int8_dither", seed=3)
    for out, order in zip(outs, ([1, 0, 3, 2], [0, 1, 2, 3], [0, 0, 0, 0])):
        want.witcert_truncate(1, [0] * 4)
        want.witcert_write(1, k[order].contiguous(), v[order].contiguous())
        assert torch.equal(out, want.decode(1, q, 1e-2, meters=False)[0])


def test_refusals():
    c = wc.Cache(1, 4, 2, 3, 64, "kivi2")
    write(c, 0, [40, 33, 5])
    want = [x.clone() for x in c.read(0, [40, 33, 5])]
    for parents, lengths in (([0, 1, 3], None), ([0, -2, 1], None), ([0, 1, 2], [40, -1, 5]), ([0, 1, 2], [31, 33, 5]),
                             ([0, 0, 2], [40, 20, 5])):
        with pytest.raises(wc.WitcertError) as e:
            c.witcert_fork(parents, lengths)
        assert e.value.status == _lib.EINVAL
    assert all(torch.equal(a, b) for a, b in zip(want, c.read(0, [40, 33, 5])))
    c.witcert_fork([0, 0, 0], [32, 33, 40])
    got = c.read(0, [32, 33, 40])[1].split([32, 33, 40])
    assert all(torch.equal(x, want[1][:len(x)]) for x in got)
    gated = wc.Cache(1, 4, 2, 2, 64, "fp8_e4m3", max_repair_blocks=8)
    with pytest.raises(wc.WitcertError, match="gated") as e:
        gated.witcert_fork([0, 0])
    assert e.value.status == _lib.EINVAL


def test_a_fork_is_not_captured():
    c = wc.Cache(1, 4, 2, 2, 64, "fp8_e4m3")
    k = rows(40)
    write(c, 0, [20, 20], k, k)
    want = [x.clone() for x in c.read(0, [20, 20])]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x = k + 1
        with pytest.raises(wc.WitcertError, match="captured") as e:
            c.witcert_fork([1, 0])
    assert e.value.status == _lib.ESTATE and x.shape == k.shape
    assert all(torch.equal(a, b) for a, b in zip(want, c.read(0, [20, 20])))
    c.witcert_fork([1, 0])
    assert all(torch.equal(a, b.view(2, 20, 2, 128).flip(0).flatten(0, 1)) for a, b in zip(want, c.read(0, [20, 20])))


@pytest.mark.parametrize("pages", [0, 8 * 8200])
def test_stores_beyond_32_bits(pages):
    """4.5 GB: the last rows of every sequence, forked, shared and appended to."""
    B, S, H = 8, 131000, 8
    c = wc.Cache(1, H, H, B, S + 8, "blackbox", max_pages=pages)
    n = [S - 7 * i for i in range(B)]
    for i in range(B):
        m = [0] * B
        m[i] = n[i]
        k = torch.randn(n[i], H, 128, device="cuda").bfloat16()
        c.witcert_write_ragged(0, k, k, m, k, k)
    at = lambda lens: [x - 40 for x in lens]
    last = [x.split(40) for x in c.read(0, [40] * B, at(n))]
    parents = [7, 5, 1, 0, 2, 3, 4, 0]
    c.witcert_fork(parents)
    n = [n[p] for p in parents]
    new = torch.randn(B, H, 128, device="cuda").bfloat16()
    c.witcert_write_ragged(0, new, new, [1] * B, new, new)
    for got, want in zip(c.read(0, [41] * B, at(n)), last):
        assert torch.equal(got, torch.cat([x for i, p in enumerate(parents) for x in (want[p], new[i:i + 1])]))
