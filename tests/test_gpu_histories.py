"""Random histories of a cache against caches that are written at once.

Appends of every kind, truncations, resets and dropped tokens that are not numbers, in any order, leave
what one ragged append of the tokens still held stores: reads and chunk attention to the bit (same codes,
same plan), decodes up to the order of their sums (splits follow the batch's history): 2^-13 of the largest
output and 2e-4 of a meter."""
import random

import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc

pytestmark = pytest.mark.gpu

SCHEMES = ["int8_dither", "fp8_e4m3", "kivi2", "int8_rtn", "blackbox"]


class History:
    def __init__(self, seed):
        self.r = r = random.Random(seed)
        torch.manual_seed(seed)
        self.scheme, self.L, self.B = SCHEMES[seed % 5], r.randint(1, 3), r.randint(1, 5)
        self.hkv, self.grp, self.cap = r.choice([1, 2, 4]), r.choice([1, 2, 4, 7]), r.choice([40, 130, 400, 900])
        self.off = r.choice([0, 16, 1000])
        self.kw = dict(seed=seed, pos_offset=self.off, v_witness=r.random() < 0.5,
                       max_pages=self.B * ((self.cap + 15) // 16) * r.randint(0, 1))
        self.cache, self.rope = self.make(), wc.Rope(128, interleaved=r.random() < 0.5)
        none = torch.empty(0, self.hkv, 128, dtype=torch.bfloat16, device="cuda")
        # keys as the cache takes them in, values, and the tensor function's keys
        self.held = [[[none, none, none] for _ in range(self.B)] for _ in range(self.L)]

    def make(self):
        return wc.Cache(self.L, self.hkv * self.grp, self.hkv, self.B, self.cap, self.scheme, **self.kw)

    def lens(self, layer):
        return [x[0].shape[0] for x in self.held[layer]]

    def hats(self, k, v):
        return ((k.float() * 0.984375).bfloat16(), (v.float() * 0.984375).bfloat16()) if self.scheme == "blackbox" else ()

    def append(self, layer):
        r, lens = self.r, self.lens(layer)
        room = [self.cap - x for x in lens]
        n = [min(x, r.choice([0, 0, 1, r.randint(0, 70), x if r.random() < 0.15 else 0])) for x in room]
        uniform = r.random() < 0.4
        if uniform:
            n = [min(room + [r.choice([1, 1, r.randint(0, 40), 300])])] * self.B
        k, v = (torch.randn(sum(n), self.hkv, 128, device="cuda").bfloat16() * s for s in (2, 1))
        h, turn = self.hats(k, v), r.random() < 0.5
        if uniform:
            k4, v4, *h4 = (x.view(self.B, n[0], self.hkv, 128) for x in (k, v) + h)
            if turn:
                self.cache.witcert_write_rope(layer, k4, v4, self.rope, *h4)
            else:
                (self.cache.witcert_write_hat if h else self.cache.witcert_write)(layer, k4, v4, *h4)
        elif turn:
            self.cache.witcert_write_rope_ragged(layer, k, v, n, self.rope, *h)
        else:
            self.cache.witcert_write_ragged(layer, k, v, n, *h)
        kh = h[0] if h else k
        if turn:
            pos = torch.cat([torch.arange(a, a + m) for a, m in zip(lens, n)]).cuda() + self.off
            k, kh = wc.witcert_rope(self.rope, pos, k), wc.witcert_rope(self.rope, pos, kh)
        for i, part in enumerate(zip(k.split(n), v.split(n), kh.split(n))):
            self.held[layer][i] = [torch.cat(x) for x in zip(self.held[layer][i], part)]

    def truncate(self, layer):
        r = self.r
        layers = range(self.L) if layer < 0 else [layer]
        to = []
        for i in range(self.B):
            now = [self.lens(x)[i] for x in layers]
            t = max(0, min(now) - r.choice([0, 0, 1, 2, 5, 17, 40]))
            if self.scheme == "kivi2" and any(t < m and t % 16 and t // 16 < m // 16 for m in now):
                t = t // 16 * 16
            to.append(t)
        self.cache.witcert_truncate(layer, to)
        for x in layers:
            self.held[x] = [[a[:t] for a in seq] for seq, t in zip(self.held[x], to)]

    def reset(self):
        i = self.r.randrange(self.B)
        self.cache.witcert_reset_sequence(i)
        for layer in self.held:
            layer[i] = [a[:0] for a in layer[i]]

    def dropped(self, layer):
        """A token that is not a number, appended to some sequences and dropped again."""
        lens = self.lens(layer)
        n = [int(x < self.cap and (self.scheme != "kivi2" or x % 16 < 15) and self.r.random() < 0.7) for x in lens]
        if any(n):
            x = torch.full((sum(n), self.hkv, 128), float(self.r.choice(["nan", "inf", "-inf", "1e30"])), device="cuda").bfloat16()
            self.cache.witcert_write_ragged(layer, x, x, n, *((x, x) if self.scheme == "blackbox" else ()))
            self.cache.witcert_truncate(layer, lens)

    def compare(self, layer):
        r, lens, c = self.r, self.lens(layer), self.cache
        assert [c.witcert_seq_length(layer, i) for i in range(self.B)] == lens
        if not any(lens):
            return
        want = self.make()
        k, v, kh = (torch.cat(x) for x in zip(*self.held[layer]))
        want.witcert_write_ragged(layer, k, v, lens, *((kh, self.hats(k, v)[1]) if self.scheme == "blackbox" else ()))
        n = [r.randint(0, x) for x in lens]
        t0 = [r.randint(0, x - m) for x, m in zip(lens, n)]
        for a, b in zip(c.read(layer, n, t0), want.read(layer, n, t0)):
            assert torch.equal(a, b)
        n = [min(x, r.choice([0, 1, 4, r.randint(0, 60), x])) for x in lens]
        q = torch.randn(sum(n), self.hkv * self.grp, 128, device="cuda").bfloat16()
        a, b = c.attend(layer, q, n), want.attend(layer, q, n)
        assert torch.equal(a, b) and a.isfinite().all()
        q = torch.randn(self.B, self.hkv * self.grp, 128, device="cuda").bfloat16()
        (a, ma), (b, mb) = c.decode(layer, q, 1e-2), want.decode(layer, q, 1e-2)
        assert (a - b).abs().max() <= 2.0 ** -13 * max(1.0, b.abs().max().item())
        for name in ma:
            if self.scheme == "int8_dither" or not name.endswith("_b"):
                assert ((ma[name] - mb[name]).abs() <= 2e-4 * mb[name] + 2.0 ** -99).all(), name
        want.close()


@pytest.mark.parametrize("seed", range(40))
def test_random_histories(seed):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    h = History(seed)
    for _ in range(40):
        layer = h.r.randrange(h.L)
        what = h.r.choice(["append"] * 6 + ["truncate"] * 2 + ["truncate all", "reset", "dropped", "dropped", "compare", "compare"])
        if what == "append":
            h.append(layer)
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
