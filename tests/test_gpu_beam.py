"""Beam selections and paths against plain implementations in 64 bits.

A candidate's score is score + x - lse.  The kernel's lse differs from log sum exp x by what its fp32 terms
round: the argument (x - m) log2 e of an exponential by two half steps of itself, the exponential by 2^-22 (the
unit's documented error, 2^-22.5, and the sum's steps), so the sum by a factor of 1 + 2^-22 + 2^-23 E|x - m|, where
E|x - m| over the softmax is at most log V + 1 (the entropy, and the largest term's share); merging the lanes' and
parts' sums is three more such factors, each below 2^-21 of what it scales, and a sum of 32 + 8 terms: 2^-19.
Scores come back in fp32: half a step of |s|.  So scores are off by at most
    TOL = 2^-18 + 2^-23 (log V + 1) + 2^-24 |s|.
Two candidates of different rows closer than twice that may change places; those of one row may not: they are
ordered by their logits and, among equal ones, by token, exactly.  `check` holds the kernel to both."""
import math

import numpy as np
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc

pytestmark = pytest.mark.gpu

INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wc.load()


def check(x, scores, got, n, done=None, eos=-1):
    """x [R, W, V], scores [R, W]: the selection in 64 bits, request by request."""
    out_s, rows, tokens, ended = (t.cpu().numpy() for t in got)
    R, W, V = x.shape
    x64, sc = x.double().cpu().numpy(), scores.double().cpu().numpy()
    done = np.zeros((R, W), bool) if done is None else done.cpu().numpy()
    assert out_s.shape == rows.shape == tokens.shape == ended.shape == (R, n)
    for r in range(R):
        offers, best = {}, []
        for w in range(W):
            if not np.isfinite(sc[r, w]):
                continue
            if done[r, w]:
                offers[w] = [(sc[r, w], eos)]
            else:
                row = x64[r, w]
                m = row.max() if not np.isnan(row).any() else np.nan
                if not np.isfinite(m):
                    continue
                # in this order nothing is lost next to a maximum of any size
                c = sc[r, w] - math.log(np.exp(row - m).sum())
                first = np.lexsort((np.arange(V), -row))[:n]
                offers[w] = [(c + (row[t] - m), int(t)) for t in first if row[t] > -INF]
            best += [s for s, _ in offers[w]]
        best = sorted(best, reverse=True)[:n]
        taken = dict.fromkeys(offers, 0)
        for k in range(n):
            if k >= len(best):
                assert rows[r, k] == -1 and tokens[r, k] == -1 and out_s[r, k] == -INF and not ended[r, k]
                continue
            w = rows[r, k] - r * W
            s, t = offers[w][taken[w]]                     # a row's candidates come in its own order
            taken[w] += 1
            assert tokens[r, k] == t, (r, k, w)
            tol = 2.0 ** -18 + 2.0 ** -23 * (math.log(V) + 1) + 2.0 ** -24 * abs(s)
            assert abs(out_s[r, k] - s) <= tol, (r, k, out_s[r, k], s)
            assert abs(s - best[k]) <= 2 * tol, (r, k, s, best[k])
            assert ended[r, k] == (done[r, w] or t == eos)
    return out_s, rows, tokens


def inputs(R, W, V, dt=torch.bfloat16, seed=0, scale=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (scale * torch.randn(R, W, V, generator=g, device="cuda")).to(dt)
    return x, -5.0 + 2.0 * torch.randn(R, W, generator=g, device="cuda")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R, W, V, n", [(1, 1, 1, 1), (1, 1, 1, 5), (3, 2, 1, 2), (1, 4, 15, 8), (2, 3, 17, 64), (1, 1, 511, 1),
                                        (2, 4, 512, 4), (2, 4, 513, 8), (1, 5, 4097, 10), (7, 3, 1000, 3), (1, 1, 32000, 1),
                                        (2, 8, 50001, 16), (1, 32, 9999, 64), (1, 128, 700, 256), (40, 4, 2050, 8), (1, 2, 152001, 256),
                                        (1, 128, 3, 256)])
def test_sizes(R, W, V, n, dt):
    x, s = inputs(R, W, V, dt, seed=V)
    check(x, s, wc.witcert_beam_select(x, s, n), n)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lay", ["offset", "padded", "beams first", "broadcast", "reversed rows"])
def test_strides(lay, dt):
    R, W, V, n = 3, 4, 3001, 8
    if lay == "offset":
        flat, s = inputs(1, 1, R * W * V + 1, dt)[0].flatten(), inputs(R, W, 1)[1]
        x = flat[1:].view(R, W, V)
    elif lay == "padded":
        x, s = inputs(R, W, V + 7, dt)
        x = x[..., 3:V + 3]
    elif lay == "beams first":
        x, s = inputs(W, R, V, dt)
        x, s = x.transpose(0, 1), s.t().contiguous()
    elif lay == "broadcast":
        x, s = inputs(R, 1, V, dt)
        x, s = x.expand(R, W, V), inputs(R, W, 1)[1]
    else:
        x, s = inputs(2 * R, 2 * W, V, dt)
        x, s = x[::2, ::2], s[::2, ::2].contiguous()
    check(x, s, wc.witcert_beam_select(x, s, n), n)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_masks(dt):
    """Allowed tokens few or in one place, rows with nothing left, the type's lowest value as a mask."""
    R, W, V, n = 9, 4, 20000, 8
    x, s = inputs(R, W, V, dt)
    low = torch.finfo(dt).min
    at = torch.arange(V, device="cuda")
    x[0, 1] = -INF                                          # a beam with nothing left
    x[1] = -INF                                             # a request with nothing left
    x[2] = x[2].masked_fill(at % 5000 != 17, -INF)          # four tokens a beam
    x[3] = x[3].masked_fill((at < 7000) | (at >= 7003), -INF)
    x[4, 2] = low                                           # a whole row of the lowest value is a uniform row
    x[5] = x[5].masked_fill(at % 100 != 3, low)
    x[6, :, 1:] = -INF                                      # one token
    x[7] = -INF
    x[7, 3, V - 1] = low
    x[8] = x[8].masked_fill(at >= 600, -INF)
    check(x, s, wc.witcert_beam_select(x, s, n), n)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_not_numbers(dt):
    """Rows that have no softmax, and absent beams whose logits are anything, do not touch the others."""
    R, W, V, n = 6, 4, 5000, 8
    x, s = inputs(R, W, V, dt)
    want = check(x[:, 2:], s[:, 2:], wc.witcert_beam_select(x[:, 2:], s[:, 2:].contiguous(), n), n)
    for k, bad in enumerate((math.nan, INF, -INF)):
        x[k, 0] = bad
        x[k, 1, 4000 + k] = bad if bad > -INF or bad != bad else math.nan
    x[3, :2], s[3, :2] = math.nan, -INF
    x[4, :2], s[4, 0], s[4, 1] = INF, INF, math.nan
    s[5, :2] = -INF
    got = wc.witcert_beam_select(x, s, n)
    out = check(x, s, got, n)
    assert np.array_equal(out[0], want[0]) and np.array_equal(out[2], want[2])
    assert np.array_equal(out[1], want[1] + 2 * np.arange(R)[:, None] + 2)
    s[:] = -INF
    assert (wc.witcert_beam_select(x, s, n)[1] == -1).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["zeros", "zeros of both signs", "two values", "ascending", "descending", "steps", "rows alike", "one chunk"])
def test_ties_and_orders(kind, dt):
    """Equal logits go by token, equal scores by row: more of them than the lists hold."""
    R, W, V, n = 2, 3, 120001, 24
    x, s = inputs(R, W, V, dt)
    at = torch.arange(V, device="cuda")
    if kind == "zeros":
        x, s = torch.zeros_like(x), torch.full_like(s, -1.5)
    elif kind == "zeros of both signs":
        x, s = torch.where(at % 3 == 0, 0.0, -0.0).expand(R, W, V).to(dt), torch.zeros_like(s)
    elif kind == "two values":
        x, s = (at % 2).float().expand(R, W, V).to(dt), torch.zeros_like(s)
    elif kind == "ascending":
        x = (at / V * 8).expand(R, W, V).to(dt)
    elif kind == "descending":
        x = (-at / V * 8).expand(R, W, V).to(dt)
    elif kind == "steps":
        x = torch.div(at, 9000, rounding_mode="floor").float().expand(R, W, V).to(dt)
    elif kind == "rows alike":
        x, s = x[:, :1].expand(R, W, V), torch.full_like(s, -2.0)
    else:
        x = x.clone()
        x[..., 60000:60512] += 30
    got = wc.witcert_beam_select(x, s, n)
    rows, tokens = check(x, s, got, n)[1:]
    if kind in ("zeros", "zeros of both signs"):
        assert (tokens == np.arange(n)).all() and (rows == np.arange(R)[:, None] * W).all()
    if kind == "rows alike":            # the rows' sums are the same to the bit: by logit, then row, then token
        for r in range(R):
            v = x[r].float().cpu().numpy().ravel()
            order = np.argsort(-v, kind="stable")[:n]
            assert (rows[r] == r * W + order // V).all() and (tokens[r] == order % V).all()


@pytest.mark.parametrize("R, W, V, n", [(2, 4, 140001, 200), (1, 64, 40000, 128), (2, 8, 131072, 16), (1, 32, 50001, 64), (3, 16, 9000, 44),
                                        (1, 2, 1500, 256)])
@pytest.mark.parametrize("kind", ["equal", "mask", "levels"])
def test_many_alike(R, W, V, n, kind):
    """More equal or nearly equal keys than any list holds, at both stages, by chunks' and rows' order and by halving."""
    x, s = inputs(R, W, V)
    if kind == "equal":
        x, s = torch.full_like(x, 0.25), torch.full_like(s, -3.0)
    elif kind == "mask":                                    # the type's lowest value everywhere but in a few places
        keep = torch.rand(x.shape, device="cuda") < 4 / V
        x = x.masked_fill(~keep, torch.finfo(x.dtype).min)
    else:                                                   # a few distinct values, rows that start alike
        x, s = x.round().clamp(-2, 2), s.round()
    check(x, s, wc.witcert_beam_select(x, s, n), n)


@pytest.mark.parametrize("V, n", [(900, 4), (120001, 24), (140001, 200)])
def test_logits_that_the_score_does_not_tell_apart(V, n):
    """Next to a score of -1e12 (2^-13 apart in 64 bits) logits 1e-7 apart vanish, but still order their row."""
    x, s = inputs(1, 3, V, torch.float32, scale=1e-3)
    s.fill_(-1e12)
    x[0, 0, 5:400] = 0.5 + 1e-7 * (torch.arange(395, device="cuda") // 2)     # pairs of equal ones among them
    rows, tokens = (t[0].cpu().numpy() for t in wc.witcert_beam_select(x, s, n)[1:3])
    order = np.lexsort((np.arange(V), -x[0, 0].cpu().numpy()))[:n]
    assert (rows == 0).all() and (tokens == order).all()


@pytest.mark.parametrize("size", [1e4, 1e20, 3e38])
def test_far_apart(size):
    """Scores and logits of any size: what 32 bits cannot tell apart, 64 do."""
    x, s = inputs(2, 4, 5000, torch.float32)
    s = torch.tensor([[-size, -size / 2, -3.0, -4.0], [-size] * 4], device="cuda")
    check(x, s, wc.witcert_beam_select(x, s, 8), 8) if size < 1e10 else None
    got = wc.witcert_beam_select(x, s, 8)
    assert (got[1][0] >= 2).all() and got[0].isfinite().all()
    x = x * 1e30
    check(x, torch.zeros_like(s), wc.witcert_beam_select(x, torch.zeros_like(s), 8), 8)


def test_finished():
    x, s = inputs(5, 6, 8000)
    done = torch.rand(5, 6, device="cuda") < 0.5
    done[0], done[1] = True, False
    x[2] = math.nan                                         # finished beams' logits are not read
    done[2] = True
    done[3, 0], s[3, 0], x[3, 1:] = True, -200.0, -INF      # what is left when nothing else is
    for n in (1, 6, 12):
        check(x, s, wc.witcert_beam_select(x, s, n, finished=done, eos=77), n, done, 77)
    x, s = inputs(1, 2, 100)
    x[0, :, 99] = 20.0
    got = wc.witcert_beam_select(x, s, eos=99)              # without finished beams the end token still counts
    check(x, s, got, 2, None, 99)
    assert got[3].any()


def test_first_step_and_in_place():
    """One live beam a request; outputs over the inputs; then the next step on them."""
    x, s = inputs(4, 5, 3333)
    s.fill_(-INF)
    s[:, 0] = 0.0
    done = torch.zeros(4, 5, dtype=torch.bool, device="cuda")
    rows, tokens = (torch.empty(4, 5, dtype=torch.int32, device="cuda") for _ in range(2))
    for step in range(3):
        x = inputs(4, 5, 3333, seed=step)[0]
        want = wc.witcert_beam_select(x, s, finished=done, eos=5)
        check(x, s, want, 5, done, 5)
        got = wc.witcert_beam_select(x, s, finished=done, eos=5, out=(s, rows, tokens, done))
        assert got[0] is s and got[3] is done
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    with pytest.raises(wc.WitcertError, match="n_out = n_beams"):
        flat = torch.zeros(4 * 10, device="cuda")
        wc.witcert_beam_select(x, flat[:20].view(4, 5), 10, out=(flat.view(4, 10), *(torch.empty(4, 10, dtype=t, device="cuda")
                               for t in (torch.int32, torch.int32, torch.bool))))


def test_logits_beyond_32_bits():
    """More than 2^31 elements, and strides as large: the requests at both ends as by themselves."""
    R, W, V = 130, 128, 131073
    x = torch.empty(R, W, V, dtype=torch.bfloat16, device="cuda").normal_(0, 3)
    s = -torch.rand(R, W, device="cuda")
    got = wc.witcert_beam_select(x, s, 16)
    for r in (0, R - 1):
        one = wc.witcert_beam_select(x[r:r + 1].clone(), s[r:r + 1].clone(), 16)
        assert torch.equal(got[2][r], one[2][0]) and torch.equal(got[1][r], one[1][0] + r * W)
        assert (got[0][r] - one[0][0]).abs().max() <= 2.0 ** -18      # the rows' parts are summed in other places
    far = x.view(-1)[:V * 2].as_strided((2, 1, V), (V * 16000, V, 1))
    check(far, s[:2, :1].contiguous(), wc.witcert_beam_select(far, s[:2, :1].contiguous(), 4), 4)


def test_no_requests():
    got = wc.witcert_beam_select(torch.empty(0, 4, 100, device="cuda"), torch.empty(0, 4, device="cuda"), 7)
    assert [tuple(t.shape) for t in got] == [(0, 7)] * 4


def test_same_every_time_and_in_graphs():
    """Bit for bit, alone, beside another call on another stream, and replayed on new inputs."""
    x, s = inputs(8, 8, 40001, torch.float32)
    y, t = inputs(8, 8, 40001, torch.float32, seed=1)
    want, other = wc.witcert_beam_select(x, s, 16), wc.witcert_beam_select(y, t, 16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a = wc.witcert_beam_select(x, s, 16)
        b = wc.witcert_beam_select(y, t, 16, stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a, want)) and all(torch.equal(p, q) for p, q in zip(b, other))
    xs, ss = x.clone(), s.clone()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]     # two that would share a workspace if it were kept
    outs = []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(wc.witcert_beam_select(xs, ss, 16))
    for a, b, w in ((x, s, want), (y, t, other), (x, s, want)):
        xs.copy_(a), ss.copy_(b)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for o in outs for p, q in zip(o, w))


# ------------------------------------------------------------------ paths

def plain_paths(rows, tokens, length, pad):
    T, R, W = rows.shape
    out = np.full((R, W, T), pad, np.int32)
    for r in range(R):
        n = T if length is None else min(max(int(length[r]), 0), T)
        for w in range(W):
            at = w
            for t in range(n - 1, -1, -1):
                p = int(rows[t, r, at]) - r * W
                if not 0 <= p < W:
                    break
                out[r, w, t] = tokens[t, r, at]
                at = p
    return out


@pytest.mark.parametrize("T, R, W", [(1, 1, 1), (1, 3, 4), (2, 2, 3), (31, 1, 8), (32, 2, 33), (33, 2, 32), (64, 5, 4), (777, 3, 31),
                                     (300, 2, 128), (2000, 1, 64), (9001, 2, 4), (4096, 1, 8), (1100, 1, 127)])
@pytest.mark.parametrize("gaps", [0.0, 0.002, 0.3])
def test_paths(T, R, W, gaps):
    g = np.random.default_rng(T * W)
    rows = g.integers(0, W, (T, R, W)) + W * np.arange(R)[:, None]
    odd = g.integers(-W - 2, R * W + W + 2, (T, R, W))      # rows of other requests, or of none
    odd[0, 0, 0] = np.iinfo(np.int32).min
    rows = np.where(g.random((T, R, W)) < gaps, odd, rows).astype(np.int32)
    tokens = g.integers(0, 2 ** 31 - 1, (T, R, W)).astype(np.int32)
    for length, pad in ((None, -1), (g.integers(-2, T + 3, R).astype(np.int32), 5)):
        got = wc.witcert_beam_paths(torch.from_numpy(rows).cuda(), torch.from_numpy(tokens).cuda(),
                                    None if length is None else torch.from_numpy(length).cuda(), pad)
        assert np.array_equal(got.cpu().numpy(), plain_paths(rows, tokens, length, pad))


def test_paths_of_nothing():
    e = torch.empty(0, 2, 3, dtype=torch.int32, device="cuda")
    assert wc.witcert_beam_paths(e, e).shape == (2, 3, 0)
    e = torch.empty(4, 0, 3, dtype=torch.int32, device="cuda")
    assert wc.witcert_beam_paths(e, e).shape == (0, 3, 4)


# ------------------------------------------------------------------ all of it together

@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("scheme", ["int8_dither", "fp8_e4m3", "kivi2", "blackbox"])
def test_search_over_a_cache(scheme, paged):
    """A model whose logits depend on the last two tokens: the search finds what a plain search in 64 bits
    finds, and every sequence of the cache holds the prompt and its own path, to the bit."""
    R, W, V, L, steps, eos = 3, 4, 50, 2, 37, 0
    g = torch.Generator().manual_seed(11)
    table = (2.5 * torch.randn(V, V, V, generator=g)).cuda()
    table[..., eos] -= 1.0
    emb = torch.randn(L, 2, V, 2, 128, generator=g).bfloat16().cuda()
    prompts = [torch.randint(1, V, (n,), generator=g).tolist() for n in (21, 3, 48)]
    S = 48 + steps
    cache = wc.Cache(L, 4, 2, R * W, S, scheme, seed=9, max_pages=R * W * ((S + 15) // 16) if paged else 0)
    hats = lambda k, v: (k, v) if scheme == "blackbox" else ()

    def feed(c, layer, ids, n):
        k, v = emb[layer, 0][ids], emb[layer, 1][ids]
        c.witcert_write_ragged(layer, k, v, n, *hats(k, v))

    n = [0] * (R * W)
    n[::W] = [len(p) for p in prompts]
    ids = torch.tensor(sum(prompts, [])).cuda()
    for layer in range(L):
        feed(cache, layer, ids, n)
    search = wc.BeamSearch(cache, W, steps, eos=eos)
    search.start()
    # the plain search: (score, path, finished) of each beam
    beams = [[(0.0, list(p), False)] for p in prompts]
    last = torch.tensor([[p[-2:]] * W for p in prompts]).cuda()
    used = None
    for step in range(steps):
        x = table[last[..., 0], last[..., 1]]
        tokens = search.step(x)
        logp = torch.log_softmax(table.double(), -1).cpu()
        for r in range(R):
            pool = []
            for s, path, end in beams[r]:
                if end:
                    pool.append((s, path + [eos], True))
                else:
                    lp = logp[path[-2], path[-1]]
                    pool += [(s + lp[t].item(), path + [t], t == eos) for t in range(V)]
            beams[r] = sorted(pool, key=lambda b: -b[0])[:W]
        assert torch.equal(tokens.cpu().long(), torch.tensor([[b[1][-1] for b in br] for br in beams])), step
        before = torch.tensor([[b[1][-2] for b in br] for br in beams]).cuda()
        last = torch.stack([before, tokens.long()], -1)
        for layer in range(L):
            feed(cache, layer, tokens.flatten().long(), [1] * (R * W))
        want = torch.tensor([[b[0] for b in br] for br in beams])
        # every step's score rounds by half a step of its size, and is off by what the selection's lse is
        assert (search.scores.cpu().double() - want).abs().max() <= (step + 1) * (2.0 ** -18 + 2.0 ** -24 * want.abs().max())
        assert torch.equal(search.finished.cpu(), torch.tensor([[b[2] for b in br] for br in beams]))
        used = cache.witcert_stats()["pages_used"]
    paths = search.paths().cpu()
    full = [prompts[i // W] + paths[i // W, i % W].tolist() for i in range(R * W)]
    assert full == [b[1] for br in beams for b in br]
    lens = [len(f) for f in full]
    want = wc.Cache(L, 4, 2, R * W, S, scheme, seed=9)
    for layer in range(L):
        feed(want, layer, torch.tensor(sum(full, [])).cuda(), lens)
        assert all(torch.equal(a, b) for a, b in zip(cache.read(layer, lens), want.read(layer, lens)))
    q = torch.randn(R * W, 4, 128, device="cuda").bfloat16()
    (a, ma), (b, mb) = cache.decode(1, q, 1e-2), want.decode(1, q, 1e-2)
    assert (a - b).abs().max() <= 2.0 ** -13 * max(1.0, b.abs().max().item())
    assert ((ma["meter_a"] - mb["meter_a"]).abs() <= 2e-4 * mb["meter_a"] + 2.0 ** -99).all()
    if paged:
        assert used < sum((n + 15) // 16 for n in lens)     # the beams share their prompts' pages
    with pytest.raises(ValueError, match="steps"):
        search.step(x)


def test_search_with_fewer_candidates_than_beams():
    cache = wc.Cache(1, 4, 2, 6, 32, "fp8_e4m3")
    k = torch.randn(2 * 5, 2, 128, device="cuda").bfloat16()
    cache.witcert_write_ragged(0, k, k, [5, 0, 0, 5, 0, 0])
    search = wc.BeamSearch(cache, 3, 4)
    search.start()
    x = torch.full((2, 3, 10), -INF, device="cuda")
    x[0, :, 4], x[1, :, 2:4] = 1.0, 1.0
    tokens = search.step(x)
    assert tokens.tolist() == [[4, -1, -1], [2, 3, -1]]
    assert [cache.witcert_seq_length(0, i) for i in range(6)] == [5] * 6
    assert search.paths(pad=9).tolist() == [[[4], [9], [9]], [[2], [3], [9]]]
    x[1] = math.nan
    assert search.step(x).tolist() == [[4, -1, -1], [-1] * 3]
    assert search.paths(pad=9).tolist() == [[[4, 4], [9, 9], [9, 9]], [[9, 9]] * 3]


def test_search_on_a_stream():
    """All of it on another stream than the current one, logits a row a sequence, as on the current stream."""
    side, out = torch.cuda.Stream(), []
    k = torch.randn(2 * 70, 2, 128, device="cuda").bfloat16()
    xs = [inputs(2, 3, 999, seed=i)[0].flatten(0, 1) for i in range(5)]
    torch.cuda.synchronize()
    for stream in (None, side):
        cache = wc.Cache(1, 4, 2, 6, 80, "int8_rtn", max_pages=30)
        cache.witcert_write_ragged(0, k, k, [70, 0, 0, 70, 0, 0], stream=stream)
        search = wc.BeamSearch(cache, 3, 5, eos=1)
        torch.cuda.synchronize()                            # what the search keeps was made on the current stream
        search.start(stream=stream)
        for x in xs:
            tokens = search.step(x, stream=stream)
            new = k[:6] * 0.5
            torch.cuda.synchronize()
            cache.witcert_write_ragged(0, new, new, [1] * 6, stream=stream)
        paths = search.paths(stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(paths[..., -1], tokens)
        out.append([paths, search.scores, *cache.read(0, [75] * 6)])
    assert all(torch.equal(a, b) for a, b in zip(*out))
    for bad in (xs[0][:5], xs[0].unflatten(0, (3, 2)), None):
        fresh = wc.BeamSearch(cache, 3, 1)
        with pytest.raises(ValueError, match="logits"):
            fresh.step(bad)
