"""Operators of a beam search over the compressed KV cache, measured in their plain form and through the library.

  select   the best continuations of each request: log-softmax over the vocabulary, candidates of all beams ranked
  fork     sequences of a cache take the state of others; every sequence gets a token; the cache is read back
  paths    the token sequences of the last beams, from each step's chosen rows and tokens

Every case is a dict of sizes; inputs come from the seed alone.  The plain forms are elementary torch operations in
32 bits, the scores that the selection ranks in 64 (two candidates may be closer than 32 bits tell apart).

select: rows (request, beam) of logits x, cumulative scores c.  s = c + x - log sum exp x; a finished beam offers one
candidate, its own score with the end token; a beam of score -inf offers none, nor do logits of -inf.  Order: score
falling, then row, then token.  Places without a candidate: score -inf, row -1, token -1.

fork: a row of the cache is a token and KV head, kept by its scheme:
  int8_dither  s (code - xi), code = rint(x / s + xi), s = fp16 up(max |x| / 127) per 32 channels, xi uniform
               on [-1/2, 1/2) from Philox4x32-10 counted by (position, channel, head, layer)
  int8_rtn     the same with xi = 0
  fp8_e4m3     the saturating E4M3 cast
  blackbox     bf16 outputs of a caller's tensor function

paths: step t chose for beam w of a request the row rows[t][w] (its parent beam) and tokens[t][w].  Beam w's sequence
ends with tokens[T-1][w] and follows the parents back; a row of -1 ends it, and all before is -1.
"""
import math

import torch

own = False

D = 128                     # head dimension
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one request's step on a small vocabulary: latency
        dict(name="select_step", op="select", R=1, W=4, V=32000, n=8, dt="bf16", start=False, masked=False, padded=False),
        # the first step of a batch: one live beam a request, logits of a packed output projection's wider rows
        dict(name="select_first", op="select", R=16, W=4, V=131072, n=4, dt="bf16", start=True, masked=False, padded=True),
        # many beams, an odd vocabulary, fp32 logits, and a grammar that allows few tokens
        dict(name="select_grammar", op="select", R=2, W=32, V=50001, n=64, dt="f32", start=False, masked=True, padded=False),
        # a serving batch: 64 requests of 8 beams, some of them finished
        dict(name="select_batch", op="select", R=64, W=8, V=131072, n=16, dt="bf16", start=False, masked=False, padded=False),
        # a short prompt handed to four beams of a paged store, rounded INT8
        dict(name="fork_short", op="fork", turn="prompt", scheme="int8_rtn", L=1, R=1, W=4, Hkv=8, ctx=100, paged=True, ragged=False),
        # prompts of a serving batch handed to their beams: pages shared, their last blocks copied
        dict(name="fork_pages", op="fork", turn="prompt", scheme="fp8_e4m3", L=4, R=4, W=4, Hkv=4, ctx=2053, paged=True, ragged=True),
        # two long prompts in a contiguous store, dithered INT8, each to eight beams
        dict(name="fork_copies", op="fork", turn="prompt", scheme="int8_dither", L=2, R=2, W=8, Hkv=8, ctx=4099, paged=False, ragged=False),
        # beams of a contiguous bf16 store that change places, and back
        dict(name="fork_places", op="fork", turn="places", scheme="blackbox", L=2, R=1, W=8, Hkv=8, ctx=8192, paged=False, ragged=False),
        # a short answer of one request
        dict(name="paths_short", op="paths", T=64, R=1, W=4),
        # long answers of a serving batch
        dict(name="paths_batch", op="paths", T=2048, R=64, W=8),
        # an odd number of steps, many beams
        dict(name="paths_wide", op="paths", T=777, R=5, W=33),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "select", "fork", "fork", "paths"])
    if op == "select":
        dt = rng.choice(["bf16", "bf16", "f32"])
        W, V = _log(rng, 1, 32), _log(rng, 500, 152000)
        most = 64 * 8 * 131072 // (W * V * (1 if dt == "bf16" else 2))
        return dict(op=op, R=_log(rng, 1, max(1, min(64, most))), W=W, V=V, n=rng.choice([W, 2 * W]), dt=dt,
                    start=rng.random() < 0.2, masked=rng.random() < 0.2, padded=rng.random() < 0.4)
    if op == "paths":
        W = _log(rng, 1, 64)
        R = _log(rng, 1, 512 // W)
        return dict(op=op, T=_log(rng, 1, 1024), R=R, W=W)
    turn = rng.choice(["prompt", "prompt", "places"])
    W, Hkv = rng.choice([2, 3, 4, 5, 8]), rng.choice([4, 8])
    R = 1 if turn == "places" else _log(rng, 1, 16 // W)
    return dict(op=op, turn=turn, scheme=rng.choice(["int8_dither", "int8_rtn", "fp8_e4m3", "blackbox"]),
                L=rng.choice([1, 2]), R=R, W=W, Hkv=Hkv, ctx=_log(rng, 1, 65536 // (R * W)), paged=rng.random() < 0.5,
                ragged=turn == "prompt" and rng.random() < 0.5)


def _lens(case):
    """Tokens of each request's prompt."""
    return [max(1, case["ctx"] - (i * case["ctx"] // (2 * case["R"]) + 5 * i if case["ragged"] else 0))
            for i in range(case["R"])]


def _places(W):
    """Beam i takes the place of beam _places(W)[i]: one chain through all of them, two trading places at its end."""
    return list(range(1, W - 2)) + [0] + [W - 1, W - 2] if W > 3 else list(range(1, W)) + [0]


CODES = {"int8_dither": 272, "int8_rtn": 272, "fp8_e4m3": 256, "blackbox": 512}     # a row's codes and scales


def work(case):
    if case["op"] == "select":
        rows = case["R"] * (1 if case["start"] else case["W"])
        e = 2 if case["dt"] == "bf16" else 4
        return {"bytes": rows * case["V"] * e + case["R"] * (case["W"] * 5 + case["n"] * 13), "flops": 4 * rows * case["V"]}
    if case["op"] == "paths":
        return {"bytes": 12 * case["T"] * case["R"] * case["W"], "flops": 0}
    held, B, W = sum(_lens(case)), case["R"] * case["W"], case["W"]
    codes = CODES[case["scheme"]]
    row = codes + 32                                    # with the witness
    if case["turn"] == "places":                        # every beam moves, there and back; pages stay where they are
        moves = codes if case["paged"] else 4 * row
        return {"bytes": case["L"] * case["Hkv"] * W * case["ctx"] * (moves + 512),
                "flops": 4 * D * case["L"] * case["Hkv"] * W * case["ctx"]}
    partial = sum(n % 16 for n in _lens(case))
    copied = partial if case["paged"] else held
    inputs = 1024 if case["scheme"] == "blackbox" else 512
    return {"bytes": case["L"] * case["Hkv"] * (held * row + copied * (W - 1) * row + B * (inputs + row) + (held * W + B) * 512),
            "flops": 4 * D * case["L"] * case["Hkv"] * (held * W + B)}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _kv(g, *shape):
    """Keys with a few strong channels and values, as bf16."""
    k = torch.randn(*shape, D, generator=g, device=DEV)
    k[..., 10:12] *= 6.0
    k[..., 74:76] *= 6.0
    return k.bfloat16(), torch.randn(*shape, D, generator=g, device=DEV).bfloat16()


def _philox(c0, c1, c2, seed):
    """Philox4x32-10 of counters (c0, c1, c2, 0), int64 tensors of 32-bit words; the four output words."""
    m = 0xFFFFFFFF
    c3 = torch.zeros_like(c0)
    k0, k1 = seed & m, seed >> 32 & m
    for _ in range(10):
        # the products' 64 bits, wrapped to a signed word: the shift's sign bits are masked away
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (p1 >> 32 & m) ^ c1 ^ k0, p1 & m, (p0 >> 32 & m) ^ c3 ^ k1, p0 & m
        k0, k1 = k0 + 0x9E3779B9 & m, k1 + 0xBB67AE85 & m
    return c0, c1, c2, c3


def _dither(S, heads, layers, tensor, seed):
    """xi [layers, 1, S, heads, 128] of positions 0 .. S - 1."""
    pos, quad = torch.arange(S, device=DEV).view(-1, 1, 1), torch.arange(D // 4, device=DEV)
    head = torch.arange(heads, device=DEV).view(1, -1, 1) | torch.arange(layers, device=DEV).view(-1, 1, 1, 1) << 16
    c0, c1, c2 = torch.broadcast_tensors(pos, quad | tensor << 16, head)
    u = torch.stack(_philox(c0, c1, c2, seed), -1).reshape(layers, 1, S, heads, D)
    return (u >> 8).float() * 2.0 ** -24 - 0.5


def _select_inputs(case, seed):
    g = _gen(seed)
    R, W, V = case["R"], case["W"], case["V"]
    x = 3.0 * torch.randn(R, W, V + (8 if case["padded"] else 0), generator=g, device=DEV)[..., :V]
    if case["masked"]:                                  # a grammar: about one token in 50, other ones in each row
        x = x.masked_fill_(torch.rand(R, W, V, generator=g, device=DEV) > 0.02, -math.inf)
    x = x.bfloat16() if case["dt"] == "bf16" else x.float()
    if case["padded"]:
        wide = torch.zeros(R, W, V + 8, dtype=x.dtype, device=DEV)
        wide[..., :V] = x
        x = wide[..., :V]
    scores = -10.0 + 2.0 * torch.randn(R, W, generator=g, device=DEV)
    done = torch.rand(R, W, generator=g, device=DEV) < 0.1
    if case["start"]:
        scores = torch.full_like(scores, -math.inf)
        scores[:, 0] = 0.0
        done = torch.zeros_like(done)
    return dict(case=case, x=x if case["padded"] else x.contiguous(), scores=scores, done=done, eos=V // 3)


def _paths_inputs(case, seed):
    g = _gen(seed)
    T, R, W = case["T"], case["R"], case["W"]
    rows = torch.randint(0, W, (T, R, W), generator=g, device=DEV)
    rows += W * torch.arange(R, device=DEV)[:, None]
    tokens = torch.randint(0, 131072, (T, R, W), generator=g, device=DEV)
    # now and then a request has fewer candidates than beams
    none = torch.rand(T, R, W, generator=g, device=DEV) < 0.25 / T
    return dict(case=case, rows=rows.masked_fill_(none, -1).int(), tokens=tokens.masked_fill_(none, -1).int())


def _fork_inputs(case, seed):
    g = _gen(seed)
    L, R, W, H = (case[k] for k in ("L", "R", "W", "Hkv"))
    lens, B = _lens(case), R * W
    st = dict(case=case, seed=int(seed), lens=lens)
    S = max(lens) + 1
    sources = B if case["turn"] == "places" else R
    st["K"], st["V"] = _kv(g, L, sources, S, H)         # the last position is the new token's: not held yet
    st["nK"], st["nV"] = _kv(g, L, B, H)
    xi = (0.0, 0.0)
    if case["scheme"] == "int8_dither":
        xi = _dither(S, H, L, 0, st["seed"]), _dither(S, H, L, 1, st["seed"])
    st["k_store"], st["v_store"] = _pack(case, st["K"], xi[0]), _pack(case, st["V"], xi[1])
    if case["turn"] == "places":
        st["from"] = torch.tensor(_places(W), device=DEV)
        held = [case["ctx"]] * W
    else:
        st["from"] = torch.arange(R, device=DEV).repeat_interleave(W)
        st["end"] = torch.tensor(lens, device=DEV).repeat_interleave(W)
        st["beam"] = torch.arange(B, device=DEV)
        held = [n + 1 for n in lens for _ in range(W)]
    st["held"] = held
    # row r of what is read back: token at[r] of sequence seq[r]
    n = torch.tensor(held)
    st["seq"] = torch.repeat_interleave(torch.arange(B), n).to(DEV)
    st["at"] = (torch.arange(int(n.sum())) - torch.repeat_interleave(n.cumsum(0) - n, n)).to(DEV)
    return st


def _inputs(case, seed):
    return {"select": _select_inputs, "paths": _paths_inputs, "fork": _fork_inputs}[case["op"]](case, seed)


def prepare(case, seed):
    state = _inputs(case, seed)
    if own and case["op"] == "fork":
        _handles(state)
    return state


def _handles(st):
    """The cache that a program of the library keeps, with the prompts (the beams, where they change places) in it."""
    import kv_cache_quantization_witcert_gb300 as wc
    case, lens = st["case"], st["lens"]
    L, R, W, H = (case[k] for k in ("L", "R", "W", "Hkv"))
    B, S = R * W, max(lens) + 1
    st["cache"] = cache = wc.Cache(L, H, H, B, S, case["scheme"], seed=st["seed"],
                                   max_pages=B * ((S + 15) // 16) if case["paged"] else 0)
    if case["turn"] == "places":
        first = [case["ctx"]] * W
        st["parents"] = _places(W)
        st["back"] = [st["parents"].index(i) for i in range(W)]
    else:
        first = [0] * B
        first[::W] = lens
        st["parents"] = [i // W * W for i in range(B)]
        st["lengths"] = [lens[i // W] for i in range(B)]
    hats = case["scheme"] == "blackbox"
    sources = st["K"].shape[1]
    held = lens if case["turn"] == "prompt" else first
    for layer in range(L):
        K, V = (torch.cat([st[k][layer, i, :held[i]] for i in range(sources)]) for k in "KV")
        cache.witcert_write_ragged(layer, K, V, first, *((K, V) if hats else ()))
    st["hats"] = [(st["nK"][layer], st["nV"][layer]) if hats else () for layer in range(L)]


# ------------------------------------------------------------------ plain forms

def _half_up(x):
    """The smallest fp16 value that is not below x (x >= 0)."""
    h = x.half()
    bits = h.view(torch.int16)
    return torch.where(h.float() < x, bits + 1, bits).view(torch.float16)


def _pack(case, x, xi):
    """The store of x [..., heads, 128]."""
    scheme = case["scheme"]
    if scheme == "blackbox":
        return dict(value=x)
    x = x.float()
    if scheme == "fp8_e4m3":
        return dict(value=x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8))
    g = x.unflatten(-1, (4, 32))
    s = _half_up(g.abs().amax(-1, True) / 127.0)
    xg = xi.unflatten(-1, (4, 32)) if isinstance(xi, torch.Tensor) else xi
    code = (g / torch.where(s > 0, s.float(), 1.0) + xg).round().clamp(-128, 127) * (s > 0)
    return dict(code=code.to(torch.int8), scale=s, xi=xg)


def _unpack(store):
    """The values of a store, in 32 bits."""
    if "value" in store:
        v = store["value"]
        return v.view(torch.float8_e4m3fn).float() if v.dtype == torch.uint8 else v.float()
    return ((store["code"].float() - store["xi"]) * store["scale"].float()).flatten(-2)


def _forked(st, name, new):
    """Layer by layer, the rows that the sequences hold once each has taken its parent's state and, unless beams
    only change places, one more token."""
    case, store = st["case"], st[name]
    moved = {k: v[:, st["from"]] for k, v in store.items() if k != "xi"}
    xi = store.get("xi")
    if case["turn"] == "prompt":
        at = xi[:, 0, st["end"]].flatten(-2) if isinstance(xi, torch.Tensor) else 0.0
        fresh = _pack(case, new, at)
        for k, v in moved.items():
            v[:, st["beam"], st["end"]] = fresh[k]
    if xi is not None:
        moved["xi"] = xi
    return list(_unpack(moved)[:, st["seq"], st["at"]].bfloat16().unbind(0))


def _select(st):
    x, scores, n = st["x"].double(), st["scores"].double(), st["case"]["n"]
    R, W, V = x.shape
    m = x.amax(-1, True)
    lse = m + (x - m).exp().sum(-1, True).log()
    s = scores[..., None] + (x - lse)
    own_end = torch.full_like(s, -math.inf)
    own_end[..., st["eos"]] = scores
    s = torch.where(st["done"][..., None], own_end, s)
    s = torch.where(scores[..., None] > -math.inf, s, -math.inf).view(R, W * V)
    best, place = s.sort(dim=-1, descending=True, stable=True)
    best, place = best[:, :n], place[:, :n]
    if best.shape[1] < n:
        best = torch.nn.functional.pad(best, (0, n - best.shape[1]), value=-math.inf)
        place = torch.nn.functional.pad(place, (0, n - place.shape[1]))
    there = best > -math.inf
    row = place // V + W * torch.arange(R, device=DEV)[:, None]
    token = place % V
    ended = st["done"].view(-1)[row] | (token == st["eos"])
    return [best.float(), torch.where(there, row, -1).int(), torch.where(there, token, -1).int(), there & ended]


def _paths(st):
    """chosen[t][w]: the beam of step t that beam w of the last step goes back to (W: none), by doubling."""
    rows, tokens = st["rows"].long(), st["tokens"]
    T, R, W = rows.shape
    rel = rows - W * torch.arange(R, device=DEV)[:, None]
    rel = torch.where((rel >= 0) & (rel < W), rel, W)
    none = torch.full((T, R, 1), W, device=DEV)
    back = torch.cat([rel, none], -1)                    # from beams of step t to beams of step t - 1
    # chosen[t] = back[T-1] o .. o back[t+1]: from the last step's beams to step t's
    same = torch.arange(W + 1, device=DEV).expand(1, R, W + 1)
    chosen = torch.cat([back[1:], same])
    span = 1
    while span < T:
        later = torch.cat([chosen[span:], same.expand(min(span, T), R, W + 1)])
        chosen = torch.gather(chosen, -1, later)
        span *= 2
    # a step without a row has no token either, and none before it
    token = torch.cat([torch.where(rel < W, tokens, -1), torch.full_like(tokens[..., :1], -1)], -1)
    return torch.gather(token, -1, chosen)[..., :W].permute(1, 2, 0).contiguous()


def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    if case["op"] == "select":
        return _select(st)
    if case["op"] == "paths":
        return _paths(st)
    return _forked(st, "k_store", st["nK"]) + _forked(st, "v_store", st["nV"])


def _run_own(st, case):
    import kv_cache_quantization_witcert_gb300 as wc
    if case["op"] == "select":
        return list(wc.witcert_beam_select(st["x"], st["scores"], case["n"], finished=st["done"], eos=st["eos"]))
    if case["op"] == "paths":
        return wc.witcert_beam_paths(st["rows"], st["tokens"])
    cache, L = st["cache"], case["L"]
    if case["turn"] == "places":
        cache.witcert_fork(st["parents"])
        got = [cache.read(layer, st["held"]) for layer in range(L)]
        cache.witcert_fork(st["back"])                   # the next pass finds the beams where they were
    else:
        cache.witcert_fork(st["parents"], st["lengths"])
        for layer in range(L):
            cache.witcert_write_ragged(layer, st["nK"][layer], st["nV"][layer], [1] * len(st["parents"]), *st["hats"][layer])
        got = [cache.read(layer, st["held"]) for layer in range(L)]
    return [k for k, _ in got] + [v for _, v in got]


# ------------------------------------------------------------------ the definitions, in 64 bits

def _exact_rows(case, st, tensor):
    """Sequence by sequence: the source's codes, and the new token quantized where it stands."""
    store, new, W = st["v_store" if tensor else "k_store"], st["nV" if tensor else "nK"], case["W"]
    out = []
    for layer in range(case["L"]):
        parts = []
        for i in range(case["R"] * W):
            src = _places(W)[i] if case["turn"] == "places" else i // W
            n = case["ctx"] if case["turn"] == "places" else st["lens"][src]
            if "value" in store:
                v = store["value"][layer, src, :n]
                v = (v.view(torch.float8_e4m3fn) if v.dtype == torch.uint8 else v).to(torch.float64)
            else:
                v = store["code"][layer, src, :n].to(torch.float64)
                if case["scheme"] == "int8_dither":
                    v = v - store["xi"][layer, 0, :n].to(torch.float64)
                v = (v * store["scale"][layer, src, :n].to(torch.float64)).reshape(n, -1, D)
            parts.append(v)
            if case["turn"] == "prompt":
                t = new[layer, i].to(torch.float64)
                if case["scheme"] == "fp8_e4m3":
                    t = t.clamp(-448, 448).float().to(torch.float8_e4m3fn).to(torch.float64)
                elif case["scheme"] != "blackbox":
                    s = _half_up((t.reshape(-1, 4, 32).abs().max(-1).values / 127.0).float()).to(torch.float64)
                    s = s.repeat_interleave(32, -1)
                    xi = store["xi"][layer, 0, n].to(torch.float64).reshape(-1, D) if case["scheme"] == "int8_dither" else 0.0
                    t = s * (torch.clamp(torch.round(t / torch.where(s > 0, s, 1.0) + xi), -128, 127) - xi)
                parts.append(t[None])
        out.append(torch.cat(parts))
    return out


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "paths":
        return None                                      # whole numbers only
    if case["op"] == "fork":
        return _exact_rows(case, st, 0) + _exact_rows(case, st, 1)
    best = torch.full((case["R"], case["n"]), -math.inf, dtype=torch.float64, device=DEV)
    for r in range(case["R"]):
        rows = []
        for w in range(case["W"]):
            c = st["scores"][r, w].to(torch.float64)
            if st["done"][r, w]:
                rows.append(c.view(1))
            elif c > -math.inf:
                rows.append(c + torch.log_softmax(st["x"][r, w].to(torch.float64), -1))
        s = torch.sort(torch.cat(rows), descending=True).values[:case["n"]]
        best[r, :len(s)] = s
    return [best, None, None, None]
