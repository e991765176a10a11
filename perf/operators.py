"""Operators around the compressed KV cache, measured in their plain form and through the library.

  rope     rotary positions of the queries and keys of a batch of tokens
  append   keys without positions, rotated and appended to a compressed cache, then read back
  read     the keys and values that a compressed cache holds
  attend   causal attention of each sequence's newest tokens over its compressed cache

Every case is a dict of sizes; inputs come from the seed alone.  The plain forms are elementary torch
operations in 32 bits (angles in 64), rounded once at the end.  Stores, by scheme:

  int8_dither  s (code - xi), code = rint(x / s + xi), s = fp16 up(max |x| / 127) per 32 channels, xi uniform
               on [-1/2, 1/2) from Philox4x32-10 counted by (position, channel, head, layer)
  int8_rtn     the same with xi = 0
  fp8_e4m3     the saturating E4M3 cast
  kivi2        zero + scale code, two bits: keys per channel over 16 tokens (the unfinished last block
               exact), values per token over 32 channels
  blackbox     bf16 outputs of a caller's tensor function
"""
import math

import torch

own = False

D = 128                     # head dimension
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a 16-sequence batch: 16 tokens, one position each
        dict(name="rope_step", op="rope", n=16, Hq=32, Hkv=8, dim=128, rot=128, inter=False, dt="bf16", base=1e4,
             scaling="none", factor=1.0, start=4096, packed=True),
        # a prefill's queries and keys at far positions, frequencies stretched for a long context
        dict(name="rope_prefill", op="rope", n=16384, Hq=32, Hkv=8, dim=128, rot=128, inter=False, dt="bf16",
             base=5e6, scaling="by_parts", factor=8.0, start=114688, packed=False),
        # interleaved pairs on half of the head, fp32, an odd token count, slices of a packed projection
        dict(name="rope_half_head", op="rope", n=1237, Hq=28, Hkv=4, dim=128, rot=64, inter=True, dt="f32",
             base=1e6, scaling="linear", factor=4.0, start=1000003, packed=True),
        # the append of a decode step: one token to each of 16 sequences of 4096
        dict(name="append_step", op="append", scheme="int8_dither", B=16, Hkv=8, ctx=4096, new=1, ragged=False,
             paged=False, rot=128, inter=False, base=1e4),
        # a prompt chunk of 2048 tokens for each of 4 sequences, raw FP8
        dict(name="append_chunk", op="append", scheme="fp8_e4m3", B=4, Hkv=8, ctx=6144, new=2048, ragged=False,
             paged=False, rot=128, inter=False, base=1e4),
        # a serving batch: ragged appends to a paged store of dithered INT8
        dict(name="append_ragged", op="append", scheme="int8_dither", B=8, Hkv=4, ctx=4099, new=517, ragged=True,
             paged=True, rot=128, inter=False, base=1e6),
        # a whole prefix handed on, dithered INT8
        dict(name="read_prefix", op="read", scheme="int8_dither", B=1, Hkv=8, ctx=32768, new=32768, ragged=False,
             paged=False),
        # prefixes of a serving batch, two-bit store
        dict(name="read_ragged", op="read", scheme="kivi2", B=8, Hkv=4, ctx=4097, new=4097, ragged=True, paged=True),
        # drafted tokens of a serving batch checked at once: four tokens a sequence
        dict(name="attend_verify", op="attend", scheme="int8_dither", B=16, Hq=28, Hkv=4, ctx=4096, new=4,
             ragged=True, paged=True),
        # eight tokens over one very long context
        dict(name="attend_long", op="attend", scheme="fp8_e4m3", B=1, Hq=32, Hkv=8, ctx=131072, new=8, ragged=False,
             paged=False),
        # a serving batch of prompt chunks over a paged cache of a caller's bf16 function
        dict(name="attend_chunks", op="attend", scheme="blackbox", B=4, Hq=32, Hkv=4, ctx=8211, new=509, ragged=True,
             paged=True),
        # the last 2048 tokens of a 32768-token prompt
        dict(name="attend_prefill", op="attend", scheme="int8_dither", B=1, Hq=32, Hkv=8, ctx=32768, new=2048,
             ragged=False, paged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attend", "attend"])
    Hq, Hkv = rng.choice([(32, 8), (28, 4), (32, 4), (16, 16)])
    if op == "rope":
        scaling = rng.choice(["none", "linear", "by_parts"])
        return dict(op=op, n=_log(rng, 1, 16384), Hq=Hq, Hkv=Hkv, dim=128, rot=rng.choice([128, 128, 64, 32]),
                    inter=rng.random() < 0.4, dt=rng.choice(["bf16", "bf16", "f32"]), base=rng.choice([1e4, 1e6, 5e6]),
                    scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 8.0]),
                    start=_log(rng, 1, 1000000), packed=rng.random() < 0.5)
    c = dict(op=op, scheme=rng.choice(["int8_dither", "int8_rtn", "fp8_e4m3", "blackbox"] + ["kivi2"] * (op != "append")))
    if op == "append":
        B = _log(rng, 1, 16)
        new = _log(rng, 1, 8192 // B)
        c.update(B=B, Hkv=Hkv, ctx=new + _log(rng, 1, 4096), new=new, rot=rng.choice([128, 128, 64]),
                 inter=rng.random() < 0.4, base=rng.choice([1e4, 1e6]))
    elif op == "read":
        B = _log(rng, 1, 16)
        ctx = _log(rng, 1, 32768 // B)
        c.update(B=B, Hkv=min(Hkv, 8), ctx=ctx, new=ctx)
    else:
        B = _log(rng, 1, 16)
        new = _log(rng, 1, 2048)
        ctx = max(new, _log(rng, 1, min(131072 // B, 2048 * 32768 // (new * B))))
        B = max(1, min(B, 2048 * 32768 // (new * ctx)))
        c.update(B=B, Hq=Hq, Hkv=Hkv, ctx=ctx, new=new)
    c.update(ragged=rng.random() < 0.5, paged=rng.random() < 0.5)
    return c


def _lens(case):
    """Tokens each sequence holds in the end, and how many of them are new (the last of a ragged batch of three
    or more adds none)."""
    B, ctx, new = case["B"], case["ctx"], case["new"]
    if not case["ragged"]:
        return [ctx] * B, [new] * B
    total = [max(1, ctx - i * ctx // (2 * B) - 5 * i) for i in range(B)]
    if case["op"] == "read":
        return total, list(total)
    fresh = [min(total[i], (new * (B - i) + B - 1) // B) for i in range(B)]
    if B > 2:
        fresh[-1] = 0
    return total, fresh


def work(case):
    if case["op"] == "rope":
        e = 2 if case["dt"] == "bf16" else 4
        heads = case["Hq"] + case["Hkv"]
        return {"bytes": case["n"] * (heads * case["dim"] * e * 2 + 8), "flops": 3 * case["n"] * heads * case["rot"]}
    total, fresh = _lens(case)
    # codes, scales and the witness row of a token and KV head (the key witness: append writes it, nobody else reads it)
    codes = {"int8_dither": 272, "int8_rtn": 272, "fp8_e4m3": 256, "kivi2": 112, "blackbox": 512}[case["scheme"]]
    rows = sum(fresh) * case["Hkv"]
    if case["op"] == "append":
        inputs = 1024 if case["scheme"] == "blackbox" else 512
        return {"bytes": rows * (inputs + codes + 32 + codes + 512), "flops": rows * (3 * case["rot"] + 8 * D)}
    if case["op"] == "read":
        return {"bytes": rows * (codes + 512), "flops": rows * 4 * D}
    pairs = sum(n * (s - n) + n * (n + 1) // 2 for s, n in zip(total, fresh))
    held = sum(s for s, n in zip(total, fresh) if n)
    return {"bytes": held * case["Hkv"] * codes + 2 * sum(fresh) * case["Hq"] * D * 2, "flops": 4 * D * case["Hq"] * pairs}


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
    for r in range(10):
        # the products' 64 bits, wrapped to a signed word: the shift's sign bits are masked away
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (p1 >> 32 & m) ^ c1 ^ k0, p1 & m, (p0 >> 32 & m) ^ c3 ^ k1, p0 & m
        k0, k1 = k0 + 0x9E3779B9 & m, k1 + 0xBB67AE85 & m
    return c0, c1, c2, c3


def _dither(pos, heads, tensor, seed):
    """xi [len(pos), heads, 128] of layer 0."""
    quad = torch.arange(D // 4, device=DEV)
    c0, c1, c2 = torch.broadcast_tensors(pos.view(-1, 1, 1), quad.view(1, 1, -1) | tensor << 16,
                                         torch.arange(heads, device=DEV).view(1, -1, 1))
    u = torch.stack(_philox(c0, c1, c2, seed), -1).reshape(len(pos), heads, D)
    return (u >> 8).float() * 2.0 ** -24 - 0.5


def _frequencies(case):
    """Radians per position of each pair (64 bits), and the factor on the rotated vector."""
    r = case["rot"]
    f = case["base"] ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    factor = case.get("factor", 1.0)
    if case.get("scaling") == "linear":
        return f / factor, 1.0
    if case.get("scaling") == "by_parts":
        # pairs that turn over 32 times in the trained 4096 tokens keep their frequency, those under one turn take
        # f / factor, a ramp between
        keep = ((4096 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        return f * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _inputs(case, seed):
    g = _gen(seed)
    if case["op"] == "rope":
        n, Hq, Hkv, d = case["n"], case["Hq"], case["Hkv"], case["dim"]
        x = torch.randn(n, (Hq + 2 * Hkv) * d, generator=g, device=DEV)
        x = x.bfloat16() if case["dt"] == "bf16" else x
        q, k = x[:, :Hq * d].view(n, Hq, d), x[:, Hq * d:(Hq + Hkv) * d].view(n, Hkv, d)
        if not case["packed"]:
            q, k = q.contiguous(), k.contiguous()
        jump = torch.randint(0, 3, (n,), generator=g, device=DEV)
        freq, gain = _frequencies(case)
        return dict(case=case, q=q, k=k, pos=case["start"] + jump.cumsum(0), freq=freq.to(DEV), gain=gain)
    total, fresh = _lens(case)
    B, H = case["B"], case["Hkv"]
    st = dict(case=case, total=total, fresh=fresh, seed=int(seed))
    # row r of the packed new tokens: token at[r] of sequence seq[r]
    st["seq"] = torch.repeat_interleave(torch.arange(B), torch.tensor(fresh)).to(DEV)
    st["at"] = torch.cat([torch.arange(s - n, s) for s, n in zip(total, fresh)]).to(DEV)
    if case["op"] == "append":
        rows = sum(fresh)
        st["K"], st["V"] = _kv(g, rows, H)
        if case["scheme"] == "blackbox":      # the caller's function: a relative error of a percent or so
            st["K_hat"] = (st["K"].float() * (1 + 0.01 * torch.randn(rows, H, D, generator=g, device=DEV))).bfloat16()
            st["V_hat"] = (st["V"].float() * (1 + 0.01 * torch.randn(rows, H, D, generator=g, device=DEV))).bfloat16()
        if case["scheme"] == "int8_dither":
            st["xi"] = _dither(st["at"], H, 0, st["seed"]), _dither(st["at"], H, 1, st["seed"])
        freq, st["gain"] = _frequencies(case)
        st["freq"] = freq.to(DEV)
        return st
    S = max(total)
    st["len"] = torch.tensor(total, device=DEV)
    K, V = _kv(g, B, S, H)
    xi = (0.0, 0.0)
    if case["scheme"] == "int8_dither":
        pos = torch.arange(S, device=DEV)
        xi = _dither(pos, H, 0, st["seed"]), _dither(pos, H, 1, st["seed"])
    # the compressed cache in a plain layout: what the library holds in its own
    st["K"], st["V"] = K, V
    st["k_store"], st["v_store"] = _pack(case, K, xi[0], st["len"]), _pack(case, V, xi[1], None)
    if case["op"] == "attend":
        st["q"] = (1.5 * torch.randn(sum(fresh), case["Hq"], D, generator=g, device=DEV)).bfloat16()
        st["row"] = torch.cat([torch.arange(n) for n in fresh]).to(DEV)
    return st


def prepare(case, seed):
    state = _inputs(case, seed)
    if own:
        _handles(state)
    return state


def _handles(st):
    """What a program of the library keeps: the rotation's plan, the cache with the tokens that precede the call."""
    import kv_cache_quantization_witcert_gb300 as wc
    case = st["case"]
    if "rot" in case:
        st["rope"] = wc.Rope(case["rot"], base=case["base"], interleaved=case["inter"],
                             scaling=None if case.get("scaling", "none") == "none" else case["scaling"],
                             factor=case.get("factor", 1.0), original_tokens=4096)
    if case["op"] == "rope":
        return
    total, fresh, H = st["total"], st["fresh"], case["Hkv"]
    blocks = sum((s + 15) // 16 for s in total)
    st["cache"] = cache = wc.Cache(1, case.get("Hq", H), H, case["B"], max(total), case["scheme"], seed=st["seed"],
                                   max_pages=blocks if case["paged"] else 0)
    if case["op"] == "append":
        before = [s - n for s, n in zip(total, fresh)]
        K, V = _kv(_gen(st["seed"] + 1), sum(before), H)
    else:
        before = total
        K = torch.cat([st["K"][i, :s] for i, s in enumerate(total)])
        V = torch.cat([st["V"][i, :s] for i, s in enumerate(total)])
    hats = (K, V) if case["scheme"] == "blackbox" else ()
    if len(set(before)) > 1:
        cache.witcert_write_ragged(0, K, V, before, *hats)
    elif before[0]:
        shape = (case["B"], before[0], H, D)
        write = cache.witcert_write_hat if hats else cache.witcert_write
        write(0, *(t.view(shape) for t in (K, V) + hats))
    st["before"] = before
    if case["op"] == "append":
        st["hats"] = tuple(st[k] for k in ("K_hat", "V_hat") if k in st)
        if not case["ragged"]:
            shape = (case["B"], fresh[0], H, D)
            st["in"] = tuple(st[k].view(shape) for k in ("K", "V"))
            st["hats"] = tuple(t.view(shape) for t in st["hats"])


# ------------------------------------------------------------------ plain forms

def _rotate(x, pos, freq, gain, rot, inter):
    """x [n, heads, d] rotated by pos [n], in 32 bits."""
    angle = pos.double()[:, None] * freq
    c, s = (gain * angle.cos()).float()[:, None], (gain * angle.sin()).float()[:, None]
    x = x.float()
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, v = a * c - b * s, b * c + a * s
    if inter:
        y[..., 0:rot:2], y[..., 1:rot:2] = u, v
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = u, v
    return y


def _half_up(x):
    """The smallest fp16 value that is not below x (x >= 0)."""
    h = x.half()
    bits = h.view(torch.int16)
    return torch.where(h.float() < x, bits + 1, bits).view(torch.float16)


def _two_bit(x, dim):
    lo, hi = x.amin(dim, True), x.amax(dim, True)
    scale, zero = ((hi - lo) / 3.0).half(), lo.half()
    s = scale.float()
    code = ((x - zero.float()) / torch.where(s > 0, s, 1.0)).round().clamp(0, 3) * (s > 0)
    return dict(code=code.to(torch.uint8), scale=scale, zero=zero)


def _pack(case, x, xi, length):
    """The store of x [..., heads, 128]; with `length` [B], x [B, S, heads, 128] are keys."""
    scheme = case["scheme"]
    if scheme == "blackbox":
        return dict(value=x)
    x = x.float()
    if scheme == "fp8_e4m3":
        return dict(value=x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn))
    if scheme == "kivi2" and length is not None:
        B, S, H, _ = x.shape
        nb = (S + 15) // 16
        blocks = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, nb * 16 - S)).view(B, nb, 16, H, D)
        st = _two_bit(blocks, 2)
        done = torch.arange(nb, device=DEV)[None] < (length // 16)[:, None]
        return dict(st, exact=x.bfloat16(), done=done)
    g = x.unflatten(-1, (4, 32))
    if scheme == "kivi2":
        return _two_bit(g, -1)
    s = _half_up(g.abs().amax(-1, True) / 127.0)
    xg = xi.unflatten(-1, (4, 32)) if isinstance(xi, torch.Tensor) else xi
    code = (g / torch.where(s > 0, s.float(), 1.0) + xg).round().clamp(-128, 127) * (s > 0)
    return dict(code=code.to(torch.int8), scale=s, xi=xg)


def _unpack(st):
    """The values of a store, in 32 bits."""
    if "value" in st:
        return st["value"].float()
    if "xi" in st:
        return ((st["code"].float() - st["xi"]) * st["scale"].float()).flatten(-2)
    x = st["zero"].float() + st["scale"].float() * st["code"].float()
    if "done" not in st:
        return x.flatten(-2)
    exact = st["exact"].float()
    done = st["done"].repeat_interleave(16, 1)[:, :exact.shape[1], None, None]
    return torch.where(done, x.flatten(1, 2)[:, :exact.shape[1]], exact)


def _attend(st):
    """Row r (token at[r] of its sequence) over the keys 0 .. at[r] of that sequence."""
    case, fresh = st["case"], st["fresh"]
    B, H, g, n = case["B"], case["Hkv"], case["Hq"] // case["Hkv"], max(st["fresh"])
    k, v = _unpack(st["k_store"]), _unpack(st["v_store"])
    S = k.shape[1]
    q = torch.zeros(B, n, H, g, D, device=DEV)
    q[st["seq"], st["row"]] = st["q"].float().unflatten(1, (H, g))
    s = q.permute(0, 2, 3, 1, 4).reshape(B, H, g * n, D) @ k.permute(0, 2, 3, 1) / math.sqrt(D)
    last = torch.full((B, n), S, device=DEV)
    last[st["seq"], st["row"]] = st["at"]
    hidden = (torch.arange(S, device=DEV) > last[..., None])[:, None, None]           # [B, 1, 1, n, S]
    s = s.view(B, H, g, n, S).masked_fill_(hidden, -math.inf)
    s = s.sub_(s.amax(-1, True)).exp_()
    total = s.sum(-1, True)
    o = (s.view(B, H, g * n, S) @ v.permute(0, 2, 1, 3)).view(B, H, g, n, D) / total
    return o.permute(0, 3, 1, 2, 4)[st["seq"], st["row"]].flatten(1, 2).bfloat16()


def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    if case["op"] == "rope":
        return [_rotate(x, st["pos"], st["freq"], st["gain"], case["rot"], case["inter"]).to(x.dtype)
                for x in (st["q"], st["k"])]
    if case["op"] == "append":
        k, v = (st.get("K_hat", st["K"]), st.get("V_hat", st["V"]))
        k = _rotate(k, st["at"], st["freq"], st["gain"], case["rot"], case["inter"]).bfloat16()
        xi = st.get("xi", (0.0, 0.0))
        return [_unpack(_pack(case, k, xi[0], None)).bfloat16(), _unpack(_pack(case, v, xi[1], None)).bfloat16()]
    if case["op"] == "read":
        return [_unpack(st[name])[st["seq"], st["at"]].bfloat16() for name in ("k_store", "v_store")]
    return _attend(st)


def _run_own(st, case):
    if case["op"] == "rope":
        import kv_cache_quantization_witcert_gb300 as wc
        return list(wc.witcert_rope(st["rope"], st["pos"], st["q"], st["k"]))
    cache = st["cache"]
    if case["op"] == "append":
        if case["ragged"]:
            cache.witcert_write_rope_ragged(0, st["K"], st["V"], st["fresh"], st["rope"], *st["hats"])
        else:
            cache.witcert_write_rope(0, *st["in"], st["rope"], *st["hats"])
        got = list(cache.read(0, st["fresh"]))
        cache.witcert_truncate(0, st["before"])          # the next pass appends at the same places
        return got
    if case["op"] == "read":
        return list(cache.read(0, st["fresh"]))
    return cache.attend(0, st["q"], st["fresh"])


# ------------------------------------------------------------------ the definitions, in 64 bits

def _exact_values(case, st, i, tensor):
    """Keys (tensor 0) or values of sequence i's cache from its codes, token by block."""
    store = st["k_store" if tensor == 0 else "v_store"]
    n = st["total"][i]
    if "value" in store:
        return store["value"][i, :n].to(torch.float64)
    code, scale = store["code"][i].to(torch.float64), store["scale"][i].to(torch.float64)
    if case["scheme"] == "kivi2":
        x = scale * code + store["zero"][i].to(torch.float64)
        if tensor:
            return x.reshape(-1, case["Hkv"], D)[:n]
        x = x.reshape(-1, case["Hkv"], D)[:n].clone()
        x[n // 16 * 16:] = st["K"][i, n // 16 * 16:n].to(torch.float64)
        return x
    if case["scheme"] == "int8_dither":
        code = code - store["xi"].to(torch.float64)
    return (scale * code).reshape(-1, case["Hkv"], D)[:n]


def _exact_rotation(x, pos, case, freq, gain):
    z = x.to(torch.float64)
    out = z.clone()
    half = case["rot"] // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if case["inter"] else (i, i + half)
        t = (pos.to(torch.float64) * freq[i])[:, None]
        out[..., a] = gain * (z[..., a] * torch.cos(t) - z[..., b] * torch.sin(t))
        out[..., b] = gain * (z[..., b] * torch.cos(t) + z[..., a] * torch.sin(t))
    return out


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "rope":
        return [_exact_rotation(x, st["pos"], case, st["freq"], st["gain"]) for x in (st["q"], st["k"])]
    if case["op"] == "append":
        got = []
        for tensor, name in enumerate("KV"):
            x = st.get(name + "_hat", st[name])
            if tensor == 0:
                x = _exact_rotation(x, st["at"], case, st["freq"], st["gain"])
                if case["scheme"] != "blackbox":
                    x = x.to(torch.bfloat16)          # the cache's keys are bf16
            x = x.to(torch.float64)
            if case["scheme"] == "fp8_e4m3":
                # a cast has jumps: a rotated key next to a border may go either way
                x = None if tensor == 0 else x.clamp(-448, 448).float().to(torch.float8_e4m3fn).to(torch.float64)
            elif case["scheme"] in ("int8_dither", "int8_rtn"):
                xi = st["xi"][tensor].to(torch.float64) if "xi" in st else torch.zeros_like(x)
                top = x.reshape(*x.shape[:-1], 4, 32).abs().max(-1).values
                s = _half_up((top / 127.0).float()).to(torch.float64).repeat_interleave(32, -1)
                codes = torch.clamp(torch.round(x / torch.where(s > 0, s, 1.0) + xi), -128, 127)
                x = torch.where(s > 0, s * (codes - xi), torch.zeros_like(x))
            got.append(x)
        return got
    if case["op"] == "read":
        return [torch.cat([_exact_values(case, st, i, t)[s - n:] for i, (s, n) in enumerate(zip(st["total"], st["fresh"]))])
                for t in (0, 1)]
    g = case["Hq"] // case["Hkv"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=DEV)
    first = 0
    for i, (s, n) in enumerate(zip(st["total"], st["fresh"])):
        if not n:
            continue
        k, v = _exact_values(case, st, i, 0), _exact_values(case, st, i, 1)
        seen = torch.arange(s, device=DEV)[None, :] <= torch.arange(s - n, s, device=DEV)[:, None]
        for h in range(case["Hq"]):
            logits = st["q"][first:first + n, h].to(torch.float64) @ k[:, h // g].T * D ** -0.5
            p = torch.softmax(logits.masked_fill(~seen, -math.inf), -1)
            out[first:first + n, h] = p @ v[:, h // g]
        first += n
    return out
