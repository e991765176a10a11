"""Rotary positions, rotated appends, truncation and cache reads on the GPU.

Rotation: against 64-bit angles reduced in rational arithmetic, every layout, dtype, stride and
position range.  A rotated value's error is half a step of its type plus the fp32 evaluation,
16 units of 2^-24 (|a| + |b|) scale: two roundings of each product pair, two of cos and sin and
their argument (2 pi 2^-27 at most, under one unit), two for the fp32 sine and cosine themselves,
doubled; plus, at position p, the frequency's own rounding to double, p f 2^-51 radians.
Rotated appends: bit for bit what the plain writers store for keys rotated beforehand.
Reads: the oracle's reconstructions, half a step of the output plus three fp32 roundings.
"""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import kv_cache_quantization_witcert_gb300 as wc
from kv_cache_quantization_witcert_gb300 import _lib
from oracle import OracleCache

from gpu_helpers import tensor_function

pytestmark = pytest.mark.gpu

SCHEMES = ["int8_dither", "fp8_e4m3", "kivi2", "int8_rtn", "blackbox"]
TWO_PI = 2 * Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    wc.load()


def want_rotation(x, pos, rope, sign=1):
    """float64 [n, heads, d] rotated, and the bound's (|a| + |b|) scale per channel."""
    x = x.double().cpu().numpy()
    y, mag = x.copy(), np.zeros_like(x)
    r = rope.rotary_dim
    for p, f in enumerate(rope.freq):
        a, b = (2 * p, 2 * p + 1) if rope.interleaved else (p, p + r // 2)
        for t, at in enumerate(pos.tolist()):
            turns = Fraction(at) * Fraction(f) / TWO_PI
            ang = sign * 2 * math.pi * float(turns - math.floor(turns))
            c, s = rope.scale * math.cos(ang), rope.scale * math.sin(ang)
            y[t, :, a], y[t, :, b] = x[t, :, a] * c - x[t, :, b] * s, x[t, :, b] * c + x[t, :, a] * s
            m = (np.abs(x[t, :, a]) + np.abs(x[t, :, b])) * abs(rope.scale)
            slack = m * (16 * 2.0 ** -24 + abs(at * f) * 2.0 ** -51)
            mag[t, :, a], mag[t, :, b] = slack, slack
    return y, mag


def check_rotation(got, x, pos, rope, sign=1):
    want, slack = want_rotation(x, pos, rope, sign)
    half = torch.finfo(got.dtype).eps / 2
    err = np.abs(got.double().cpu().numpy() - want)
    bound = slack + half * (np.abs(want) + slack)
    bound[..., rope.rotary_dim:] = 0.0
    assert np.all(err <= bound), (float(err.max()), np.argwhere(err > bound)[:3])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,hq,hkv,dim,rot", [(1, 4, 1, 128, 128), (7, 5, 2, 128, 64), (19, 28, 4, 128, 24),
                                              (3, 2, 2, 256, 256), (5, 1, 1, 66, 8)])
def test_rotation(dtype, inter, n, hq, hkv, dim, rot):
    g = torch.Generator().manual_seed(n * rot)
    q = torch.randn(n, hq, dim, generator=g).to("cuda", dtype)
    k = torch.randn(n, hkv, dim, generator=g).to("cuda", dtype)
    pos = torch.randint(0, 200000, (n,), generator=g)
    rope = wc.Rope(rot, base=1e4, interleaved=inter, scaling="by_parts", factor=4.0)
    qo, ko = wc.witcert_rope(rope, pos.cuda(), q, k)
    check_rotation(qo, q, pos, rope)
    check_rotation(ko, k, pos, rope)
    alone = wc.witcert_rope(rope, pos.cuda(), q)
    assert torch.equal(alone, qo)
    back = wc.witcert_rope(rope, pos.cuda(), q, inverse=True)
    check_rotation(back, q, pos, rope, sign=-1)
    wc.witcert_rope(rope, pos.cuda(), q, k, q_out=q, k_out=k)             # in place
    assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
def test_strides_and_alignment(dtype, inter):
    """Slices of a packed projection, head-major tensors, and rows that start on odd elements."""
    g = torch.Generator().manual_seed(5)
    rope, n, pos = wc.Rope(48, interleaved=inter), 9, torch.arange(100, 109)
    packed = torch.randn(n, 6 * 80 + 3, generator=g).to("cuda", dtype)
    heads = torch.randn(4, n, 80, generator=g).to("cuda", dtype).transpose(0, 1)
    for q in (packed[:, :320].view(n, 4, 80) if packed.shape[1] == 320 else packed[:, :320].unflatten(1, (4, 80)),
              packed[:, 1:321].unflatten(1, (4, 80)), heads):
        want = wc.witcert_rope(rope, pos.cuda(), q.contiguous())
        check_rotation(want, q, pos, rope)
        assert torch.equal(wc.witcert_rope(rope, pos.cuda(), q), want)
        out = torch.zeros(n, 4, 81, dtype=dtype, device="cuda")[..., :80]
        assert torch.equal(wc.witcert_rope(rope, pos.cuda(), q, q_out=out), want)


def test_far_and_negative_positions():
    rope = wc.Rope(128, base=1e6)
    pos = torch.tensor([0, 1, -1, -70000, 2 ** 24 + 1, 2 ** 31 + 7, -2 ** 33, 2 ** 36 + 12345])
    q = torch.randn(len(pos), 2, 128, generator=torch.Generator().manual_seed(1)).cuda()
    check_rotation(wc.witcert_rope(rope, pos.cuda(), q), q, pos, rope)


def test_many_tokens_many_heads_and_none():
    """Both launch shapes, against each other, token by token; and an empty call."""
    rope = wc.Rope(128)
    q = torch.randn(1500, 33, 128, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    pos = torch.arange(1500, device="cuda") * 3
    whole = wc.witcert_rope(rope, pos, q)
    parts = torch.cat([wc.witcert_rope(rope, pos[a:a + 100], q[a:a + 100]) for a in range(0, 1500, 100)])
    assert torch.equal(whole, parts)
    assert wc.witcert_rope(rope, pos[:0], q[:0]).shape == (0, 33, 128)


def test_gradient_is_the_inverse():
    """d/dx of <y, w> is the inverse rotation of w, also by central differences (fp32)."""
    rope = wc.Rope(32, scaling="by_parts", factor=2.0)
    g = torch.Generator().manual_seed(3)
    x, w = torch.randn(2, 1, 32, generator=g).cuda(), torch.randn(2, 1, 32, generator=g).cuda()
    pos = torch.tensor([5, 1000], device="cuda")
    grad = wc.witcert_rope(rope, pos, w, inverse=True)
    f = lambda z: (wc.witcert_rope(rope, pos, z).double() * w.double()).sum().item()
    for t, c in ((0, 0), (0, 17), (1, 3), (1, 31)):
        d = torch.zeros_like(x)
        d[t, 0, c] = 0.5
        # the map is linear: a central difference has no truncation error, only the rounding of 64 values
        # of a few units (16 2^-24 (|a| + |b|) each), under 1e-4 in all
        assert (f(x + d) - f(x - d)) == pytest.approx(grad[t, 0, c].item(), abs=1e-4)


# ------------------------------------------------------------------ rotated appends

def store(cache, layer, scheme):
    kinds = [_lib.X_K_CODES, _lib.X_V_CODES, _lib.X_WITNESS]
    kinds += [_lib.X_K_SCALES, _lib.X_V_SCALES] if scheme in ("int8_dither", "int8_rtn") else []
    kinds += [_lib.X_V_SCALES, _lib.X_V_ZEROS, _lib.X_KIVI_K_SCALE, _lib.X_KIVI_K_ZERO] if scheme == "kivi2" else []
    kinds += [_lib.X_V_WITNESS] if cache.v_witness else []
    return [cache.export(layer, k) for k in kinds]


def draws(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    k = torch.randn(*shape, 128, generator=g)
    k[..., 10:12] *= 6
    return k, torch.randn(*shape, 128, generator=g)


def hats(scheme, K, V, seed):
    if scheme != "blackbox":
        return None, None
    f = lambda x, s: torch.from_numpy(tensor_function(x.float().cpu().numpy(), s)).to(x.device, x.dtype)
    return f(K, seed), f(V, seed + 1)


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("dtype,rot,inter,hkv", [(torch.bfloat16, 128, False, 4), (torch.bfloat16, 72, False, 3),
                                                 (torch.bfloat16, 40, True, 2), (torch.float32, 128, True, 1),
                                                 (torch.float32, 64, False, 5)])
def test_rotated_append_stores_what_rotating_first_does(scheme, dtype, rot, inter, hkv):
    B, off = 2, 1000
    rope = wc.Rope(rot, base=1e4, interleaved=inter)
    mk = lambda: wc.Cache(1, hkv, hkv, B, 160, scheme, dtype=dtype, seed=9, pos_offset=off, v_witness=True)
    fused, plain = mk(), mk()
    at = 0
    for step, n in enumerate((1, 37, 1, 70, 16)):
        K, V = (x.to("cuda", dtype) for x in draws(100 + step, B, n, hkv))
        Kh, Vh = hats(scheme, K, V, step)
        pos = off + at + torch.arange(n, device="cuda").repeat(B)
        turn = lambda x: wc.witcert_rope(rope, pos, x.view(B * n, hkv, 128)).view(x.shape)
        fused.witcert_write_rope(0, K, V, rope, Kh, Vh)
        if Kh is None:
            plain.witcert_write(0, turn(K), V)
        else:
            plain.witcert_write_hat(0, turn(K), V, turn(Kh), Vh)
        at += n
        for a, b in zip(store(fused, 0, scheme), store(plain, 0, scheme)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    q = torch.randn(B, hkv, 128, generator=torch.Generator().manual_seed(7)).to("cuda", dtype)
    a, b = fused.decode(0, q, 1e-2), plain.decode(0, q, 1e-2)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1]["raw_a"], b[1]["raw_a"])


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("pages", [0, 40])
def test_rotated_ragged_append(scheme, pages):
    B, hkv = 4, 2
    rope = wc.Rope(128, base=1e6)
    mk = lambda: wc.Cache(1, hkv, hkv, B, 120, scheme, seed=3, max_pages=pages)
    fused, plain = mk(), mk()
    lens = [0] * B
    for step, n in enumerate(([5, 0, 33, 16], [1, 1, 1, 1], [0, 64, 3, 0], [2, 0, 0, 90])):
        K, V = (x.to("cuda", torch.bfloat16) for x in draws(step, sum(n), hkv))
        Kh, Vh = hats(scheme, K, V, step)
        pos = torch.cat([torch.arange(a, a + m) for a, m in zip(lens, n)]).cuda()
        fused.witcert_write_rope_ragged(0, K, V, n, rope, Kh, Vh)
        K2 = wc.witcert_rope(rope, pos, K)
        plain.witcert_write_ragged(0, K2, V, n, None if Kh is None else wc.witcert_rope(rope, pos, Kh), Vh)
        lens = [a + m for a, m in zip(lens, n)]
    for i in range(B):
        assert fused.witcert_seq_length(0, i) == lens[i]
    for a, b in zip(fused.read(0, lens), plain.read(0, lens)):
        assert torch.equal(a, b)
    q = torch.randn(B, hkv, 128, generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
    a, b = fused.decode(0, q, 1e-2), plain.decode(0, q, 1e-2)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1]["raw_a"], b[1]["raw_a"])


@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("pages", [0, 200])
@pytest.mark.parametrize("turn", [False, True])
def test_long_ragged_appends_equal_short_ones(scheme, pages, turn):
    """Appends that go by whole blocks (many rows at once) store what appends of few tokens do."""
    lens, hkv, at0 = [900, 0, 1307, 30], 16, [5, 3, 0, 16]
    rope = wc.Rope(128)
    mk = lambda: wc.Cache(1, hkv, hkv, 4, 1400, scheme, seed=8, max_pages=pages, v_witness=True)
    whole, parts = mk(), mk()
    K, V = (x.to("cuda", torch.bfloat16) for x in draws(3, sum(lens) + sum(at0), hkv))
    Kh, Vh = (K * 0.984375, V * 0.984375) if scheme == "blackbox" else (None, None)

    def write(c, rows, n):
        hat = (None, None) if Kh is None else (Kh[rows], Vh[rows])
        if turn:
            c.witcert_write_rope_ragged(0, K[rows], V[rows], n, rope, *hat)
        else:
            c.witcert_write_ragged(0, K[rows], V[rows], n, *hat)

    first = [sum(lens[:i]) for i in range(4)]
    head = torch.arange(sum(at0), device="cuda") + sum(lens)
    for c in (whole, parts):
        write(c, head, at0)
    write(whole, torch.arange(sum(lens), device="cuda"), lens)
    done = [0] * 4
    while done != lens:                                    # at most 301 tokens a sequence and call
        n = [min(301, a - b) for a, b in zip(lens, done)]
        rows = torch.cat([torch.arange(f + d, f + d + m) for f, d, m in zip(first, done, n)]).cuda()
        write(parts, rows, n)
        done = [a + b for a, b in zip(done, n)]
    total = [a + b for a, b in zip(lens, at0)]
    for a, b in zip(whole.read(0, total), parts.read(0, total)):
        assert torch.equal(a, b)
    for a, b in zip(store(whole, 0, scheme), store(parts, 0, scheme)):
        for i, m in enumerate(total):
            m = m // 16 if scheme == "kivi2" and a.shape[1] < 200 else m
            assert torch.equal(a[i, :m], b[i, :m])


@pytest.mark.parametrize("scheme", SCHEMES)
def test_long_uniform_appends_equal_short_ones(scheme):
    B, hkv, n = 2, 9, 1900                                 # 34200 rows: by whole blocks; 500 tokens: one by one
    whole, parts = (wc.Cache(1, hkv, hkv, B, n + 7, scheme, seed=8) for _ in range(2))
    K, V = (x.to("cuda", torch.bfloat16) for x in draws(4, B, n + 7, hkv))
    rope = wc.Rope(96, interleaved=True)
    for c, cuts in ((whole, [0, 7, n + 7]), (parts, [0, 7, 500, 1000, 1500, n + 7])):
        for a, b in zip(cuts, cuts[1:]):
            k, v = K[:, a:b].contiguous(), V[:, a:b].contiguous()
            c.witcert_write_rope(0, k, v, rope, *((k, v) if scheme == "blackbox" else ()))
    for a, b in zip(store(whole, 0, scheme), store(parts, 0, scheme)):
        assert torch.equal(a, b)


def test_rotated_keys_reach_the_backing_store():
    """A gated cache pages in the rotated exact keys, after bulk and single appends alike."""
    B, hkv, n = 1, 1, 80
    rope = wc.Rope(128)
    cache = wc.Cache(1, 1, 1, B, 96, "fp8_e4m3", max_repair_blocks=16)
    K, V = (x.to("cuda", torch.bfloat16) for x in draws(1, B, n + 1, hkv))
    cache.witcert_write_rope(0, K[:, :n].contiguous(), V[:, :n].contiguous(), rope)
    cache.witcert_write_rope(0, K[:, n:].contiguous(), V[:, n:].contiguous(), rope)
    cache.decode(0, torch.randn(1, 1, 128).bfloat16().cuda(), 1e-2)
    cache.witcert_gate(0, 0.0)
    assert cache.witcert_gate_stats()["blocks_paged_in"] == 6
    got = cache.read(0, [n + 1])[0]
    want = wc.witcert_rope(rope, torch.arange(n + 1, device="cuda"), K[0])
    assert torch.equal(got, want)


# ------------------------------------------------------------------ reads

@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_read_gives_the_oracle_values(scheme, dtype):
    B, hkv, n = 2, 3, 45
    cache = wc.Cache(2, hkv, hkv, B, 64, scheme, dtype=dtype, seed=(5 << 33) + 11, pos_offset=7 if scheme != "int8_dither" else 0)
    ref = OracleCache(2, hkv, hkv, B, scheme, (5 << 33) + 11, 1)
    K, V = (x.to(dtype).float() for x in draws(4, B, n, hkv))
    Kh, Vh = hats(scheme, K.to(dtype), V.to(dtype), 3)
    dev = lambda x: x.to("cuda", dtype)
    if Kh is None:
        cache.witcert_write(1, dev(K), dev(V))
        ref.write(1, K.numpy(), V.numpy())
    else:
        cache.witcert_write_hat(1, dev(K), dev(V), dev(Kh), dev(Vh))
        ref.write(1, K.numpy(), V.numpy(), Kh.float().numpy(), Vh.float().numpy())
    half = torch.finfo(dtype).eps / 2
    for t0, cnt in ((None, [n, n]), ([0, 0], [n, n]), ([3, 44], [20, 1]), ([0, 16], [0, 29]), (None, [1, 0])):
        got = cache.read(1, cnt, t0)
        for x, full in zip(got, (ref.khat[1], ref.vhat[1])):
            first = [n - c for c in cnt] if t0 is None else t0
            want = np.concatenate([full[i, a:a + c] for i, (a, c) in enumerate(zip(first, cnt))])
            assert tuple(x.shape) == want.shape
            # code - xi and zero + scale code are formed from operands of up to 128 scale (|x| <= 40 here):
            # three fp32 roundings of at most 2^-24 x 40, then half a step of the output
            err = np.abs(x.double().cpu().numpy() - want)
            assert np.all(err <= half * np.abs(want) * (1 + 2.0 ** -20) + 3 * 2.0 ** -24 * 40), float(err.max())


def test_read_refuses_rows_that_are_not_there():
    cache = wc.Cache(1, 1, 1, 2, 64, "fp8_e4m3")
    K = torch.zeros(2, 5, 1, 128, dtype=torch.bfloat16, device="cuda")
    cache.witcert_write(0, K, K)
    for n, t0 in (([6, 0], None), ([1, 1], [5, 0]), ([1, 1], [0, -1]), ([-1, 1], None)):
        with pytest.raises((wc.WitcertError, ValueError)):
            cache.read(0, n, t0)
    assert cache.read(0, [0, 0])[0].shape == (0, 1, 128)


# ------------------------------------------------------------------ truncation

@pytest.mark.parametrize("scheme", SCHEMES)
@pytest.mark.parametrize("pages", [0, 24])
@pytest.mark.parametrize("lens", [[48, 48, 48], [33, 48, 70]])
def test_truncated_rows_are_written_anew(scheme, pages, lens):
    """Append, drop the tail, append other tokens: the cache equals one that never held the tail."""
    B, hkv, n = 3, 2, 70
    keep = [min(a // 16 * 16, 64) for a in lens] if scheme == "kivi2" else lens
    mk = lambda: wc.Cache(1, hkv, hkv, B, 100, scheme, seed=2, max_pages=pages)
    a, b = mk(), mk()
    K, V = (x.to("cuda", torch.bfloat16) for x in draws(1, B, n, hkv))
    K2, V2 = (x.to("cuda", torch.bfloat16) for x in draws(2, B, 21, hkv))
    H = hats(scheme, K, V, 1) if scheme == "blackbox" else ()
    H2 = hats(scheme, K2, V2, 3) if scheme == "blackbox" else ()
    cut = lambda x: torch.cat([x[i, :m] for i, m in enumerate(keep)])
    flat = lambda x: x.reshape(-1, hkv, 128)
    write = (lambda c, *t: c.witcert_write_hat(0, *t)) if H else (lambda c, *t: c.witcert_write(0, *t))
    write(a, K, V, *H)
    a.witcert_truncate(-1, keep)
    b.witcert_write_ragged(0, cut(K), cut(V), keep, *(cut(h) for h in H))
    for c in (a, b):
        assert [c.witcert_seq_length(0, i) for i in range(B)] == keep
        c.witcert_write_ragged(0, flat(K2), flat(V2), [21] * B, *(flat(h) for h in H2))
    total = [m + 21 for m in keep]
    for x, y in zip(a.read(0, total), b.read(0, total)):
        assert torch.equal(x, y)
    q = torch.randn(B, hkv, 128, generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
    for x, y in zip(a.decode(0, q, 1e-2)[1].values(), b.decode(0, q, 1e-2)[1].values()):
        assert torch.equal(x, y) or (x.isnan().all() and y.isnan().all())


def test_truncate_refuses_and_ignores():
    cache = wc.Cache(2, 1, 1, 2, 64, "kivi2")
    K = torch.zeros(2, 40, 1, 128, dtype=torch.bfloat16, device="cuda")
    cache.witcert_write(0, K, K)
    for bad in ([31, 40], [40, -1]):
        with pytest.raises(wc.WitcertError):
            cache.witcert_truncate(0, bad)
        assert cache.witcert_length(0) == 40
    cache.witcert_truncate(0, [50, 40])               # nothing is longer: nothing changes
    assert cache.witcert_seq_length(0, 0) == 40
    cache.witcert_truncate(-1, [33, 32])              # within the unfinished block, and to a block's end
    assert [cache.witcert_seq_length(0, i) for i in (0, 1)] == [33, 32]
    with pytest.raises(wc.WitcertError):
        cache.witcert_truncate(2, [0, 0])


def test_truncate_makes_block_risks_stale():
    cache = wc.Cache(1, 1, 1, 1, 64, "fp8_e4m3", max_repair_blocks=4)
    K = torch.randn(1, 40, 1, 128, device="cuda").bfloat16()
    cache.witcert_write(0, K, K)
    cache.decode(0, K[:, 0], 1e-2)
    cache.witcert_truncate(0, [20])
    with pytest.raises(wc.WitcertError) as e:
        cache.witcert_gate(0, 0.5)
    assert e.value.status == _lib.ESTATE
