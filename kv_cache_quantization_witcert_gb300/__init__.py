"""Python binding of libwitcert (GB300 metered KV-cache decode).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch provides device memory and streams.  Function names follow
the C ABI (include/witcert.h): witcert_create / write / decode / gate / ...
"""
from __future__ import annotations

import array
import ctypes
import math

import torch

from . import _lib
from ._lib import (BF16, BLACKBOX, EINVAL, ENOMEM, EPAGEIN, ESTATE, ETIMEDOUT, F32, FP8_E4M3, INT8_DITHER,  # noqa: F401
                   INT8_RTN, KIVI2, SCHEMES, WitcertError, check, load)

__all__ = ["Cache", "Rope", "witcert_rope", "witcert_dither", "witcert_merge_partials", "witcert_gate_select", "witcert_beam_select",
           "witcert_beam_paths", "BeamSearch", "WitcertError", "load", "SCHEMES", "PART_STRIDE"]

_TORCH_DT = {F32: torch.float32, BF16: torch.bfloat16}


def _stream_ptr(stream) -> int:
    if stream is None:          # the current stream's handle, without a Stream object around it
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return int(stream.cuda_stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _torch_stream(stream):
    """The torch stream of a call's stream argument (None for the current one)."""
    return stream if stream is None or isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream.cuda_stream)


def _empty(stream, shape, dtype, device="cuda"):
    """An output or workspace of a call on `stream` (None: the current stream).  It comes from that
    stream's memory: a block freed on the current stream may still be in use by work queued there, which
    another stream does not wait for.  It may be used on the current stream too (ordering is the caller's)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    stream = _torch_stream(stream)
    here = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(here)
    return t


def _extent(t, i):
    """Extent i of a tensor argument, or None when it has none (_need then rejects it)."""
    return t.shape[i] if isinstance(t, torch.Tensor) and t.dim() > i else None


def _need(*specs):
    """Check the tensors a call hands the library, each spec (name, tensor, dtype, shape[,
    optional]) with None in shape for any extent: contiguous tensors of that dtype and shape,
    then all on a CUDA device.  The C ABI takes bare pointers, so a host tensor or a short
    buffer would reach a kernel; the binding raises ValueError instead."""
    for spec in specs:                          # what nearly every call passes: nothing to complain about
        t = spec[1]
        if t is None:
            if len(spec) > 4 and spec[4]:
                continue
            break
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == spec[2] and t.shape == spec[3] and t.is_contiguous()):
            break
    else:
        return
    given = []
    for name, t, dtype, shape, *opt in specs:
        if t is None:
            if opt and opt[0]:
                continue
            raise ValueError(f"{name} must not be None")
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.dim() != len(shape) or any(e is not None and e != x for e, x in zip(shape, t.shape)):
            want = tuple("*" if e is None else e for e in shape)
            raise ValueError(f"{name} must have shape {want}, got {tuple(t.shape)}")
        given.append((name, t))
    for name, t in given:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")


class Rope:
    """Rotary positions: the first `rotary_dim` channels of a head, pairs (p, p + rotary_dim/2) or,
    interleaved, (2p, 2p + 1), pair p turning base^(-2p / rotary_dim) radians a position.

    scaling None: as above.  "linear": every frequency / factor (position interpolation, Chen et
    al., 2023).  "by_parts" (Peng et al., "YaRN", 2023): pairs that turn more than `fast` times in
    the original_tokens the model was trained on keep their frequency, those under `slow` turns take
    frequency / factor, a linear ramp between; the vectors are scaled by 0.1 ln(factor) + 1.
    freq (rotary_dim / 2 radians per position) and scale override what these give."""

    def __init__(self, rotary_dim=128, base=10000.0, interleaved=False, scaling=None, factor=1.0,
                 original_tokens=4096, fast=32.0, slow=1.0, freq=None, scale=None):
        rotary_dim = int(rotary_dim)
        if rotary_dim < 8 or rotary_dim % 8 or rotary_dim > 256:
            raise ValueError(f"rotary_dim must be a multiple of 8 in [8, 256], got {rotary_dim}")
        if scaling not in (None, "linear", "by_parts"):
            raise ValueError(f'scaling must be None, "linear" or "by_parts", got {scaling!r}')
        if not (base > 0 and math.isfinite(base) and factor > 0 and math.isfinite(factor)):
            raise ValueError("base and factor must be positive and finite")
        gain = 1.0
        if freq is None:
            freq = [base ** (-2.0 * p / rotary_dim) for p in range(rotary_dim // 2)]
            if scaling == "linear":
                freq = [f / factor for f in freq]
            elif scaling == "by_parts":
                if not (fast > slow >= 0 and original_tokens > 0):
                    raise ValueError("by_parts needs fast > slow >= 0 and original_tokens > 0")
                keep = [min(max((original_tokens * f / (2 * math.pi) - slow) / (fast - slow), 0.0), 1.0) for f in freq]
                freq = [f * (k + (1 - k) / factor) for f, k in zip(freq, keep)]
                gain = 0.1 * math.log(factor) + 1.0
        elif len(freq) != rotary_dim // 2:
            raise ValueError(f"freq needs one entry per pair ({rotary_dim // 2}), got {len(freq)}")
        self.freq = tuple(float(f) for f in freq)
        self.scale = gain if scale is None else float(scale)
        if not (math.isfinite(self.scale) and all(math.isfinite(f) for f in self.freq)):
            raise ValueError("freq and scale must be finite")
        self.rotary_dim, self.interleaved = rotary_dim, bool(interleaved)
        self._cfg = _lib.witcert_rope_config(rotary_dim, int(self.interleaved), self.scale,
                                             (ctypes.c_double * 128)(*self.freq))

    @property
    def _ref(self):
        """Where this plan's own configuration lies (a copy has its own)."""
        return ctypes.addressof(self._cfg)


def _need_rope(rope, head_dim):
    if not isinstance(rope, Rope):
        raise ValueError(f"rope must be a Rope, got {type(rope).__name__}")
    if rope.rotary_dim > head_dim:
        raise ValueError(f"rope turns {rope.rotary_dim} channels of a head of {head_dim}")


def _rope_tensor(name, x, y, n_tok, like, stream=None):
    """A tensor [n_tok, heads, head_dim] with adjacent channels and its output (None: a new contiguous
    one): the output and what witcert_rope takes."""
    if isinstance(x, torch.Tensor) and y is None:
        y = _empty(stream if x.is_cuda else None, x.shape, x.dtype, x.device)
    for nm, t in ((name, x), (name + "_out", y)):
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{nm} must be a torch.Tensor, got {type(t).__name__}")
    xs, shape = x.stride(), x.shape
    ys = y.stride()
    if not (len(shape) == 3 and y.shape == shape and shape[0] == n_tok and shape[2] == like.shape[2] and
            x.dtype == like.dtype == y.dtype and xs[2] == 1 == ys[2] and x.is_cuda and y.is_cuda):
        for nm, t in ((name, x), (name + "_out", y)):
            if t.dim() != 3 or t.shape[0] != n_tok or t.shape[2] != like.shape[2] or t.shape[1] != x.shape[1]:
                raise ValueError(f"{nm} must have shape ({n_tok}, {x.shape[1] if x.dim() == 3 else '*'}, "
                                 f"{like.shape[2]}), got {tuple(t.shape)}")
            if t.dtype != like.dtype:
                raise ValueError(f"{nm} must be {like.dtype}, got {t.dtype}")
            if t.stride(2) != 1:
                raise ValueError(f"{nm} must have adjacent channels (stride 1), got stride {t.stride(2)}")
        raise ValueError(f"{name if not x.is_cuda else name + '_out'} must be a CUDA tensor")
    return y, _lib.witcert_rope_tensor(x.data_ptr(), y.data_ptr(), shape[1], xs[0], xs[1], ys[0], ys[1])


def witcert_rope(rope, positions, q, k=None, q_out=None, k_out=None, inverse=False, stream=None):
    """Rotate q [n_tok, heads, head_dim] and, if given, k [n_tok, kv_heads, head_dim] (bf16 or fp32, any
    token and head strides) by int64 positions [n_tok], in one launch.  Returns q_out, or (q_out, k_out);
    outputs are new contiguous tensors unless given (the input itself rotates in place).  inverse turns
    back: the gradient of the inputs from that of the outputs.  See witcert_rope in include/witcert.h."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a torch.Tensor [n_tok, heads, head_dim]")
    if q.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"q must be torch.bfloat16 or torch.float32, got {q.dtype}")
    n_tok, _, head_dim = q.shape
    _need_rope(rope, head_dim)
    _need(("positions", positions, torch.int64, (n_tok,)))
    q_out, tq = _rope_tensor("q", q, q_out, n_tok, q, stream)
    if k is not None:
        k_out, tk = _rope_tensor("k", k, k_out, n_tok, q, stream)
    elif k_out is not None:
        raise ValueError("k_out needs k")
    check(load().witcert_rope(rope._ref, BF16 if q.dtype == torch.bfloat16 else F32, head_dim, n_tok,
                              _ptr(positions), ctypes.addressof(tq), None if k is None else ctypes.addressof(tk),
                              int(bool(inverse)), _stream_ptr(stream)), "witcert_rope")
    return q_out if k is None else (q_out, k_out)


class Cache:
    """One WitCert cache: compressed K/V store, witnesses, optional gate state."""

    def __init__(self, n_layers, n_q_heads, n_kv_heads, batch, max_tokens, scheme="int8_dither",
                 dtype=torch.bfloat16, seed=0, total_steps=1, n_splits=0, max_repair_blocks=0, pos_offset=0,
                 v_witness=False, max_pages=0):
        lib = load()
        self.dtype = dtype
        self.cfg = _lib.witcert_config(n_layers, n_q_heads, n_kv_heads, 128, batch, max_tokens,
                                       SCHEMES[scheme] if isinstance(scheme, str) else scheme,
                                       BF16 if dtype == torch.bfloat16 else F32, seed, total_steps, n_splits,
                                       max_repair_blocks, pos_offset, int(bool(v_witness)), max_pages)
        self.scheme = scheme
        self.v_witness = bool(v_witness)
        h = ctypes.c_void_p()
        check(lib.witcert_create(ctypes.byref(self.cfg), ctypes.byref(h)), "witcert_create")
        self._h = h

    # ------------------------------------------------------------------ ABI calls
    def _kv_shape(self, n_tok=None):
        return (self.cfg.batch, n_tok, self.cfg.n_kv_heads, 128)

    def _q_shape(self, last=128):
        return (self.cfg.batch, self.cfg.n_q_heads, last)

    def _decode_args(self, q, out, meters):
        names = ("meter_a", "meter_b", "raw_a", "raw_b", "meter_v")
        _need(("q", q, self.dtype, self._q_shape()), ("out", out, torch.float32, self._q_shape()),
              *((n, m, torch.float32, self._q_shape()[:2], True) for n, m in zip(names, meters)))

    def witcert_write(self, layer, K, V, stream=None):
        """Append K, V [batch, n_tok, n_kv_heads, 128] to every sequence of `layer`."""
        n_tok = _extent(K, 1)
        _need(("K", K, self.dtype, self._kv_shape(n_tok)), ("V", V, self.dtype, self._kv_shape(n_tok)))
        check(load().witcert_write(self._h, layer, _ptr(K), _ptr(V), n_tok, _stream_ptr(stream)), "witcert_write")

    def witcert_write_hat(self, layer, K, V, K_hat, V_hat, stream=None):
        """Black-box scheme: K_hat, V_hat are the tensor function's outputs f(K), f(V)."""
        n_tok = _extent(K, 1)
        _need(*((name, t, self.dtype, self._kv_shape(n_tok)) for name, t in
                (("K", K), ("V", V), ("K_hat", K_hat), ("V_hat", V_hat))))
        check(load().witcert_write_hat(self._h, layer, _ptr(K), _ptr(V), _ptr(K_hat), _ptr(V_hat), n_tok,
                                       _stream_ptr(stream)), "witcert_write_hat")

    def _counts(self, name, values):
        """One host integer per sequence, as the library takes them."""
        batch = self.cfg.batch
        if type(values) is list and len(values) == batch:
            try:                                # whole numbers that fit: what nearly every call passes
                arr = array.array("i", values)
                return arr.tolist(), (ctypes.c_int32 * batch).from_buffer(arr)
            except (TypeError, OverflowError):
                pass
        counts = [int(x) for x in values]
        if len(counts) != batch:
            raise ValueError(f"{name} needs one count per sequence ({batch}), got {len(counts)}")
        try:
            return counts, (ctypes.c_int32 * batch).from_buffer(array.array("i", counts))
        except OverflowError:
            raise ValueError(f"{name} must fit 32 bits, got {counts}") from None

    def witcert_write_rope(self, layer, K, V, rope, K_hat=None, V_hat=None, stream=None):
        """witcert_write (witcert_write_hat with K_hat, V_hat) of keys without positions: each is turned by
        its position in the sequence on the way into the cache."""
        n_tok = _extent(K, 1)
        _need_rope(rope, 128)
        shape = self._kv_shape(n_tok)
        _need(("K", K, self.dtype, shape), ("V", V, self.dtype, shape), ("K_hat", K_hat, self.dtype, shape, True),
              ("V_hat", V_hat, self.dtype, shape, True))
        check(load().witcert_write_rope(self._h, layer, _ptr(K), _ptr(V), _ptr(K_hat), _ptr(V_hat), n_tok, rope._ref,
                                        _stream_ptr(stream)), "witcert_write_rope")

    def witcert_write_rope_ragged(self, layer, K, V, n_tok, rope, K_hat=None, V_hat=None, stream=None):
        """witcert_write_ragged of keys without positions (see witcert_write_rope)."""
        counts, arr = self._counts("n_tok", n_tok)
        _need_rope(rope, 128)
        shape = (sum(counts), self.cfg.n_kv_heads, 128)
        _need(("K", K, self.dtype, shape), ("V", V, self.dtype, shape), ("K_hat", K_hat, self.dtype, shape, True),
              ("V_hat", V_hat, self.dtype, shape, True))
        check(load().witcert_write_rope_ragged(self._h, layer, _ptr(K), _ptr(V), _ptr(K_hat), _ptr(V_hat), arr,
                                               rope._ref, _stream_ptr(stream)), "witcert_write_rope_ragged")

    def witcert_truncate(self, layer, lengths, stream=None):
        """Keep the first lengths[i] tokens of sequence i in `layer` (-1: every layer)."""
        _, arr = self._counts("lengths", lengths)
        check(load().witcert_truncate(self._h, layer, arr, _stream_ptr(stream)), "witcert_truncate")

    def witcert_fork(self, parents, lengths=None, stream=None):
        """Sequence i takes, in every layer, the first lengths[i] tokens (None: all) of what sequence parents[i]
        holds (-1: none, it is empty then).  See witcert_fork in include/witcert.h."""
        _, arr = self._counts("parents", parents)
        cut = None if lengths is None else self._counts("lengths", lengths)[1]
        check(load().witcert_fork(self._h, arr, cut, _stream_ptr(stream)), "witcert_fork")

    def witcert_read(self, layer, t0, n_tok, K, V, stream=None):
        """Tokens t0[i] .. t0[i] + n_tok[i] - 1 of every sequence (t0 None: the last n_tok[i]) as rows
        K, V [sum(n_tok), Hkv, 128] of the cache's dtype."""
        counts, arr = self._counts("n_tok", n_tok)
        start = None if t0 is None else self._counts("t0", t0)[1]
        shape = (sum(counts), self.cfg.n_kv_heads, 128)
        _need(("K", K, self.dtype, shape), ("V", V, self.dtype, shape))
        self._read(layer, start, arr, K, V, stream)

    def _read(self, layer, start, arr, K, V, stream):
        check(load().witcert_read(self._h, layer, start, arr, _ptr(K), _ptr(V), _stream_ptr(stream)), "witcert_read")

    def witcert_attend_workspace(self, layer, n_tok):
        """Bytes of workspace that witcert_attend needs for these counts."""
        _, arr = self._counts("n_tok", n_tok)
        n = ctypes.c_size_t()
        check(load().witcert_attend_workspace(self._h, layer, arr, ctypes.byref(n)), "witcert_attend_workspace")
        return n.value

    def witcert_attend(self, layer, q, n_tok, out, workspace, stream=None):
        """Causal attention of each sequence's last n_tok[i] tokens, q [sum(n_tok), Hq, 128] bf16, over the
        cache, into out (q's shape, bf16)."""
        counts, arr = self._counts("n_tok", n_tok)
        shape = (sum(counts), self.cfg.n_q_heads, 128)
        _need(("q", q, torch.bfloat16, shape), ("out", out, torch.bfloat16, shape),
              ("workspace", workspace, torch.uint8, (None,)))
        self._attend(layer, q, arr, out, workspace, stream)

    def _attend(self, layer, q, arr, out, workspace, stream):
        check(load().witcert_attend(self._h, layer, _ptr(q), arr, _ptr(out), _ptr(workspace), workspace.numel(),
                                    _stream_ptr(stream)), "witcert_attend")

    def attend(self, layer, q, n_tok, stream=None):
        """Chunk attention with a fresh output and workspace (see witcert_attend)."""
        counts, arr = self._counts("n_tok", n_tok)
        n = ctypes.c_size_t()
        check(load().witcert_attend_workspace(self._h, layer, arr, ctypes.byref(n)), "witcert_attend_workspace")
        _need(("q", q, torch.bfloat16, (sum(counts), self.cfg.n_q_heads, 128)))
        out = _empty(stream, q.shape, q.dtype, q.device)
        workspace = _empty(stream, n.value, torch.uint8, q.device)
        self._attend(layer, q, arr, out, workspace, stream)
        return out

    def witcert_write_ragged(self, layer, K, V, n_tok, K_hat=None, V_hat=None, stream=None):
        """Ragged append: n_tok[i] tokens to sequence i; K, V (and K_hat, V_hat for black-box
        caches) packed sequence by sequence, [sum(n_tok), Hkv, 128]."""
        counts, arr = self._counts("n_tok", n_tok)
        shape = (sum(counts), self.cfg.n_kv_heads, 128)
        _need(("K", K, self.dtype, shape), ("V", V, self.dtype, shape), ("K_hat", K_hat, self.dtype, shape, True),
              ("V_hat", V_hat, self.dtype, shape, True))
        check(load().witcert_write_ragged(self._h, layer, _ptr(K), _ptr(V), _ptr(K_hat), _ptr(V_hat), arr,
                                          _stream_ptr(stream)), "witcert_write_ragged")

    def witcert_reset_sequence(self, seq, stream=None):
        check(load().witcert_reset_sequence(self._h, int(seq), _stream_ptr(stream)), "witcert_reset_sequence")

    def witcert_seq_length(self, layer, seq):
        n = ctypes.c_int()
        check(load().witcert_seq_length(self._h, layer, int(seq), ctypes.byref(n)), "witcert_seq_length")
        return n.value

    def witcert_decode(self, layer, q, delta_req, out, meter_a=None, meter_b=None, raw_a=None, raw_b=None,
                       meter_v=None, stream=None):
        self._decode_args(q, out, (meter_a, meter_b, raw_a, raw_b, meter_v))
        check(load().witcert_decode(self._h, layer, _ptr(q), float(delta_req), _ptr(out), _ptr(meter_a),
                                    _ptr(meter_b), _ptr(raw_a), _ptr(raw_b), _ptr(meter_v), _stream_ptr(stream)),
              "witcert_decode")

    def witcert_decode_noalloc(self, layer, q, delta_req, out, meter_a=None, meter_b=None, raw_a=None, raw_b=None,
                               meter_v=None, stream=None):
        self._decode_args(q, out, (meter_a, meter_b, raw_a, raw_b, meter_v))
        check(load().witcert_decode_noalloc(self._h, layer, _ptr(q), float(delta_req), _ptr(out), _ptr(meter_a),
                                            _ptr(meter_b), _ptr(raw_a), _ptr(raw_b), _ptr(meter_v),
                                            _stream_ptr(stream)), "witcert_decode_noalloc")

    def witcert_decode_partial(self, layer, q, delta_req, s_total, part, stream=None):
        _need(("q", q, self.dtype, self._q_shape()), ("part", part, torch.float32, self._q_shape(PART_STRIDE)))
        check(load().witcert_decode_partial(self._h, layer, _ptr(q), float(delta_req), int(s_total), _ptr(part),
                                            _stream_ptr(stream)), "witcert_decode_partial")

    def decode_partial(self, layer, q, delta_req, s_total, stream=None):
        """This shard's per-cell records [B, Hq, 136] (see witcert_decode_partial)."""
        part = _empty(stream, (q.shape[0], q.shape[1], PART_STRIDE), torch.float32, q.device)
        self.witcert_decode_partial(layer, q, delta_req, s_total, part, stream=stream)
        return part

    def witcert_gate(self, layer, tau, stream=None):
        check(load().witcert_gate(self._h, layer, float(tau), _stream_ptr(stream)), "witcert_gate")

    def witcert_inject_fault(self, fault, layer):
        """Host-side fault injection (see witcert_inject_fault in include/witcert.h)."""
        check(load().witcert_inject_fault(self._h, int(fault), int(layer)), "witcert_inject_fault")

    def witcert_gate_stats(self, timeout_ms=10000):
        s = _lib.witcert_gate_counters()
        check(load().witcert_gate_stats(self._h, ctypes.byref(s), timeout_ms), "witcert_gate_stats")
        return {f: getattr(s, f) for f, _ in s._fields_}

    def witcert_stats(self):
        s = _lib.witcert_stats_t()
        check(load().witcert_stats(self._h, ctypes.byref(s)), "witcert_stats")
        return {f: getattr(s, f) for f, _ in s._fields_}

    def witcert_set_profiling(self, on):
        check(load().witcert_set_profiling(self._h, int(bool(on))), "witcert_set_profiling")

    def witcert_set_launch_overlap(self, on):
        check(load().witcert_set_launch_overlap(self._h, int(bool(on))), "witcert_set_launch_overlap")

    def witcert_length(self, layer):
        n = ctypes.c_int()
        check(load().witcert_length(self._h, layer, ctypes.byref(n)), "witcert_length")
        return n.value

    def witcert_export(self, layer, what, dst, stream=None):
        _need(("dst", dst, getattr(dst, "dtype", None), tuple(getattr(dst, "shape", ()))))   # the library checks the size
        check(load().witcert_export(self._h, layer, what, _ptr(dst), dst.numel() * dst.element_size(),
                                    _stream_ptr(stream)), "witcert_export")

    def close(self):
        if getattr(self, "_h", None):
            check(load().witcert_destroy(self._h), "witcert_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------------ conveniences (allocation + the calls above)
    def decode(self, layer, q, delta_req, meters=True, stream=None):
        B, Hq = q.shape[0], q.shape[1]
        out = _empty(stream, (B, Hq, 128), torch.float32, q.device)
        if not meters:
            self.witcert_decode(layer, q, delta_req, out, stream=stream)
            return out, None
        m = _empty(stream, (5, B, Hq), torch.float32, q.device)
        self.witcert_decode(layer, q, delta_req, out, m[0], m[1], m[2], m[3], m[4] if self.v_witness else None,
                            stream=stream)
        meters = {"meter_a": m[0], "meter_b": m[1], "raw_a": m[2], "raw_b": m[3]}
        if self.v_witness:
            meters["meter_v"] = m[4]
        return out, meters

    def read(self, layer, n_tok, t0=None, stream=None):
        """Keys and values the cache stands for, packed [sum(n_tok), Hkv, 128] (see witcert_read)."""
        counts, arr = self._counts("n_tok", n_tok)
        start = None if t0 is None else self._counts("t0", t0)[1]
        shape = (max(sum(counts), 0), self.cfg.n_kv_heads, 128)      # the library refuses negative counts
        K, V = _empty(stream, shape, self.dtype), _empty(stream, shape, self.dtype)
        self._read(layer, start, arr, K, V, stream)
        return K, V

    def export(self, layer, what, stream=None):
        B, Hkv, Hq = self.cfg.batch, self.cfg.n_kv_heads, self.cfg.n_q_heads
        S = self.witcert_length(layer)
        nblk = (S + 15) // 16
        dev = torch.device("cuda", torch.cuda.current_device())
        code_dt = torch.bfloat16 if self.cfg.scheme == BLACKBOX else torch.uint8
        shapes = {
            _lib.X_K_CODES: ((B, S, Hkv, 128), code_dt), _lib.X_V_CODES: ((B, S, Hkv, 128), code_dt),
            _lib.X_K_SCALES: ((B, S, Hkv, 4), torch.float16), _lib.X_V_SCALES: ((B, S, Hkv, 4), torch.float16),
            _lib.X_V_ZEROS: ((B, S, Hkv, 4), torch.float16),
            _lib.X_KIVI_K_SCALE: ((B, nblk, Hkv, 128), torch.float16),
            _lib.X_KIVI_K_ZERO: ((B, nblk, Hkv, 128), torch.float16),
            _lib.X_WITNESS: ((B, S, Hkv, 16), torch.float16), _lib.X_SLOTS: ((B, Hkv, nblk), torch.int32),
            _lib.X_BLOCK_RISK: ((B, Hq, nblk), torch.float32), _lib.X_V_WITNESS: ((B, S, Hkv), torch.float16),
        }
        shape, dt = shapes[what]
        dst = _empty(stream, shape, dt, dev)
        if dst.numel():
            self.witcert_export(layer, what, dst, stream=stream)
        return dst


PART_STRIDE = 136     # floats per (sequence, query head) record: m, Z, S_A, S_B, S_V, 3 unused, 128 value sums


def witcert_merge_partials(parts, scheme, out=None, meters=True, stream=None):
    """Merge shard records parts [B, Hq, n_parts, 136] (device fp32) into the output [B, Hq, 128]
    and, with meters, {"meter_a", "meter_b", "raw_a", "raw_b", "meter_v"} (see witcert_merge_partials)."""
    _need(("parts", parts, torch.float32, (None, None, None, PART_STRIDE)))
    B, Hq, n = parts.shape[0], parts.shape[1], parts.shape[2]
    if out is None:
        out = _empty(stream, (B, Hq, 128), torch.float32, parts.device)
    _need(("out", out, torch.float32, (B, Hq, 128)))
    m = _empty(stream, (5, B, Hq), torch.float32, parts.device) if meters else None
    ptrs = tuple(_ptr(m[k]) for k in range(5)) if meters else (None,) * 5
    check(load().witcert_merge_partials(_ptr(parts), n, B, Hq, SCHEMES[scheme] if isinstance(scheme, str) else scheme,
                                        _ptr(out), *ptrs, _stream_ptr(stream)), "witcert_merge_partials")
    return out, ({"meter_a": m[0], "meter_b": m[1], "raw_a": m[2], "raw_b": m[3], "meter_v": m[4]}
                 if meters else None)


def witcert_gate_select(risk, n_kv_heads, tau, repaired=None, selected=None, stream=None):
    """The gate's block selection on caller arrays: risk [B, Hq, nblk] float32 (device), repaired
    [B, Hkv, nblk] uint8 or None; returns the selection bitmap [B, Hkv, nblk // 32 + 1] int32
    (see witcert_gate_select)."""
    _need(("risk", risk, torch.float32, (None, None, None)))
    B, Hq, nblk = risk.shape
    _need(("repaired", repaired, torch.uint8, (B, n_kv_heads, nblk), True))
    if selected is None:
        selected = _empty(stream, (B, n_kv_heads, nblk // 32 + 1), torch.int32, risk.device)
    _need(("selected", selected, torch.int32, (B, n_kv_heads, nblk // 32 + 1)))
    check(load().witcert_gate_select(_ptr(risk), _ptr(repaired), B, Hq, n_kv_heads, nblk, float(tau), _ptr(selected),
                                     _stream_ptr(stream)), "witcert_gate_select")
    return selected


def _here(name, t, *others):
    """Check that a call's tensors lie on the current CUDA device, where the library launches."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    dev = torch._C._cuda_getDevice()
    for x in (t, *others):
        if x is not None and x.get_device() != dev:
            raise ValueError(f"{name} and what goes with it must be on the current device (cuda:{dev}), got {x.device}")


def witcert_beam_select(logits, scores, n_out=None, finished=None, eos=-1, out=None, stream=None):
    """Each request's n_out (None: as many as beams) best continuations: logits [R, W, V] bf16 or float32 (any
    request and beam strides, tokens adjacent), cumulative log-probabilities scores [R, W] float32, finished
    [R, W] bool or None.  Returns (scores float32, rows int32, tokens int32, finished bool), each [R, n_out]: a
    row is request * W + beam, -1 where there is no candidate.  out: a tuple of four tensors to write, the
    last of them or the input's own for scores and finished as witcert_beam_step in include/witcert.h allows."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 3:
        raise ValueError("logits must be a torch.Tensor [requests, beams, vocabulary]")
    R, W, V = logits.shape
    xs, dev = logits.stride(), logits.device
    n = W if n_out is None else int(n_out)
    if logits.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"logits must be torch.bfloat16 or torch.float32, got {logits.dtype}")
    if V != 1 and xs[2] != 1:
        raise ValueError(f"logits must have adjacent tokens (stride 1), got stride {xs[2]}")
    _need(("scores", scores, torch.float32, (R, W)), ("finished", finished, torch.bool, (R, W), True))
    if out is not None:
        if not isinstance(out, (tuple, list)) or len(out) != 4:
            raise ValueError("out needs a tuple of four tensors (scores, rows, tokens, finished)")
        _need(*((name, t, dt, (R, n)) for name, t, dt in zip(("out scores", "rows", "tokens", "out finished"), out,
                                                            (torch.float32, torch.int32, torch.int32, torch.bool))))
    _here("logits", logits, scores, finished, *(out or ()))
    if out is None:
        shape = (R, max(n, 0))
        out = (_empty(stream, shape, torch.float32, dev), _empty(stream, shape, torch.int32, dev),
               _empty(stream, shape, torch.int32, dev), _empty(stream, shape, torch.bool, dev))
    step = _lib.witcert_beam_step(BF16 if logits.dtype == torch.bfloat16 else F32, R, W, V, n, int(eos), logits.data_ptr(),
                                  xs[0], xs[1], scores.data_ptr(), _ptr(finished), *[t.data_ptr() for t in out])
    size = 12 * R * W * (V // 512 + 2)                     # what witcert_beam_workspace says is at most this
    workspace = _empty(stream, size, torch.uint8, dev)
    check(load().witcert_beam_select(ctypes.addressof(step), workspace.data_ptr(), size, _stream_ptr(stream)),
          "witcert_beam_select")
    return tuple(out)


def witcert_beam_paths(rows, tokens, length=None, pad=-1, out=None, stream=None):
    """The token sequences [R, W, T] int32 of the last beams: rows, tokens [T, R, W] int32 as witcert_beam_select
    chose them step by step, length [R] int32 steps that count (None: all), pad elsewhere (see
    witcert_beam_paths in include/witcert.h)."""
    T, R, W = (_extent(rows, i) for i in range(3))
    _need(("rows", rows, torch.int32, (T, R, W)), ("tokens", tokens, torch.int32, (T, R, W)),
          ("length", length, torch.int32, (R,), True), ("out", out, torch.int32, (R, W, T), True))
    _here("rows", rows, tokens, length, out)
    if out is None:
        out = _empty(stream, (R, W, T), torch.int32, rows.device)
    check(load().witcert_beam_paths(_ptr(rows), _ptr(tokens), T, R, W, _ptr(length), int(pad), _ptr(out),
                                    _stream_ptr(stream)), "witcert_beam_paths")
    return out


class BeamSearch:
    """A beam search of n_beams a request over a cache: sequence r * n_beams + b is beam b of request r.

    Write each request's prompt to its first beam's sequence, then start(); every step() takes the logits of
    all beams, chooses their continuations, and moves the cache's sequences to where the chosen beams are.
    It returns the tokens [R, W] int32 (-1: the request has no beam there) that the next step appends.  A
    finished beam keeps its score and goes on with eos; paths() gives the sequences so far, scores the
    beams' log-probabilities, falling."""

    def __init__(self, cache, n_beams, max_steps, eos=-1):
        batch = cache.cfg.batch
        if n_beams < 1 or batch % n_beams:
            raise ValueError(f"the cache's batch ({batch}) must be a multiple of n_beams ({n_beams})")
        if max_steps < 1:
            raise ValueError(f"max_steps must be at least 1, got {max_steps}")
        self.cache, self.eos, self.steps = cache, int(eos), 0
        self.shape = R, W = batch // n_beams, int(n_beams)
        dev = torch.device("cuda", torch.cuda.current_device())
        self._rows = torch.empty((int(max_steps), R, W), dtype=torch.int32, device=dev)
        self._tokens = torch.empty_like(self._rows)
        self.scores = torch.empty((R, W), dtype=torch.float32, device=dev)
        self.finished = torch.empty((R, W), dtype=torch.bool, device=dev)
        self._restart()

    def _restart(self):
        self.steps = 0
        self.scores.fill_(-math.inf)
        self.scores[:, 0] = 0.0
        self.finished.fill_(False)

    def start(self, stream=None):
        """Hand each request's prompt, in its first beam's sequence, to the other beams."""
        W = self.shape[1]
        self.cache.witcert_fork([i // W * W for i in range(self.cache.cfg.batch)], stream=stream)
        with torch.cuda.stream(_torch_stream(stream)):
            self._restart()

    def step(self, logits, stream=None):
        """Choose the continuations of all beams from logits [R, W, V] (or [R * W, V], a row a sequence of the
        cache) and move the cache's sequences."""
        if self.steps == len(self._rows):
            raise ValueError(f"the search was made for {len(self._rows)} steps")
        if isinstance(logits, torch.Tensor) and logits.dim() == 2 and logits.shape[0] == self.shape[0] * self.shape[1]:
            logits = logits.unflatten(0, self.shape)
        if not isinstance(logits, torch.Tensor) or tuple(logits.shape[:2]) != self.shape:
            raise ValueError(f"logits must be a torch.Tensor [{self.shape[0]}, {self.shape[1]}, vocabulary]")
        rows, tokens = self._rows[self.steps], self._tokens[self.steps]
        done = self.finished if self.eos >= 0 else None
        witcert_beam_select(logits, self.scores, finished=done, eos=self.eos,
                            out=(self.scores, rows, tokens, self.finished), stream=stream)
        with torch.cuda.stream(_torch_stream(stream)):
            parents = rows.flatten().tolist()
        # a request with fewer candidates than beams leaves the others where they are
        self.cache.witcert_fork([i if p < 0 else p for i, p in enumerate(parents)], stream=stream)
        self.steps += 1
        return tokens

    def paths(self, pad=-1, stream=None):
        """The beams' tokens so far, [R, W, steps] int32."""
        return witcert_beam_paths(self._rows[:self.steps], self._tokens[:self.steps], pad=pad, stream=stream)


def witcert_quotient_selftest(n_f32=4096, seed=0, stream=None):
    """Differing quotients between the writers' x / s and the IEEE quotient over every positive
    fp16 scale (see witcert_quotient_selftest); expected 0."""
    n = ctypes.c_uint64()
    check(load().witcert_quotient_selftest(int(n_f32), int(seed), ctypes.byref(n), _stream_ptr(stream)),
          "witcert_quotient_selftest")
    return n.value


def witcert_wait_selftest(limit_ns, stream=None):
    """Run the bounded device wait against a barrier nothing completes; returns the status code."""
    return load().witcert_wait_selftest(int(limit_ns), _stream_ptr(stream))


def witcert_dither(seed, layer, kv_head, t0, n, tensor, out=None, stream=None):
    """Device dither xi [n, 128] float32 (see witcert_dither in include/witcert.h)."""
    if out is None:
        out = _empty(stream, (n, 128), torch.float32)
    _need(("out", out, torch.float32, (n, 128)))
    check(load().witcert_dither(seed, layer, kv_head, t0, n, tensor, _ptr(out), _stream_ptr(stream)),
          "witcert_dither")
    return out
