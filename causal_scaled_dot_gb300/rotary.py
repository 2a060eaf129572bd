"""Rotary positions and norms of heads over libattn's entry points (``attn_rope``, ``attn_rope_bwd`` in
include/attn.h): what stands between a layer's QKV projection and its attention, in one pass.

    rotary = Rotary.from_base(128)                       # the model's positions, once
    q, k, v = rotary.heads(qkv, Hq, Hkv)                 # qkv [B, S, (Hq + 2 Hkv) D] bf16, as projected
    o = native.attention_trainable(q, k, v)              # takes q, k, v [B, H, S, D] contiguous
    q, k = rotary.rotate(q, k, q_norm=wq, k_norm=wk)     # heads by themselves, any strides; norms before the rotation

Gradients flow to the heads and to the norms' weights.  For text after a prompt ``KVCache.append``
(kv_cache.py) takes the same plan and writes the rotated K straight into the 8-bit cache.

Argument marshalling only: the work runs in the CUDA library.
"""
from __future__ import annotations

import ctypes
import math
import weakref

import torch

from . import native
from .autograd import refuse_tangents, tied

# 1 / (2 pi) to 256 bits, from pi to 100 decimals (OEIS A000796).
_PER_TURN = (10**100 << 255) // int("31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679")
_STRIDES = ctypes.c_longlong * 3
_BF16 = torch.bfloat16
_INDEX = {torch.int32: 0, torch.int64: 1}
# The current stream's handle by device index, without a Stream object.
_stream_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None) or torch.cuda.is_current_stream_capturing


def _frequencies(rotary_dim: int, base: float, stretch: float) -> list[float]:
    if rotary_dim % 2 or not base > 0 or not stretch > 0:
        raise ValueError("rotary_dim must be even, base and stretch positive")
    return [base ** (-2 * i / rotary_dim) for i in range(rotary_dim // 2)]


def _turns(x: float) -> int:
    """x / (2 pi) in 2^-64 turns, to nearest, whole turns dropped: the angle of position p is then p times it, mod 2^64."""
    n, d = x.as_integer_ratio()  # d is a power of two
    return ((n * _PER_TURN >> d.bit_length() - 1 + 256 - 65) + 1 >> 1) % 2**64


class Rotary:
    """How a model's heads turn with their position: pair i of a head's first ``2 * len(frequencies)``
    elements turns by ``position * frequencies[i]`` radians, and is scaled by ``factor``.  The pairs are
    (i, i + len(frequencies)), or neighbours (2i, 2i + 1) when ``interleaved``; the rest of the head stays.
    No frequencies: no rotation (norms and the change of layout remain).

    The frequencies are held as 64-bit fractions of a turn, and there is no table: cos and sin of position p
    are within 2^-22 + abs(p) 2^-62.  A Rotary holds no device memory, so it serves every device."""

    def __init__(self, frequencies, interleaved: bool = False, factor: float = 1.0):
        f = [float(x) for x in (frequencies.tolist() if hasattr(frequencies, "tolist") else frequencies)]
        if len(f) > 64 or len(f) % (4 if interleaved else 8):
            raise ValueError(f"{len(f)} frequencies: at most 64, in multiples of {4 if interleaved else 8}, are needed "
                             f"({'neighbouring' if interleaved else 'half-way'} pairs)")
        if not all(map(math.isfinite, f)) or not math.isfinite(factor):
            raise ValueError("frequencies and factor must be finite")
        self.frequencies = tuple(f)
        self.rotary_dim = 2 * len(f)
        self.interleaved = bool(interleaved)
        self.factor = float(factor)
        turns = [_turns(x) for x in f]
        self._c = native.AttnRope((ctypes.c_ulonglong * 64)(*turns), self.rotary_dim, int(self.interleaved), self.factor)

    def __reduce__(self):  # the struct of the C calls is made again
        return type(self), (self.frequencies, self.interleaved, self.factor)

    def __repr__(self):
        return f"Rotary({self.rotary_dim} elements, {'neighbouring' if self.interleaved else 'half-way'} pairs, factor {self.factor:g})"

    @classmethod
    def from_base(cls, rotary_dim: int, base: float = 10000.0, stretch: float = 1.0, interleaved: bool = False):
        """frequencies[i] = base^(-2i / rotary_dim) / stretch: a stretch of s puts s positions where one was."""
        return cls([f / stretch for f in _frequencies(rotary_dim, base, stretch)], interleaved)

    @classmethod
    def raised_base(cls, rotary_dim: int, stretch: float, base: float = 10000.0, interleaved: bool = False):
        """The base raised so that the slowest pair is stretched by ``stretch`` and the fastest stays."""
        if rotary_dim < 4:
            raise ValueError("rotary_dim must be 4 or more")
        if not stretch > 0:
            raise ValueError("stretch must be positive")
        return cls(_frequencies(rotary_dim, base * stretch ** (rotary_dim / (rotary_dim - 2)), 1.0), interleaved)

    @classmethod
    def by_parts(cls, rotary_dim: int, stretch: float, original_length: float, base: float = 10000.0, slow: float = 1.0,
                 fast: float = 32.0, interleaved: bool = False, factor: float | None = None):
        """Pairs with at most ``slow`` turns over the original length are stretched, those with at least ``fast``
        stay, and between them the share that stays grows with the turns ("YaRN: Efficient Context Window
        Extension of Large Language Models", Peng et al., 2023, section 3.2; section 3.3's factor
        0.1 ln(stretch) + 1, unless another is given)."""
        if not fast > slow:
            raise ValueError("fast must be larger than slow")
        out = []
        for f in _frequencies(rotary_dim, base, stretch):
            keep = min(max((original_length * f / math.tau - slow) / (fast - slow), 0.0), 1.0)
            out.append(f * (keep + (1 - keep) / stretch))
        return cls(out, interleaved, 0.1 * math.log(stretch) + 1 if factor is None else factor)

    # ------------------------------------------------------------------ arguments of the C calls
    def _plan(self, device, B, S, D, positions, first, q_norm, k_norm, eps):
        """attn_rope_t for a call on tensors of `device`."""
        if self.rotary_dim > D:
            raise ValueError(f"{self.rotary_dim} elements are rotated, and a head has {D}")
        if positions is None and q_norm is None and k_norm is None and not first:
            return self._c  # never changed
        c = native.AttnRope.from_buffer_copy(self._c)
        c.first = first
        if positions is not None:
            if first:
                raise ValueError("first goes with positions that are not given")
            if positions.device != device or positions.dtype not in _INDEX:
                raise ValueError(f"positions must be an int32 or int64 tensor on {device}")
            shape = tuple(positions.shape)
            if shape != (S,) and shape != (B, S) and shape != (1, S):
                raise ValueError(f"positions must be [{S}] or [{B}, {S}], got {list(shape)}")
            if S > 1 and positions.stride(-1) != 1:
                raise ValueError("positions must be contiguous along the sequence")
            c.positions = positions.data_ptr()
            c.positions_64 = _INDEX[positions.dtype]
            c.position_stride = positions.stride(0) if len(shape) == 2 and shape[0] > 1 else 0
        if q_norm is not None or k_norm is not None:
            c.eps = eps
            dtype = (k_norm if q_norm is None else q_norm).dtype
            if dtype is not _BF16 and dtype is not torch.float32:
                raise ValueError(f"{'k_norm' if q_norm is None else 'q_norm'} must be bf16 or fp32")
            c.weight_format = native.ATTN_WEIGHT_BF16 if dtype is _BF16 else native.ATTN_WEIGHT_F32
            if q_norm is not None:
                c.q_weight = _weight("q_norm", q_norm, dtype, D, device)
            if k_norm is not None:
                c.k_weight = _weight("k_norm", k_norm, dtype, D, device)
        return c

    # ------------------------------------------------------------------ calls
    def heads(self, qkv, q_heads: int, kv_heads: int, positions=None, first: int = 0, q_norm=None, k_norm=None,
              eps: float = 1e-6):
        """q, k, v (bf16 [B, H, S, D], contiguous) of a projection's output qkv (bf16 [B, S, (Hq + 2 Hkv) D]:
        q's heads, then k's, then v's; strides of 16 bytes with the last dimension contiguous), q and k
        normed where ``q_norm`` / ``k_norm`` ([D], bf16 or fp32) are given, and rotated.  Row s of sequence b
        stands at ``positions[b, s]`` (int32 or int64 [B, S] or [S] on the device), or at first + s.
        Gradients flow to qkv and the norms' weights, once: a gradient made with ``create_graph=True`` raises where
        it is differentiated again (RuntimeError).  Forward-mode tangents are refused (ValueError).  Runs with
        qkv's device current, on its current stream.

        Captured into a graph, a step with its backward pass must not share leaves (qkv or weights that are
        nobody's result) with an eager graph of the default stream that still lives: torch keeps one node per
        leaf, on the stream of the first use, and a backward pass that meets one of the default stream, which
        cannot be captured, breaks the capture or ends the process.  The backward pass is refused where that
        eager graph is of these functions (ValueError); let it go first, warm up on another stream, pass
        ``leaf.detach().requires_grad_()``, or capture ``heads_backward``, which needs no autograd."""
        x = _packed(qkv, q_heads, kv_heads)
        refuse_tangents(qkv, q_norm, k_norm)
        c = self._plan(qkv.device, x.B, x.S, x.D, positions, first, q_norm, k_norm, eps)
        if torch.is_grad_enabled() and _any_grad(qkv, q_norm, k_norm):
            return _functions()[0].apply(qkv, q_norm, k_norm, positions, self, x, c, (q_heads, kv_heads, first, eps))
        return self._heads(qkv, x, c)

    def rotate(self, q, k=None, positions=None, first: int = 0, q_norm=None, k_norm=None, eps: float = 1e-6):
        """q (and k), bf16 [B, H, S, D] of any strides of 16 bytes with D contiguous, normed and rotated as by
        ``heads``, in new contiguous tensors.  Gradients flow to q, k and the norms' weights."""
        x = _apart(q, k, k_norm)
        refuse_tangents(q, k, q_norm, k_norm)
        c = self._plan(q.device, x.B, x.S, x.D, positions, first, q_norm, k_norm, eps)
        if torch.is_grad_enabled() and _any_grad(q, k, q_norm, k_norm):
            out = _functions()[1].apply(q, k, q_norm, k_norm, positions, self, x, c, (first, eps))
        else:
            out = self._rotate(q, k, x, c)
        return out if k is not None else out[0]

    def heads_backward(self, dq, dk, dv, qkv, q_heads: int, kv_heads: int, positions=None, first: int = 0, q_norm=None,
                       k_norm=None, eps: float = 1e-6, weight_grads: bool = True):
        """(dqkv, dq_norm, dk_norm) for upstream gradients of what ``heads`` returned with the same arguments.
        Without norms qkv's values are not read.  ``weight_grads=False`` leaves the norms' out (None).  Outside
        autograd: nothing is recorded, whatever the arguments require."""
        x = _packed(qkv, q_heads, kv_heads)
        for name, t, shape in (("dq", dq, x.q_shape), ("dk", dk, x.k_shape), ("dv", dv, x.k_shape)):
            _upstream(name, t, shape, qkv.device)
        c = self._plan(qkv.device, x.B, x.S, x.D, positions, first, q_norm, k_norm, eps)
        rows = None if q_norm is None and k_norm is None else x.at(qkv)
        return self._heads_backward(dq, dk, dv, rows, x, c, *((q_norm, k_norm) if weight_grads else (None, None)))

    def rotate_backward(self, dq, dk, q, k, positions=None, first: int = 0, q_norm=None, k_norm=None, eps: float = 1e-6,
                        weight_grads: bool = True):
        """(dq, dk, dq_norm, dk_norm): gradients of ``rotate``'s inputs, laid out as those are, for upstream
        ones of its outputs.  k and dk may be None together.  Outside autograd, as ``heads_backward``."""
        x = _apart(q, k, k_norm)
        if (k is None) != (dk is None):
            raise ValueError("k and dk go together")
        _upstream("dq", dq, x.q_shape, q.device)
        if k is not None:
            _upstream("dk", dk, x.k_shape, q.device)
        c = self._plan(q.device, x.B, x.S, x.D, positions, first, q_norm, k_norm, eps)
        rows = None if q_norm is None and k_norm is None else x.rows(q, k)
        return self._rotate_backward(dq, dk, rows, x, c, *((q_norm, k_norm) if weight_grads else (None, None)))

    # ------------------------------------------------------------------ the C calls
    def _heads(self, qkv, x, c):
        index = qkv.get_device()
        if _current_device() != index:
            with torch.cuda.device(index):
                return self._heads(qkv, x, c)
        q, k, v = qkv.new_empty(x.q_shape), qkv.new_empty(x.k_shape), qkv.new_empty(x.k_shape)
        rc = _lib().attn_rope(c, x.at(qkv), x.dense(q.data_ptr(), k.data_ptr(), v.data_ptr()), x.B, x.Hq, x.Hkv, x.S, x.D,
                              _stream_handle(index))
        if rc:
            raise native.AttnError(rc, "attn_rope")
        return q, k, v

    def _rotate(self, q, k, x, c):
        index = q.get_device()
        if _current_device() != index:
            with torch.cuda.device(index):
                return self._rotate(q, k, x, c)
        yq, yk = q.new_empty(x.q_shape), None if k is None else q.new_empty(x.k_shape)
        rc = _lib().attn_rope(c, x.rows(q, k), x.dense(yq.data_ptr(), None if k is None else yk.data_ptr(), None), x.B, x.Hq, x.Hkv, x.S,
                              x.D, _stream_handle(index))
        if rc:
            raise native.AttnError(rc, "attn_rope")
        return yq, yk

    # `rows`: the forward's, where they have norms; None without any.
    def _heads_backward(self, dq, dk, dv, rows, x, c, q_norm, k_norm):
        index = dq.get_device()
        if _current_device() != index:
            with torch.cuda.device(index):
                return self._heads_backward(dq, dk, dv, rows, x, c, q_norm, k_norm)
        dqkv = dq.new_empty(x.qkv_shape)
        return (dqkv, *self._backward(index, (dq, dk, dv), x, rows, x.at_dense(dqkv), c, q_norm, k_norm))

    def _rotate_backward(self, dq, dk, rows, x, c, q_norm, k_norm):
        index = dq.get_device()
        if _current_device() != index:
            with torch.cuda.device(index):
                return self._rotate_backward(dq, dk, rows, x, c, q_norm, k_norm)
        sq, sk = x.grad_strides()
        out = dq.new_empty_strided(x.q_shape, sq), None if dk is None else dq.new_empty_strided(x.k_shape, sk)
        return (*out, *self._backward(index, (dq, dk, None), x, rows, _heads_of(*out, None), c, q_norm, k_norm))

    def _backward(self, index, up, x, rows, out, c, q_norm, k_norm):
        """Fills `out` from upstream gradients and the forward's rows; returns the gradients of the weights given."""
        dwq = dwk = w = None
        need = 0
        if q_norm is not None or k_norm is not None:
            need = x.need(c)
            w = up[0].new_empty((need + 1) // 2)  # elements of two bytes
            if q_norm is not None:
                dwq = torch.empty_like(q_norm)
            if k_norm is not None:
                dwk = torch.empty_like(k_norm)
        rc = _lib().attn_rope_bwd(c, x.upstream(*up), rows, out, None if dwq is None else dwq.data_ptr(),
                                  None if dwk is None else dwk.data_ptr(), x.B, x.Hq, x.Hkv, x.S, x.D, None if w is None else w.data_ptr(),
                                  need, _stream_handle(index))
        if rc:
            raise native.AttnError(rc, "attn_rope_bwd")
        return dwq, dwk


_library = None


def _lib():
    global _library
    if _library is None:
        _library = native.load()
    return _library


def _any_grad(*tensors):
    for t in tensors:
        if t is not None and t.requires_grad:
            return True
    return False


def _weight(name, w, dtype, D, device):
    if w.dtype is not dtype:
        raise ValueError("q_norm and k_norm must have one type")
    if w.device != device or w.shape != (D,) or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor [{D}] on {device}")
    return w.data_ptr()


class _Sizes:
    """What calls of one set of sizes and strides have in common: checked once, with the structs of the C calls but
    for their addresses (a call fills a copy of its own)."""

    def __init__(self, B, S, Hq, Hkv, D, strides):
        self.B, self.S, self.Hq, self.Hkv, self.D = B, S, Hq, Hkv, D
        self.q_shape, self.k_shape, self.qkv_shape = (B, Hq, S, D), (B, Hkv, S, D), (B, S, (Hq + 2 * Hkv) * D)
        self._strides, self._grad_strides = strides, None
        self._in = native.AttnHeads(None, None, None, *(_STRIDES(*st) for st in strides))
        self._dense = native.AttnHeads(None, None, None, *(_STRIDES(H * S * D, S * D, D) for H in (Hq, Hkv, Hkv)))
        W = (Hq + 2 * Hkv) * D
        self._packed = native.AttnHeads(None, None, None, *(_STRIDES(S * W, D, W) for _ in range(3)))
        self._k_at, self._v_at = 2 * Hq * D, 2 * (Hq + Hkv) * D
        self._need = {}

    def _packed_at(self, c, p):
        c = native.AttnHeads.from_buffer_copy(c)
        c.q, c.k, c.v = p, p + self._k_at, p + self._v_at
        return c

    def at(self, qkv):
        """The heads as they lie in qkv."""
        return self._packed_at(self._in, qkv.data_ptr())

    def at_dense(self, dqkv):
        """The heads as they lie in a contiguous tensor of qkv's sizes."""
        return self._packed_at(self._packed, dqkv.data_ptr())

    def rows(self, q, k):
        c = native.AttnHeads.from_buffer_copy(self._in)
        c.q = q.data_ptr()
        if k is not None:
            c.k = k.data_ptr()
        return c

    def dense(self, q, k, v):
        """Contiguous heads at these addresses."""
        c = native.AttnHeads.from_buffer_copy(self._dense)
        c.q, c.k, c.v = q, k, v
        return c

    def grad_strides(self):
        """Strides of new tensors with the order of q's and k's dimensions in memory, D contiguous."""
        if self._grad_strides is None:
            def like(shape, stride):
                y = torch.empty_like(torch.empty_strided(shape, (*stride, 1), device="meta"))
                return y.stride() if y.stride(3) == 1 else torch.empty(shape, device="meta").stride()
            self._grad_strides = like(self.q_shape, self._strides[0]), like(self.k_shape, self._strides[1])
        return self._grad_strides

    def upstream(self, dq, dk, dv):
        """attn_heads_t of upstream gradients, made dense where their strides or addresses do not fit (`held` keeps
        those alive with it)."""
        given = (dq, dk, dv)
        at = [None if t is None else t.data_ptr() for t in given]
        if all(t is None or (t.is_contiguous() and p % 16 == 0) for t, p in zip(given, at)):
            return self.dense(*at)
        held = [None if t is None else _aligned(t) for t in given]
        c = _heads_of(*held)
        c.held = held
        return c

    def need(self, c):
        """Bytes of the backward's workspace."""
        key = bool(c.q_weight), bool(c.k_weight)
        need = self._need.get(key)
        if need is None:
            n = ctypes.c_ulonglong(0)
            rc = _lib().attn_rope_workspace(c, self.B, self.Hq, self.Hkv, self.S, self.D, n)
            if rc:
                raise native.AttnError(rc, "attn_rope_workspace")
            need = self._need[key] = n.value
        return need


_sizes: dict = {}  # _Sizes by the sizes and strides of a call


def _kept(key, made):
    if len(_sizes) >= 4096:
        _sizes.clear()
    _sizes[key] = made
    return made


def _packed(qkv, Hq, Hkv):
    """_Sizes of a projection's output, checked."""
    if not qkv.is_cuda or qkv.dtype is not _BF16:
        raise ValueError("qkv must be a bf16 CUDA tensor [B, S, (Hq + 2 Hkv) D]")
    key = qkv.shape, qkv.stride(), Hq, Hkv
    x = _sizes.get(key)
    if x is not None:
        return x
    if qkv.dim() != 3:
        raise ValueError("qkv must be a bf16 CUDA tensor [B, S, (Hq + 2 Hkv) D]")
    B, S, W = qkv.shape
    if Hq < 1 or Hkv < 1 or W % (Hq + 2 * Hkv) or W // (Hq + 2 * Hkv) not in (64, 128):
        raise ValueError(f"qkv holds {W} elements a token: not {Hq} + 2 * {Hkv} heads of 64 or 128")
    if B < 1 or S < 1:
        raise ValueError("at least one sequence and one token are needed")
    if qkv.stride(2) != 1:
        raise ValueError("qkv's last dimension must be contiguous")
    D = W // (Hq + 2 * Hkv)
    return _kept(key, _Sizes(B, S, Hq, Hkv, D, [(qkv.stride(0), D, qkv.stride(1))] * 3))


def _apart(q, k, k_norm):
    """_Sizes of q and k (or None) by themselves, checked."""
    if not q.is_cuda or q.dtype is not _BF16:
        raise ValueError("q must be a bf16 CUDA tensor [B, H, S, D]")
    if k is None:
        if k_norm is not None:
            raise ValueError("k_norm without k")
    elif k.dtype is not _BF16 or k.device != q.device:
        raise ValueError(f"k must be a bf16 tensor on {q.device}")
    key = q.shape, q.stride(), None if k is None else (k.shape, k.stride())
    x = _sizes.get(key)
    if x is not None:
        return x
    for name, t in (("q", q), ("k", k)):
        if t is None:
            continue
        if t.dim() != 4 or 0 in t.shape:
            raise ValueError(f"{name} must be a bf16 CUDA tensor [B, H, S, D]")
        if t.shape[3] not in (64, 128):
            raise ValueError(f"heads of 64 or 128 elements are needed, got {t.shape[3]}")
        if t.stride(3) != 1:
            raise ValueError(f"{name}'s last dimension must be contiguous")
        if (t.shape[0], t.shape[2], t.shape[3]) != (q.shape[0], q.shape[2], q.shape[3]):
            raise ValueError(f"{name} must be [{q.shape[0]}, H, {q.shape[2]}, {q.shape[3]}]")
    B, Hq, S, D = q.shape
    strides = [q.stride()[:3], (0, 0, 0) if k is None else k.stride()[:3], (0, 0, 0)]
    return _kept(key, _Sizes(B, S, Hq, 1 if k is None else k.shape[1], D, strides))


def _upstream(name, t, shape, device):
    if t is None or t.device != device or t.dtype is not _BF16 or t.shape != shape:
        raise ValueError(f"{name} must be a bf16 tensor {list(shape)} on {device}")


def _aligned(t):
    """An upstream gradient as the library takes it: as it is, or dense where its strides or address do not fit."""
    if t.stride(3) == 1 and t.data_ptr() % 16 == 0 and not any(t.stride(i) % 8 for i in range(3) if t.shape[i] > 1):
        return t
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _heads_of(q, k, v):
    """attn_heads_t of rows [B, H, S, D]; None: absent."""
    pointers = [None if x is None else x.data_ptr() for x in (q, k, v)]
    strides = [_STRIDES() if x is None else _STRIDES(*x.stride()[:3]) for x in (q, k, v)]
    return native.AttnHeads(*pointers, *strides)


# Nodes of the eager calls on a default stream whose graphs live, by id, as weak references.
_live: dict = {}


def _watch(ctx, index):
    """Notes an eager forward on the default stream."""
    if _stream_handle(index) == 0 and not _capturing():
        key = id(ctx)
        _live[key] = weakref.ref(ctx, lambda _: _live.pop(key, None))


def _leaves(node):
    return [f.variable for f, _ in node.next_functions if f is not None and hasattr(f, "variable")]


def _check(ctx):
    """Refuses a captured backward whose leaves an eager graph of the default stream holds."""
    if not _live or not _capturing():
        return
    mine = _leaves(ctx)
    for ref in list(_live.values()):
        node = ref()
        if node is not None and any(t is x for t in mine for x in _leaves(node)):
            raise ValueError("an eager graph of the same leaf lives, whose backward node belongs to the default stream: capturing "
                             "would break. Let it go first, warm up on another stream, pass leaf.detach().requires_grad_(), or "
                             "capture the *_backward call")


def _functions():
    global _FUNCTIONS
    if _FUNCTIONS is None:
        _FUNCTIONS = _make_functions()
    return _FUNCTIONS


_FUNCTIONS = None


def _make_functions():
    """torch.autograd.Functions over the calls above.  What is saved is q and k, or qkv, only where they have norms; a
    backward takes sizes, strides and addresses from what it gets back, which hooks may have moved.  In a backward that is
    itself recorded each gradient is tied to what it depends on, and cannot be differentiated again."""

    def heads_backward(ctx, saved, dq, dk, dv):
        _check(ctx)
        qkv, q_norm, k_norm, positions = saved
        rotary, x, (Hq, Hkv, first, eps) = ctx.args
        _, need_q, need_k, *_ = ctx.needs_input_grad
        rows = None
        if qkv is not None:
            x = _packed(qkv, Hq, Hkv)
            rows = x.at(qkv)
        c = rotary._plan(dq.device, x.B, x.S, x.D, positions, first, q_norm, k_norm, eps)
        return rotary._heads_backward(dq, dk, dv, rows, x, c, q_norm if need_q else None, k_norm if need_k else None)

    def rotate_backward(ctx, saved, dq, dk):
        _check(ctx)
        q, k, q_norm, k_norm, positions = saved
        rotary, x, (first, eps), has_k = ctx.args
        _, _, need_q, need_k, *_ = ctx.needs_input_grad
        rows = None if q is None else _apart(q, k, k_norm).rows(q, k)
        c = rotary._plan(dq.device, x.B, x.S, x.D, positions, first, q_norm, k_norm, eps)
        return rotary._rotate_backward(dq, dk if has_k else None, rows, x, c, q_norm if need_q else None, k_norm if need_k else None)

    class HeadsFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, qkv, q_norm, k_norm, positions, rotary, x, c, args):
            _watch(ctx, qkv.get_device())
            normed = q_norm is not None or k_norm is not None
            ctx.save_for_backward(qkv if normed else None, q_norm, k_norm, positions)
            ctx.args = rotary, x, args
            return rotary._heads(qkv, x, c)

        @staticmethod
        def backward(ctx, dq, dk, dv):
            saved = ctx.saved_tensors  # once: hooks may make them anew each time, or refuse to
            if torch.is_grad_enabled():
                qkv, q_norm, k_norm, _ = saved
                with torch.no_grad():
                    dqkv, dq_norm, dk_norm = heads_backward(ctx, saved, dq, dk, dv)
                got = tied(dqkv, dq, dk, dv, qkv, q_norm, k_norm), tied(dq_norm, dq, qkv), tied(dk_norm, dk, qkv)
            else:
                got = heads_backward(ctx, saved, dq, dk, dv)
            return (*got, None, None, None, None, None)

    class RotateFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, q_norm, k_norm, positions, rotary, x, c, args):
            _watch(ctx, q.get_device())
            normed = q_norm is not None or k_norm is not None
            ctx.save_for_backward(*((q, k) if normed else (None, None)), q_norm, k_norm, positions)
            ctx.args = rotary, x, args, k is not None
            return rotary._rotate(q, k, x, c)

        @staticmethod
        def backward(ctx, dq, dk):
            saved = ctx.saved_tensors
            if torch.is_grad_enabled():
                q, k, q_norm, k_norm, _ = saved
                with torch.no_grad():
                    gq, gk, dq_norm, dk_norm = rotate_backward(ctx, saved, dq, dk)
                of_q = () if q_norm is None else (q, q_norm)  # without a norm a gradient depends on the upstream one alone
                of_k = () if k_norm is None else (k, k_norm)
                got = tied(gq, dq, *of_q), tied(gk, dk, *of_k), tied(dq_norm, dq, q), tied(dk_norm, dk, k)
            else:
                got = rotate_backward(ctx, saved, dq, dk)
            return (*got, None, None, None, None, None)

    return HeadsFunction, RotateFunction
