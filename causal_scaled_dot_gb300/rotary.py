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

import contextlib
import ctypes
import math
import weakref
from fractions import Fraction

import torch

from . import native

# pi to 60 decimals (OEIS A000796): a frequency's share of a turn is taken to nearest from its exact double value.
_PI = Fraction(3141592653589793238462643383279502884197169399375105820974945, 10**60)
_STRIDES = ctypes.c_longlong * 3
_BF16 = torch.bfloat16
_WEIGHT = {torch.bfloat16: native.ATTN_WEIGHT_BF16, torch.float32: native.ATTN_WEIGHT_F32}
_INDEX = {torch.int32: 0, torch.int64: 1}
# The current stream's handle by device index, without a Stream object.
_stream_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _frequencies(rotary_dim: int, base: float) -> list[float]:
    if rotary_dim % 2 or not base > 0:
        raise ValueError("rotary_dim must be even and base positive")
    return [base ** (-2 * i / rotary_dim) for i in range(rotary_dim // 2)]


class Rotary:
    """How a model's heads turn with their position: pair i of a head's first ``2 * len(frequencies)``
    elements turns by ``position * frequencies[i]`` radians, and is scaled by ``factor``.  The pairs are
    (i, i + len(frequencies)), or neighbours (2i, 2i + 1) when ``interleaved``; the rest of the head stays.
    No frequencies: no rotation (norms and the change of layout remain).

    Angles are exact at any position (the frequencies are held as 64-bit fractions of a turn); there is no
    table and no longest position.  A Rotary holds no device memory, so it serves every device."""

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
        turns = [round(Fraction(x) / (2 * _PI) * 2**64) % 2**64 for x in f]
        self._c = native.AttnRope((ctypes.c_ulonglong * 64)(*turns), self.rotary_dim, int(self.interleaved), self.factor)
        self._workspace_bytes = {}

    @classmethod
    def from_base(cls, rotary_dim: int, base: float = 10000.0, stretch: float = 1.0, interleaved: bool = False):
        """frequencies[i] = base^(-2i / rotary_dim) / stretch: a stretch of s puts s positions where one was."""
        return cls([f / stretch for f in _frequencies(rotary_dim, base)], interleaved)

    @classmethod
    def raised_base(cls, rotary_dim: int, stretch: float, base: float = 10000.0, interleaved: bool = False):
        """The base raised so that the slowest pair is stretched by ``stretch`` and the fastest stays."""
        if rotary_dim < 4:
            raise ValueError("rotary_dim must be 4 or more")
        return cls(_frequencies(rotary_dim, base * stretch ** (rotary_dim / (rotary_dim - 2))), interleaved)

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
        for f in _frequencies(rotary_dim, base):
            keep = min(max((original_length * f / math.tau - slow) / (fast - slow), 0.0), 1.0)
            out.append(f * (keep + (1 - keep) / stretch))
        return cls(out, interleaved, 0.1 * math.log(stretch) + 1 if factor is None else factor)

    # ------------------------------------------------------------------ arguments of the C calls
    def _plan(self, device, B, S, D, positions, first, q_norm, k_norm, eps):
        """attn_rope_t for a call on tensors of `device`."""
        if self.rotary_dim > D:
            raise ValueError(f"{self.rotary_dim} elements are rotated, and a head has {D}")
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
            formats = set()
            for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
                if w is None:
                    continue
                if w.device != device or w.dtype not in _WEIGHT or tuple(w.shape) != (D,) or not w.is_contiguous():
                    raise ValueError(f"{name} must be a contiguous bf16 or fp32 tensor [{D}] on {device}")
                formats.add(_WEIGHT[w.dtype])
            if len(formats) > 1:
                raise ValueError("q_norm and k_norm must have one type")
            c.weight_format = formats.pop()
            c.q_weight = None if q_norm is None else q_norm.data_ptr()
            c.k_weight = None if k_norm is None else k_norm.data_ptr()
        return c

    def _need(self, c, B, Hq, Hkv, S, D) -> int:
        key = (bool(c.q_weight), bool(c.k_weight), B, Hq, Hkv, S, D)
        need = self._workspace_bytes.get(key)
        if need is None:
            n = ctypes.c_ulonglong(0)
            _ok(native.load().attn_rope_workspace(ctypes.byref(c), B, Hq, Hkv, S, D, ctypes.byref(n)), "attn_rope_workspace")
            if len(self._workspace_bytes) > 256:
                self._workspace_bytes.clear()
            need = self._workspace_bytes[key] = n.value
        return need

    # ------------------------------------------------------------------ calls
    def heads(self, qkv, q_heads: int, kv_heads: int, positions=None, first: int = 0, q_norm=None, k_norm=None,
              eps: float = 1e-6):
        """q, k, v (bf16 [B, H, S, D], contiguous) of a projection's output qkv (bf16 [B, S, (Hq + 2 Hkv) D]:
        q's heads, then k's, then v's; strides of 16 bytes with the last dimension contiguous), q and k
        normed where ``q_norm`` / ``k_norm`` ([D], bf16 or fp32) are given, and rotated.  Row s of sequence b
        stands at ``positions[b, s]`` (int32 or int64 [B, S] or [S] on the device), or at first + s.
        Gradients flow to qkv and the norms' weights.  Runs with qkv's device current, on its current stream.

        Captured into a graph, a step with its backward pass must not share leaves (qkv or weights that are
        nobody's result) with an eager graph that still lives: torch keeps one node per leaf, on the stream
        of the first use, and a backward pass that meets it breaks the capture or ends the process.  A call
        that would is refused where that eager graph is of these functions (ValueError); let it go first,
        pass ``leaf.detach().requires_grad_()``, or capture ``heads_backward``, which needs no autograd."""
        _packed(qkv, q_heads, kv_heads)
        if torch.is_grad_enabled() and _any_grad(qkv, q_norm, k_norm):
            return _functions()[0].apply(qkv, q_norm, k_norm, self, q_heads, kv_heads, positions, first, eps)
        return self._heads(qkv, q_heads, kv_heads, positions, first, q_norm, k_norm, eps)

    def rotate(self, q, k=None, positions=None, first: int = 0, q_norm=None, k_norm=None, eps: float = 1e-6):
        """q (and k), bf16 [B, H, S, D] of any strides of 16 bytes with D contiguous, normed and rotated as by
        ``heads``, in new contiguous tensors.  Gradients flow to q, k and the norms' weights."""
        _rows("q", q)
        if k is not None:
            _rows("k", k, q)
        elif k_norm is not None:
            raise ValueError("k_norm without k")
        if torch.is_grad_enabled() and _any_grad(q, k, q_norm, k_norm):
            out = _functions()[1].apply(q, k, q_norm, k_norm, self, positions, first, eps)
        else:
            out = self._rotate(q, k, positions, first, q_norm, k_norm, eps)
        return out if k is not None else out[0]

    def heads_backward(self, dq, dk, dv, qkv, q_heads: int, kv_heads: int, positions=None, first: int = 0, q_norm=None,
                       k_norm=None, eps: float = 1e-6, weight_grads: bool = True):
        """(dqkv, dq_norm, dk_norm) for upstream gradients of what ``heads`` returned with the same arguments.
        Without norms qkv's values are not read.  ``weight_grads=False`` leaves the norms' out (None)."""
        B, S, W = _packed(qkv, q_heads, kv_heads)
        D = W // (q_heads + 2 * kv_heads)
        for name, t, H in (("dq", dq, q_heads), ("dk", dk, kv_heads), ("dv", dv, kv_heads)):
            _upstream(name, t, (B, H, S, D), qkv.device)
        with _on(qkv):
            dqkv = torch.empty((B, S, W), dtype=_BF16, device=qkv.device)
            got = self._backward((dq, dk, dv), _split(qkv, q_heads, kv_heads), _split(dqkv, q_heads, kv_heads), positions, first,
                                 q_norm, k_norm, eps, weight_grads)
        return (dqkv, *got)

    def rotate_backward(self, dq, dk, q, k, positions=None, first: int = 0, q_norm=None, k_norm=None, eps: float = 1e-6,
                        weight_grads: bool = True):
        """(dq, dk, dq_norm, dk_norm): gradients of ``rotate``'s inputs, laid out as those are, for upstream
        ones of its outputs.  k and dk may be None together."""
        _rows("q", q)
        _upstream("dq", dq, tuple(q.shape), q.device)
        if (k is None) != (dk is None):
            raise ValueError("k and dk go together")
        if k is not None:
            _rows("k", k, q)
            _upstream("dk", dk, tuple(k.shape), q.device)
        elif k_norm is not None:
            raise ValueError("k_norm without k")
        with _on(q):
            out = tuple(None if x is None else _like(x) for x in (q, k))
            got = self._backward((dq, dk, None), (q, k, None), (*out, None), positions, first, q_norm, k_norm, eps, weight_grads)
        return (*out, *got)

    # ------------------------------------------------------------------ the C calls
    def _heads(self, qkv, Hq, Hkv, positions, first, q_norm, k_norm, eps):
        B, S, W = qkv.shape
        D = W // (Hq + 2 * Hkv)
        c = self._plan(qkv.device, B, S, D, positions, first, q_norm, k_norm, eps)
        with _on(qkv) as st:
            q = torch.empty((B, Hq, S, D), dtype=_BF16, device=qkv.device)
            k = torch.empty((B, Hkv, S, D), dtype=_BF16, device=qkv.device)
            v = torch.empty((B, Hkv, S, D), dtype=_BF16, device=qkv.device)
            _ok(native.load().attn_rope(c, _packed_heads(qkv, Hq, Hkv, D), _dense_heads(q, k, v), B, Hq, Hkv, S, D, st), "attn_rope")
        return q, k, v

    def _rotate(self, q, k, positions, first, q_norm, k_norm, eps):
        B, Hq, S, D = q.shape
        c = self._plan(q.device, B, S, D, positions, first, q_norm, k_norm, eps)
        with _on(q) as st:
            out = tuple(None if x is None else torch.empty(x.shape, dtype=_BF16, device=q.device) for x in (q, k))
            _ok(native.load().attn_rope(c, _heads_of(q, k, None), _heads_of(*out, None), B, Hq, 1 if k is None else k.shape[1], S, D,
                                        st), "attn_rope")
        return out

    def _backward(self, up, x, out, positions, first, q_norm, k_norm, eps, weight_grads):
        """Fills `out` (q, k, v rows) from upstream gradients and the forward's rows; the weights' gradients."""
        B, Hq, S, D = x[0].shape
        Hkv = 1 if x[1] is None else x[1].shape[1]
        c = self._plan(x[0].device, B, S, D, positions, first, q_norm, k_norm, eps)
        st = _stream_handle(x[0].device.index)
        dw = [None if w is None or not weight_grads else torch.empty_like(w) for w in (q_norm, k_norm)]
        w, need = None, 0
        if any(t is not None for t in dw):
            need = self._need(c, B, Hq, Hkv, S, D)
            w = torch.empty(need, dtype=torch.uint8, device=x[0].device)
        up = [None if t is None else _aligned(t) for t in up]
        normed = q_norm is not None or k_norm is not None
        _ok(native.load().attn_rope_bwd(c, _heads_of(*up), _heads_of(*x) if normed else None, _heads_of(*out),
                                        *(None if t is None else t.data_ptr() for t in dw), B, Hq, Hkv, S, D,
                                        None if w is None else w.data_ptr(), need, st), "attn_rope_bwd")
        return dw


def _ok(rc, where):
    if rc != native.ATTN_OK:
        raise native.AttnError(rc, where)


@contextlib.contextmanager
def _switched(index):
    with torch.cuda.device(index):
        yield _stream_handle(index)


def _on(x):
    """x's device current; yields its current stream's handle."""
    index = x.device.index
    return contextlib.nullcontext(_stream_handle(index)) if _current_device() == index else _switched(index)


def _any_grad(*tensors):
    return any(t is not None and t.requires_grad for t in tensors)


def _packed(qkv, Hq, Hkv):
    if not qkv.is_cuda or qkv.dtype is not _BF16 or qkv.dim() != 3:
        raise ValueError("qkv must be a bf16 CUDA tensor [B, S, (Hq + 2 Hkv) D]")
    B, S, W = qkv.shape
    if Hq < 1 or Hkv < 1 or W % (Hq + 2 * Hkv) or W // (Hq + 2 * Hkv) not in (64, 128):
        raise ValueError(f"qkv holds {W} elements a token: not {Hq} + 2 * {Hkv} heads of 64 or 128")
    if B < 1 or S < 1:
        raise ValueError("at least one sequence and one token are needed")
    if qkv.stride(2) != 1:
        raise ValueError("qkv's last dimension must be contiguous")
    return B, S, W


def _rows(name, x, like=None):
    if not x.is_cuda or x.dtype is not _BF16 or x.dim() != 4 or 0 in x.shape:
        raise ValueError(f"{name} must be a bf16 CUDA tensor [B, H, S, D]")
    if x.shape[3] not in (64, 128):
        raise ValueError(f"heads of 64 or 128 elements are needed, got {x.shape[3]}")
    if x.stride(3) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    if like is not None and (x.device != like.device or (x.shape[0], *x.shape[2:]) != (like.shape[0], *like.shape[2:])):
        raise ValueError(f"{name} must be [{like.shape[0]}, H, {like.shape[2]}, {like.shape[3]}] on {like.device}")


def _upstream(name, t, shape, device):
    if t.device != device or t.dtype is not _BF16 or tuple(t.shape) != shape:
        raise ValueError(f"{name} must be a bf16 tensor {list(shape)} on {device}")


def _aligned(t):
    """An upstream gradient as the library takes it: as it is, or dense where its strides or address do not fit."""
    if t.stride(3) == 1 and t.data_ptr() % 16 == 0 and not any(t.stride(i) % 8 for i in range(3) if t.shape[i] > 1):
        return t
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _like(x):
    """A new tensor with x's order of dimensions in memory, D contiguous."""
    y = torch.empty_like(x)
    return y if y.stride(3) == 1 else torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _split(qkv, Hq, Hkv):
    """q, k, v [B, H, S, D] as they lie in qkv."""
    x = qkv.unflatten(2, (Hq + 2 * Hkv, -1)).transpose(1, 2)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _packed_heads(qkv, Hq, Hkv, D):
    b, s, _ = qkv.stride()
    at, st = qkv.data_ptr(), _STRIDES(b, D, s)
    return native.AttnHeads(at, at + 2 * Hq * D, at + 2 * (Hq + Hkv) * D, st, st, st)


def _dense_heads(q, k, v):
    _, Hq, S, D = q.shape
    qs, ks = _STRIDES(Hq * S * D, S * D, D), _STRIDES(k.shape[1] * S * D, S * D, D)
    return native.AttnHeads(q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, ks)


def _heads_of(q, k, v):
    """attn_heads_t of rows [B, H, S, D]; None: absent."""
    pointers = [None if x is None else x.data_ptr() for x in (q, k, v)]
    strides = [_STRIDES() if x is None else _STRIDES(*x.stride()[:3]) for x in (q, k, v)]
    return native.AttnHeads(*pointers, *strides)


# The live eager graphs of these functions by leaf (id): (leaf, node, stream), the first two as weak references.
_live: dict = {}


def _watch(ctx, leaves, index):
    """Notes an eager call's leaves, or refuses a captured one that shares a leaf with an eager graph of another stream."""
    leaves = [t for t in leaves if t is not None and t.requires_grad and t.is_leaf]
    if not leaves:
        return
    capturing, st = torch.cuda.is_current_stream_capturing(), _stream_handle(index)
    for t in leaves:
        held = [x for x in _live.get(id(t), ()) if x[0]() is t and x[1]() is not None]
        if capturing:
            if any(x[2] != st for x in held):
                raise ValueError("an eager graph of the same leaf lives, whose backward node belongs to another stream: capturing "
                                 "would break. Let it go first, pass leaf.detach().requires_grad_(), or capture the *_backward call")
        else:
            held.append((weakref.ref(t), weakref.ref(ctx), st))
            if len(_live) > 4096:  # leaves that are gone
                for key in [k for k, v in _live.items() if all(x[0]() is None or x[1]() is None for x in v)]:
                    del _live[key]
        _live[id(t)] = held


def _functions():
    global _FUNCTIONS
    if _FUNCTIONS is None:
        _FUNCTIONS = _make_functions()
    return _FUNCTIONS


_FUNCTIONS = None


def _make_functions():
    """torch.autograd.Functions over the calls above."""
    once = torch.autograd.function.once_differentiable

    class HeadsFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, qkv, q_norm, k_norm, rotary, Hq, Hkv, positions, first, eps):
            _watch(ctx, (qkv, q_norm, k_norm), qkv.device.index)
            ctx.save_for_backward(qkv, q_norm, k_norm, positions)
            ctx.args = (rotary, Hq, Hkv, first, eps)
            return rotary._heads(qkv, Hq, Hkv, positions, first, q_norm, k_norm, eps)

        @staticmethod
        @once
        def backward(ctx, dq, dk, dv):
            qkv, q_norm, k_norm, positions = ctx.saved_tensors
            rotary, Hq, Hkv, first, eps = ctx.args
            got = rotary.heads_backward(dq, dk, dv, qkv, Hq, Hkv, positions, first, q_norm, k_norm, eps, any(ctx.needs_input_grad[1:3]))
            return (*got, None, None, None, None, None, None)

    class RotateFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, q_norm, k_norm, rotary, positions, first, eps):
            _watch(ctx, (q, k, q_norm, k_norm), q.device.index)
            ctx.save_for_backward(q, k, q_norm, k_norm, positions)
            ctx.args = (rotary, first, eps)
            return rotary._rotate(q, k, positions, first, q_norm, k_norm, eps)

        @staticmethod
        @once
        def backward(ctx, dq, dk):
            q, k, q_norm, k_norm, positions = ctx.saved_tensors
            rotary, first, eps = ctx.args
            got = rotary.rotate_backward(dq, dk if k is not None else None, q, k, positions, first, q_norm, k_norm, eps,
                                         any(ctx.needs_input_grad[2:4]))
            return (*got, None, None, None, None)

    return HeadsFunction, RotateFunction
