"""A paged key/value cache in 8 bits over libattn's cache entry points
(``attn_cache_write``, ``attn_cache_append``, ``attn_cache_read``, ``attn_cache_fwd`` in include/attn.h).

    cache = KVCache.empty(batch, kv_heads, head_dim, max_tokens, device="cuda")
    cache.seq_lens.add_(n)             # the step's n new tokens count from here on
    cache.write(k, v)                  # k, v [B, Hkv, n, D] bf16, quantised into the cache
    out, lse = cache.attention(q)      # q [B, Hq, n, D] bf16 over everything held

or, with rotary positions (and norms of the heads) on the way into the cache, from the
heads as projected:

    q = cache.append(k, v, rotary, q=q)          # rotary: a rotary.Rotary

Argument marshalling only: the tensors are the caller's (or ``empty``'s), the work runs
in the CUDA library.  There are no gradients through a cache.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from . import native
from .autograd import refuse_tangents
from .rotary import _heads_of

_DIMS3 = ctypes.c_longlong * 3
# The current stream's handle by device index.  A step calls write and attention once per layer, and
# building a Stream object takes longer than the rest of a call's checks.
_stream_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_BF16 = torch.bfloat16
# Every thread's own default stream has this handle: streams that it does not tell apart.
_PER_THREAD = 2
# Workspaces by (device, stream): calls on one stream run one after the other, so they share one.
# Captured calls do not take part: each has its own from the graph's memory, as graphs may be
# replayed on any stream.
_workspaces: dict = {}


def _strides(name, x):
    """{batch, head, token} strides of [B, H, S, D] for the C call (NULL stands for contiguous)."""
    if x.shape[3] > 1 and x.stride(3) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    # The stride of a dimension of one element is never used, and may be any number.
    return _DIMS3(*(x.stride(i) if x.shape[i] > 1 else 0 for i in range(3)))


class KVCache:
    """The tensors of one layer's cache and the calls on it.

    k, v              float8_e4m3fn codes [num_blocks, Hkv, block_size, D], contiguous
    k_scale, v_scale  float32 [num_blocks, Hkv]
    block_table       int32 [B, max_blocks]: sequence b's token t is in block
                      block_table[b, t // block_size], slot t % block_size
    seq_lens          int32 [B]: tokens held, the current step's included

    All on one CUDA device.  ``block_table`` and ``seq_lens`` may be shared between
    layers and are updated in place by their owner; the tensors themselves stay the
    same for the cache's lifetime.  Calls run with the tensors' device current, on
    ``stream`` (a torch.cuda.Stream of that device or a handle, not the per-thread
    default stream's; default: that device's current stream), and do not synchronise unless
    ``check_status`` asks for it: it then raises AttnError if a device-side wait ran
    out or a block number or length lay outside the cache (one status word per
    device, shared by every stream on it).  Attention over more than 1024 tokens a
    sequence keeps a workspace of up to 40 MB for each device and stream, for the
    process's lifetime; captured calls take theirs from their graph's memory."""

    def __init__(self, k, v, k_scale, v_scale, block_table, seq_lens):
        named = dict(k=k, v=v, k_scale=k_scale, v_scale=v_scale, block_table=block_table, seq_lens=seq_lens)
        dtypes = dict(k=torch.float8_e4m3fn, v=torch.float8_e4m3fn, k_scale=torch.float32, v_scale=torch.float32,
                      block_table=torch.int32, seq_lens=torch.int32)
        if k.dim() != 4:
            raise ValueError("k must be [num_blocks, Hkv, block_size, D]")
        num_blocks, Hkv, block_size, D = k.shape
        if block_table.dim() != 2:
            raise ValueError("block_table must be [B, max_blocks]")
        B, max_blocks = block_table.shape
        shapes = dict(k=tuple(k.shape), v=tuple(k.shape), k_scale=(num_blocks, Hkv), v_scale=(num_blocks, Hkv),
                      block_table=(B, max_blocks), seq_lens=(B,))
        for name, t in named.items():
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            if t.dtype != dtypes[name]:
                raise ValueError(f"{name} must be {dtypes[name]}, got {t.dtype}")
            if tuple(t.shape) != shapes[name]:
                raise ValueError(f"{name} must have shape {list(shapes[name])}, got {list(t.shape)}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            if t.device != k.device:
                raise ValueError(f"{name} is on {t.device} but k is on {k.device}: all tensors of one cache "
                                 "must be on the same device")
        if block_size not in (16, 32, 64, 128) or D not in (64, 128):
            raise ValueError(f"block_size must be 16, 32, 64 or 128 and D 64 or 128, got {block_size} and {D}")
        if 0 in (num_blocks, Hkv, B, max_blocks):
            raise ValueError("a cache needs at least one block, head and sequence")
        self._tensors = named
        self._device = k.device
        self._index = k.device.index
        self._sizes = (B, Hkv, D)
        self._capacity = max_blocks * block_size
        self._c = native.AttnCache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                   block_table.data_ptr(), seq_lens.data_ptr(), num_blocks, block_size, max_blocks, B,
                                   Hkv, D)
        self._ref = ctypes.byref(self._c)
        self._lib = native.load()
        self._workspace_bytes = {}
        self._steps = {}

    @classmethod
    def empty(cls, batch: int, kv_heads: int, head_dim: int, max_tokens: int, block_size: int = 64, device="cuda"):
        """A cache without tokens (seq_lens = 0) with room for max_tokens in every
        sequence, sequence b's blocks in order at b * ceil(max_tokens / block_size)."""
        per = -(-max_tokens // block_size)
        shape = (batch * per, kv_heads, block_size, head_dim)
        code = lambda: torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)  # noqa: E731
        scale = lambda: torch.ones(shape[:2], dtype=torch.float32, device=device)  # noqa: E731
        table = torch.arange(batch * per, dtype=torch.int32, device=device).view(batch, per)
        return cls(code(), code(), scale(), scale(), table, torch.zeros(batch, dtype=torch.int32, device=device))

    k = property(lambda self: self._tensors["k"])
    v = property(lambda self: self._tensors["v"])
    k_scale = property(lambda self: self._tensors["k_scale"])
    v_scale = property(lambda self: self._tensors["v_scale"])
    block_table = property(lambda self: self._tensors["block_table"])
    seq_lens = property(lambda self: self._tensors["seq_lens"])
    capacity = property(lambda self: self._capacity, doc="tokens a sequence can hold")

    def _rows(self, name, x, heads, S=None, strided=True):
        """Checks a bf16 tensor [B, heads, S, D] on the cache's device; returns S and its strides."""
        if x.dtype is not _BF16 or x.device != self._device:
            raise ValueError(f"{name} must be a bf16 tensor on {self._device}")
        B, Hkv, D = self._sizes
        shape = x.shape
        if len(shape) != 4 or shape[0] != B or shape[3] != D or shape[2] < 1 or (heads and shape[1] != heads) or (
                S is not None and shape[2] != S):
            raise ValueError(f"{name} must be [{B}, {heads or 'Hq'}, {S or 'S'}, {D}], got {list(shape)}")
        contiguous = x.is_contiguous()
        if not strided:
            if not contiguous:
                raise ValueError(f"{name} must be contiguous")
        else:
            if x.requires_grad and torch.is_grad_enabled():
                raise ValueError(f"{name} requires a gradient, and none flows through an 8-bit cache: detach it")
            refuse_tangents(x)
        return shape[2], None if contiguous else _strides(name, x)

    def _counts(self, name, t):
        if t is None:
            return None
        if t.device != self._device or t.dtype != torch.int32 or tuple(t.shape) != (self._sizes[0],) \
                or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 tensor [{self._sizes[0]}] on {self._device}")
        return t.data_ptr()

    @contextlib.contextmanager
    def _on(self, stream):
        """The cache's device current, and `stream` (a torch.cuda.Stream, a handle, or None for the
        device's current stream) current on it, so that memory allocated within belongs to that
        stream; yields its handle."""
        if stream == _PER_THREAD or getattr(stream, "cuda_stream", None) == _PER_THREAD:
            raise ValueError("the per-thread default stream is another one in each thread, which memory that belongs to "
                             "a stream does not tell apart: pass a stream of its own")
        if not isinstance(stream, (int, type(None))) and stream.device != self._device:
            raise ValueError(f"stream is on {stream.device} but the cache is on {self._device}")
        with torch.cuda.device(self._device):
            if stream is None:
                stream = torch.cuda.current_stream(self._device)
            elif isinstance(stream, int):
                # 0 and 1 stand for the default stream, which an ExternalStream of 0 is not.
                stream = torch.cuda.default_stream(self._device) if stream in (0, 1) else torch.cuda.ExternalStream(
                    stream, device=self._device)
            with torch.cuda.stream(stream):
                yield stream.cuda_stream

    def _here(self, stream) -> bool:
        """Whether a call can run as things are: on the current device's current stream."""
        return stream is None and _current_device() == self._index

    def _done(self, where, rc, handle, check_status) -> None:
        if rc != native.ATTN_OK:
            raise native.AttnError(rc, where)
        if check_status:
            with torch.cuda.device(self._device):
                native.attn_sync_status(handle)

    def write(self, k, v, new_lens=None, stream=None, check_status: bool = False) -> None:
        """Quantise the step's new tokens k, v (bf16 [B, Hkv, S, D], any strides of
        16 bytes with D contiguous) into the cache (``attn_cache_write``).  They stand for the last
        positions that ``seq_lens`` counts: sequence b's ``new_lens[b]`` (int32 [B];
        default S each) first rows for positions seq_lens[b] - new_lens[b] ...."""
        S, ks = self._rows("k", k, self._sizes[1])
        _, vs = self._rows("v", v, self._sizes[1], S)
        n = self._counts("new_lens", new_lens)
        if self._here(stream):
            st = _stream_handle(self._index)
            rc = self._lib.attn_cache_write(self._ref, k.data_ptr(), ks, v.data_ptr(), vs, n, S, st)
        else:
            with self._on(stream) as st:
                rc = self._lib.attn_cache_write(self._ref, k.data_ptr(), ks, v.data_ptr(), vs, n, S, st)
        self._done("attn_cache_write", rc, st, check_status)

    def append(self, k, v, rotary, q=None, new_lens=None, positions=None, first: int = 0, q_norm=None, k_norm=None,
               eps: float = 1e-6, q_out=None, stream=None, check_status: bool = False):
        """``write`` of the step's heads as projected: K normed (``k_norm``, [D] bf16 or fp32, if given) and
        rotated by ``rotary`` (a rotary.Rotary) before it is quantised, V as it is, in one launch with the
        step's queries q (bf16 [B, Hq, S, D], strides as k's), which come back normed and rotated,
        contiguous, for ``attention`` (``attn_cache_append``).  A token stands at its place in the cache
        plus ``first``, or at ``positions[b, i]`` (int32 or int64 [B, S] or [S] on the device).  Rows of q
        past ``new_lens[b]`` are left as they were in ``q_out`` when given, and unspecified otherwise."""
        B, Hkv, D = self._sizes
        key = k.shape, k.stride(), v.shape, v.stride(), None if q is None else (q.shape, q.stride())
        x = self._steps.get(key)
        if x is None:
            x = self._step(key, q, k, v)
        S, Hq, like = x
        at = self._device
        if k.dtype is not _BF16 or v.dtype is not _BF16 or k.device != at or v.device != at or (
                q is not None and (q.dtype is not _BF16 or q.device != at)):
            raise ValueError(f"k, v and q must be bf16 tensors on {at}")
        if q is None and (q_out is not None or q_norm is not None):
            raise ValueError("q_out and q_norm go with q")
        if q_out is not None:
            self._rows("q_out", q_out, Hq, S, strided=False)
        if torch.is_grad_enabled():
            for name, t in (("k", k), ("v", v), ("q", q), ("q_norm", q_norm), ("k_norm", k_norm)):
                if t is not None and t.requires_grad:
                    raise ValueError(f"{name} requires a gradient, and none flows through an 8-bit cache: detach it")
        refuse_tangents(k, v, q, q_norm, k_norm)
        n = None if new_lens is None else self._counts("new_lens", new_lens)
        c = rotary._plan(self._device, B, S, D, positions, first, q_norm, k_norm, eps)
        heads = native.AttnHeads.from_buffer_copy(like)
        heads.k, heads.v = k.data_ptr(), v.data_ptr()
        if q is not None:
            heads.q = q.data_ptr()
        if self._here(stream):
            st = _stream_handle(self._index)
            q_out, rc = self._append(c, heads, q, q_out, n, Hq, S, st)
        else:
            with self._on(stream) as st:
                q_out, rc = self._append(c, heads, q, q_out, n, Hq, S, st)
        if rc or check_status:
            self._done("attn_cache_append", rc, st, check_status)
        return q_out

    def _step(self, key, q, k, v):
        """(S, Hq, attn_heads_t without addresses) of an append's heads, checked and kept by their sizes and strides."""
        S, _ = self._rows("k", k, self._sizes[1])
        self._rows("v", v, self._sizes[1], S)
        if q is not None:
            self._rows("q", q, 0, S)
        heads = _heads_of(q, k, v)
        heads.q = heads.k = heads.v = None
        if len(self._steps) >= 256:
            self._steps.clear()
        x = self._steps[key] = S, 0 if q is None else q.shape[1], heads
        return x

    def _append(self, c, heads, q, q_out, n, Hq, S, st):
        if q is not None and q_out is None:
            q_out = q.new_empty((self._sizes[0], Hq, S, self._sizes[2]))
        rc = self._lib.attn_cache_append(self._ref, c, heads, None if q_out is None else q_out.data_ptr(), n, Hq, S, st)
        return q_out, rc

    def read(self, S: int, first: int = 0, k_out=None, v_out=None, stream=None, check_status: bool = False):
        """Positions first .. first+S-1 of every sequence as bf16 (k, v), each
        [B, Hkv, S, D] (``attn_cache_read``).  Rows past a sequence's length are left as
        they were in ``k_out`` / ``v_out`` when given, and are zero otherwise."""
        B, Hkv, D = self._sizes
        S, first = int(S), int(first)
        if S < 1 or first < 0:
            raise ValueError("read needs S >= 1 and first >= 0")
        for name, t in (("k_out", k_out), ("v_out", v_out)):
            if t is not None:
                self._rows(name, t, Hkv, S, strided=False)

        with contextlib.nullcontext(_stream_handle(self._index)) if self._here(stream) else self._on(stream) as st:
            if k_out is None:
                k_out = torch.zeros((B, Hkv, S, D), dtype=torch.bfloat16, device=self._device)
            if v_out is None:
                v_out = torch.zeros((B, Hkv, S, D), dtype=torch.bfloat16, device=self._device)
            rc = self._lib.attn_cache_read(self._ref, k_out.data_ptr(), v_out.data_ptr(), first, S, st)
        self._done("attn_cache_read", rc, st, check_status)
        return k_out, v_out

    def attention(self, q, causal: bool = True, scale: float | None = None, q_lens=None, out=None, lse=None,
                  return_lse: bool = True, stream=None, check_status: bool = False):
        """O (and LSE) of the step's queries q (bf16 [B, Hq, Sq, D], strides as in
        ``write``) over the cache (``attn_cache_fwd``).  Sequence b's ``q_lens[b]``
        (int32 [B]; default Sq each) first rows stand for its last positions; rows past
        them are left as they were in ``out`` / ``lse`` when given, and unspecified
        otherwise."""
        B, Hkv, D = self._sizes
        Sq, qs = self._rows("q", q, 0)
        Hq = q.shape[1]
        if Hq < 1 or Hq % Hkv:
            raise ValueError(f"q has {Hq} heads: a multiple of the cache's {Hkv} is needed")
        if out is not None:
            self._rows("out", out, Hq, Sq, strided=False)
        if lse is not None and (lse.device != self._device or lse.dtype != torch.float32
                                or tuple(lse.shape) != (B, Hq, Sq) or not lse.is_contiguous()):
            raise ValueError(f"lse must be a contiguous float32 tensor [{B}, {Hq}, {Sq}] on {self._device}")
        n = self._counts("q_lens", q_lens)
        if scale is None:
            scale = 1.0 / math.sqrt(D)

        if self._here(stream):
            st = _stream_handle(self._index)
            out, lse, rc = self._attend(q, qs, out, lse, n, Hq, Sq, scale, causal, return_lse, st)
        else:
            with self._on(stream) as st:
                out, lse, rc = self._attend(q, qs, out, lse, n, Hq, Sq, scale, causal, return_lse, st)
        self._done("attn_cache_fwd", rc, st, check_status)
        return (out, lse) if return_lse else out

    def _attend(self, q, qs, out, lse, n, Hq, Sq, scale, causal, return_lse, st):
        need = self._workspace_bytes.get((Hq, Sq))
        if need is None:
            c = ctypes.c_ulonglong(0)
            rc = self._lib.attn_cache_workspace(self._ref, Hq, Sq, ctypes.byref(c))
            if rc != native.ATTN_OK:
                return None, None, rc
            need = self._workspace_bytes[Hq, Sq] = c.value
        if out is None:
            out = torch.empty((self._sizes[0], Hq, Sq, self._sizes[2]), dtype=torch.bfloat16, device=self._device)
        if lse is None and return_lse:
            lse = torch.empty((self._sizes[0], Hq, Sq), dtype=torch.float32, device=self._device)
        w = None
        if need:
            if st == _PER_THREAD:
                raise ValueError("attention over a cache of this length needs a workspace, which belongs to a stream, and "
                                 "the per-thread default stream is another one in each thread")
            if torch.cuda.is_current_stream_capturing():
                w = torch.empty(need, dtype=torch.uint8, device=self._device)
            else:
                w = _workspaces.get((self._index, st))
                if w is None or w.numel() < need:
                    w = _workspaces[self._index, st] = torch.empty(need, dtype=torch.uint8, device=self._device)
        rc = self._lib.attn_cache_fwd(self._ref, q.data_ptr(), qs, out.data_ptr(), None if lse is None else lse.data_ptr(), n,
                                      Hq, Sq, scale, 1 if causal else 0, None if w is None else w.data_ptr(), need, st)
        return out, lse, rc
