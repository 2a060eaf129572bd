"""The append to the 8-bit cache on the GPU against its definition in float64: scales exactly, K's codes within half a
step of E4M3 and the rotation's fp32 error, V's exactly, q as the rotation gives it."""
import math

import numpy as np
import pytest
import torch

from causal_scaled_dot_gb300 import native
from causal_scaled_dot_gb300.kv_cache import KVCache
from causal_scaled_dot_gb300.rotary import Rotary
from tests import rope_util
from tests.cache_util import PlainCache, attention, codes_of, make, rows, scale_of, to_f64
from tests.test_cache_gpu import ints, set_lens
from tests.test_rope_gpu import weights

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def projected(B, S, Hq, Hkv, D, seed):
    """A projection's output and its heads [B, H, S, D], on the device."""
    x = rows((B, S, (Hq + 2 * Hkv) * D), seed).cuda()
    h = x.unflatten(2, (Hq + 2 * Hkv, D)).transpose(1, 2)
    return h[:, :Hq], h[:, Hq:Hq + Hkv], h[:, Hq + Hkv:]


class Expected:
    """What a cache holds after appends: float64 values of K with their fp32 error, and a PlainCache for V.  K's codes are
    compared after each call; what a block held before comes from the device's own cache, so that one code that fell on
    the other side of a border does not count twice."""

    def __init__(self, cache):
        total, Hkv, block, D = cache.k.shape
        self.cache, self.plain = cache, PlainCache(total, Hkv, block, D)

    def append(self, table, lens, new, q, k, v, rotary, wq, wk, positions=None, first=0, q_out=None, **call):
        cache, block = self.cache, self.plain.block
        B, Hkv, S, D = k.shape
        codes, scales = to_f64(cache.k.float()), to_f64(cache.k_scale)
        set_lens(cache, lens)
        at = np.array([[t - n + i for i in range(S)] for t, n in zip(lens, new)]) + first
        if positions is not None:
            at = np.broadcast_to(positions.cpu().numpy(), (B, S))
        got = cache.append(k, v, rotary, q=q, new_lens=None if min(new) == S else ints(new), positions=positions, first=first, q_norm=wq,
                           k_norm=wk, q_out=q_out, check_status=call.pop("check_status", True), **call)
        f = lambda w: None if w is None else to_f64(w)  # noqa: E731
        if q is not None:
            want, tol, _ = rope_util.forward(to_f64(q), at, rotary, f(wq))
            for b, n in enumerate(new):
                assert (np.abs(to_f64(got[b, :, :n]) - want[b, :, :n]) <= tol[b, :, :n]).all()
        y, _, fp32 = rope_util.forward(to_f64(k), at, rotary, f(wk))
        now, now_scale = to_f64(cache.k.float()), to_f64(cache.k_scale)
        self.plain.write(np.zeros_like(to_f64(v)), to_f64(v), table, lens, new)
        touched = np.zeros(codes.shape[:3], bool)
        for b, (t, n) in enumerate(zip(lens, new)):
            p = max(t - n, 0)
            while p < t:
                to = min(t, (p // block + 1) * block)
                page, a, row = table[b][p // block], p % block, p - (t - n)
                for h in range(Hkv):
                    x, e = y[b, h, row:row + to - p], fp32[b, h, row:row + to - p]
                    s = scale_of(x)
                    if a:
                        s = max(s, scales[page, h])
                    assert now_scale[page, h] == s, (b, p, h)
                    moved = codes_of(codes[page, h, :a] * (scales[page, h] / s)) if a else codes[page, h, :0]
                    assert np.array_equal(now[page, h, :a], moved, equal_nan=True)
                    put, finite = now[page, h, a:a + to - p], np.isfinite(x)
                    assert np.array_equal(np.isnan(put), ~finite)
                    # half a step of E4M3: 2^-4 of the value, 2^-10 (times the scale) below its normal numbers
                    tol = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s) + e
                    assert (np.abs(put * s - x)[finite] <= tol[finite]).all()
                    # and all but those next to a border are the code itself
                    same = (put == codes_of(x / s)) | ~finite
                    border = np.abs(codes_of((x - e) / s) - codes_of((x + e) / s)) > 0
                    assert (same | border).all()
                    touched[page, h, :a + to - p] = True
                p = to
        assert np.array_equal(now[~touched], codes[~touched], equal_nan=True), "something else was written"
        code_v = to_f64(cache.v.float())
        for b, (t, n) in enumerate(zip(lens, new)):
            for i in range(-(-t // block)) if n else ():
                m = min(block, t - i * block)
                assert np.array_equal(code_v[table[b][i]][:, :m], self.plain.v[table[b][i]][:, :m], equal_nan=True)
        return got


CACHES = [(64, 16), (64, 64), (64, 128), (128, 16), (128, 32), (128, 128)]


@pytest.mark.parametrize("D,block", CACHES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [None, torch.bfloat16, torch.float32])
def test_prompts_chunks_and_tokens(D, block, interleaved, norm):
    """Uneven prompts, then a padded chunk, then single tokens; one slot idle."""
    B, Hq, Hkv = 3, 6, 2
    r = Rotary.from_base(D, interleaved=interleaved)
    w = [t.cuda() for t in weights(D, norm)] if norm else (None, None)
    cache, table = make(B, Hkv, D, block, 400, seed=D + block)
    e, lens = Expected(cache), [0] * B
    for i, new in enumerate(([150, 0, 37], [70, 0, 101], [1, 0, 1], [1, 0, 1], [3, 0, 2])):
        lens = [t + n for t, n in zip(lens, new)]
        e.append(table, lens, new, *projected(B, max(new), Hq, Hkv, D, 10 + i), r, *w)


@pytest.mark.parametrize("rotary", [Rotary([]), Rotary.from_base(16), Rotary.from_base(48), Rotary.from_base(72, interleaved=True),
                                    Rotary.by_parts(64, 16, 512), Rotary([0.1] * 8, factor=3.0)])
@pytest.mark.parametrize("norm", [None, torch.float32])
def test_parts_and_scalings(rotary, norm):
    D = 128
    w = [t.cuda() for t in weights(D, norm)] if norm else (None, None)
    cache, table = make(2, 3, D, 64, 200, seed=3)
    e = Expected(cache)
    e.append(table, [90, 61], [90, 61], *projected(2, 90, 3, 3, D, 1), rotary, *w)
    e.append(table, [97, 68], [7, 7], *projected(2, 7, 3, 3, D, 2), rotary, *w)


@pytest.mark.parametrize("S", [1, 5, 100])
def test_without_rotation_it_is_the_write(S):
    """No frequencies and no norm: every bit as attn_cache_write has it, and q as it was."""
    D, Hkv = 128, 2
    a, table = make(2, Hkv, D, 32, 300, seed=1)
    b, _ = make(2, Hkv, D, 32, 300, seed=1)
    for step in range(3):
        q, k, v = projected(2, S, 4, Hkv, D, step)
        for c in (a, b):
            c.seq_lens.add_(S)
        got = a.append(k, v, Rotary([]), q=q, check_status=True)
        b.write(k, v, check_status=True)
        assert torch.equal(got, q)
        for name in ("k", "v"):
            assert torch.equal(getattr(a, name).view(torch.uint8), getattr(b, name).view(torch.uint8))
            x, y = getattr(a, name + "_scale"), getattr(b, name + "_scale")
            assert torch.equal(x.nan_to_num(-1), y.nan_to_num(-1))


@pytest.mark.parametrize("kind", ["each", "shared", "first"])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_given_positions(kind, dtype):
    """Positions of drafted tokens that share one, or an offset."""
    D = 64
    cache, table = make(2, 1, D, 16, 64, seed=5)
    e, r = Expected(cache), Rotary.from_base(D)
    p = torch.tensor([[40, 41, 41, 42, 42], [7, 8, 8, 8, 9]], dtype=dtype, device="cuda")
    e.append(table, [15, 26], [15, 26], *projected(2, 26, 2, 1, D, 2), r, None, None)  # what the blocks hold before
    more = {"each": dict(positions=p), "shared": dict(positions=p[0]), "first": dict(first=1000)}[kind]
    e.append(table, [20, 31], [5, 5], *projected(2, 5, 2, 1, D, 1), r, None, None, **more)


def test_rows_past_the_last_are_left():
    D = 64
    cache, table = make(3, 2, D, 16, 64, seed=5)
    q, k, v = projected(3, 9, 4, 2, D, 1)
    out = torch.full((3, 4, 9, D), 7.0, dtype=torch.bfloat16, device="cuda")
    w = [t.cuda() for t in weights(D, torch.float32)]
    got = Expected(cache).append(table, [9, 20, 3], [9, 0, 3], q, k, v, Rotary.from_base(D), *w, q_out=out)
    assert got is out and (out[1] == 7).all() and (out[2, :, 3:] == 7).all() and not (out[2, :, :3] == 7).all()


def test_without_q():
    D = 64
    cache, table = make(2, 2, D, 16, 64, seed=5)
    _, k, v = projected(2, 20, 1, 2, D, 1)
    assert Expected(cache).append(table, [20, 20], [20, 20], None, k, v, Rotary.from_base(D), None, None) is None


@pytest.mark.parametrize("layout", ["dense", "by token", "heads apart"])
def test_layouts(layout):
    D = 128
    cache, table = make(2, 2, D, 64, 128, seed=5)
    q, k, v = projected(2, 70, 4, 2, D, 1)
    if layout == "dense":
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    elif layout == "heads apart":
        wide = torch.full((2, 70, 4, D + 8), math.nan, dtype=torch.bfloat16, device="cuda")
        wide[:, :, :2, :D], wide[:, :, 2:, :D] = k.transpose(1, 2), v.transpose(1, 2)
        k, v = wide[:, :, :2, :D].transpose(1, 2), wide[:, :, 2:, :D].transpose(1, 2)
    Expected(cache).append(table, [70, 70], [70, 70], q, k, v, Rotary.from_base(D), None, None)


def test_values_that_are_not_finite():
    """They become NaN and do not count for the scale; a norm spreads NaN over its row."""
    D = 64
    r = Rotary.from_base(32)
    q, k, v = projected(1, 12, 1, 2, D, 1)
    k[0, 0, 3, 2], k[0, 1, 5, 40], v[0, 0, 7, 9] = math.inf, math.nan, -math.inf
    for w in (None, weights(D, torch.float32)[0].cuda()):
        cache, table = make(1, 2, D, 16, 16, seed=5)
        cache.seq_lens.fill_(12)
        cache.append(k, v, r, k_norm=w, check_status=True)
        got = to_f64(cache.k.float())[table[0][0]][:, :12]
        y, _, _ = rope_util.forward(to_f64(k), np.arange(12)[None], r, None if w is None else to_f64(w))
        assert np.array_equal(np.isnan(got), ~np.isfinite(y[0]))
        for h in range(2):
            assert float(cache.k_scale[table[0][0], h]) == scale_of(y[0, h])
        assert np.isnan(to_f64(cache.v.float())[table[0][0], 0, 7, 9])


@pytest.mark.parametrize("s", [0.3, 1e-3, 5.0])
def test_a_callers_scale(s):
    """A block under a scale that is no power of two keeps it: the codes are x / s to nearest."""
    D = 64
    cache, table = make(1, 1, D, 16, 32, seed=5)
    page = table[0][0]
    cache.k_scale[page], cache.v_scale[page] = s, s
    cache.k.view(torch.uint8)[page, :, :4] = 0x38  # 1.0
    cache.v.view(torch.uint8)[page, :, :4] = 0x38
    cache.seq_lens.fill_(10)
    q, k, v = projected(1, 6, 1, 1, D, 1)
    k, v = k * (s * 10), v * (s * 10)
    r = Rotary.from_base(D)
    cache.append(k, v, r, check_status=True)
    f = float(np.float32(s))
    y, _, fp32 = rope_util.forward(to_f64(k), np.arange(4, 10)[None], r)
    assert float(cache.k_scale[page, 0]) == f and float(cache.v_scale[page, 0]) == f
    got = to_f64(cache.k.float())[page, 0, 4:10]
    border = codes_of((y[0, 0] - fp32[0, 0]) / f) != codes_of((y[0, 0] + fp32[0, 0]) / f)
    assert ((got == codes_of(y[0, 0] / f)) | border).all()
    assert np.array_equal(to_f64(cache.v.float())[page, 0, 4:10], codes_of(to_f64(v)[0, 0] / f))


@pytest.mark.parametrize("what", ["table", "length", "count"])
def test_bad_device_data_is_reported(what):
    """A page outside the cache or a length past its end: nothing is written there, and the status says so."""
    D = 64
    cache, table = make(2, 1, D, 16, 64, seed=5)
    q, k, v = projected(2, 20, 2, 1, D, 1)
    set_lens(cache, [20, 20])
    new = ints([20, 20])
    if what == "table":
        cache.block_table[0, 1] = 10**6
    elif what == "length":
        cache.seq_lens[1] = 1000
    else:
        new[1] = 21
    with pytest.raises(native.AttnError) as e:
        cache.append(k, v, Rotary.from_base(D), q=q, new_lens=new, check_status=True)
    assert e.value.code == native.ATTN_ERR_BAD_CACHE
    native.attn_sync_status()  # cleared
    put = to_f64(cache.k.float())
    if what == "table":
        assert np.isfinite(put[table[0][0]]).all() and np.isnan(put[table[0][1]]).all() and np.isfinite(put[table[1][1], 0, :4]).all()
    elif what == "length":  # taken as the cache's end, 64
        assert np.isfinite(put[table[1][3]]).all() and np.isnan(put[table[1][0]]).all()


def test_more_tokens_than_the_sequence_holds():
    """Rows before the first position are dropped; their queries are rotated all the same."""
    D = 64
    cache, table = make(1, 1, D, 16, 64, seed=5)
    Expected(cache).append(table, [7], [12], *projected(1, 12, 2, 1, D, 1), Rotary.from_base(D), None, None)


@pytest.mark.parametrize("D,block,Hq,Hkv", [(64, 16, 4, 2), (128, 64, 8, 2)])
def test_generating(D, block, Hq, Hkv):
    """Prompt, drafted tokens and single tokens: append, then attention over what the cache holds."""
    B = 3
    r, w = Rotary.from_base(D), [t.cuda() for t in weights(D, torch.bfloat16)]
    cache, table = make(B, Hkv, D, block, 300, seed=9)
    lens, e = [0] * B, Expected(cache)
    for step, new in enumerate(([130, 80, 0], [4, 2, 30], [1, 1, 1], [1, 1, 1])):
        lens = [t + n for t, n in zip(lens, new)]
        S = max(new)
        x = projected(B, S, Hq, Hkv, D, 100 + step)
        q = e.append(table, lens, new, *x, r, *w)
        out, lse = cache.attention(q, q_lens=ints(new), check_status=True)
        kv = [to_f64(t) for t in cache.read(max(lens))]
        for b, (t, n) in enumerate(zip(lens, new)):
            if n == 0:
                continue
            want, want_l, tol, tol_l = attention(to_f64(q[b, :, :n]), kv[0][b, :, :t], kv[1][b, :, :t], 1 / math.sqrt(D), t - n, True)
            assert (np.abs(to_f64(out[b, :, :n]) - want) <= tol).all()
            assert (np.abs(to_f64(lse[b, :, :n]) - want_l) <= tol_l).all()


def test_prompt_then_cache_agrees_with_attention_on_all():
    """What a user does: a prompt through heads and attention, its heads appended, then a token over the cache.  The queries
    are the same bits.  The cache's K is the rotated fp32 value to E4M3, half a step of which is 2^-4 of it or 2^-10 of the
    scale, and heads' k the same value to bf16, 2^-8 of it: they differ by no more than both, taken of |k| / (1 - 2^-8),
    and the fp32 error, 2^-19 of two elements' magnitudes.
    (How far E4M3 moves the output depends on the scores' spread, so the output is compared over what the cache holds.)"""
    D, Hq, Hkv, S = 64, 4, 2, 161
    r, w = Rotary.from_base(D), [t.cuda() for t in weights(D, torch.float32)]
    qkv = (rows((1, S, (Hq + 2 * Hkv) * D), 4) * 0.5).cuda()
    q, k, v = r.heads(qkv, Hq, Hkv, q_norm=w[0], k_norm=w[1])
    o = native.attention(q, k, v, return_lse=False)
    cache = KVCache.empty(1, Hkv, D, 256, block_size=32)
    h = qkv.unflatten(2, (Hq + 2 * Hkv, D)).transpose(1, 2)
    parts = lambda a, z: (h[:, Hq:Hq + Hkv, a:z], h[:, Hq + Hkv:, a:z], r)  # noqa: E731
    cache.seq_lens.fill_(S - 1)
    prompt = cache.append(*parts(0, S - 1), q=h[:, :Hq, :S - 1], q_norm=w[0], k_norm=w[1])
    assert torch.equal(prompt, q[:, :, :S - 1])
    cache.seq_lens.add_(1)
    last = cache.append(*parts(S - 1, S), q=h[:, :Hq, S - 1:], q_norm=w[0], k_norm=w[1])
    assert torch.equal(last, q[:, :, S - 1:])
    got, _ = cache.attention(last, check_status=True)
    held = cache.read(S)
    for x, y, scale in zip(held, (k, v), (cache.k_scale, cache.v_scale)):
        x, y = to_f64(x), to_f64(y)
        s = to_f64(scale)[: -(-S // 32)].repeat(32, 0)[:S].T[None, :, :, None]
        big = np.abs(y) / (1 - 2.0 ** -8)
        assert (np.abs(x - y) <= np.maximum(2.0 ** -4 * big, 2.0 ** -10 * s) + 2.0 ** -8 * big + 2.0 ** -18 * big.max(-1, keepdims=True)).all()
    want, _, tol, _ = attention(to_f64(last)[0], *(to_f64(t)[0] for t in held), 1 / math.sqrt(D), S - 1, True)
    assert (np.abs(to_f64(got)[0] - want) <= tol).all()
    assert o.isfinite().all()


def test_captured_steps_follow_the_lengths():
    D, Hq, Hkv = 128, 8, 2
    r, w = Rotary.from_base(D), [t.cuda() for t in weights(D, torch.bfloat16)]
    a, table = make(2, Hkv, D, 64, 200, seed=9)
    b, _ = make(2, Hkv, D, 64, 200, seed=9)
    x = rows((2, 1, (Hq + 2 * Hkv) * D), 1).cuda()
    h = x.unflatten(2, (Hq + 2 * Hkv, D)).transpose(1, 2)
    parts = h[:, Hq:Hq + Hkv], h[:, Hq + Hkv:], r

    def step(c):
        c.seq_lens.add_(1)
        q = c.append(*parts, q=h[:, :Hq], q_norm=w[0], k_norm=w[1])
        return c.attention(q)

    for c in (a, b):
        set_lens(c, [60, 3])
        p = projected(2, 60, Hq, Hkv, D, 7)
        c.append(p[1], p[2], r, k_norm=w[1], new_lens=ints([60, 3]))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(a)
    torch.cuda.current_stream().wait_stream(s)
    step(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(a)
    for i in range(12):  # over a block's end
        x.copy_(rows(x.shape, 20 + i))
        graph.replay()
        want = step(b)
        for y, z in zip(got, want):
            assert torch.equal(y, z)
    assert torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8)) and torch.equal(a.seq_lens, b.seq_lens)
    native.attn_sync_status()


def test_on_other_streams():
    """stream= as a Stream and as a handle, after a copy that is still under way there."""
    D = 64
    r = Rotary.from_base(D)
    want, _ = make(2, 1, D, 16, 64, seed=5)
    q, k, v = projected(2, 30, 2, 1, D, 1)
    want.seq_lens.fill_(30)
    ref = want.append(k, v, r, q=q)
    for handle in (False, True):
        cache, _ = make(2, 1, D, 16, 64, seed=5)
        cache.seq_lens.fill_(30)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            big = torch.zeros(1 << 26, device="cuda")
            for _ in range(10):
                big.add_(1)
            q2, k2, v2 = (t * 1 for t in (q, k, v))
        got = cache.append(k2, v2, r, q=q2, stream=s.cuda_stream if handle else s)
        s.synchronize()
        assert torch.equal(got, ref) and torch.equal(cache.k.view(torch.uint8), want.k.view(torch.uint8))
    with pytest.raises(ValueError, match="per-thread"):
        want.append(k, v, r, stream=2)


def test_offsets_past_32_bits():
    """A cache whose blocks lie more than 2^31 elements from its start, and heads as far apart."""
    D, block, Hkv = 128, 128, 2
    total = (1 << 31) // (Hkv * block * D) + 4
    shape = (total, Hkv, block, D)
    k, v = (torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = torch.ones(shape[:2], device="cuda"), torch.ones(shape[:2], device="cuda")
    far = KVCache(k, v, ks, vs, torch.tensor([[total - 1, total - 3]], dtype=torch.int32, device="cuda"), ints([140]))
    near_ = KVCache.empty(1, Hkv, D, 256, block_size=block)
    near_.seq_lens.fill_(140)
    x = projected(1, 140, 4, Hkv, D, 3)
    r = Rotary.from_base(D)
    a, b = far.append(x[1], x[2], r, q=x[0], check_status=True), near_.append(x[1], x[2], r, q=x[0], check_status=True)
    assert torch.equal(a, b)
    for p, q in zip(far.read(140), near_.read(140)):
        assert torch.equal(p, q)


def test_two_streams_at_once():
    """Appends to two caches that run side by side."""
    D, Hq, Hkv = 64, 4, 2
    r, w = Rotary.from_base(D), [t.cuda() for t in weights(D, torch.float32)]
    sets = []
    for i in range(2):
        c, _ = make(3, Hkv, D, 32, 400, seed=i)
        ref, _ = make(3, Hkv, D, 32, 400, seed=i)
        for x in (c, ref):
            set_lens(x, [300, 17, 211])
        sets.append((c, ref, projected(3, 211, Hq, Hkv, D, 40 + i), ints([211, 17, 100])))
    call = lambda c, x, n: c.append(x[1], x[2], r, q=x[0], new_lens=n, q_norm=w[0], k_norm=w[1])  # noqa: E731
    # rows past a sequence's own are left unspecified in a new tensor: compare those that are there
    want = [call(ref, x, n) for _, ref, x, n in sets]
    torch.cuda.synchronize()
    got, streams = [None, None], [torch.cuda.Stream() for _ in sets]
    for _ in range(10):
        for i, (c, _, x, n) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                got[i] = call(c, x, n)
    torch.cuda.synchronize()
    for i, (c, ref, _, n) in enumerate(sets):
        for b, m in enumerate(n.tolist()):
            assert torch.equal(got[i][b, :, :m], want[i][b, :, :m])
        assert torch.equal(c.k.view(torch.uint8), ref.k.view(torch.uint8)) and torch.equal(c.v.view(torch.uint8), ref.v.view(torch.uint8))


def test_the_same_tokens_again():
    """An append that is made twice leaves what the first one left."""
    D = 64
    c, table = make(2, 2, D, 16, 100, seed=3)
    r = Rotary.from_base(D)
    e = Expected(c)
    e.append(table, [40, 21], [40, 21], *projected(2, 40, 2, 2, D, 1), r, None, None)
    x = projected(2, 30, 2, 2, D, 2)
    set_lens(c, [70, 51])
    c.append(x[1], x[2], r)
    once = [t.clone() for t in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale.nan_to_num(-1), c.v_scale.nan_to_num(-1))]
    c.append(x[1], x[2], r, check_status=True)
    for a, b in zip((c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale.nan_to_num(-1), c.v_scale.nan_to_num(-1)), once):
        assert torch.equal(a, b)


def test_gradients_are_refused_and_no_grad_is_taken():
    D = 64
    c, _ = make(1, 1, D, 16, 32, seed=3)
    c.seq_lens.fill_(3)
    q, k, v = projected(1, 3, 1, 1, D, 1)
    w = torch.ones(D, device="cuda", requires_grad=True)
    r = Rotary.from_base(D)
    with pytest.raises(ValueError, match="gradient"):
        c.append(k.requires_grad_() if k.is_leaf else k.detach().requires_grad_(), v, r)
    with pytest.raises(ValueError, match="k_norm"):
        c.append(k.detach(), v, r, k_norm=w)
    with torch.no_grad():
        c.append(k, v, r, k_norm=w, check_status=True)
