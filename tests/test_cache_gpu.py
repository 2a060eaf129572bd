"""The 8-bit key/value cache on the GPU against its definitions in float64
(tests/cache_util.py): codes and scales exactly, values read back exactly,
attention within the roundings that cache_util.attention adds up."""
import math

import numpy as np
import pytest
import torch

from causal_scaled_dot_gb300.kv_cache import KVCache
from tests.cache_util import PlainCache, attention, make, rows, to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def set_lens(cache, lens):
    cache.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def fill(cache, table, lens, seed, chunk=None, plain=None):
    """Write lens[b] tokens in calls of at most `chunk` tokens; returns the plain cache beside it."""
    B, Hkv, D = cache._sizes
    total, _, block, _ = cache.k.shape
    plain = plain or PlainCache(total, Hkv, block, D)
    done, step = [0] * B, 0
    while any(d < t for d, t in zip(done, lens)):
        new = [min(t - d, chunk or t - d) for d, t in zip(done, lens)]
        done = [d + n for d, n in zip(done, new)]
        k, v = rows((B, Hkv, max(new), D), seed + step), rows((B, Hkv, max(new), D), seed + 1000 + step, 0.5)
        set_lens(cache, done)
        cache.write(k.cuda(), v.cuda(), new_lens=None if min(new) == max(new) else ints(new), check_status=True)
        plain.write(to_f64(k), to_f64(v), table, done, new)
        step += 1
    set_lens(cache, lens)
    return plain


def assert_same_cache(cache, plain, table, lens):
    _, _, block, _ = cache.k.shape
    for name in ("k", "v"):
        code, scale = to_f64(getattr(cache, name).float()), to_f64(getattr(cache, name + "_scale"))
        want, want_scale = getattr(plain, name), getattr(plain, name + "_scale")
        for b, t in enumerate(lens):
            for i in range(-(-t // block)):
                p, n = table[b][i], min(block, t - i * block)
                assert np.array_equal(scale[p], want_scale[p]), (name, b, i)
                assert np.array_equal(code[p][:, :n], want[p][:, :n], equal_nan=True), (name, b, i)
                assert np.isnan(code[p][:, n:]).all(), "a slot past the last token was written"
    used = {table[b][i] for b, t in enumerate(lens) for i in range(-(-t // block))}
    rest = [p for p in range(cache.k.shape[0]) if p not in used]
    assert torch.isnan(cache.k.float()[rest]).all() and torch.isnan(cache.k_scale[rest]).all(), "an unused block was written"


def check_attention(cache, plain, table, lens, Hq, Sq, q_lens=None, causal=True, seed=77, sigma=1.0, q=None, **call):
    B, Hkv, D = cache._sizes
    q = rows((B, Hq, Sq, D), seed, sigma) if q is None else q
    out = torch.full((B, Hq, Sq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Hq, Sq), 7.0, device="cuda")
    scale = 1 / math.sqrt(D)
    cache.attention(q.cuda() if not q.is_cuda else q, causal=causal, q_lens=ints(q_lens), out=out, lse=lse,
                    check_status=True, **call)
    o, l, qf = to_f64(out), to_f64(lse), to_f64(q)
    for b, t in enumerate(lens):
        n = q_lens[b] if q_lens else Sq
        assert (o[b, :, n:] == 7).all() and (l[b, :, n:] == 7).all(), "a row past the last query was written"
        if n == 0:
            continue
        want, want_l, tol, tol_l = attention(qf[b, :, :n], plain.values("k", table[b], t), plain.values("v", table[b], t),
                                             scale, t - n, causal)
        err = np.abs(o[b, :, :n] - want)
        assert (err <= tol).all(), (b, float((err / tol).max()), float(err.max()))
        empty = np.isneginf(want_l)
        assert np.array_equal(np.isneginf(l[b, :, :n]), empty) and (o[b, :, :n][empty] == 0).all()
        assert (np.abs(l[b, :, :n][~empty] - want_l[~empty]) <= tol_l[~empty]).all()
        norm = np.linalg.norm(want)
        # bf16's rounding and the weights' (each at most 2^-8, evenly spread: / sqrt 3), both, and a quarter more
        assert norm == 0 or np.linalg.norm(o[b, :, :n] - want) <= 4e-3 * norm
    return out, lse


# ------------------------------------------------------------------ write and read back
@pytest.mark.parametrize("D,block", [(64, 16), (64, 128), (128, 16), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("chunk", [1, 7, 50, None])
def test_write_codes_and_scales(D, block, chunk):
    lens = [100, 0, 37, 130] if chunk == 1 else [301, 0, 128, 517]
    cache, table = make(4, 3, D, block, 517, seed=block + D)
    plain = fill(cache, table, lens, seed=5, chunk=chunk)
    assert_same_cache(cache, plain, table, lens)


def test_write_growing_scale_moves_earlier_codes():
    cache, table = make(1, 1, 64, 64, 64, seed=1)
    plain = PlainCache(4, 1, 64, 64)
    for i, size in enumerate([2.0 ** -20, 1.0, 3e-3, 448.0, 449.0, 2.0 ** 60, 0.0, 2.0 ** 126]):
        x = rows((1, 1, 1, 64), 40 + i)
        x = (x / x.abs().max() * size).to(torch.bfloat16)
        set_lens(cache, [i + 1])
        cache.write(x.cuda(), (-x).cuda(), check_status=True)
        plain.write(to_f64(x), -to_f64(x), table, [i + 1], [1])
        assert_same_cache(cache, plain, table, [i + 1])


def test_write_zeros_extremes_and_non_finite():
    cache, table = make(1, 2, 64, 16, 48, seed=2)
    x = torch.zeros(1, 2, 48, 64)
    x[0, 0, 16:32] = 2.0 ** -133  # bf16's smallest subnormal: below the smallest scale's reach
    x[0, 1, :16] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1.5]).repeat(16)
    x[0, 1, 16:32] = float("inf")
    x[0, 1, 32:48, 0] = -float(torch.finfo(torch.bfloat16).max) / 2
    x = x.to(torch.bfloat16)
    plain = PlainCache(6, 2, 16, 64)
    set_lens(cache, [48])
    cache.write(x.cuda(), x.cuda(), check_status=True)
    plain.write(to_f64(x), to_f64(x), table, [48], [48])
    assert_same_cache(cache, plain, table, [48])


def test_write_more_rows_than_tokens_and_padding():
    """Rows for positions before 0 are dropped; padding rows (NaN here) are not read."""
    cache, table = make(3, 2, 128, 32, 64, seed=3)
    k = rows((3, 2, 9, 128), 9)
    k[1, :, 4:] = float("nan")
    plain = PlainCache(9, 2, 32, 128)
    lens, new = [5, 4, 0], [9, 4, 0]
    set_lens(cache, lens)
    cache.write(k.cuda(), k.cuda(), new_lens=ints(new), check_status=True)
    plain.write(to_f64(k), to_f64(k), table, lens, new)
    assert_same_cache(cache, plain, table, lens)


def test_write_and_attend_strided_rows():
    """K, V and q as slices of one fused projection [B, S, (Hq + 2 Hkv) D]."""
    B, Hq, Hkv, S, D = 2, 4, 2, 21, 128
    x = rows((B, S, (Hq + 2 * Hkv) * D), 11).cuda().view(B, S, Hq + 2 * Hkv, D).transpose(1, 2)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    cache, table = make(B, Hkv, D, 16, S, seed=4)
    set_lens(cache, [S] * B)
    cache.write(k, v, check_status=True)
    plain = PlainCache(cache.k.shape[0], Hkv, 16, D)
    plain.write(to_f64(k), to_f64(v), table, [S] * B, [S] * B)
    assert_same_cache(cache, plain, table, [S] * B)
    check_attention(cache, plain, table, [S] * B, Hq, S, q=q)
    # one key/value row for all heads and tokens (stride 0)
    one = rows((B, 1, 1, D), 12).cuda()
    cache.write(one.expand(B, Hkv, S, D), one.expand(B, Hkv, S, D), check_status=True)
    back, _ = cache.read(S)
    assert (back == back[:, :1, :1]).all()


@pytest.mark.parametrize("D,block,first,S", [(64, 16, 0, 300), (128, 64, 37, 100), (128, 128, 299, 5), (64, 32, 290, 500)])
def test_read_back(D, block, first, S):
    lens = [300, 0, 120]
    cache, table = make(3, 2, D, block, 300, seed=6)
    plain = fill(cache, table, lens, seed=21, chunk=90)
    k = torch.full((3, 2, S, D), 7.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    cache.read(S, first=first, k_out=k, v_out=v, check_status=True)
    for name, got in (("k", to_f64(k)), ("v", to_f64(v))):
        for b, t in enumerate(lens):
            n = max(0, min(S, t - first))
            want = plain.values(name, table[b], t)[:, first:first + n]
            assert np.array_equal(got[b, :, :n], want)  # 4 bits times a power of two: exact in bf16
            assert (got[b, :, n:] == 7).all()
    k2, v2 = cache.read(S, first=first)
    assert torch.equal(k2[0, :, :max(0, 300 - first)], k[0, :, :max(0, 300 - first)])
    assert (k2[1] == 0).all() and (v2[1] == 0).all()


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("D,block", [(64, 16), (64, 64), (128, 16), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (6, 2), (5, 1)])
def test_attention_one_token(D, block, Hq, Hkv):
    lens = [1, 0, 127, 128, 129, 300, 641]
    cache, table = make(7, Hkv, D, block, 641, seed=8)
    plain = fill(cache, table, lens, seed=31)
    check_attention(cache, plain, table, lens, Hq, 1)


@pytest.mark.parametrize("D,block,Hq,Hkv,Sq", [(128, 64, 8, 2, 3), (64, 16, 4, 4, 5), (128, 32, 32, 1, 2),
                                                (64, 128, 12, 2, 11), (128, 16, 6, 2, 90), (64, 32, 3, 1, 200)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_several_tokens(D, block, Hq, Hkv, Sq, causal):
    lens = [Sq, 0, 260, Sq + 130, 401, 2]
    q_lens = [Sq, 0, 1, Sq, max(1, Sq // 2), Sq]  # the last has more rows than tokens: its first rows see nothing
    cache, table = make(6, Hkv, D, block, 512, seed=9)
    plain = fill(cache, table, lens, seed=41)
    check_attention(cache, plain, table, lens, Hq, Sq, q_lens=q_lens, causal=causal)
    check_attention(cache, plain, table, lens, Hq, Sq, causal=causal)


@pytest.mark.parametrize("lens,Hq,Hkv,D,block,Sq", [([20011], 8, 1, 128, 64, 1), ([9000, 5], 4, 2, 64, 16, 2),
                                                    ([2500], 64, 1, 128, 128, 2), ([9000, 700], 40, 1, 128, 64, 1),
                                                    ([12345], 9, 1, 64, 32, 1), ([20011, 3000], 50, 2, 64, 64, 4)])
def test_attention_long_cache_is_joined(lens, Hq, Hkv, D, block, Sq):
    cache, table = make(len(lens), Hkv, D, block, max(lens), seed=10)
    plain = fill(cache, table, lens, seed=51)
    check_attention(cache, plain, table, lens, Hq, Sq)


@pytest.mark.parametrize("Hq,Hkv,Sq", [(33, 1, 1), (64, 2, 1), (128, 1, 1), (129, 1, 1), (300, 1, 1), (8, 1, 5), (6, 2, 43),
                                       (200, 1, 2), (2, 2, 129)])
@pytest.mark.parametrize("D,block", [(128, 64), (64, 16)])
def test_attention_many_rows(D, block, Hq, Hkv, Sq):
    """Around the sizes where a key/value head's rows (query heads x queries) fill units of 32 and 128,
    over caches with and without joined pieces."""
    for lens in ([0, 450, Sq + 63, 64], [2100, Sq, 1]):
        cache, table = make(len(lens), Hkv, D, block, max(lens), seed=12)
        plain = fill(cache, table, lens, seed=71)
        check_attention(cache, plain, table, lens, Hq, Sq)
        check_attention(cache, plain, table, lens, Hq, Sq, q_lens=[max(Sq - 1 - b, 0) for b in range(len(lens))], causal=False)


def test_attention_large_batch_of_short_sequences():
    lens = [(37 * b) % 200 for b in range(300)]
    cache, table = make(300, 2, 64, 16, 200, seed=11)
    plain = fill(cache, table, lens, seed=61)
    check_attention(cache, plain, table, lens, 4, 1)


@pytest.mark.parametrize("Hq,Sq", [(4, 1), (4, 20)])
def test_attention_one_long_sequence_among_empty_and_short_ones(Hq, Sq):
    """Units are split here, and most are smaller than what a CTA is given."""
    lens = [0 if b % 3 else (29 * b) % 260 for b in range(150)]
    lens[77] = 2900
    cache, table = make(150, 2, 64, 64, 2900, seed=11)
    plain = fill(cache, table, lens, seed=62)
    check_attention(cache, plain, table, lens, Hq, Sq)


def test_attention_sharp_scores_and_scales_far_apart():
    """Large queries (one key takes nearly all the weight, the running maximum moves often) over
    blocks whose scales differ by 2^40, for K and V alike."""
    B, Hkv, D, block, t = 1, 2, 128, 16, 700
    cache, table = make(B, Hkv, D, block, t, seed=12)
    k, v = rows((B, Hkv, t, D), 71), rows((B, Hkv, t, D), 72)
    size = 2.0 ** torch.randint(-20, 20, (t // block + 1,), generator=torch.Generator().manual_seed(3))
    v = (v * size.repeat_interleave(block)[:t, None]).to(torch.bfloat16)
    k = (k * (0.05 + torch.arange(t) / 200)[:, None]).to(torch.bfloat16)
    plain = PlainCache(cache.k.shape[0], Hkv, block, D)
    set_lens(cache, [t])
    cache.write(k.cuda(), v.cuda(), check_status=True)
    plain.write(to_f64(k), to_f64(v), table, [t], [t])
    for sigma in (0.01, 1.0, 20.0):
        check_attention(cache, plain, table, [t], 4, 1, sigma=sigma)
        check_attention(cache, plain, table, [t], 4, 30, sigma=sigma)


@pytest.mark.parametrize("Hq,Hkv,D,Sq", [(2, 2, 64, 1), (32, 2, 128, 1), (8, 1, 128, 4), (16, 2, 64, 8), (8, 1, 128, 40)])
@pytest.mark.parametrize("at", [0, 1500])
def test_attention_one_key_far_above_the_rest(Hq, Hkv, D, Sq, at):
    """A key that every row attends to, e^14 times the others, with values of zero: O is what the rest
    of a long sequence adds up to.  The others' scores differ by 1 at most and their values are
    positive, so O's relative error is at most a weight's: 2^-10 (half a step of the smallest codes) of
    0.25 / e where the row's maximum just does not fall, 2^-6.5, and the bf16 of O and the weights, 2^-8
    each; the 127 keys in that key's own tile may be lost."""
    length, block, B = 4000, 64, 40  # 40 sequences over the same blocks: a CTA's share of one is long
    rng = np.random.default_rng(7)
    one, table = make(1, Hkv, D, block, length, 3)
    set_lens(one, [length])
    plain = PlainCache(one.k.shape[0], Hkv, block, D)
    k = torch.tensor(rng.uniform(-0.5, 0.5, (1, Hkv, length, D)) * (np.arange(D) == 1), dtype=torch.bfloat16)
    v = torch.tensor(rng.uniform(1, 2, (1, Hkv, length, D)), dtype=torch.bfloat16)
    k[:, :, at, 0] = 14.0
    v[:, :, at] = 0
    one.write(k.cuda(), v.cuda())
    plain.write(to_f64(k), to_f64(v), table, [length], [length])
    cache = KVCache(one.k, one.v, one.k_scale, one.v_scale, one.block_table.repeat(B, 1), one.seq_lens.repeat(B))
    q = torch.zeros(B, Hq, Sq, D, dtype=torch.bfloat16)
    q[..., :2] = 1.0
    o = to_f64(cache.attention(q.cuda(), scale=1.0)[0])
    ks, vs = plain.values("k", table[0], length), plain.values("v", table[0], length)
    for i in range(Sq):
        n = length - Sq + i + 1
        for h in range(Hq):
            p = np.exp(ks[h * Hkv // Hq][:n, :2].sum(1))
            ref = (p / p.sum()) @ vs[h * Hkv // Hq][:n]
            assert (np.abs(o[:, h, i] - ref) <= (2 ** -6.5 + 2 ** -7 + 127 / n) * ref).all()


def test_attention_ignores_what_no_row_may_see():
    """NaN in keys and values after a row's position, and in slots past the length, reach only the
    rows that see them."""
    B, Hq, Hkv, D, block, t, Sq = 1, 2, 1, 64, 32, 150, 20
    cache, table = make(B, Hkv, D, block, t, seed=13)
    plain = fill(cache, table, [t], seed=81)
    q = rows((B, Hq, Sq, D), 82).cuda()
    clean = cache.attention(q)[0]
    bad = t - 8  # position of a token with NaN in one element of V, visible to the last 8 rows
    for which in ("v", "k"):
        code = getattr(cache, which).view(torch.uint8)
        page, slot = table[0][bad // block], bad % block
        had = int(code[page, 0, slot, 5])
        code[page, 0, slot, 5] = 0x7F if which == "v" else 0xFF
        o, lse = cache.attention(q, check_status=True)
        code[page, 0, slot, 5] = had
        sees = torch.arange(t - Sq, t) >= bad
        assert torch.equal(o[:, :, ~sees], clean[:, :, ~sees])
        hit = o[:, :, sees].isnan().cpu()
        if which == "v":
            assert hit[..., 5].all() and not hit[..., :5].any() and not hit[..., 6:].any()
            assert lse.isfinite().all()
        else:
            assert hit.all() and lse[:, :, sees].isnan().all() and lse[:, :, ~sees].isfinite().all()


def test_attention_non_finite_queries_stay_in_their_row():
    cache, table = make(1, 1, 128, 64, 200, seed=14)
    fill(cache, table, [200], seed=91)
    q = rows((1, 4, 3, 128), 92)
    clean = cache.attention(q.cuda())[0]
    q[0, 1, 1, 7], q[0, 2, 0, 3] = float("nan"), float("inf")
    o = cache.attention(q.cuda())[0]
    bad = torch.zeros(4, 3, dtype=torch.bool)
    bad[1, 1] = bad[2, 0] = True
    assert o[0, bad].isnan().all() and torch.equal(o[0, ~bad], clean[0, ~bad])
    zero = torch.zeros_like(q)
    o, lse = cache.attention(zero.cuda())  # all scores 0: plain means, LSE = ln of the keys seen
    want = torch.log(torch.tensor([198.0, 199.0, 200.0])).cuda()
    assert (lse - want).abs().max() <= 2.0 ** -18


def test_bad_blocks_and_lengths_are_reported_and_masked():
    from causal_scaled_dot_gb300 import native
    cache, table = make(2, 1, 64, 16, 64, seed=15)
    plain = fill(cache, table, [64, 64], seed=101)
    cache.block_table[0, 1], cache.block_table[1, 2] = 10 ** 6, -1
    bad = [r[:] for r in table]
    bad[0][1], bad[1][2] = 10 ** 6, -1
    q = rows((2, 2, 3, 64), 102)
    o, lse = cache.attention(q.cuda())
    with pytest.raises(native.AttnError) as e:
        native.attn_sync_status()
    assert e.value.code == native.ATTN_ERR_BAD_CACHE
    native.attn_sync_status()  # read and cleared
    for b in range(2):
        want, want_l, tol, tol_l = attention(to_f64(q)[b], plain.values("k", bad[b], 64),
                                             np.nan_to_num(plain.values("v", bad[b], 64)), 0.125, 61, True)
        assert (np.abs(to_f64(o)[b] - want) <= tol).all() and (np.abs(to_f64(lse)[b] - want_l) <= tol_l).all()
    before = cache.k.view(torch.uint8).clone()
    x = rows((2, 1, 64, 64), 103).cuda()
    cache.write(x, x)
    with pytest.raises(native.AttnError):
        native.attn_sync_status()
    changed = (cache.k.view(torch.uint8) != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert set(changed) <= {p for r in bad for p in r if 0 <= p < cache.k.shape[0]}
    k, _ = cache.read(64)
    with pytest.raises(native.AttnError):
        native.attn_sync_status()
    assert (k[0, :, 16:32] == 0).all() and (k[1, :, 32:48] == 0).all()
    # lengths outside the cache are taken as the nearer bound
    cache.block_table.copy_(torch.tensor(table, dtype=torch.int32))
    set_lens(cache, [64, 64])
    want = cache.attention(q.cuda())[0][0]
    set_lens(cache, [10 ** 9, -5])
    o, lse = cache.attention(q.cuda())
    with pytest.raises(native.AttnError):
        native.attn_sync_status()
    assert torch.equal(o[0], want) and (o[1] == 0).all() and torch.isneginf(lse[1]).all()
    cache.attention(q.cuda(), q_lens=ints([99, -3]))
    with pytest.raises(native.AttnError):
        native.attn_sync_status()


def test_prompt_then_tokens_against_the_forward():
    """As a program uses them together: a prompt's K and V enter the cache after attn_fwd, tokens
    follow one by one, and every step's attention equals attn_fwd over the values read back."""
    from causal_scaled_dot_gb300 import native
    from causal_scaled_dot_gb300.kv_cache import KVCache
    B, Hq, Hkv, D, prompt, steps = 2, 8, 2, 128, 200, 6
    cache = KVCache.empty(B, Hkv, D, 256, block_size=32)
    q, k, v = rows((B, Hq, prompt + steps, D), 1).cuda(), rows((B, Hkv, prompt + steps, D), 2).cuda(), \
        rows((B, Hkv, prompt + steps, D), 3).cuda()
    native.attention(q[:, :, :prompt].contiguous(), k[:, :, :prompt].contiguous(), v[:, :, :prompt].contiguous())
    cache.seq_lens.add_(prompt)
    cache.write(k[:, :, :prompt], v[:, :, :prompt])
    for t in range(prompt, prompt + steps):
        cache.seq_lens.add_(1)
        cache.write(k[:, :, t:t + 1], v[:, :, t:t + 1])
        o, lse = cache.attention(q[:, :, t:t + 1], check_status=True)
        kb, vb = cache.read(t + 1)
        want, want_l = native.attention(q[:, :, :t + 1].contiguous(), kb, vb)
        # both round weights and output to 8 bits: at most 2^-8 of the weights' share each, twice, and O twice
        assert (o[:, :, 0].float() - want[:, :, t].float()).abs().max() <= 4 * 2.0 ** -8 * vb.abs().max().float()
        assert (lse[:, :, 0] - want_l[:, :, t]).abs().max() <= 1e-3
    # the prompt's last rows again, as one chunk over the cache
    n = 50
    cache.seq_lens.fill_(prompt)
    o, _ = cache.attention(q[:, :, prompt - n:prompt])
    kb, vb = cache.read(prompt)
    want, _ = native.attention(q[:, :, :prompt].contiguous(), kb, vb)
    assert (o.float() - want[:, :, prompt - n:].float()).abs().max() <= 4 * 2.0 ** -8 * vb.abs().max().float()


def test_captured_graph_replays_with_new_lengths_and_data():
    """Lengths, tables and data live on the device: a captured step replays on whatever they hold
    then; two graphs replayed at once each have their own workspace."""
    B, Hq, Hkv, D = 2, 8, 2, 128
    cache, table = make(B, Hkv, D, 64, 3000, seed=16)
    fill(cache, table, [2000, 900], seed=111)
    q, k, v = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((B, Hq, 1, D), (B, Hkv, 1, D), (B, Hkv, 1, D)))
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            cache.attention(q)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            if not graphs:
                cache.write(k, v)
            outs.append(cache.attention(q))
        graphs.append(g)
    for step, lens in enumerate(([2001, 901], [2500, 1], [3000, 129])):
        q.copy_(rows(q.shape, 112 + step)), k.copy_(rows(k.shape, 122 + step)), v.copy_(rows(v.shape, 132 + step))
        plain_lens = [t - 1 for t in lens]
        fill(cache, table, plain_lens, seed=140 + step)
        set_lens(cache, lens)
        torch.cuda.synchronize()
        graphs[0].replay()  # writes the token and attends
        torch.cuda.synchronize()
        for _ in range(5):
            for g, s in zip(graphs[1:] + graphs[1:], streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        want = cache.attention(q, check_status=True)
        for o in outs:
            assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])


def test_results_do_not_depend_on_stream_or_repetition():
    cache, table = make(3, 2, 128, 32, 1500, seed=17)
    fill(cache, table, [1500, 3, 700], seed=151)
    q = rows((3, 8, 4, 128), 152).cuda()
    want = cache.attention(q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream, None):
        got = cache.attention(q, stream=stream, check_status=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(cache.attention(q, return_lse=False), want[0])


def test_workspace_contents_do_not_matter():
    """One workspace for calls of different shapes, full of whatever was there: zeros, ones, random
    bytes, the last call's partial results."""
    import ctypes
    from causal_scaled_dot_gb300 import native
    cache, table = make(2, 2, 64, 64, 5000, seed=18)
    fill(cache, table, [5000, 800], seed=161)
    lib, n = native.load(), ctypes.c_ulonglong(0)
    st = torch.cuda.current_stream().cuda_stream
    sizes = [(2, 1), (4, 7), (16, 4), (2, 90)]
    need = 0
    for Hq, Sq in sizes:
        assert lib.attn_cache_workspace(ctypes.byref(cache._c), Hq, Sq, ctypes.byref(n)) == 0
        need = max(need, n.value)
    work = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for round_, content in enumerate((0, 255, None, "random", "random", None)):
        for Hq, Sq in sizes:
            q = rows((2, Hq, Sq, 64), 162 + round_).cuda()
            if content == "random":
                work.random_(0, 256)
            elif content is not None:
                work.fill_(content)
            want = cache.attention(q)
            o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
            assert lib.attn_cache_fwd(ctypes.byref(cache._c), q.data_ptr(), None, o.data_ptr(), lse.data_ptr(), None, Hq, Sq,
                                      0.125, 1, work.data_ptr(), need, st) == 0
            native.attn_sync_status()
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_offsets_past_32_bits():
    """Blocks on both sides of 2^32 bytes of codes, and the cache's last one."""
    Hkv, block, D = 8, 128, 128
    total = 2 ** 32 // (Hkv * block * D) + 5
    code = lambda: torch.empty((total, Hkv, block, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)  # noqa: E731
    scale = lambda: torch.empty((total, Hkv), device="cuda")  # noqa: E731
    table = [[total - 1, 0, total - 5], [1, total - 3, total - 2]]
    cache = KVCache(code(), code(), scale(), scale(), ints(table), ints([0, 0]))
    small = [[0, 1, 2], [3, 4, 5]]  # the plain cache's own numbers for the same blocks
    lens, plain = [300, 384], PlainCache(6, Hkv, block, D)
    k, v = rows((2, Hkv, 384, D), 5), rows((2, Hkv, 384, D), 6)
    set_lens(cache, lens)
    cache.write(k.cuda(), v.cuda(), new_lens=ints(lens), check_status=True)
    plain.write(to_f64(k), to_f64(v), small, lens, lens)
    got_k, got_v = cache.read(384)
    for b, t in enumerate(lens):
        assert np.array_equal(to_f64(got_k)[b, :, :t], to_f64(torch.from_numpy(plain.values("k", small[b], t)).bfloat16()))
        assert np.array_equal(to_f64(got_v)[b, :, :t], to_f64(torch.from_numpy(plain.values("v", small[b], t)).bfloat16()))
    for Sq in (1, 20):
        check_attention(cache, plain, small, lens, 16, Sq)


@pytest.mark.parametrize("Hq,Sq", [(2, 1), (6, 3), (2, 70)])
def test_attention_takes_any_positive_scale(Hq, Sq):
    """Scales that no write makes: not powers of two, far apart between blocks and heads."""
    lens = [700, 33]
    cache, table = make(2, 2, 128, 32, 700, seed=13)
    plain = fill(cache, table, lens, seed=81)
    g = torch.Generator().manual_seed(3)
    for name, spread in (("k_scale", 0.3), ("v_scale", 6.0)):
        by = torch.exp(torch.randn(cache.k_scale.shape, generator=g) * spread).float()
        getattr(cache, name).mul_(by.cuda())
        setattr(plain, name, np.where(np.isfinite(to_f64(getattr(cache, name))), to_f64(getattr(cache, name)), 1.0))
    check_attention(cache, plain, table, lens, Hq, Sq)


@pytest.mark.parametrize("Hq,Sq", [(2, 1), (2, 40)])
@pytest.mark.parametrize("zero", ["some", "all"])
def test_attention_over_blocks_of_zeros(Hq, Sq, zero):
    """Blocks whose values are all zero have the smallest scale; their keys count all the same."""
    lens = [600, 90]
    cache, table = make(2, 2, 64, 16, 600, seed=14)
    plain = PlainCache(cache.k.shape[0], 2, 16, 64)
    k, v = rows((2, 2, 600, 64), 91), rows((2, 2, 600, 64), 92)
    v[:, :, 64:330] = 0
    if zero == "all":
        v.zero_()
    set_lens(cache, lens)
    cache.write(k.cuda(), v.cuda(), new_lens=ints(lens))
    plain.write(to_f64(k), to_f64(v), table, lens, lens)
    check_attention(cache, plain, table, lens, Hq, Sq)


def test_calls_on_two_streams_at_once():
    """Two caches, each on its own stream with its own workspace, run side by side as they run alone."""
    made, want = [], []
    for i, (lens, Hq, Sq) in enumerate((([9000, 200], 8, 1), ([5000, 4000], 4, 64))):
        cache, table = make(2, 2, 128, 64, max(lens), seed=15 + i)
        fill(cache, table, lens, seed=95 + i)
        q = rows((2, Hq, Sq, 128), 96 + i).cuda()
        made.append((cache, q, torch.cuda.Stream()))
        want.append(cache.attention(q))
    torch.cuda.synchronize()
    for _ in range(20):
        got = [cache.attention(q, stream=stream) for cache, q, stream in made]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_among_copies_and_on_a_side_stream():
    """A graph of copies, clears and cache calls in turn, with a read on a side stream, gives what the calls give one by one."""
    B, Hq, Hkv, D, n = 3, 8, 2, 128, 4
    cache, _ = make(B, Hkv, D, 32, 2000, seed=21)
    fill(cache, cache.block_table.tolist(), [1500, 700, 40], seed=201)
    src = [rows((B, h, n, D), 210 + i).cuda() for i, h in enumerate((Hkv, Hkv, Hq))]
    k, v, q = (torch.empty_like(x) for x in src)
    out = torch.empty_like(q)
    kept, lse = torch.empty_like(q), torch.empty((B, Hq, n), device="cuda")
    back = [torch.zeros((B, Hkv, 300, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    start = cache.seq_lens.clone()

    def step(side):
        cache.seq_lens.copy_(start)
        cache.seq_lens.add_(n)
        for to, x in zip((k, v, q), src):
            to.copy_(x)
        out.zero_()
        cache.write(k, v)
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            for x in back:
                x.zero_()
            cache.read(300, 450, *back)
        cache.attention(q, out=out, lse=lse)
        kept.copy_(out)
        here.wait_stream(side)

    side = torch.cuda.Stream()
    step(side)
    torch.cuda.synchronize()
    want = [x.clone() for x in (kept, lse, *back)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(side)
    for i in range(6):
        for x in (kept, lse, *back):
            x.fill_(3)
        src[2].add_(0)  # a kernel right before the replay
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((kept, lse, *back), want):
            assert torch.equal(a, b), i
