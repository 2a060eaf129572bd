"""The 8-bit cache's attention where many small weights add up, where scores or V's scales are far
apart, and where a row is not finite: against float64 on the same codes."""
import math

import numpy as np
import pytest
import torch

from causal_scaled_dot_gb300.kv_cache import KVCache
from tests.cache_util import PlainCache, attention, make, rows, to_f64

pytestmark = pytest.mark.gpu

LN2 = math.log(2.0)
# Query heads and queries over one key/value head: 1, 4, 8 | 16 | 20, 32 rows of the forms for few
# rows, and 40, 128 of the form for many.
SHAPES = [(1, 1), (4, 1), (8, 1), (16, 1), (4, 5), (32, 1), (8, 5), (128, 1)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def one_channel(scores, values, D, block=64, sequences=1):
    """A cache of one key/value head whose key j has `scores[j]` in channel 0 and `values[j]` in every
    channel of V, for `sequences` sequences over the same blocks, and its values in float64.  Many
    sequences make a thread block's share of one of them long."""
    n = len(scores)
    one, table = make(1, 1, D, block, n, seed=3)
    k, v = np.zeros((1, 1, n, D)), np.zeros((1, 1, n, D))
    k[0, 0, :, 0] = scores
    v[0, 0] = np.asarray(values)[:, None]
    k, v = (torch.tensor(x, dtype=torch.bfloat16) for x in (k, v))
    one.seq_lens.fill_(n)
    one.write(k.cuda(), v.cuda(), check_status=True)
    plain = PlainCache(one.k.shape[0], 1, block, D)
    plain.write(to_f64(k), to_f64(v), table, [n], [n])
    cache = KVCache(one.k, one.v, one.k_scale, one.v_scale, one.block_table.repeat(sequences, 1), one.seq_lens.repeat(sequences))
    return cache, plain.values("k", table[0], n)[0, :, 0], plain.values("v", table[0], n)[0, :, 0]


def ask(cache, Hq, Sq):
    """O and LSE for queries that take a key's channel 0 as its score in powers of two."""
    B, _, D = cache._sizes
    q = torch.zeros(B, Hq, Sq, D, dtype=torch.bfloat16)
    q[..., 0] = 1
    o, lse = cache.attention(q.cuda(), scale=LN2, causal=False, check_status=True)
    return to_f64(o), to_f64(lse)


def want(scores, values):
    top = scores.max()
    w = np.exp2(scores - top)
    return w @ values / w.sum(), (top + math.log2(w.sum())) * LN2


def lost(scores):
    """What weights that are too small add up to, at the most, as a share of the sum: 2^-7 of the largest
    weight among each 128 keys."""
    w = np.exp2(scores - scores.max())
    return 2.0 ** -7 * w.reshape(-1, 128).max(1).sum() / w.sum()


@pytest.mark.parametrize("Hq,Sq", SHAPES)
@pytest.mark.parametrize("near,every", [(10, None), (10, 128), (5, 64), (9, 64), (3, 64)])
@pytest.mark.parametrize("low", [0.0, -1.0, -3.0])
def test_small_weights_add_up(Hq, Sq, near, every, low):
    """One key 2^15 above the rest, some 2^-10 .. 2^-5 of it, and thousands that matter only together: with
    V = 1 the answer is 1, and with V = 1 for those thousands alone it is their share."""
    n = 42 * 128
    scores = np.full(n, low)
    scores[0] = 15
    if every is None:
        scores[[128 + 5, 9 * 128 + 7]] = near
    else:
        scores[3::every] = near
        scores[0] = 15
    for values in (np.ones(n), np.where(scores == low, 1.0, 0.0)):
        cache, s, v = one_channel(scores, values, 64, sequences=320)
        o, lse = ask(cache, Hq, Sq)
        ref, ref_lse = want(s, v)
        # the weights' rounding (2^-8 of each), O's (2^-9, as bf16), and what is lost
        assert np.abs(o - ref).max() <= (2.0 ** -8 + 2.0 ** -9) * ref + lost(s), (ref, o.min(), o.max())
        assert np.abs(lse - ref_lse).max() <= 2.0 ** -16 * abs(ref_lse)


@pytest.mark.parametrize("Hq,Sq", SHAPES)
@pytest.mark.parametrize("n", [200, 257, 384, 130])
def test_keys_of_the_last_tile_keep_their_weights(Hq, Sq, n):
    """A first key 2^22 above the rest, with V = 1 from the second tile of 128 on alone: what is left of that tile is
    a tile whose weights are measured against its own largest, also where it is the last and cut short."""
    scores, values = np.zeros(n), np.ones(n)
    scores[0], values[:128] = 22, 0
    for sequences in (1, 320):
        cache, s, v = one_channel(scores, values, 64, sequences=sequences)
        o, _ = ask(cache, Hq, Sq)
        ref = want(s, v)[0]
        assert np.abs(o / ref - 1).max() <= 2.0 ** -8 + 2.0 ** -9 + 2.0 ** -7


@pytest.mark.parametrize("Hq,Sq", SHAPES)
def test_normal_tails_add_up(Hq, Sq):
    """Scores of deviation 2 nats under one key 10 nats above: O of V = 1 stays 1."""
    rng = np.random.default_rng(5)
    n = 8192
    for _ in range(3):
        scores = rng.standard_normal(n) * 2 / LN2
        scores[0] = 10 / LN2
        cache, s, v = one_channel(scores, np.ones(n), 128, sequences=160)
        o, lse = ask(cache, Hq, Sq)
        ref, ref_lse = want(s, v)
        assert np.abs(o - 1).max() <= 2.0 ** -8 + 2.0 ** -9 + lost(s)
        assert np.abs(lse - ref_lse).max() <= 2.0 ** -16 * abs(ref_lse)


@pytest.mark.parametrize("Hq,Sq", SHAPES)
@pytest.mark.parametrize("jump", [30, 44, 56, 80, 96, 120])
@pytest.mark.parametrize("tile", [0, 4, 20])
def test_a_jump_of_the_scores_over_values_of_zero(Hq, Sq, jump, tile):
    """V of zeros has the smallest scale, whose inverse a key's weight is multiplied by for the sum: a key
    far above the ones before it leaves O = 0 and LSE its score."""
    n = 30 * 128
    scores = np.zeros(n)
    scores[tile * 128 + 17] = jump
    cache, s, v = one_channel(scores, np.zeros(n), 64, sequences=320)
    o, lse = ask(cache, Hq, Sq)
    assert (o == 0).all()
    assert np.abs(lse - want(s, v)[1]).max() <= 2.0 ** -16 * jump


@pytest.mark.parametrize("Hq,Sq", SHAPES)
@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 24, 2.0 ** 28])
def test_values_of_zero_before_large_ones(Hq, Sq, size):
    """Keys whose V is zero keep their share of the sum beside keys whose V is large."""
    n = 20 * 128
    values = np.zeros(n)
    values[12 * 128:] = size
    cache, s, v = one_channel(np.zeros(n), values, 64, sequences=320)
    o, lse = ask(cache, Hq, Sq)
    ref, ref_lse = want(s, v)
    assert np.abs(o / ref - 1).max() <= 2.0 ** -8 + 2.0 ** -9
    assert np.abs(lse - ref_lse).max() <= 2.0 ** -16 * abs(ref_lse)


@pytest.mark.parametrize("Hq,Sq", [(2, 1), (6, 3), (4, 16), (2, 70)])
def test_large_keys_and_a_small_scale(Hq, Sq):
    """Scores are moderate though K alone is near the type's largest value."""
    B, Hkv, D, block, t = 1, 2, 128, 32, 700
    cache, table = make(B, Hkv, D, block, t, seed=12)
    k, v = (rows((B, Hkv, t, D), 71).double() * 2.0 ** 114).bfloat16(), rows((B, Hkv, t, D), 72)
    q = (rows((B, Hq, Sq, D), 73).double() * 2.0 ** -100).bfloat16()
    plain = PlainCache(cache.k.shape[0], Hkv, block, D)
    cache.seq_lens.fill_(t)
    cache.write(k.cuda(), v.cuda(), check_status=True)
    plain.write(to_f64(k), to_f64(v), table, [t], [t])
    scale = 2.0 ** -14 / math.sqrt(D)
    o, lse = cache.attention(q.cuda(), scale=scale, check_status=True)
    ref, ref_l, tol, tol_l = attention(to_f64(q)[0], plain.values("k", table[0], t), plain.values("v", table[0], t), scale, t - Sq,
                                       True)
    assert (np.abs(to_f64(o)[0] - ref) <= tol).all() and (np.abs(to_f64(lse)[0] - ref_l) <= tol_l).all()


@pytest.mark.parametrize("Hq,Sq", [(8, 9), (4, 40), (130, 1), (2, 200)])
def test_non_finite_queries_stay_in_their_row_of_many(Hq, Sq):
    cache, table = make(1, 1, 128, 64, 1900, seed=14)
    n = 1900
    k, v = rows((1, 1, n, 128), 91), rows((1, 1, n, 128), 92)
    cache.seq_lens.fill_(n)
    cache.write(k.cuda(), v.cuda())
    q = rows((1, Hq, Sq, 128), 93)
    clean, clean_lse = cache.attention(q.cuda())
    bad = torch.zeros(Hq, Sq, dtype=torch.bool)
    for h, i, d, x in ((0, 0, 7, float("nan")), (Hq - 1, Sq - 1, 3, float("inf")), (1, Sq // 2, 127, float("-inf"))):
        q[0, h, i, d] = x
        bad[h, i] = True
    o, lse = cache.attention(q.cuda(), check_status=True)
    assert o[0, bad].isnan().all() and lse[0, bad].isnan().all()
    # a row's maximum may move with its neighbours', so its weights may be rounded at another place
    assert (o[0, ~bad].float() - clean[0, ~bad].float()).abs().max() <= 2.0 ** -7 * v.abs().max()
    assert (lse[0, ~bad] - clean_lse[0, ~bad]).abs().max() <= 2.0 ** -16 * clean_lse[0, ~bad].abs().max()
