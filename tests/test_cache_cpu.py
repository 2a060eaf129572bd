"""The cache entry points' refusals, the checked index arithmetic, and the definitions
that the GPU tests compare with.  No GPU."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from causal_scaled_dot_gb300 import native
from causal_scaled_dot_gb300.native import ATTN_ERR_INVALID_ARG, ATTN_ERR_MISALIGNED, ATTN_ERR_UNSUPPORTED
from tests.cache_util import codes_of, scale_of

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
T = 1 << 40  # fake, never-dereferenced addresses, 2^40 bytes apart


def cache(**kw):
    a = dict(k=T, v=2 * T, k_scale=3 * T, v_scale=4 * T, block_table=5 * T, seq_lens=6 * T, num_blocks=100, block_size=64,
             max_blocks=20, B=2, Hkv=2, D=128)  # 1280 tokens: the attention needs a workspace
    a.update(kw)
    return native.AttnCache(*(a[n] for n, _ in native.AttnCache._fields_))


def strides(s):
    return None if s is None else (ctypes.c_longlong * 3)(*s)


def call_write(c=None, k=7 * T, v=8 * T, ks=None, vs=None, new_lens=None, S=4):
    return native.load().attn_cache_write(c, k, strides(ks), v, strides(vs), new_lens, S, None)


def call_read(c=None, k=7 * T, v=8 * T, first=0, S=4):
    return native.load().attn_cache_read(c, k, v, first, S, None)


def call_fwd(c=None, q=7 * T, qs=None, out=8 * T, lse=9 * T, q_lens=None, Hq=4, Sq=3, scale=0.1, ws=10 * T, wb=1 << 30):
    return native.load().attn_cache_fwd(c, q, strides(qs), out, lse, q_lens, Hq, Sq, scale, 1, ws, wb, None)


BAD_CACHES = [
    (dict(k=None), ATTN_ERR_INVALID_ARG), (dict(v_scale=None), ATTN_ERR_INVALID_ARG),
    (dict(block_table=None), ATTN_ERR_INVALID_ARG), (dict(seq_lens=None), ATTN_ERR_INVALID_ARG),
    (dict(num_blocks=0), ATTN_ERR_INVALID_ARG), (dict(max_blocks=0), ATTN_ERR_INVALID_ARG),
    (dict(B=0), ATTN_ERR_INVALID_ARG), (dict(Hkv=-1), ATTN_ERR_INVALID_ARG),
    (dict(D=96), ATTN_ERR_UNSUPPORTED), (dict(block_size=48), ATTN_ERR_UNSUPPORTED),
    (dict(block_size=256), ATTN_ERR_UNSUPPORTED), (dict(max_blocks=1 << 24), ATTN_ERR_UNSUPPORTED),
    (dict(num_blocks=(1 << 30)), ATTN_ERR_UNSUPPORTED), (dict(k=T + 8), ATTN_ERR_MISALIGNED),
    (dict(k_scale=3 * T + 2), ATTN_ERR_MISALIGNED), (dict(seq_lens=6 * T + 1), ATTN_ERR_MISALIGNED),
]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
@pytest.mark.parametrize("call", [call_write, call_read, call_fwd])
def test_bad_caches_are_refused(call, kw, code):
    assert call(cache(**kw)) == code


@pytest.mark.parametrize("call", [call_write, call_read, call_fwd])
def test_null_cache_is_refused(call):
    assert call(None) == ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), ATTN_ERR_INVALID_ARG), (dict(v=None), ATTN_ERR_INVALID_ARG), (dict(S=0), ATTN_ERR_INVALID_ARG),
    (dict(k=7 * T + 8), ATTN_ERR_MISALIGNED), (dict(new_lens=11 * T + 2), ATTN_ERR_MISALIGNED),
    (dict(ks=(1024, -128, 128)), ATTN_ERR_INVALID_ARG), (dict(vs=(1024, 128, 132)), ATTN_ERR_MISALIGNED),
    (dict(ks=(1 << 50, 0, 0)), ATTN_ERR_UNSUPPORTED), (dict(S=(1 << 29) + 1), ATTN_ERR_UNSUPPORTED),
    (dict(k=T), ATTN_ERR_INVALID_ARG), (dict(v=2 * T + 1600), ATTN_ERR_INVALID_ARG),
    (dict(new_lens=4 * T), ATTN_ERR_INVALID_ARG),
    (dict(k=T - 4096, ks=(0, 0, 128), S=64), ATTN_ERR_INVALID_ARG),  # its last row lies in the cache
])
def test_write_refusals(kw, code):
    assert call_write(cache(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=None, v=None), ATTN_ERR_INVALID_ARG), (dict(S=0), ATTN_ERR_INVALID_ARG), (dict(first=-1), ATTN_ERR_INVALID_ARG),
    (dict(k=7 * T + 2), ATTN_ERR_MISALIGNED), (dict(v=7 * T + 1024), ATTN_ERR_INVALID_ARG),
    (dict(k=T + 1024), ATTN_ERR_INVALID_ARG), (dict(v=5 * T), ATTN_ERR_INVALID_ARG), (dict(v=6 * T), ATTN_ERR_INVALID_ARG),
    (dict(first=(1 << 29) + 1), ATTN_ERR_UNSUPPORTED),
])
def test_read_refusals(kw, code):
    assert call_read(cache(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), ATTN_ERR_INVALID_ARG), (dict(out=None), ATTN_ERR_INVALID_ARG), (dict(ws=None, wb=0), ATTN_ERR_INVALID_ARG),
    (dict(Hq=3), ATTN_ERR_INVALID_ARG), (dict(Hq=0), ATTN_ERR_INVALID_ARG), (dict(Sq=0), ATTN_ERR_INVALID_ARG),
    (dict(scale=0.0), ATTN_ERR_INVALID_ARG), (dict(scale=float("nan")), ATTN_ERR_INVALID_ARG),
    (dict(scale=-1.0), ATTN_ERR_INVALID_ARG), (dict(q=7 * T + 8), ATTN_ERR_MISALIGNED),
    (dict(lse=9 * T + 2), ATTN_ERR_MISALIGNED), (dict(qs=(0, 128, 4)), ATTN_ERR_MISALIGNED),
    (dict(out=7 * T), ATTN_ERR_INVALID_ARG), (dict(out=T), ATTN_ERR_INVALID_ARG), (dict(lse=8 * T), ATTN_ERR_INVALID_ARG),
    (dict(lse=6 * T), ATTN_ERR_INVALID_ARG), (dict(ws=8 * T), ATTN_ERR_INVALID_ARG),
    (dict(q_lens=9 * T), ATTN_ERR_INVALID_ARG), (dict(ws=7 * T), ATTN_ERR_INVALID_ARG),
    (dict(Hq=1 << 20, Sq=1 << 20), ATTN_ERR_UNSUPPORTED),
])
def test_attention_refusals(kw, code):
    assert call_fwd(cache(), **kw) == code


def test_workspace_refusals():
    n = ctypes.c_ulonglong(7)
    f = native.load().attn_cache_workspace
    assert f(cache(), 8, 1, None) == ATTN_ERR_INVALID_ARG
    assert f(None, 8, 1, ctypes.byref(n)) == ATTN_ERR_INVALID_ARG
    for bad in ((0, 1), (9, 1), (8, 0)):
        assert f(cache(), *bad, ctypes.byref(n)) == ATTN_ERR_INVALID_ARG
    assert f(cache(D=80), 8, 1, ctypes.byref(n)) == ATTN_ERR_UNSUPPORTED
    for blocks in (8, 16):  # up to 1024 tokens: no unit is split
        assert f(cache(max_blocks=blocks), 8, 1, ctypes.byref(n)) == 0 and n.value == 0


def test_status_string_of_a_bad_cache():
    assert native.attn_status_string(native.ATTN_ERR_BAD_CACHE).startswith("ATTN_ERR_BAD_CACHE")


def test_struct_layout_matches_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    names = [n for n, _ in native.AttnCache._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include "attn.h"\n#include <stddef.h>\n#include <stdio.h>\nint main(void) {\n' + "".join(
        f'printf("%zu ", offsetof(attn_cache_t, {n}));\n' for n in names) + 'printf("%zu", sizeof(attn_cache_t)); return 0; }\n')
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(tmp_path / "layout"), str(src)], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True).stdout.split()]
    assert got == [getattr(native.AttnCache, n).offset for n in names] + [ctypes.sizeof(native.AttnCache)]


def test_host_tensors_are_refused():
    from causal_scaled_dot_gb300.kv_cache import KVCache
    with pytest.raises(ValueError, match="CUDA"):
        KVCache.empty(1, 1, 64, 100, device="cpu")
    code = torch.zeros(4, 1, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        KVCache(code, code, code, code, code, code)


class _Fake:
    """A CUDA tensor's description without one."""

    def __init__(self, shape, dtype, index=0, contiguous=True):
        self.shape, self.dtype, self.is_cuda, self.device = torch.Size(shape), dtype, True, torch.device("cuda", index)
        self.contiguous_ = contiguous

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return self.contiguous_

    def data_ptr(self):
        return 1 << 40


def _fake_cache(**kw):
    from causal_scaled_dot_gb300.kv_cache import KVCache
    t = dict(k=_Fake((9, 2, 16, 64), torch.float8_e4m3fn), v=_Fake((9, 2, 16, 64), torch.float8_e4m3fn),
             k_scale=_Fake((9, 2), torch.float32), v_scale=_Fake((9, 2), torch.float32),
             block_table=_Fake((3, 4), torch.int32), seq_lens=_Fake((3,), torch.int32))
    t.update(kw)
    return KVCache(**t)


@pytest.mark.parametrize("kw", [
    dict(k=_Fake((9, 2, 16, 64), torch.uint8)), dict(v=_Fake((9, 2, 16, 128), torch.float8_e4m3fn)),
    dict(k_scale=_Fake((9, 3), torch.float32)), dict(block_table=_Fake((3, 4), torch.int64)),
    dict(block_table=_Fake((3,), torch.int32)), dict(seq_lens=_Fake((4,), torch.int32)),
    dict(seq_lens=_Fake((3,), torch.int32, index=1)), dict(k=_Fake((9, 2, 16, 64), torch.float8_e4m3fn, contiguous=False)),
    dict(k=_Fake((9, 2, 24, 64), torch.float8_e4m3fn), v=_Fake((9, 2, 24, 64), torch.float8_e4m3fn)),
    dict(k=_Fake((9, 2, 64), torch.float8_e4m3fn)), dict(block_table=_Fake((3, 0), torch.int32)),
])
def test_cache_tensors_are_checked(kw):
    with pytest.raises(ValueError):
        _fake_cache(**kw)


def test_call_tensors_are_checked():
    c = _fake_cache()
    assert c.capacity == 64
    bf = torch.bfloat16
    good = _Fake((3, 2, 5, 64), bf)
    good.requires_grad = False
    for bad in (_Fake((3, 2, 5, 64), torch.float16), _Fake((3, 2, 5, 64), bf, index=1), _Fake((2, 2, 5, 64), bf),
                _Fake((3, 1, 5, 64), bf), _Fake((3, 2, 5, 128), bf), _Fake((3, 2, 64), bf)):
        with pytest.raises(ValueError):
            c.write(bad, good)
        with pytest.raises(ValueError):
            c.write(good, bad)
    other = _Fake((3, 2, 6, 64), bf)
    other.requires_grad = False
    with pytest.raises(ValueError):
        c.write(good, other)
    for n in (_Fake((3,), torch.int64), _Fake((2,), torch.int32), _Fake((3,), torch.int32, index=1)):
        with pytest.raises(ValueError, match="new_lens"):
            c.write(good, good, new_lens=n)
    odd = _Fake((3, 3, 5, 64), bf)
    odd.requires_grad = False
    with pytest.raises(ValueError, match="heads"):
        c.attention(odd)
    with pytest.raises(ValueError, match="out"):
        c.attention(good, out=_Fake((3, 2, 4, 64), bf))
    with pytest.raises(ValueError, match="lse"):
        c.attention(good, lse=_Fake((3, 2, 5), torch.float64))
    grad = _Fake((3, 2, 5, 64), bf)
    grad.requires_grad = True
    with pytest.raises(ValueError, match="gradient"):
        c.attention(grad)
    for kw in (dict(S=0), dict(S=4, first=-1), dict(S=4, k_out=_Fake((3, 2, 5, 64), bf))):
        with pytest.raises(ValueError):
            c.read(**kw)


def test_the_definition_rounds_as_the_type_does():
    x = np.concatenate([np.linspace(-448, 448, 4001), np.geomspace(1e-4, 448, 4001), [0.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    want = torch.tensor(x, dtype=torch.float32).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes_of(x.astype(np.float32).astype(np.float64)), want)
    for big, s in ((448.0, 1.0), (449.0, 2.0), (224.0, 0.5), (225.0, 1.0), (0.0, 2.0 ** -126), (3e-38, 2.0 ** -126), (1.75, 2.0 ** -8),
                   (1.76, 2.0 ** -7)):
        assert scale_of(np.array([big, -big / 2])) == s, big


PROGRAM = r"""
#include "cache_index.h"
#include <cstdio>
#include <initializer_list>
using namespace attn;
#define CHECK(c) do { if (!(c)) { std::printf("FAIL line %d: %s\n", __LINE__, #c); return 1; } } while (0)
int main() {
    const int big = 2147483647;
    for (int entry : {-big - 1, -1, 0, 6, 7, big}) {
        bool bad = false;
        const int b = cache_block(entry, 7, &bad);
        CHECK(bad == (entry < 0 || entry >= 7) && b == (bad ? -1 : entry));
    }
    for (int len : {-big - 1, -1, 0, 5, 64, 65, big})
        for (int count : {-big - 1, -1, 0, 3, 9, 10, big}) {
            bool bad = false;
            const CacheSpan s = cache_span(len, count, 64, 9, &bad);
            CHECK(s.len >= 0 && s.len <= 64 && s.count >= 0 && s.count <= 9 && s.first == s.len - s.count);
            CHECK(bad == (len < 0 || len > 64 || count < 0 || count > 9));
        }
    CHECK(cache_offset(1 << 20, 3, 5, 8, 128, 128) == (((1ull << 20) * 8 + 3) * 128 + 5) * 128);  // past 32 bits
    std::printf("OK\n");
    return 0;
}
"""


def test_checked_index_arithmetic(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    src = tmp_path / "index.cpp"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(ROOT, "causal_scaled_dot_gb300", "csrc"), "-o",
                    str(tmp_path / "index"), str(src)], check=True)
    res = subprocess.run([str(tmp_path / "index")], capture_output=True, text=True)
    assert res.returncode == 0 and res.stdout.startswith("OK"), res.stdout


PLAN_PROGRAM = r"""
#include "cache_index.h"
#include <cstdio>
#include <cstdlib>
#include <vector>
using namespace attn;
#define CHECK(c) do { if (!(c)) { std::printf("FAIL line %d: %s\n", __LINE__, #c); return 1; } } while (0)
// Every unit's tiles are taken exactly once and in order, for each count of CTAs, with the plan summed
// by `threads` threads in chunks as the kernel does it.
int main() {
    for (int total : {1, 303, 304, 70000, 0x7ffffffe, 0x7fffffff})
        for (int ctas : {1, 152, 304, 32767})
            for (int c = 0; c <= ctas; ++c) {
                const int t = plan_begin(total, c, ctas);
                CHECK(t == (int)((long long)total * c / ctas));
                if (ctas <= total && c < ctas) CHECK(plan_cta(total, t, ctas) == c);
                if (ctas <= total && c > 0) CHECK(plan_cta(total, t - 1, ctas) == c - 1);
            }
    std::srand(7);
    for (int round = 0; round < 400; ++round) {
        CachePlan p{};
        p.B = 1 + std::rand() % 9;
        p.Sq = 1 + std::rand() % 40;
        p.capacity = 128 * (1 + std::rand() % 8);
        p.causal = std::rand() % 2;
        p.qper = 1 + std::rand() % 16;
        p.q_tiles = (p.Sq + p.qper - 1) / p.qper;
        p.heads = 1 + std::rand() % 5;
        p.whole = std::rand() % 2 ? 0 : std::rand() % 3;
        p.least = 1 + std::rand() % 6;
        p.start = p.whole == 1 ? 0 : std::rand() % 4;
        std::vector<int> lens(p.B), counts(p.B);
        for (int b = 0; b < p.B; ++b) {
            lens[b] = std::rand() % 5 == 0 ? 0 : std::rand() % (p.capacity + 1);
            if (std::rand() % 9 == 0) lens[b] = -3;
            if (std::rand() % 9 == 0) lens[b] = 2147483647;
            counts[b] = std::rand() % (p.Sq + 1);
        }
        p.seq_lens = lens.data();
        p.q_lens = std::rand() % 3 ? counts.data() : nullptr;
        // the units, written down one by one
        struct U { int b, qt, h, tiles, keys, at; };
        std::vector<U> want;
        int total = 0;
        for (int b = 0; b < p.B; ++b) {
            const int len = lens[b] < 0 ? 0 : lens[b] > p.capacity ? p.capacity : lens[b];
            const int count = p.q_lens ? counts[b] : p.Sq;
            for (int qt = 0; qt * p.qper < count; ++qt) {
                const int last = (qt + 1) * p.qper < count ? (qt + 1) * p.qper : count;
                int keys = p.causal ? len - count + last : len;
                if (keys < 0) keys = 0;
                const int tiles = keys <= 128 ? 1 : (keys + 127) / 128;
                for (int h = 0; h < p.heads; ++h) {
                    want.push_back({b, qt, h, tiles, keys, total + p.start});
                    total += p.whole == 1 ? 1 : p.start + tiles;
                }
            }
        }
        const int pairs = p.B * p.q_tiles, threads = 1 + std::rand() % 20, per = (pairs + threads - 1) / threads;
        std::vector<int> sum(threads);
        int all = 0;
        bool bad = false;
        for (int t = 0; t < threads; ++t) {
            const int a = t * per < pairs ? t * per : pairs, z = a + per < pairs ? a + per : pairs;
            all += sum[t] = plan_chunk(p, a, z, &bad);
        }
        CHECK(all == total);
        const int given = 1 + std::rand() % 70, ctas = plan_ctas(p, total, given);
        size_t unit = 0;
        int tile = 0, pieces = 0, expect_first = -1, expect_last = -1;
        for (int c = 0; c < given; ++c) {
            const int begin = plan_begin(total, c, ctas), end = plan_begin(total, c + 1, ctas);
            CHECK((begin == end) == (c >= ctas));  // no CTA without a place among those that share them
            if (begin == end) continue;
            int before = 0;
            int t = 0;
            while (begin >= before + sum[t]) before += sum[t++];
            CacheCursor cur = cursor_at(p, plan_find(p, t * per, begin - before), begin, end - begin);
            CacheUnit u;
            int seen = begin;  // places up to the last tile taken
            while (cursor_next(p, cur, u)) {
                CHECK(unit < want.size());
                const U& w = want[unit];
                CHECK(u.b == w.b && u.qt == w.qt && u.h == w.h && u.tiles == w.tiles && u.keys == w.keys && u.t == tile && u.n > 0);
                CHECK(u.at == w.at);
                if (!p.whole) CHECK(u.at + u.t >= seen && u.at + u.t + u.n <= end && (u.t == 0 || u.at + u.t == begin));
                if (p.whole) CHECK(u.at - p.start >= begin && u.at - p.start < end);
                seen = p.whole == 1 ? u.at + 1 : u.at + u.t + u.n;
                CHECK(u.t + u.n <= u.tiles);
                tile += u.n;
                ++pieces;
                if (pieces == 1 && tile < u.tiles) {
                    CHECK(!p.whole);
                    expect_first = c;
                    expect_last = plan_cta(total, u.at + u.tiles - 1, ctas);
                }
                if (pieces > 1) CHECK(plan_cta(total, u.at, ctas) == expect_first);  // every piece finds the first
                if (tile == u.tiles) {
                    CHECK(pieces == 1 || (expect_last == c && pieces == expect_last - expect_first + 1));
                    tile = pieces = 0;
                    ++unit;
                }
            }
            if (!p.whole) CHECK(end - seen <= p.start);
        }
        CHECK(unit == want.size() && tile == 0);
    }
    std::printf("OK\n");
    return 0;
}
"""


def test_attention_work_is_split_exactly(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    src = tmp_path / "plan.cpp"
    src.write_text(PLAN_PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=address,undefined", "-I",
                    os.path.join(ROOT, "causal_scaled_dot_gb300", "csrc"), "-o", str(tmp_path / "plan"), str(src)], check=True)
    res = subprocess.run([str(tmp_path / "plan")], capture_output=True, text=True)
    assert res.returncode == 0 and res.stdout.startswith("OK"), res.stdout + res.stderr
