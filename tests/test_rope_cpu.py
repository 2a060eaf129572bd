"""Rotary positions without a GPU: refusals of the entry points and of the Python calls, the layout of the structs, the
split of the work, frequencies, and the definitions that the GPU tests compare with."""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from causal_scaled_dot_gb300 import native
from causal_scaled_dot_gb300.native import ATTN_ERR_INVALID_ARG, ATTN_ERR_MISALIGNED, ATTN_ERR_UNSUPPORTED, AttnHeads, AttnRope
from causal_scaled_dot_gb300.rotary import Rotary
from tests import rope_util

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
T = 1 << 40  # fake, never-dereferenced addresses, 2^40 bytes apart
B, HQ, HKV, S, D = 2, 4, 2, 10, 128


def rope(**kw):
    r = AttnRope.from_buffer_copy(Rotary.from_base(128)._c)
    r.eps = 1e-6
    for n, v in kw.items():
        setattr(r, n, v)
    return r


def dense(q=None, k=None, v=None, Hq=HQ, Hkv=HKV, **kw):
    st = lambda H: (ctypes.c_longlong * 3)(H * S * D, S * D, D)  # noqa: E731
    h = AttnHeads(q, k, v, st(Hq), st(Hkv), st(Hkv))
    for n, v in kw.items():
        setattr(h, n, (ctypes.c_longlong * 3)(*v))
    return h


def packed(at, q=True, k=True, v=True, W=(HQ + 2 * HKV) * D, shift=0):
    """Views of a projection's output [B, S, W] at `at`."""
    st = (ctypes.c_longlong * 3)(S * W, D, W)
    p = [at, at + 2 * HQ * D + shift, at + 2 * (HQ + HKV) * D]
    return AttnHeads(*(x if on else None for x, on in zip(p, (q, k, v))), st, st, st)


def call_fwd(r="default", x="default", y="default", sizes=(B, HQ, HKV, S, D)):
    return native.load().attn_rope(rope() if r == "default" else r, packed(T) if x == "default" else x,
                                   dense(2 * T, 3 * T, 4 * T) if y == "default" else y, *sizes, None)


def call_bwd(r="default", up="default", x="default", y="default", dqw=None, dkw=None, sizes=(B, HQ, HKV, S, D), ws=None, wb=0):
    return native.load().attn_rope_bwd(rope() if r == "default" else r, dense(2 * T, 3 * T, 4 * T) if up == "default" else up,
                                       packed(T) if x == "default" else x, packed(5 * T) if y == "default" else y, dqw, dkw, *sizes, ws, wb,
                                       None)


BAD_SIZES = [((0, HQ, HKV, S, D), ATTN_ERR_INVALID_ARG), ((B, 0, HKV, S, D), ATTN_ERR_INVALID_ARG),
             ((B, HQ, -1, S, D), ATTN_ERR_INVALID_ARG), ((B, HQ, HKV, 0, D), ATTN_ERR_INVALID_ARG),
             ((B, HQ, HKV, S, 96), ATTN_ERR_UNSUPPORTED), ((1 << 16, HQ, HKV, 1 << 16, D), ATTN_ERR_UNSUPPORTED),
             ((B, (1 << 20) + 1, HKV, S, D), ATTN_ERR_UNSUPPORTED)]


@pytest.mark.parametrize("sizes,code", BAD_SIZES)
@pytest.mark.parametrize("call", [call_fwd, call_bwd])
def test_bad_sizes_are_refused(call, sizes, code):
    assert call(sizes=sizes) == code
    n = ctypes.c_ulonglong(0)
    assert native.load().attn_rope_workspace(rope(), *sizes, ctypes.byref(n)) == code


BAD_ROPES = [
    (dict(rotary_dim=-16), ATTN_ERR_INVALID_ARG), (dict(rotary_dim=144), ATTN_ERR_INVALID_ARG),
    (dict(rotary_dim=24), ATTN_ERR_UNSUPPORTED), (dict(rotary_dim=20, interleaved=1), ATTN_ERR_UNSUPPORTED),
    (dict(factor=float("nan")), ATTN_ERR_INVALID_ARG), (dict(factor=float("inf")), ATTN_ERR_INVALID_ARG),
    (dict(q_weight=8 * T, eps=0.0), ATTN_ERR_INVALID_ARG), (dict(k_weight=8 * T, eps=-1.0), ATTN_ERR_INVALID_ARG),
    (dict(q_weight=8 * T, eps=float("nan")), ATTN_ERR_INVALID_ARG), (dict(q_weight=8 * T, weight_format=2), ATTN_ERR_INVALID_ARG),
    (dict(q_weight=8 * T + 8), ATTN_ERR_MISALIGNED), (dict(k_weight=8 * T + 2), ATTN_ERR_MISALIGNED),
    (dict(positions=8 * T + 2), ATTN_ERR_MISALIGNED), (dict(positions=8 * T + 4, positions_64=1), ATTN_ERR_MISALIGNED),
    (dict(positions=8 * T, position_stride=-1), ATTN_ERR_INVALID_ARG),
    (dict(positions=8 * T, position_stride=1 << 41), ATTN_ERR_UNSUPPORTED),
]


def call_append(r="default", **kw):
    from tests.test_cache_cpu import cache
    a = dict(c=cache(B=B, Hkv=HKV, D=D), x=packed(7 * T), q_out=8 * T + (1 << 30), new_lens=None, Hq=HQ, S=S)
    a.update(kw)
    return native.load().attn_cache_append(a["c"], rope() if r == "default" else r, a["x"], a["q_out"], a["new_lens"], a["Hq"], a["S"],
                                           None)


@pytest.mark.parametrize("kw,code", BAD_ROPES)
@pytest.mark.parametrize("call", [call_fwd, call_bwd, call_append])
def test_bad_ropes_are_refused(call, kw, code):
    assert call(rope(**kw)) == code


@pytest.mark.parametrize("call", [call_fwd, call_bwd, call_append])
def test_null_rope_is_refused(call):
    assert call(None) == ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), ATTN_ERR_INVALID_ARG), (dict(y=None), ATTN_ERR_INVALID_ARG),
    (dict(x=packed(T, k=False)), ATTN_ERR_INVALID_ARG), (dict(y=dense(2 * T, 3 * T)), ATTN_ERR_INVALID_ARG),
    (dict(x=dense(), y=dense()), ATTN_ERR_INVALID_ARG),
    (dict(x=packed(T + 8)), ATTN_ERR_MISALIGNED), (dict(y=dense(2 * T + 2, 3 * T, 4 * T)), ATTN_ERR_MISALIGNED),
    (dict(x=packed(T, W=1028)), ATTN_ERR_MISALIGNED), (dict(x=dense(T, 6 * T, 7 * T, q_strides=(-8, 0, 0))), ATTN_ERR_INVALID_ARG),
    (dict(x=dense(T, 6 * T, 7 * T, v_strides=(1 << 47, 0, 0))), ATTN_ERR_UNSUPPORTED),
    (dict(x=dense(T, 6 * T, 7 * T, k_strides=(0, 0, 1 << 45))), ATTN_ERR_UNSUPPORTED),  # ten tokens
    (dict(y=dense(2 * T, 2 * T, 4 * T)), ATTN_ERR_INVALID_ARG),               # outputs share
    (dict(y=dense(T, 3 * T, 4 * T)), ATTN_ERR_INVALID_ARG),                   # over the input, of another layout
    (dict(y=dense(2 * T, 3 * T, T - 1024)), ATTN_ERR_INVALID_ARG),
    (dict(y=dense(2 * T, 3 * T, 4 * T, q_strides=(0, S * D, D))), ATTN_ERR_INVALID_ARG),   # an element twice
    (dict(y=dense(2 * T, 3 * T, 4 * T, k_strides=(HKV * S * D, S * D, 64))), ATTN_ERR_INVALID_ARG),
    (dict(y=packed(T, shift=256), x=packed(T)), ATTN_ERR_INVALID_ARG),        # k over the input's k and v
    (dict(y=packed(2 * T, shift=-64)), ATTN_ERR_INVALID_ARG),                 # q's and k's rows share
    (dict(r=rope(positions=2 * T + 64)), ATTN_ERR_INVALID_ARG), (dict(r=rope(q_weight=3 * T)), ATTN_ERR_INVALID_ARG),
])
def test_forward_refusals(kw, code):
    assert call_fwd(**kw) == code


NORM = dict(q_weight=9 * T, k_weight=9 * T + 4096)


@pytest.mark.parametrize("kw,code", [
    (dict(up=None), ATTN_ERR_INVALID_ARG), (dict(y=None), ATTN_ERR_INVALID_ARG),
    (dict(r=rope(**NORM), x=None), ATTN_ERR_INVALID_ARG), (dict(r=rope(**NORM), x=packed(T, k=False)), ATTN_ERR_INVALID_ARG),
    (dict(up=dense(2 * T, 3 * T)), ATTN_ERR_INVALID_ARG), (dict(y=packed(5 * T, q=False)), ATTN_ERR_INVALID_ARG),
    (dict(up=dense(), y=dense()), ATTN_ERR_INVALID_ARG),
    (dict(dqw=10 * T, ws=11 * T, wb=1 << 30), ATTN_ERR_INVALID_ARG),          # no such weight
    (dict(r=rope(**NORM), dqw=10 * T), ATTN_ERR_INVALID_ARG),                 # no workspace
    (dict(r=rope(**NORM), dqw=10 * T, ws=11 * T, wb=64), ATTN_ERR_INVALID_ARG),
    (dict(r=rope(**NORM), dqw=10 * T + 4, ws=11 * T, wb=1 << 30), ATTN_ERR_MISALIGNED),
    (dict(r=rope(**NORM), dqw=10 * T, ws=11 * T + 8, wb=1 << 30), ATTN_ERR_MISALIGNED),
    (dict(r=rope(**NORM), dqw=10 * T, dkw=10 * T, ws=11 * T, wb=1 << 30), ATTN_ERR_INVALID_ARG),
    (dict(r=rope(**NORM), dqw=T, ws=11 * T, wb=1 << 30), ATTN_ERR_INVALID_ARG),
    (dict(r=rope(**NORM), dqw=9 * T, ws=11 * T, wb=1 << 30), ATTN_ERR_INVALID_ARG),
    (dict(r=rope(**NORM), dqw=10 * T, ws=5 * T, wb=1 << 30), ATTN_ERR_INVALID_ARG),
    (dict(r=rope(**NORM), dqw=10 * T, ws=2 * T, wb=1 << 30), ATTN_ERR_INVALID_ARG),
    (dict(y=packed(2 * T)), ATTN_ERR_INVALID_ARG),                            # over the gradients, of another layout
    (dict(r=rope(**NORM), y=packed(T, shift=256)), ATTN_ERR_INVALID_ARG),
    (dict(up=packed(6 * T, W=1028)), ATTN_ERR_MISALIGNED),
])
def test_backward_refusals(kw, code):
    assert call_bwd(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(c=None), ATTN_ERR_INVALID_ARG), (dict(x=None), ATTN_ERR_INVALID_ARG), (dict(S=0), ATTN_ERR_INVALID_ARG),
    (dict(x=packed(7 * T, k=False)), ATTN_ERR_INVALID_ARG), (dict(x=packed(7 * T, v=False)), ATTN_ERR_INVALID_ARG),
    (dict(x=packed(7 * T, q=False)), ATTN_ERR_INVALID_ARG), (dict(q_out=None), ATTN_ERR_INVALID_ARG), (dict(Hq=0), ATTN_ERR_INVALID_ARG),
    (dict(x=packed(7 * T + 8)), ATTN_ERR_MISALIGNED), (dict(q_out=8 * T + 4), ATTN_ERR_MISALIGNED),
    (dict(new_lens=9 * T + 2), ATTN_ERR_MISALIGNED), (dict(x=packed(7 * T, W=1028)), ATTN_ERR_MISALIGNED),
    (dict(S=(1 << 29) + 1), ATTN_ERR_UNSUPPORTED), (dict(x=packed(T)), ATTN_ERR_INVALID_ARG), (dict(q_out=T), ATTN_ERR_INVALID_ARG),
    (dict(q_out=6 * T), ATTN_ERR_INVALID_ARG), (dict(q_out=7 * T + 1024), ATTN_ERR_INVALID_ARG),
    (dict(new_lens=3 * T), ATTN_ERR_INVALID_ARG), (dict(new_lens=8 * T + (1 << 30)), ATTN_ERR_INVALID_ARG),
    (dict(r=rope(k_weight=2 * T)), ATTN_ERR_INVALID_ARG), (dict(r=rope(positions=4 * T)), ATTN_ERR_INVALID_ARG),
    (dict(r=rope(positions=8 * T + (1 << 30) + 64)), ATTN_ERR_INVALID_ARG),
])
def test_append_refusals(kw, code):
    assert call_append(**kw) == code


def test_append_refuses_bad_caches():
    from tests.test_cache_cpu import BAD_CACHES, cache
    for kw, code in BAD_CACHES:
        assert call_append(c=cache(**{**dict(B=B, Hkv=HKV, D=D), **kw})) == code


@pytest.mark.skipif(torch.cuda.is_available(), reason="reaches the device")
@pytest.mark.parametrize("kw", [
    dict(x=packed(T), y=packed(T)),                                           # in place
    dict(y=packed(2 * T)),                                                    # packed to packed: ranges interleave
    dict(x=dense(T, T, T)),                                                   # the same rows read three times
    dict(x=dense(T, 6 * T, 7 * T, q_strides=(0, 0, 0))),
])
def test_views_that_share_nothing_are_taken(kw):
    assert call_fwd(**kw) == native.ATTN_ERR_DEVICE


@pytest.mark.skipif(torch.cuda.is_available(), reason="reaches the device")
def test_heads_side_by_side_are_taken():
    """q, k and v of each head next to each other: [B, S, H, 3, D]."""
    def grouped(at):
        st = (ctypes.c_longlong * 3)(S * 6 * D, 3 * D, 6 * D)
        return AttnHeads(at, at + 2 * D, at + 4 * D, st, st, st)
    assert call_fwd(x=grouped(T), y=grouped(2 * T), sizes=(B, 2, 2, S, D)) == native.ATTN_ERR_DEVICE
    bad = grouped(2 * T)
    bad.v = 2 * T + 3 * D
    assert call_fwd(x=grouped(T), y=bad, sizes=(B, 2, 2, S, D)) == ATTN_ERR_INVALID_ARG


def test_workspace():
    n = ctypes.c_ulonglong(7)
    f = native.load().attn_rope_workspace
    assert f(rope(), B, HQ, HKV, S, D, ctypes.byref(n)) == 0 and n.value == 0
    assert f(rope(**NORM), B, HQ, HKV, S, D, None) == ATTN_ERR_INVALID_ARG
    assert f(rope(q_weight=T), B, HQ, HKV, S, D, ctypes.byref(n)) == 0 and n.value > 0
    q = n.value
    assert f(rope(**NORM), B, HQ, HKV, S, D, ctypes.byref(n)) == 0 and n.value > q


@pytest.mark.parametrize("struct,name", [(AttnRope, "attn_rope_t"), (AttnHeads, "attn_heads_t")])
def test_struct_layout_matches_the_header(tmp_path, struct, name):
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    names = [n for n, _ in struct._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include "attn.h"\n#include <stddef.h>\n#include <stdio.h>\nint main(void) {\n' + "".join(
        f'printf("%zu ", offsetof({name}, {n}));\n' for n in names) + f'printf("%zu", sizeof({name})); return 0; }}\n')
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(tmp_path / "layout"), str(src)], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True).stdout.split()]
    assert got == [getattr(struct, n).offset for n in names] + [ctypes.sizeof(struct)]


PLAN = r"""
#include "rope_index.h"
#include <cstdio>
#include <cstdlib>
using namespace attn;
int main(int argc, char** argv) {
    if (argc == 3) {  // blocks of K and of q: which is which
        const unsigned ks = atoi(argv[1]), qs = atoi(argv[2]);
        for (unsigned i = 0; i < ks + qs; ++i) {
            unsigned index;
            const int k = append_is_k(append_share(ks, qs), i, &index);
            printf("%d %u\n", k, index);
        }
        return 0;
    }
    if (argc == 4) {  // D rot interleaved: each lane's vectors
        const int D = atoi(argv[1]);
        for (int l = 0; l < D / 16; ++l) {
            const RopeLane x = rope_lane(l, D, atoi(argv[2]), atoi(argv[3]));
            printf("%d %d %d %d\n", x.a, x.b, x.turn_a, x.turn_b);
        }
        return 0;
    }
    const RopePlan p = rope_plan(atoll(argv[1]), atoi(argv[2]), atoi(argv[3]), atoi(argv[4]), atoi(argv[5]), atoi(argv[6]), atoi(argv[7]), atoll(argv[8]));
    const long long units = rope_tiles(p) * rope_chunks(p);
    printf("%lld %d %d %d\n", units, p.tokens, p.groups, p.per);
    for (long long i = 0; i < units; ++i) {
        const RopeUnit u = rope_unit(p, (unsigned)i);
        printf("%u %d %d\n", u.tile, u.kind, u.chunk);
    }
}
"""


@pytest.fixture(scope="module")
def plan_program(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    at = tmp_path_factory.mktemp("rope")
    (at / "plan.cpp").write_text(PLAN)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(ROOT, "causal_scaled_dot_gb300", "csrc"), "-o",
                    str(at / "plan"), str(at / "plan.cpp")], check=True)

    def run(*args):
        out = subprocess.run([str(at / "plan"), *map(str, args)], capture_output=True, text=True, check=True).stdout
        return [[int(x) for x in line.split()] for line in out.splitlines()]

    return run


@pytest.mark.parametrize("head", [64, 128])
@pytest.mark.parametrize("interleaved", [0, 1])
def test_lanes_hold_every_element_once_and_pairs_together(plan_program, head, interleaved):
    for rot in range(0, head + 1, 8 if interleaved else 16):
        lanes = plan_program(head, rot, interleaved)
        assert sorted(v for a, b, _, _ in lanes for v in (a, b)) == list(range(head // 8))
        partner = {}
        for i, (a, b) in enumerate(zip(*rope_util.pairs(rot, interleaved))):
            partner[a], partner[b] = (b, i), (a, i)
        for l, (a, b, turn_a, turn_b) in enumerate(lanes):
            mine = {8 * a + j for j in range(8)} | {8 * b + j for j in range(8)}
            for v, turned in ((a, turn_a), (b, turn_b)):
                for e in range(8 * v, 8 * v + 8):
                    assert (e in partner) == bool(turned)
                    if turned:
                        assert partner[e][0] in mine
                        assert partner[e][1] == (e // 2 if interleaved else 8 * l + e % 8)


@pytest.mark.parametrize("case", [(1, 2, 2, 2, 64), (1, 32, 8, 8, 128), (37, 12, 4, 4, 64), (64, 32, 8, 8, 128), (33, 5, 1, 0, 128),
                                  (1000, 7, 7, 7, 64), (4096, 16, 16, 16, 128), (3, 33, 1, 1, 128), (31, 40, 40, 0, 64)])
@pytest.mark.parametrize("threads,per,least", [(256, 1, 1), (128, 8, 1216), (256, 5, 100), (128, 16, 1)])
def test_units_hold_every_row_once(plan_program, case, threads, per, least):
    total, Hq, Hk, Hv, head = case
    (units, tokens, groups, heads), *listed = plan_program(total, Hq, Hk, Hv, head, threads, per, least)
    assert len(listed) == units and tokens * groups == threads // (head // 16) and 1 <= heads <= per
    seen = np.zeros((total, 3, max(Hq, Hk, Hv)), int)
    for tile, kind, chunk in listed:
        H = (Hq, Hk, Hv)[kind]
        for side in range(groups):
            for i in range(heads):
                h = chunk * groups * heads + side + i * groups
                if h < min(H, (chunk + 1) * groups * heads):
                    seen[tile * tokens:(tile + 1) * tokens, kind, h] += 1
    for kind, H in enumerate((Hq, Hk, Hv)):
        assert (seen[:, kind, :H] == 1).all() and (seen[:, kind, H:] == 0).all()


@pytest.mark.parametrize("ks,qs", [(1, 0), (7, 0), (1, 1), (1, 1000), (1000, 1), (512, 1024), (1024, 512), (333, 1000), (999, 1001), (40000, 7)])
def test_an_appends_blocks_are_each_there_once(plan_program, ks, qs):
    got = plan_program(ks, qs)
    assert [i for k, i in got if k] == list(range(ks)) and [i for k, i in got if not k] == list(range(qs))
    done = np.cumsum([k for k, _ in got])
    assert (np.abs(done - np.arange(1, ks + qs + 1) * ks / (ks + qs)) <= 1 + 1e-6).all()  # evenly


# ------------------------------------------------------------------ frequencies
def test_frequencies():
    assert Rotary.from_base(64).frequencies == tuple(10000.0 ** (-i / 32) for i in range(32))
    assert Rotary.from_base(64, 5e5, stretch=4).frequencies[3] == 5e5 ** (-6 / 64) / 4
    near = Rotary.raised_base(128, 8.0).frequencies
    assert near[0] == 1.0 and near[-1] == pytest.approx(Rotary.from_base(128).frequencies[-1] / 8, rel=1e-12)
    parts, plain = Rotary.by_parts(128, 16, 4096), Rotary.from_base(128).frequencies
    assert parts.factor == pytest.approx(0.1 * math.log(16) + 1)
    for f, g in zip(parts.frequencies, plain):
        turns = 4096 * g / (2 * math.pi)
        assert f == pytest.approx(g if turns >= 32 else g / 16 if turns <= 1 else g * (1 / 16 + (turns - 1) / 31 * 15 / 16))
    assert Rotary.by_parts(64, 4, 4096, factor=1.0).factor == 1.0
    assert Rotary([]).rotary_dim == 0
    assert Rotary(torch.ones(8)).rotary_dim == 16


def test_a_plan_is_copied_and_pickled():
    """As part of a model that is."""
    import copy
    import pickle
    r = Rotary.by_parts(64, 4, 2048, interleaved=True)
    for other in (copy.copy(r), copy.deepcopy(r), pickle.loads(pickle.dumps(r))):
        assert bytes(other._c) == bytes(r._c) and other.frequencies == r.frequencies and repr(other) == repr(r)


def test_turns_are_exact():
    """Positions times the stored fractions, modulo a turn, against the angle in rationals."""
    from fractions import Fraction
    _PI = Fraction(31415926535897932384626433832795028841971693993751, 10**49)
    r = Rotary([1.0, 0.3, 1e-9, 7.5, -2.0, 1e-4, 0.0, 3.0])
    for p in (0, 1, 12345, 2**20 + 1, 2**31 - 1, -5):
        for f, t in zip(r.frequencies, r._c.turns):
            want = (Fraction(f) * p / (2 * _PI)) % 1
            got = Fraction(p * t % 2**64, 2**64)
            off = abs(want - got)
            assert min(off, 1 - off) <= Fraction(abs(p) + 1, 2**65)


@pytest.mark.parametrize("call", [
    lambda: Rotary([1.0] * 7), lambda: Rotary([1.0] * 3, interleaved=True), lambda: Rotary([1.0] * 72),
    lambda: Rotary([float("nan")] * 8), lambda: Rotary([1.0] * 8, factor=float("inf")), lambda: Rotary.from_base(63),
    lambda: Rotary.from_base(64, base=0.0), lambda: Rotary.raised_base(2, 4.0), lambda: Rotary.by_parts(64, 4, 4096, slow=3, fast=3),
    lambda: Rotary.from_base(64, stretch=0.0), lambda: Rotary.raised_base(64, -1.0), lambda: Rotary.by_parts(64, -4, 4096),
])
def test_bad_frequencies_are_refused(call):
    with pytest.raises(ValueError):
        call()


# ------------------------------------------------------------------ the Python calls
def test_host_tensors_are_refused():
    r, x = Rotary.from_base(64), torch.zeros(2, 5, 4 * 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        r.heads(x, 2, 1)
    with pytest.raises(ValueError, match="CUDA"):
        r.rotate(x.view(2, 5, 4, 64))


class Fake:
    """A CUDA tensor's description without one."""

    def __init__(self, shape, dtype=torch.bfloat16, index=0, last=1, requires_grad=False):
        self.shape, self.dtype, self.is_cuda, self.device = torch.Size(shape), dtype, True, torch.device("cuda", index)
        self.requires_grad = requires_grad
        self.st = [1] * len(shape)
        for i in range(len(shape) - 2, -1, -1):
            self.st[i] = self.st[i + 1] * shape[i + 1]
        self.st[-1] = last

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return tuple(self.st) if i is None else self.st[i]

    def is_contiguous(self):
        return self.st[-1] == 1

    def data_ptr(self):
        return 1 << 40


@pytest.mark.parametrize("x", [Fake((2, 5, 4 * 64), torch.float16), Fake((2, 5, 4, 64)), Fake((2, 5, 5 * 64)), Fake((2, 5, 4 * 96)),
                               Fake((0, 5, 4 * 64)), Fake((2, 0, 4 * 64)), Fake((2, 5, 4 * 64), last=2)])
def test_bad_projections_are_refused(x):
    with pytest.raises(ValueError):
        Rotary.from_base(64).heads(x, 2, 1)


@pytest.mark.parametrize("kw,match", [
    (dict(positions=Fake((5,), torch.int16)), "positions"), (dict(positions=Fake((5,), torch.int32, index=1)), "positions"),
    (dict(positions=Fake((4,), torch.int32)), "positions"), (dict(positions=Fake((3, 5), torch.int64)), "positions"),
    (dict(positions=Fake((2, 5), torch.int64, last=2)), "contiguous"), (dict(positions=Fake((5,), torch.int32), first=3), "first"),
    (dict(q_norm=Fake((128,))), "q_norm"), (dict(k_norm=Fake((64,), torch.float16)), "k_norm"), (dict(k_norm=Fake((64,), index=1)), "k_norm"),
    (dict(q_norm=Fake((64,), last=2)), "q_norm"), (dict(q_norm=Fake((64,)), k_norm=Fake((64,), torch.float32)), "one type"),
])
def test_bad_positions_and_weights_are_refused(kw, match):
    with pytest.raises(ValueError, match=match):
        Rotary.from_base(64).heads(Fake((2, 5, 4 * 64)), 2, 1, **kw)


def test_more_elements_than_the_head_has_are_refused():
    with pytest.raises(ValueError, match="rotated"):
        Rotary.from_base(128).heads(Fake((2, 5, 4 * 64)), 2, 1)


def test_rows_are_checked():
    r, q = Rotary.from_base(64), Fake((2, 4, 5, 64))
    for k in (Fake((2, 2, 6, 64)), Fake((1, 2, 5, 64)), Fake((2, 2, 5, 128)), Fake((2, 2, 5, 64), index=1), Fake((2, 2, 5, 64), torch.float32),
              Fake((2, 2, 5, 64), last=2), Fake((2, 0, 5, 64))):
        with pytest.raises(ValueError):
            r.rotate(q, k)
    with pytest.raises(ValueError, match="k_norm"):
        r.rotate(q, k_norm=Fake((64,)))
    with pytest.raises(ValueError, match="64 or 128"):
        r.rotate(Fake((2, 4, 5, 96)))
    with pytest.raises(ValueError, match="dq"):
        r.rotate_backward(Fake((2, 4, 6, 64)), None, q, None)
    with pytest.raises(ValueError, match="together"):
        r.rotate_backward(q, q, q, None)
    with pytest.raises(ValueError, match="dk"):
        r.heads_backward(Fake((2, 2, 5, 64)), None, Fake((2, 1, 5, 64)), Fake((2, 5, 4 * 64)), 2, 1)
    with pytest.raises(ValueError, match="dv"):
        r.heads_backward(Fake((2, 2, 5, 64)), Fake((2, 1, 5, 64)), Fake((2, 2, 5, 64)), Fake((2, 5, 4 * 64)), 2, 1)


def test_append_arguments_are_checked():
    from tests.test_cache_cpu import _fake_cache
    c, r = _fake_cache(), Rotary.from_base(64)
    k, q = Fake((3, 2, 5, 64)), Fake((3, 4, 5, 64))
    for call in (lambda: c.append(k, Fake((3, 2, 6, 64)), r), lambda: c.append(Fake((3, 1, 5, 64)), k, r),
                 lambda: c.append(k, k, r, q=Fake((3, 4, 6, 64))), lambda: c.append(k, k, r, q_out=q),
                 lambda: c.append(k, k, r, q_norm=Fake((64,))), lambda: c.append(k, k, r, q=q, q_out=Fake((3, 4, 5, 64), last=2)),
                 lambda: c.append(k, k, r, new_lens=Fake((2,), torch.int32)), lambda: c.append(k, k, r, positions=Fake((4,), torch.int32)),
                 lambda: c.append(k, k, Rotary.from_base(128)), lambda: c.append(Fake((3, 2, 5, 64), requires_grad=True), k, r),
                 lambda: c.append(k, k, r, k_norm=Fake((64,), requires_grad=True))):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ the definitions
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weight", [False, True])
def test_definitions_agree_with_differences(interleaved, weight):
    """The tests' backward against the differences of the tests' forward, and scores that depend on distances alone."""
    rng = np.random.default_rng(3)
    r = Rotary.by_parts(32, 4.0, 64, interleaved=interleaved)
    x, dy = rng.normal(size=(1, 2, 3, 64)), rng.normal(size=(1, 2, 3, 64))
    at, w = np.array([[5, 2, 9]]), rng.uniform(0.5, 1.5, 64) if weight else None
    f = lambda x, w: float((rope_util.forward(x, at, r, w)[0] * dy).sum())  # noqa: E731
    dx, _, dw, _ = rope_util.backward(dy, x, at, r, w)
    for _ in range(10):
        d, h = rng.normal(size=x.shape), 1e-5
        assert (f(x + h * d, w) - f(x - h * d, w)) / (2 * h) == pytest.approx((dx * d).sum(), rel=1e-6, abs=1e-6)
        if weight:
            d = rng.normal(size=64)
            assert (f(x, w + h * d) - f(x, w - h * d)) / (2 * h) == pytest.approx((dw * d).sum(), rel=1e-6, abs=1e-6)
    q, k = rng.normal(size=(1, 1, 1, 64)), rng.normal(size=(1, 1, 1, 64))
    score = lambda i, j: float((rope_util.turn(q, [[i]], r) * rope_util.turn(k, [[j]], r)).sum())  # noqa: E731
    assert score(7, 3) == pytest.approx(score(1007, 1003), abs=1e-9) and score(7, 3) != pytest.approx(score(7, 4), abs=1e-3)


ROWS = r"""
#include "rows.h"
#include <cstdio>
#include <cstdlib>
#include <set>
using namespace attn::host;
static unsigned long long state = 12345;
static int below(int n) { state = state * 6364136223846793005ull + 1442695040888963407ull; return (int)((state >> 33) % n); }
static std::multiset<long long> elements(const RowsBox& x) {
    std::multiset<long long> all;
    for (int b = 0; b < x.n[0]; ++b)
        for (int h = 0; h < x.n[1]; ++h)
            for (int s = 0; s < x.n[2]; ++s)
                for (int d = 0; d < x.D; d += 8)  // strides and addresses are multiples of 8 elements
                    all.insert((long long)(size_t)x.p / 2 + b * x.stride[0] + h * x.stride[1] + s * x.stride[2] + d);
    return all;
}
int main() {
    int apart = 0, told_apart = 0, distinct = 0, told_distinct = 0;
    for (int i = 0; i < 20000; ++i) {
        RowsBox box[2];
        const int common = below(2), D = 16;  // half of the pairs: views of one tensor
        long long st[3] = {8ll * below(200), 8ll * below(20), 8ll * below(60)};
        for (int k = 0; k < 2; ++k) {
            box[k] = RowsBox{(const void*)(size_t)(4096 + 16 * below(300)), {1 + below(3), 1 + below(3), 1 + below(4)}, {0, 0, 0}, D};
            for (int d = 0; d < 3; ++d)
                if (box[k].n[d] > 1) box[k].stride[d] = common ? st[d] : 8ll * below(d == 0 ? 200 : 40);
        }
        const auto a = elements(box[0]), b = elements(box[1]);
        const std::set<long long> only(a.begin(), a.end());
        bool share = false;
        for (long long e : b) share = share || only.count(e);
        const bool once = only.size() == a.size();
        if (rows_apart(box[0], box[1]) && share) { printf("apart %d\n", i); return 1; }
        if (rows_apart(box[0], box[1]) != rows_apart(box[1], box[0])) { printf("order %d\n", i); return 1; }
        if (rows_distinct(box[0]) && !once) { printf("distinct %d\n", i); return 1; }
        apart += !share;
        told_apart += rows_apart(box[0], box[1]);
        distinct += once;
        told_distinct += rows_distinct(box[0]);
    }
    printf("%d %d %d %d\n", apart, told_apart, distinct, told_distinct);
}
"""


def test_shared_elements_are_never_overlooked(tmp_path):
    """Random strided tensors against their elements one by one: what is called apart shares none, what is called
    distinct has each once, and few that would do are refused."""
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    (tmp_path / "rows.cpp").write_text(ROWS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "causal_scaled_dot_gb300", "csrc"), "-o", str(tmp_path / "rows"),
                    str(tmp_path / "rows.cpp")], check=True)
    r = subprocess.run([str(tmp_path / "rows")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    apart, told_apart, distinct, told_distinct = map(int, r.stdout.split())
    assert told_apart > 0.5 * apart and told_distinct > 0.5 * distinct, r.stdout
