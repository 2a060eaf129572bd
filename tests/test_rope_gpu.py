"""Rotary positions and norms of heads on the GPU against their definitions in float64 (tests/rope_util.py)."""
import math

import numpy as np
import pytest
import torch

from causal_scaled_dot_gb300 import native
from causal_scaled_dot_gb300.rotary import Rotary
from tests import rope_util
from tests.cache_util import rows
from tests.rope_util import HALF_BF16, to_f64

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def weights(D, dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    return [(0.4 + 1.2 * torch.rand(D, generator=g)).mul(torch.where(torch.rand(D, generator=g) > 0.9, -3.0, 1.0)).to(dtype) for _ in range(2)]


def split(qkv, Hq, Hkv):
    """float64 q, k, v [B, H, S, D] of a projection's output."""
    B, S, W = qkv.shape
    x = to_f64(qkv).reshape(B, S, Hq + 2 * Hkv, -1).transpose(0, 2, 1, 3)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def near(got, want, tol, what=""):
    got = to_f64(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((np.abs(got - want) / tol)[bad].max()))


def check_heads(rotary, B, S, Hq, Hkv, D, norm=None, positions=None, first=0, seed=0, eps=EPS):
    """heads and heads_backward of one set of sizes, against the definitions."""
    qkv = rows((B, S, (Hq + 2 * Hkv) * D), seed)
    wq, wk = weights(D, norm) if norm else (None, None)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    more = dict(positions=dev(positions), first=first, q_norm=dev(wq), k_norm=dev(wk), eps=eps)
    q, k, v = rotary.heads(qkv.cuda(), Hq, Hkv, **more)
    at = np.broadcast_to(np.arange(S) + first if positions is None else positions.numpy(), (B, S))
    xq, xk, xv = split(qkv, Hq, Hkv)
    fw = [None if w is None else to_f64(w) for w in (wq, wk)]
    for got, x, w, name in ((q, xq, fw[0], "q"), (k, xk, fw[1], "k")):
        want, tol, _ = rope_util.forward(x, at, rotary, w, eps)
        assert got.is_contiguous() and got.dtype == torch.bfloat16
        near(got, want, tol, name)
    assert np.array_equal(to_f64(v), xv)

    up = [rows((B, H, S, D), seed + 10 + i, 0.1) for i, H in enumerate((Hq, Hkv, Hkv))]
    dqkv, dwq, dwk = rotary.heads_backward(*(u.cuda() for u in up), qkv.cuda(), Hq, Hkv, **more)
    assert dqkv.shape == qkv.shape and dqkv.is_contiguous()
    d = split(dqkv, Hq, Hkv)
    for i, (x, w, dw, name) in enumerate(((xq, fw[0], dwq, "dq"), (xk, fw[1], dwk, "dk"))):
        want, tol, want_w, tol_w = rope_util.backward(to_f64(up[i]), x, at, rotary, w, eps)
        assert (np.abs(d[i] - want) <= tol).all(), (name, float((np.abs(d[i] - want) / tol).max()))
        if w is None:
            assert dw is None
        else:
            assert dw.dtype == norm and dw.shape == (D,)
            near(dw, want_w, tol_w + (HALF_BF16 * np.abs(want_w) if norm == torch.bfloat16 else 0), name + "_norm")
    assert np.array_equal(d[2], to_f64(up[2]))
    return q, k, v


SIZES = [(1, 1, 1, 1), (1, 1, 32, 8), (2, 5, 3, 1), (1, 256, 2, 2), (3, 37, 12, 4), (5, 33, 5, 5), (64, 1, 8, 2), (2, 300, 9, 3)]


@pytest.mark.parametrize("B,S,Hq,Hkv", SIZES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [None, torch.bfloat16, torch.float32])
def test_heads(B, S, Hq, Hkv, D, interleaved, norm):
    check_heads(Rotary.from_base(D, interleaved=interleaved), B, S, Hq, Hkv, D, norm, seed=S)


@pytest.mark.parametrize("D,rot,interleaved", [(64, r, False) for r in (0, 16, 32, 48)] + [(128, r, False) for r in (0, 16, 32, 48, 112)]
                         + [(64, r, True) for r in (0, 8, 24, 40)] + [(128, r, True) for r in (0, 8, 64, 72, 120)])
@pytest.mark.parametrize("norm", [None, torch.float32])
def test_part_of_the_head(D, rot, interleaved, norm):
    """Elements past the rotated ones come back bit for bit without a norm."""
    r = Rotary.from_base(rot, interleaved=interleaved) if rot else Rotary([], interleaved=interleaved)
    q, _, _ = check_heads(r, 2, 41, 3, 1, D, norm, seed=rot)
    if norm is None:
        x = rows((2, 41, 5 * D), rot).view(2, 41, 5, D).transpose(1, 2)[:, :3]
        assert torch.equal(q.cpu()[..., rot:], x[..., rot:])


@pytest.mark.parametrize("rotary", [Rotary.from_base(128, 5e5, stretch=8), Rotary.raised_base(64, 4.0), Rotary.by_parts(128, 32, 4096),
                                    Rotary.by_parts(64, 4, 2048, interleaved=True, factor=0.5), Rotary([0.5] * 8, factor=-2.0),
                                    Rotary([7.0, 100.0, -3.0, 0.0] * 2)])
def test_scalings(rotary):
    check_heads(rotary, 2, 70, 4, 2, 128, torch.float32)


@pytest.mark.parametrize("first", [1, 131071, 2**24 + 1, 2**31 - 300, -77])
def test_far_positions(first):
    """Angles of hundreds of millions of radians."""
    check_heads(Rotary.from_base(64), 1, 50, 2, 1, 64, first=first)


@pytest.mark.parametrize("kind", ["shared", "each", "one row", "expanded", "wide"])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_positions(kind, dtype):
    g = torch.Generator().manual_seed(4)
    p = torch.randint(-1000, 1 << 20, (3, 45), generator=g).to(dtype)
    p = {"shared": p[0], "each": p, "one row": p[1:2], "expanded": p[:1].expand(3, 45), "wide": torch.cat((p, p), 1)[:, 20:65]}[kind]
    check_heads(Rotary.from_base(128), 3, 45, 4, 2, 128, torch.bfloat16, positions=p)


def test_same_position_twice():
    check_heads(Rotary.from_base(64), 2, 8, 2, 2, 64, positions=torch.zeros(8, dtype=torch.int32))


def test_int64_positions_past_32_bits():
    check_heads(Rotary.from_base(64), 1, 4, 2, 1, 64, positions=torch.tensor([2**31, 2**32 + 7, 2**33, 2**34 - 1]))


@pytest.mark.parametrize("only", ["q", "k"])
def test_norm_of_one_of_them(only):
    r, x = Rotary.from_base(64), rows((2, 30, 4 * 64), 3).cuda()
    w = weights(64, torch.float32)[0].cuda()
    q, k, v = r.heads(x, 2, 1, **{only + "_norm": w})
    bare, normed = r.heads(x, 2, 1), r.heads(x, 2, 1, q_norm=w, k_norm=w)
    assert torch.equal(q, normed[0] if only == "q" else bare[0]) and torch.equal(k, normed[1] if only == "k" else bare[1])
    up = [rows(t.shape, 5).cuda() for t in (q, k, v)]
    dx, dwq, dwk = r.heads_backward(*up, x, 2, 1, **{only + "_norm": w})
    dn, nq, nk = r.heads_backward(*up, x, 2, 1, q_norm=w, k_norm=w)
    db, _, _ = r.heads_backward(*up, x, 2, 1)
    at = slice(0, 128) if only == "q" else slice(128, 192)
    want = db.clone()
    want[..., at] = dn[..., at]
    assert torch.equal(dx, want)
    assert torch.equal(dwq, nq) and dwk is None if only == "q" else torch.equal(dwk, nk) and dwq is None


@pytest.mark.parametrize("size,eps", [(1e18, 1e-6), (3e38, 1e-6), (1e-20, 1e-6), (1e-20, 2.0 ** -100), (0.0, 1e-6), (1.0, 1e30)])
def test_norms_of_very_large_and_very_small_rows(size, eps):
    """Squares beyond fp32, rows of zeros, and eps far above or below the squares."""
    r = Rotary.from_base(64)
    base = rows((1, 20, 4 * 64), 8).clamp(-1, 1)
    x = (base.double() * size).to(torch.bfloat16)
    w = weights(64, torch.float32)
    q, k, _ = r.heads(x.cuda(), 2, 1, q_norm=w[0].cuda(), k_norm=w[1].cuda(), eps=eps)
    xq, xk, _ = split(x, 2, 1)
    at = np.arange(20)[None]
    eps = float(np.float32(eps))
    for got, y, wi in ((q, xq, w[0]), (k, xk, w[1])):
        want, tol, _ = rope_util.forward(y, at, r, to_f64(wi), eps)
        near(got, want, tol)
    up = [rows(t.shape, 5).cuda() for t in (q, k, k)]
    dx, dwq, _ = r.heads_backward(*up, x.cuda(), 2, 1, q_norm=w[0].cuda(), k_norm=w[1].cuda(), eps=eps)
    want, tol, want_w, tol_w = rope_util.backward(to_f64(up[0]), xq, at, r, to_f64(w[0]), eps)
    got = split(dx, 2, 1)[0]
    assert (np.abs(got - want) <= tol).all()
    near(dwq, want_w, tol_w + 1e-38)


def test_values_that_are_not_finite_stay_in_their_row():
    r = Rotary.from_base(32)  # half of the head is not rotated
    x = rows((1, 6, 3 * 64), 2)
    clean = x.clone()
    x[0, 1, 5], x[0, 2, 40], x[0, 3, 64 + 63] = math.inf, math.nan, -math.inf
    w = weights(64, torch.float32)
    for norm in (None, w):
        more = {} if norm is None else dict(q_norm=w[0].cuda(), k_norm=w[1].cuda())
        q, k, _ = (t.float().cpu() for t in r.heads(x.cuda(), 1, 1, **more))
        q0, k0, _ = (t.float().cpu() for t in r.heads(clean.cuda(), 1, 1, **more))
        for s in (0, 4, 5):
            assert torch.equal(q[0, 0, s], q0[0, 0, s]) and torch.equal(k[0, 0, s], k0[0, 0, s])
        if norm is None:
            hurt = torch.zeros(64, dtype=torch.bool)
            hurt[[5, 21]] = True  # the element and its partner
            assert torch.equal(q[0, 0, 1][~hurt], q0[0, 0, 1][~hurt]) and not q[0, 0, 1][hurt].isfinite().any()
            hurt[:] = False
            hurt[40] = True
            assert torch.equal(q[0, 0, 2][~hurt], q0[0, 0, 2][~hurt]) and q[0, 0, 2, 40].isnan()
            assert torch.equal(k[0, 0, 3][:63], k0[0, 0, 3][:63]) and k[0, 0, 3, 63] == -math.inf
        else:
            assert q[0, 0, 2].isnan().all()
            # 1 / sqrt(inf) is 0: the others are 0, and the infinity itself NaN
            assert k[0, 0, 3, 63].isnan() and (k[0, 0, 3, 32:63] == 0).all()


# ------------------------------------------------------------------ layouts
def views(B, H, S, D, seed):
    """The same rows in different layouts."""
    x = rows((B, H, S, D), seed)
    wide = torch.full((B, S, H, D + 24), math.nan, dtype=torch.bfloat16)
    wide[..., 8:8 + D] = x.transpose(1, 2)
    return x, {"dense": x.cuda(), "by token": x.transpose(1, 2).contiguous().cuda().transpose(1, 2),
               "batch last": x.permute(1, 2, 0, 3).contiguous().cuda().permute(2, 0, 1, 3), "wide": wide.cuda()[..., 8:8 + D].transpose(1, 2)}


@pytest.mark.parametrize("D", [64, 128])
def test_rotate_takes_any_layout(D):
    r, w = Rotary.from_base(D), [t.cuda() for t in weights(D, torch.bfloat16)]
    xq, qs = views(3, 5, 21, D, 1)
    xk, ks = views(3, 2, 21, D, 2)
    at = np.broadcast_to(np.arange(21), (3, 21))
    dq, dk = rows(xq.shape, 7).cuda(), rows(xk.shape, 8).cuda()
    first = None
    for a in qs:
        for b in ks:
            q, k = r.rotate(qs[a], ks[b], q_norm=w[0], k_norm=w[1])
            back = r.rotate_backward(dq, dk, qs[a], ks[b], q_norm=w[0], k_norm=w[1])
            if first is None:
                first = q, k, *back
                for got, x, wi in ((q, xq, w[0]), (k, xk, w[1])):
                    want, tol, _ = rope_util.forward(to_f64(x), at, r, to_f64(wi))
                    near(got, want, tol)
            else:
                for x, y in zip((q, k, *back), first):
                    assert torch.equal(x, y), (a, b)
            assert q.is_contiguous() and k.is_contiguous()
            if a == "by token":
                assert back[0].stride() == qs[a].stride()
    alone = r.rotate(qs["by token"], q_norm=w[0])
    assert torch.equal(alone, first[0])
    da, none, dwa, _ = r.rotate_backward(dq, None, qs["wide"], None, q_norm=w[0])
    assert none is None and torch.equal(da, first[2]) and torch.equal(dwa, first[4])


def test_expanded_and_odd_gradients():
    """Upstream gradients with strides of 0, of another order, and at an odd address."""
    r, x = Rotary.from_base(64), rows((2, 33, 4 * 64), 3).cuda()
    one = rows((1, 1, 1, 64), 4).cuda()
    up = [one.expand(2, 2, 33, 64), rows((2, 33, 64, 1), 5).cuda().permute(0, 3, 1, 2), rows((2 * 33 * 64 + 3,), 6).cuda()[3:].view(2, 1, 33, 64)]
    got = r.heads_backward(*up, x, 2, 1)
    want = r.heads_backward(*(u.contiguous().clone() for u in up), x, 2, 1)
    assert torch.equal(got[0], want[0])
    scalar = torch.ones((), dtype=torch.bfloat16, device="cuda").expand(2, 2, 33, 64)
    assert torch.equal(r.heads_backward(scalar, *up[1:], x, 2, 1)[0], r.heads_backward(scalar.contiguous(), *up[1:], x, 2, 1)[0])


def test_qkv_of_other_strides_and_bad_addresses():
    r, x = Rotary.from_base(64), rows((2, 9, 8 * 64), 3).cuda()
    want = r.heads(x[:, :, :256].contiguous(), 2, 1)
    for y in (x[:, :, :256], x[:, :, :256].transpose(0, 1).contiguous().transpose(0, 1)):
        for a, b in zip(r.heads(y, 2, 1), want):
            assert torch.equal(a, b)
    shared = x[:1, :, :256].expand(2, 9, 256)
    for a, b in zip(r.heads(shared, 2, 1), r.heads(shared.contiguous(), 2, 1)):
        assert torch.equal(a, b)
    with pytest.raises(native.AttnError, match="MISALIGNED"):
        r.heads(x.view(-1)[4:4 + 256].view(1, 1, 256), 2, 1)
    with pytest.raises(native.AttnError, match="MISALIGNED"):
        r.heads(torch.zeros(1, 4, 260, dtype=torch.bfloat16, device="cuda")[:, :, :256], 2, 1)


def c_heads(q, k, v):
    from causal_scaled_dot_gb300.rotary import _heads_of
    return _heads_of(q, k, v)


def test_in_place():
    """The C call on rows that are written where they are read."""
    r, lib = Rotary.from_base(128, interleaved=True), native.load()
    q, k = rows((2, 3, 50, 128), 1).cuda(), rows((2, 1, 50, 128), 2).cuda()
    want = r.rotate(q, k)
    c = r._plan(q.device, 2, 50, 128, None, 0, None, None, EPS)
    st = torch.cuda.current_stream().cuda_stream
    assert lib.attn_rope(c, c_heads(q, k, None), c_heads(q, k, None), 2, 3, 1, 50, 128, st) == 0
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_nothing_else_is_written():
    """Rows among others: what lies between them keeps its values."""
    r, lib = Rotary.from_base(64), native.load()
    x, w = rows((2, 35, 4 * 64), 1).cuda(), [t.cuda() for t in weights(64, torch.float32)]
    out = torch.full((2, 37, 6 * 64), 7.0, dtype=torch.bfloat16, device="cuda")
    y = out[:, 1:36, 64:64 + 256].unflatten(2, (4, 64)).transpose(1, 2)
    c = r._plan(x.device, 2, 35, 64, None, 0, *w, EPS)
    rows_in = x.unflatten(2, (4, 64)).transpose(1, 2)
    st = torch.cuda.current_stream().cuda_stream
    parts = lambda t: c_heads(t[:, :2], t[:, 2:3], t[:, 3:])  # noqa: E731
    assert lib.attn_rope(c, parts(rows_in), parts(y), 2, 2, 1, 35, 64, st) == 0
    for got, want in zip((y[:, :2], y[:, 2:3], y[:, 3:]), r.heads(x, 2, 1, q_norm=w[0], k_norm=w[1])):
        assert torch.equal(got, want)
    y.fill_(7.0)
    assert (out == 7.0).all()


def test_only_weight_gradients():
    """Rows' gradients left out, and one of the two weights' too."""
    import ctypes
    r, lib, x = Rotary.from_base(64), native.load(), rows((2, 100, 4 * 64), 1).cuda()
    w = [t.cuda() for t in weights(64, torch.bfloat16)]
    up = [rows((2, H, 100, 64), H + i).cuda() for i, H in enumerate((2, 1, 1))]
    _, want, _ = r.heads_backward(*up, x, 2, 1, q_norm=w[0], k_norm=w[1])
    c = r._plan(x.device, 2, 100, 64, None, 0, *w, EPS)
    n = ctypes.c_ulonglong(0)
    assert lib.attn_rope_workspace(c, 2, 2, 1, 100, 64, n) == 0
    ws, got = torch.empty(n.value, dtype=torch.uint8, device="cuda"), torch.zeros_like(w[0])
    q = x.unflatten(2, (4, 64)).transpose(1, 2)[:, :2]
    st = torch.cuda.current_stream().cuda_stream
    assert lib.attn_rope_bwd(c, c_heads(up[0], None, None), c_heads(q, None, None), c_heads(None, None, None), got.data_ptr(), None, 2, 2, 1,
                             100, 64, ws.data_ptr(), n.value, st) == 0
    assert torch.equal(got, want)
    dx, dwq, dwk = r.heads_backward(*up, x, 2, 1, q_norm=w[0], k_norm=w[1], weight_grads=False)
    assert dwq is None and dwk is None and torch.equal(dx, r.heads_backward(*up, x, 2, 1, q_norm=w[0], k_norm=w[1])[0])


# ------------------------------------------------------------------ gradients through autograd
@pytest.mark.parametrize("D,interleaved", [(64, False), (128, True)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_autograd(D, interleaved, dtype):
    r = Rotary.by_parts(D // 2, 4, 64, interleaved=interleaved)
    x = rows((2, 31, 7 * D), 2).cuda().requires_grad_()
    w = [t.cuda().requires_grad_() for t in weights(D, dtype)]
    out = r.heads(x, 3, 2, q_norm=w[0], k_norm=w[1], first=5)
    up = [rows(t.shape, 20 + i).cuda() for i, t in enumerate(out)]
    torch.autograd.backward(out, up)
    want = r.heads_backward(*up, x.detach(), 3, 2, q_norm=w[0].detach(), k_norm=w[1].detach(), first=5)
    for leaf, g in zip((x, *w), want):
        assert torch.equal(leaf.grad, g)
    # q and k by themselves
    q, k = (t.detach().requires_grad_() for t in (x.detach()[:, :, :3 * D].unflatten(2, (3, D)).transpose(1, 2),
                                                  x.detach()[:, :, 3 * D:5 * D].unflatten(2, (2, D)).transpose(1, 2)))
    for t in w:
        t.grad = None
    out = r.rotate(q, k, q_norm=w[0], k_norm=w[1], first=5)
    torch.autograd.backward(out, up[:2])
    got = want[0].unflatten(2, (7, D)).transpose(1, 2)
    assert torch.equal(q.grad, got[:, :3]) and torch.equal(k.grad, got[:, 3:5])
    assert torch.equal(w[0].grad, want[1]) and torch.equal(w[1].grad, want[2])


def test_autograd_of_parts():
    """Outputs that nothing depends on, inputs without gradients, and no second derivatives."""
    r, x = Rotary.from_base(64), rows((1, 12, 4 * 64), 2).cuda()
    w = weights(64, torch.float32)[0].cuda().requires_grad_()
    q, k, v = r.heads(x, 2, 1, q_norm=w)
    (q.float() ** 2).sum().backward()
    assert w.grad is not None and x.grad is None
    y = x.clone().requires_grad_()
    k = r.heads(y, 2, 1)[1]
    g, = torch.autograd.grad(k.float().sum(), y, create_graph=True)
    assert (g[..., :128] == 0).all() and (g[..., 192:] == 0).all() and g[..., 128:192].any()
    with pytest.raises(RuntimeError):
        torch.autograd.grad((g.float() ** 2).sum(), y)
    with torch.no_grad():
        assert not r.heads(y, 2, 1)[0].requires_grad
    y2 = x.clone().requires_grad_()
    q = r.rotate(y2[:, :, :128].unflatten(2, (2, 64)).transpose(1, 2))
    q.sum().backward()
    assert (y2.grad[..., 128:] == 0).all() and y2.grad[..., :128].any()


def test_differences():
    """The gradient against differences of the float64 forward's scalar."""
    rng = np.random.default_rng(0)
    r, D = Rotary.from_base(64), 64
    x, w = rows((1, 9, 4 * D), 2), weights(D, torch.float32)
    up = [rows(s, 3 + i) for i, s in enumerate(((1, 2, 9, D), (1, 1, 9, D), (1, 1, 9, D)))]
    dx, dwq, dwk = (to_f64(t) for t in r.heads_backward(*(u.cuda() for u in up), x.cuda(), 2, 1, q_norm=w[0].cuda(), k_norm=w[1].cuda()))
    at = np.arange(9)[None]

    def f(x, wq, wk):
        h = x.reshape(1, 9, 4, D).transpose(0, 2, 1, 3)
        parts = rope_util.forward(h[:, :2], at, r, wq, EPS)[0], rope_util.forward(h[:, 2:3], at, r, wk, EPS)[0], h[:, 3:]
        return sum((p * to_f64(u)).sum() for p, u in zip(parts, up))

    x0, w0 = to_f64(x), [to_f64(t) for t in w]
    for _ in range(8):
        d, dw, h = rng.normal(size=x0.shape), [rng.normal(size=D) for _ in w], 1e-5
        moved = [f(x0 + s * h * d, *(a + s * h * b for a, b in zip(w0, dw))) for s in (1, -1)]
        got = [(dx * d).sum(), (dwq * dw[0]).sum(), (dwk * dw[1]).sum()]
        # roundings of dx: half a step each, none with a preferred sign (a deviation of 1 / sqrt 3 of it), six deviations
        tol = 6 * HALF_BF16 / math.sqrt(3) * np.linalg.norm(dx * d) + 1e-4 * sum(map(abs, got))
        assert abs((moved[0] - moved[1]) / (2 * h) - sum(got)) <= tol


def test_deterministic():
    r, x = Rotary.from_base(128), rows((3, 700, 10 * 128), 2).cuda()
    w = [t.cuda() for t in weights(128, torch.float32)]
    up = [rows((3, H, 700, 128), H).cuda() for H in (4, 3, 3)]
    first = r.heads_backward(*up, x, 4, 3, q_norm=w[0], k_norm=w[1])
    for _ in range(3):
        for a, b in zip(r.heads_backward(*up, x, 4, 3, q_norm=w[0], k_norm=w[1]), first):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ with the attention
def test_a_training_layer():
    """Projection, norms, rotation and attention together, against the same in float64 through torch's own gradients.
    Relative errors count bf16's roundings on the way (projection, q, k and v, weights, O; back as many), each 2^-9 of the
    norm at most in the mean: under ten of them add up to 2e-2 even if all point one way."""
    B, S, Hq, Hkv, D, E = 2, 192, 4, 2, 64, 96
    r = Rotary.from_base(D)
    g = torch.Generator().manual_seed(1)
    h, proj = torch.randn(B, S, E, generator=g), torch.randn((Hq + 2 * Hkv) * D, E, generator=g) / math.sqrt(E)
    up = torch.randn(B, Hq, S, D, generator=g)
    w = weights(D, torch.float32)
    leaves = [t.to(torch.bfloat16).cuda().requires_grad_() for t in (h, proj)] + [t.cuda().requires_grad_() for t in w]
    qkv = leaves[0] @ leaves[1].T
    q, k, v = r.heads(qkv, Hq, Hkv, q_norm=leaves[2], k_norm=leaves[3])
    o = native.attention_trainable(q, k, v, check_status=True)
    o.backward(up.to(torch.bfloat16).cuda())

    ref = [t.detach().double().requires_grad_() for t in leaves]
    x = (ref[0] @ ref[1].T).unflatten(2, (Hq + 2 * Hkv, D)).transpose(1, 2)
    angle = torch.arange(S, device="cuda").double()[:, None] * torch.tensor(r.frequencies, dtype=torch.float64, device="cuda")
    turned = lambda t: torch.cat((t[..., :32] * angle.cos() - t[..., 32:] * angle.sin(), t[..., 32:] * angle.cos() + t[..., :32] * angle.sin()), -1)  # noqa: E731
    normed = lambda t, wi: t * (t.square().mean(-1, keepdim=True) + EPS).rsqrt() * wi  # noqa: E731
    q, k, v = turned(normed(x[:, :Hq], ref[2])), turned(normed(x[:, Hq:Hq + Hkv], ref[3])), x[:, Hq + Hkv:]
    k, v = (t.repeat_interleave(Hq // Hkv, 1) for t in (k, v))
    s = (q @ k.transpose(2, 3) / math.sqrt(D)).masked_fill(torch.ones(S, S, dtype=torch.bool, device="cuda").triu(1), -math.inf)
    want = torch.softmax(s, -1) @ v
    want.backward(up.to(torch.bfloat16).double().cuda())
    for got, ref_, name in [(o, want, "o")] + [(a.grad, b.grad, n) for a, b, n in zip(leaves, ref, ("h", "proj", "wq", "wk"))]:
        assert float((got.detach().double() - ref_.detach()).norm() / ref_.detach().norm()) <= 2e-2, name


# ------------------------------------------------------------------ streams, graphs, other callers
def test_on_another_stream():
    r, x = Rotary.from_base(128), rows((2, 500, 6 * 128), 2).cuda()
    want = r.heads(x, 4, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = r.heads(x * 1, 4, 1)  # after the copy, on the same stream
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    r = Rotary.from_base(64)
    w = [t.cuda() for t in weights(64, torch.float32)]
    xs = [rows((2, 900, 4 * 64), 30 + i).cuda() for i in range(2)]
    ups = [[rows((2, H, 900, 64), 40 + i + H).cuda() for H in (2, 1, 1)] for i in range(2)]
    want = [r.heads_backward(*u, x, 2, 1, q_norm=w[0], k_norm=w[1]) for x, u in zip(xs, ups)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(r.heads_backward(*ups[i], xs[i], 2, 1, q_norm=w[0], k_norm=w[1]))
    torch.cuda.synchronize()
    for i in range(2):
        for one in got[i]:
            for a, b in zip(one, want[i]):
                assert torch.equal(a, b)


def test_captured_step():
    """Forward, attention and backward in a graph, replayed on new inputs and positions."""
    r, Hq, Hkv, D, S = Rotary.from_base(64), 2, 1, 64, 130
    x = rows((1, S, 4 * D), 2).cuda().requires_grad_()
    w = [t.cuda().requires_grad_() for t in weights(D, torch.float32)]
    at = torch.arange(S, device="cuda")
    up = rows((1, Hq, S, D), 3).cuda()

    def step():
        q, k, v = r.heads(x, Hq, Hkv, positions=at, q_norm=w[0], k_norm=w[1])
        o = native.attention_trainable(q, k, v)
        return (o, *torch.autograd.grad(o, (x, *w), up))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        with torch.no_grad():
            x.copy_(rows((1, S, 4 * D), 50 + i))
            at.copy_(torch.arange(S) + 100 * i)
        graph.replay()
        torch.cuda.synchronize()
        held = [t.clone() for t in got]
        for a, b in zip(held, step()):
            assert torch.equal(a, b)


def test_captured_while_an_eager_graph_lives():
    """Through autograd the backward is refused, the forward captured; the backward call itself is captured and replayed."""
    r, x = Rotary.from_base(64), rows((1, 50, 4 * 64), 2).cuda()
    w = weights(64, torch.float32)[0].cuda().requires_grad_()
    eager = r.heads(x, 2, 1, q_norm=w)
    up = [rows(t.shape, 5).cuda() for t in eager]
    for call in (lambda: r.heads(x, 2, 1, q_norm=w), lambda: (r.rotate(x.unflatten(2, (4, 64)).transpose(1, 2), q_norm=w),)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        graph.replay()
        assert torch.equal(out[0][:, :2], eager[0])
        del out
        graph = torch.cuda.CUDAGraph()
        with pytest.raises(ValueError, match="eager graph"):
            with torch.cuda.graph(graph):
                torch.autograd.grad(call()[0].float().sum(), w)
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = r.heads_backward(*up, x, 2, 1, q_norm=w.detach())
    graph.replay()
    want, = torch.autograd.grad(eager, w, up)
    assert torch.equal(got[1], want)
    # another leaf of the same values, and the same one once the eager graph is gone
    torch.cuda.synchronize()
    alias = w.detach().requires_grad_()
    for leaf in (alias, w):
        if leaf is w:
            del eager
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got, = torch.autograd.grad(r.heads(x, 2, 1, q_norm=leaf), leaf, up)
        graph.replay()
        assert torch.equal(got, want)


def test_two_captured_backwards_at_once():
    """Two graphs of the same sizes share no workspace."""
    r, D = Rotary.from_base(64), 64
    w = [t.cuda() for t in weights(D, torch.float32)]
    sets = [[rows((2, 600, 4 * D), 60 + i).cuda()] + [rows((2, H, 600, D), 70 + i + H).cuda() for H in (2, 1, 1)] for i in range(2)]
    call = lambda t: r.heads_backward(*t[1:], t[0], 2, 1, q_norm=w[0], k_norm=w[1])  # noqa: E731
    want = [call(t) for t in sets]
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in sets], []
    for g, t in zip(graphs, sets):
        with torch.cuda.graph(g):
            outs.append(call(t))
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, want):
        for a, b in zip(got, ref):
            assert torch.equal(a, b)


def test_from_a_new_thread():
    import threading
    r, x = Rotary.from_base(64), rows((1, 40, 4 * 64), 2).cuda()
    want, got = r.heads(x, 2, 1), []
    torch.cuda.synchronize()
    t = threading.Thread(target=lambda: got.extend(r.heads(x, 2, 1)) or torch.cuda.synchronize())
    t.start()
    t.join()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements apart."""
    r, D = Rotary.from_base(64), 64
    far = torch.empty((1 << 31) + 4096, dtype=torch.bfloat16, device="cuda")
    x = rows((2, 3, 4 * D), 2)
    view = far.as_strided((2, 3, 4 * D), ((1 << 31) + 8, 4 * D, 1))
    view.copy_(x)
    for a, b in zip(r.heads(view, 2, 1), r.heads(x.cuda(), 2, 1)):
        assert torch.equal(a, b)


def test_many_tokens_of_one_head():
    """More rows than one wave of blocks holds, odd counts."""
    check_heads(Rotary.from_base(64), 7, 1771, 1, 1, 64, torch.float32)


def test_rows_past_32_bits_of_elements():
    """More than 2^31 elements in the input, the outputs and the gradient: rows at both ends and in the middle."""
    B, S, Hq, Hkv, D = 1, 270_001, 64, 1, 128
    r, w = Rotary.from_base(D), [t.cuda() for t in weights(D, torch.float32)]
    at = [0, 1, 131_072, 262_143, 262_145, S - 1]
    few = rows((1, len(at), (Hq + 2 * Hkv) * D), 5).cuda()
    x = torch.zeros((B, S, (Hq + 2 * Hkv) * D), dtype=torch.bfloat16, device="cuda")
    x[:, at] = few
    positions = torch.tensor(at, device="cuda")
    got, want = r.heads(x, Hq, Hkv, q_norm=w[0], k_norm=w[1]), r.heads(few, Hq, Hkv, positions=positions, q_norm=w[0], k_norm=w[1])
    for a, b in zip(got, want):
        assert torch.equal(a[:, :, at], b)
    up = [torch.zeros_like(t) for t in got]
    few_up = [rows(t.shape, 6 + i).cuda() for i, t in enumerate(want)]
    for t, u in zip(up, few_up):
        t[:, :, at] = u
    dx, dwq, dwk = r.heads_backward(*up, x, Hq, Hkv, q_norm=w[0], k_norm=w[1])
    want = r.heads_backward(*few_up, few, Hq, Hkv, positions=positions, q_norm=w[0], k_norm=w[1])
    assert torch.equal(dx[:, at], want[0]) and not dx[:, 2:1000].any()
    for a, b in zip((dwq, dwk), want[1:]):  # the same terms in another order
        assert float((a - b).abs().max()) <= 2.0 ** -17 * float(b.abs().max()) * len(at) * Hq


def test_two_threads_at_once():
    """Calls of one plan from two threads, each on a stream of its own."""
    import threading
    r = Rotary.by_parts(64, 4, 128)
    w = [t.cuda() for t in weights(64, torch.bfloat16)]
    xs = [rows((2, 64 + 3 * i, 6 * 64), 80 + i).cuda() for i in range(2)]
    call = lambda x: (*r.heads(x, 2, 2, q_norm=w[0], k_norm=w[1]), *r.heads_backward(*r.heads(x, 2, 2), x, 2, 2, q_norm=w[0], k_norm=w[1]))  # noqa: E731
    want = [call(x) for x in xs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(100):
                if not all(torch.equal(a, b) for a, b in zip(call(xs[i]), want[i])):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad


def test_rotate_backward_without_weight_gradients():
    r, w = Rotary.from_base(64), [t.cuda() for t in weights(64, torch.float32)]
    q, k = rows((2, 3, 20, 64), 1).cuda(), rows((2, 1, 20, 64), 2).cuda()
    dq, dk = rows(q.shape, 3).cuda(), rows(k.shape, 4).cuda()
    full = r.rotate_backward(dq, dk, q, k, q_norm=w[0], k_norm=w[1])
    bare = r.rotate_backward(dq, dk, q, k, q_norm=w[0], k_norm=w[1], weight_grads=False)
    assert torch.equal(full[0], bare[0]) and torch.equal(full[1], bare[1]) and bare[2] is None and bare[3] is None


def test_frozen_weights_under_autograd():
    """A norm's weight that needs no gradient gets none, the other does."""
    r, x = Rotary.from_base(64), rows((1, 30, 4 * 64), 2).cuda().requires_grad_()
    w = [t.cuda() for t in weights(64, torch.float32)]
    w[1].requires_grad_()
    out = r.heads(x, 2, 1, q_norm=w[0], k_norm=w[1])
    up = [rows(t.shape, 5).cuda() for t in out]
    dx, dwk = torch.autograd.grad(out, (x, w[1]), up)
    want = r.heads_backward(*up, x.detach(), 2, 1, q_norm=w[0], k_norm=w[1].detach())
    assert torch.equal(dx, want[0]) and torch.equal(dwk, want[2]) and w[0].grad is None


def test_inputs_changed_before_the_backward_are_noticed():
    r, x = Rotary.from_base(64), rows((1, 30, 4 * 64), 2).cuda()
    w = weights(64, torch.float32)[0].cuda().requires_grad_()
    at = torch.arange(30, device="cuda")
    q = r.heads(x, 2, 1, positions=at, q_norm=w)[0]
    at.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        q.float().sum().backward()


@pytest.mark.parametrize("norm", [False, True])
def test_saved_tensors_that_move(norm):
    """Hooks that keep what is saved elsewhere and bring it back as another tensor, dense where it was a view, while the
    positions of the forward are gone."""
    r = Rotary.from_base(64)
    wide = rows((3, 40, 9 * 64), 2).cuda()
    w = [t.cuda().requires_grad_() for t in weights(64, torch.float32)] if norm else [None, None]
    up = [rows((3, H, 40, 64), 5 + H).cuda() for H in (2, 1, 1)]

    def step():
        x = wide.clone().requires_grad_()
        view = x[:, :, 64:320]
        q, k, v = r.heads(view, 2, 1, positions=torch.arange(40, device="cuda") * 3, q_norm=w[0], k_norm=w[1])
        h = view.unflatten(2, (4, 64)).transpose(1, 2)
        q2, k2 = r.rotate(h[:, :2], h[:, 2:3], positions=torch.arange(40, device="cuda") + 7, q_norm=w[0], k_norm=w[1])
        torch.full((1 << 16,), -1, dtype=torch.int64, device="cuda")  # where the positions were
        return torch.autograd.grad((q, k, v, q2, k2), [x, *(t for t in w if norm)], (*up, up[0], up[1]))

    want = step()
    with torch.autograd.graph.save_on_cpu():
        got = step()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_what_is_kept_for_the_backward():
    """Without norms the projection's output is not."""
    r, x = Rotary.from_base(64), rows((1, 30, 4 * 64), 2).cuda().requires_grad_()
    h = x.unflatten(2, (4, 64)).transpose(1, 2)
    kept = lambda out: [t for t in out[0].grad_fn.saved_tensors if t is not None]  # noqa: E731
    assert kept(r.heads(x, 2, 1)) == [] and kept(r.rotate(h[:, :2], h[:, 2:3])) == []
    w = torch.ones(64, device="cuda")
    assert len(kept(r.heads(x, 2, 1, q_norm=w))) == 2 and len(kept(r.rotate(h[:, :2], h[:, 2:3], k_norm=w))) == 3


@pytest.mark.parametrize("which", ["q", "k", "v", "qk", "qv", "kv", "qkv"])
@pytest.mark.parametrize("packed", [False, True])
def test_c_calls_of_some_tensors(which, packed):
    """Any of q, k and v, from a projection's output to new tensors or in place, and the gradients of the same ones."""
    from causal_scaled_dot_gb300.native import AttnHeads
    r, lib = Rotary.from_base(32), native.load()
    B, S, Hq, Hkv, D = 2, 45, 3, 2, 64
    x = rows((B, S, 7 * D), 3).cuda()
    w = [t.cuda() for t in weights(D, torch.bfloat16)]
    want = r.heads(x, Hq, Hkv, q_norm=w[0], k_norm=w[1])
    c = r._plan(x.device, B, S, D, None, 0, *w, EPS)
    split_ = lambda t: (lambda h: (h[:, :Hq], h[:, Hq:Hq + Hkv], h[:, Hq + Hkv:]))(t.unflatten(2, (7, D)).transpose(1, 2))  # noqa: E731
    some = lambda ts: c_heads(*(t if n in which else None for n, t in zip("qkv", ts)))  # noqa: E731
    st = torch.cuda.current_stream().cuda_stream
    held = x.clone()
    to = split_(held) if packed else tuple(torch.full_like(t, 7.0) for t in want)
    assert lib.attn_rope(c, some(split_(held)), some(to), B, Hq, Hkv, S, D, st) == 0
    for n, got, ref, was in zip("qkv", to, want, split_(x)):
        assert torch.equal(got, ref if n in which else was if packed else torch.full_like(ref, 7.0))
    up = [rows(t.shape, 8).cuda() for t in want]
    dx = r.heads_backward(*up, x, Hq, Hkv, q_norm=w[0], k_norm=w[1], weight_grads=False)[0]
    out = torch.full_like(x, 7.0)
    assert isinstance(some(up), AttnHeads)
    assert lib.attn_rope_bwd(c, some(up), some(split_(x)), some(split_(out)), None, None, B, Hq, Hkv, S, D, None, 0, st) == 0
    for n, got, ref in zip("qkv", split_(out), split_(dx)):
        assert torch.equal(got, ref if n in which else torch.full_like(ref, 7.0))


def test_captured_after_a_warm_up_whose_results_live():
    """The usual way: a few steps on a side stream, whose last results are still held, then the capture of a whole step with
    .backward() into the leaves' gradients."""
    r, D, S = Rotary.from_base(64), 64, 96
    x = rows((1, S, 4 * D), 2).cuda()
    w = [t.cuda().requires_grad_() for t in weights(D, torch.float32)]

    def step():
        q, k, v = r.heads(x, 2, 1, q_norm=w[0], k_norm=w[1])
        o = native.attention_trainable(q, k, v)
        (o.float() ** 2).sum().backward()
        return q, k, v, o

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            for t in w:
                t.grad = None
            held = step()
    torch.cuda.current_stream().wait_stream(s)
    for t in w:
        t.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    grads = [t.grad for t in w]
    for i in range(2):
        x.copy_(rows(x.shape, 30 + i).cuda())
        graph.replay()
        torch.cuda.synchronize()
        alias = [t.detach().requires_grad_() for t in w]
        q, k, v = r.heads(x, 2, 1, q_norm=alias[0], k_norm=alias[1])
        o = native.attention_trainable(q, k, v)
        want = torch.autograd.grad((o.float() ** 2).sum(), alias)
        assert torch.equal(got[3], o)
        for a, b in zip(grads, want):
            assert torch.equal(a, b)
        del q, k, v, o
    assert all(t.isfinite().all() for t in held)
