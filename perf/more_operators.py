"""Cases that measure what stands between a layer's QKV projection and its attention: norms of queries and
keys per head, rotary positions, the change to the attention's layout, and the append to the 8-bit cache.

A row is one head of one token: D elements x at position p.  Its pairs are rotated by a_i = p f_i:

* half layout: pairs (i, i + rot/2), interleaved: pairs (2i, 2i + 1), i < rot/2; the elements from rot on stay;
* y_a = m (u_a cos a - u_b sin a), y_b = m (u_b cos a + u_a sin a), where u = x, or with a norm
  u_d = x_d w_d / sqrt(mean(x^2) + eps) over the whole head.
* f_i = base^(-2i/rot); with a stretch s > 1 over an original length L, t_i = L f_i / (2 pi) and
  g = clamp((t_i - 1) / 31, 0, 1), f_i is multiplied by g + (1 - g) / s, and m = 0.1 ln s + 1 (else m = 1).

fwd: the projection's output [B, S, (Hq + 2 Hkv) D] (or q and k [B, S, H, D] by themselves) to contiguous
q, k, v [B, H, S, D].  bwd: upstream gradients of those to the gradient of the projection's output and of the
norms' weights.  step: both, through autograd.  append: the step's tokens into the paged 8-bit cache (K rotated
and rounded once, to its code), and the rotated q; the cache as in ``operators.py``, a token's position its place.

``run`` computes each in elementary torch operations, or with ``own`` set calls the library."""
import math
import random

import torch

own = False
EPS = 1e-6
LENGTH = 4096  # the original length L of stretched positions


def listed():
    def case(name, op, B, S, Hq, Hkv, D, rot, interleaved=False, norm="", packed=True, stretch=1.0, first=0, docs=False,
             block=0, ctx=0, ragged=False):
        return dict(name=name, op=op, B=B, S=S, Hq=Hq, Hkv=Hkv, D=D, rot=rot, interleaved=interleaved, norm=norm, packed=packed,
                    stretch=stretch, first=first, docs=docs, block=block, ctx=ctx, ragged=ragged)

    return [
        # The smallest workload's layer before its attention: launch and latency.
        case("rotate_small", "fwd", 1, 256, 2, 2, 64, 64),
        # The profiling workload's layer.
        case("rotate_profile", "fwd", 4, 4096, 16, 16, 128, 128),
        # The long workload, q and k from projections of their own, half of each head rotated in neighbouring
        # pairs, positions stretched and far from the start (a chunk of a very long prompt).
        case("rotate_long_part", "fwd", 2, 8192, 32, 32, 128, 64, True, packed=False, stretch=16.0, first=57001),
        # The grouped-query workload's gradients on their way back to the projection.
        case("rotate_bwd_gqa", "bwd", 2, 4096, 32, 8, 128, 128),
        # A few tokens of a small model with norms, odd sizes.
        case("norm_small_d64", "fwd", 1, 37, 12, 4, 64, 32, True, "fp32"),
        # The 7B layer's forward with norms of its queries and keys.
        case("norm_7b", "fwd", 1, 2048, 32, 32, 128, 128, norm="bf16"),
        # A training step of the grouped-query workload: forward, then gradients of the projection and the norms.
        case("norm_step_gqa", "step", 2, 4096, 32, 8, 128, 128, norm="bf16"),
        # Gradients of packed documents whose positions start over, odd lengths, heads of 64.
        case("norm_bwd_docs_d64", "bwd", 3, 1237, 12, 4, 64, 64, norm="fp32", docs=True),
        # One token of the 7B layer enters its cache: latency counts.
        case("append_token_7b", "append", 1, 1, 32, 32, 128, 128, block=64, ctx=2048),
        # One token for each sequence of a serving batch, with norms, uneven lengths.
        case("append_token_b64", "append", 64, 1, 32, 8, 128, 128, norm="bf16", block=64, ctx=4096, ragged=True),
        # Two whole prompts of the grouped-query workload.
        case("append_prompt_gqa", "append", 2, 4096, 32, 8, 128, 128, norm="bf16", block=64, ctx=4096),
        # Chunks of uneven prompts (padded batch), small pages, part of each head in neighbouring pairs.
        case("append_chunk_d64", "append", 8, 700, 16, 4, 64, 32, True, block=16, ctx=2500, ragged=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("fwd", "bwd", "step", "append")}
    while True:
        op = rng.choice(["fwd", "fwd", "bwd", "step", "append", "append"])
        Hkv, D = rng.choice([1, 2, 3, 4, 8, 16, 32]), rng.choice([64, 128])
        append = op == "append"
        ctx = _spread(rng, 17, 65536) if append else 0
        S = 1 if append and rng.random() < 0.5 else _spread(rng, 1, min(ctx, 4096) if append else 8192)
        case = dict(op=op, B=_spread(rng, 1, 64), S=S, Hq=Hkv * rng.choice([1, 2, 3, 4, 5, 8]), Hkv=Hkv, D=D,
                    rot=rng.choice([D, D, D, D // 2, D // 4, 48]), interleaved=rng.random() < 0.4,
                    norm=rng.choice(["", "bf16", "fp32"]), packed=append or rng.random() < 0.7,
                    stretch=rng.choice([1.0, 1.0, 4.0, 32.0]), first=0 if append else rng.choice([0, 0, _spread(rng, 1, 1 << 20)]),
                    docs=not append and rng.random() < 0.3, block=rng.choice([16, 32, 64, 128]) if append else 0, ctx=ctx,
                    ragged=append and rng.random() < 0.6)
        if case["B"] * ctx * Hkv * D <= 1 << 28 and _cost(case) <= top[op]:
            return case


def _lens(case):
    """(tokens held, new tokens) of each sequence.  Uneven batches have one idle slot from three sequences on."""
    B, S, ctx = case["B"], case["S"], case["ctx"]
    if not case["ragged"]:
        return [ctx] * B, [S] * B
    rng = random.Random(B * 1000003 + ctx * 1009 + S)
    lens = [ctx] + [rng.randint(max(1, ctx // 4), ctx) for _ in range(B - 1)]
    new = [S] + [rng.randint(1, S) for _ in range(B - 1)]
    if B >= 3:
        lens[1] = 0
    return lens, [min(n, t) for n, t in zip(new, lens)]


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 60e12)


def work(case):
    """Bytes: each input once, each output once.  Operations: 3 an element rotated, 4 one that is normed, 8 its gradient."""
    D, Hq, Hkv, op = case["D"], case["Hq"], case["Hkv"], case["op"]
    normed = 1 if case["norm"] else 0
    if op == "append":
        lens, new = _lens(case)
        tokens = sum(new)
        pages = sum(-(-t // case["block"]) - (t - n) // case["block"] for t, n in zip(lens, new) if n)
        return {"bytes": tokens * D * (4 * Hq + 6 * Hkv) + 8 * pages * Hkv + 8 * case["B"],
                "flops": tokens * D * ((Hq + Hkv) * (3 + 4 * normed) + 4 * Hkv)}
    tokens = case["B"] * case["S"]
    qk, v = tokens * (Hq + Hkv) * D, tokens * Hkv * D if case["packed"] else 0
    positions = 8 * tokens if case["docs"] else 0
    fwd = {"bytes": 4 * (qk + v) + positions, "flops": qk * (3 + 4 * normed)}
    bwd = {"bytes": (4 + 2 * normed) * qk + 4 * v + positions, "flops": qk * (3 + 8 * normed)}
    if op == "step":
        return {k: fwd[k] + bwd[k] for k in fwd}
    return fwd if op == "fwd" else bwd


def _values(g, shape, sigma):
    """bf16 rows as a projection gives them: heads of different size, a few strong channels."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= sigma * (1 + 4 * (torch.rand(shape[-1], generator=g, device="cuda") > 0.97))
    return x.to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, S, Hq, Hkv, D, op = (case[x] for x in ("B", "S", "Hq", "Hkv", "D", "op"))
    st = dict(case=case, q_norm=None, k_norm=None, positions=None)
    if case["packed"]:
        st["qkv"] = _values(g, (B, S, (Hq + 2 * Hkv) * D), 1.2)
    else:
        st["q"], st["k"] = _values(g, (B, S, Hq, D), 1.2), _values(g, (B, S, Hkv, D), 1.0)
    if case["norm"]:
        weight = lambda: (0.6 + 0.8 * torch.rand(D, generator=g, device="cuda")).to(  # noqa: E731
            torch.bfloat16 if case["norm"] == "bf16" else torch.float32)
        st["q_norm"], st["k_norm"] = weight(), weight()
    if case["docs"]:  # documents one after another, each from position `first` on
        start = torch.rand((B, S), generator=g, device="cuda") < 4.0 / S
        at = torch.arange(S, device="cuda").expand(B, S)
        st["positions"] = case["first"] + at - torch.cummax(torch.where(start, at, 0), 1).values
    if op in ("bwd", "step"):
        up = lambda H: torch.randn((B, H, S, D), generator=g, device="cuda").mul(0.05).to(torch.bfloat16)  # noqa: E731
        st["dq"], st["dk"] = up(Hq), up(Hkv)
        st["dv"] = up(Hkv) if case["packed"] else None
    if op == "append":
        lens, new = _lens(case)
        per = -(-case["ctx"] // case["block"])
        total = B * per + 3
        st["block"] = case["block"]
        st["k_cache"], st["k_scale"] = _codes(g, (total, Hkv, case["block"], D), 1.0)
        st["v_cache"], st["v_scale"] = _codes(g, (total, Hkv, case["block"], D), 0.7)
        st["table"] = torch.randperm(total, generator=g, device="cuda")[:B * per].view(B, per).to(torch.int32)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["new"] = torch.tensor(new, dtype=torch.int32, device="cuda") if new != [S] * B else None
        st["q_out"] = torch.zeros((B, Hq, S, D), dtype=torch.bfloat16, device="cuda")
    if own:  # the plan of the model's positions, and the handle over its cache
        from causal_scaled_dot_gb300.rotary import Rotary
        if case["stretch"] > 1:
            st["rotary"] = Rotary.by_parts(case["rot"], case["stretch"], LENGTH, interleaved=case["interleaved"])
        else:
            st["rotary"] = Rotary.from_base(case["rot"], interleaved=case["interleaved"])
        if op == "append":
            from causal_scaled_dot_gb300.kv_cache import KVCache
            st["cache"] = KVCache(st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["table"], st["lens"])
    if op == "step":
        for x in ("qkv", "q", "k", "q_norm", "k_norm"):
            if st.get(x) is not None:
                st[x].requires_grad_()
    return st


def _codes(g, shape, sigma):
    """Pages as an earlier write left them."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= sigma * (0.5 + torch.rand((1, shape[1], 1, 1), generator=g, device="cuda"))
    s = _scale_of(x.abs().amax((2, 3)))
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn), s


def _scale_of(amax):
    """The smallest power of two s (at least 2^-126) with amax <= 448 s."""
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.ldexp(torch.ones_like(amax), e.clamp(min=-126))


# ------------------------------------------------------------------ the plain form
def _frequencies(case):
    """fp64 [rot / 2] and the factor m."""
    i = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
    f, s = 10000.0 ** (-2 * i / case["rot"]), case["stretch"]
    if s == 1:
        return f, 1.0
    g = ((LENGTH * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
    return f * (g + (1 - g) / s), 0.1 * math.log(s) + 1


def _waves(case, positions):
    """m cos and m sin [B or 1, 1, S, rot / 2] in fp32, from angles in fp64."""
    f, m = _frequencies(case)
    a = positions.double()[:, None, :, None] * f
    return (m * torch.cos(a)).float(), (m * torch.sin(a)).float()


def _split(case, x):
    """The parts (a, b, rest) of a head."""
    r = case["rot"]
    if case["interleaved"]:
        return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]
    return x[..., :r // 2], x[..., r // 2:r], x[..., r:]


def _join(case, a, b, rest):
    pairs = torch.stack((a, b), -1).flatten(-2) if case["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((pairs, rest), -1)


def _turn(case, x, cos, sin):
    a, b, rest = _split(case, x)
    return _join(case, a * cos - b * sin, b * cos + a * sin, rest)


def _forward(case, x, weight, cos, sin):
    """fp32 y of bf16 rows x [B, H, S, D]."""
    x = x.float()
    if weight is not None:
        x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * weight.float()
    return _turn(case, x, cos, sin)


def _backward(case, dy, x, weight, cos, sin):
    """The gradient of a row, bf16, and of the weight in its type."""
    d = _turn(case, dy.float(), cos, -sin)
    if weight is None:
        return d.to(torch.bfloat16), None
    x = x.float()
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    n = x * r
    dw = (d * n).double().sum((0, 1, 2))
    d = d * weight.float()
    return (r * (d - n * (d * n).mean(-1, keepdim=True))).to(torch.bfloat16), dw.to(weight.dtype)


def _heads(case, qkv):
    """q, k, v [B, H, S, D] of the projection's output."""
    B, S, Hq, Hkv, D = (case[x] for x in ("B", "S", "Hq", "Hkv", "D"))
    x = qkv.detach().view(B, S, Hq + 2 * Hkv, D).transpose(1, 2)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]


def _rows(case, st):
    if case["packed"]:
        return _heads(case, st["qkv"])
    return st["q"].detach().transpose(1, 2), st["k"].detach().transpose(1, 2), None


def _positions(case, st):
    if st["positions"] is not None:
        return st["positions"]
    return case["first"] + torch.arange(case["S"], device="cuda")[None]


def _plain_fwd(st):
    case = st["case"]
    q, k, v = _rows(case, st)
    cos, sin = _waves(case, _positions(case, st))
    out = {"q": _forward(case, q, st["q_norm"], cos, sin).to(torch.bfloat16),
           "k": _forward(case, k, st["k_norm"], cos, sin).to(torch.bfloat16)}
    if v is not None:
        out["v"] = v.contiguous()
    return out


def _plain_bwd(st):
    case = st["case"]
    q, k, v = _rows(case, st)
    cos, sin = _waves(case, _positions(case, st))
    dq, dq_norm = _backward(case, st["dq"], q, st["q_norm"], cos, sin)
    dk, dk_norm = _backward(case, st["dk"], k, st["k_norm"], cos, sin)
    if v is None:
        out = {"dq": dq.transpose(1, 2).contiguous(), "dk": dk.transpose(1, 2).contiguous()}
    else:
        out = {"dqkv": torch.cat((dq, dk, st["dv"]), 1).transpose(1, 2).reshape(st["qkv"].shape)}
    return {**out, "dq_norm": dq_norm, "dk_norm": dk_norm}


def _plain_append(st):
    case, block, S = st["case"], st["block"], st["case"]["S"]
    q, k, v = _heads(case, st["qkv"])
    lens = st["lens"].long()
    new = st["new"].long() if st["new"] is not None else torch.full_like(lens, S)
    step = torch.arange(S, device="cuda")
    pos = (lens - new)[:, None] + step
    cos, sin = _waves(case, pos)
    mine = step < new[:, None]
    st["q_out"].copy_(torch.where(mine[:, None, :, None], _forward(case, q, st["q_norm"], cos, sin).to(torch.bfloat16), st["q_out"]))
    b, s = torch.nonzero(mine, as_tuple=True)
    page, slot = st["table"][b, pos[b, s] // block].long(), pos[b, s] % block
    begin = lens - new
    held = begin % block  # tokens that the first block holds already
    part = torch.nonzero((held > 0) & (lens > begin), as_tuple=True)[0]
    part_page, old = st["table"][part, begin[part] // block].long(), torch.arange(block, device="cuda") < held[part, None]

    def one(code, scale, x):
        x = x[b, :, s]
        amax = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")
        before = torch.zeros_like(scale)
        before[part_page] = scale[part_page]
        fresh = torch.maximum(_scale_of(amax), before)
        bits = code.view(torch.uint8)
        had = bits[part_page].view(torch.float8_e4m3fn).float()
        moved = (had * (scale[part_page] / fresh[part_page])[:, :, None, None]).to(torch.float8_e4m3fn)
        bits[part_page] = torch.where(old[:, None, :, None], moved.view(torch.uint8), bits[part_page])
        bits[page, :, slot] = (x / fresh[page][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scale[page] = fresh[page]

    one(st["k_cache"], st["k_scale"], _forward(case, k, st["k_norm"], cos, sin))
    one(st["v_cache"], st["v_scale"], v.float())
    return {x: st[x] for x in ("q_out", "k_cache", "v_cache", "k_scale", "v_scale")}


# ------------------------------------------------------------------ the library's calls
def _own_fwd(st):
    case = st["case"]
    more = dict(positions=st["positions"], first=case["first"] if st["positions"] is None else 0, q_norm=st["q_norm"],
                k_norm=st["k_norm"], eps=EPS)
    if case["packed"]:
        q, k, v = st["rotary"].heads(st["qkv"], case["Hq"], case["Hkv"], **more)
        return {"q": q, "k": k, "v": v}
    q, k = st["rotary"].rotate(st["q"].transpose(1, 2), st["k"].transpose(1, 2), **more)
    return {"q": q, "k": k}


def _own_bwd(st):
    case = st["case"]
    more = dict(positions=st["positions"], first=case["first"] if st["positions"] is None else 0, q_norm=st["q_norm"],
                k_norm=st["k_norm"], eps=EPS)
    if case["packed"]:
        dqkv, dq_norm, dk_norm = st["rotary"].heads_backward(st["dq"], st["dk"], st["dv"], st["qkv"], case["Hq"], case["Hkv"], **more)
        return {"dqkv": dqkv, "dq_norm": dq_norm, "dk_norm": dk_norm}
    dq, dk, dq_norm, dk_norm = st["rotary"].rotate_backward(st["dq"], st["dk"], st["q"].transpose(1, 2), st["k"].transpose(1, 2),
                                                            **more)
    return {"dq": dq.transpose(1, 2), "dk": dk.transpose(1, 2), "dq_norm": dq_norm, "dk_norm": dk_norm}


def _own_step(st):
    out = _own_fwd(st)
    names = [x for x in ("qkv", "q", "k", "q_norm", "k_norm") if st.get(x) is not None]
    grads = torch.autograd.grad(list(out.values()), [st[x] for x in names], [st["d" + x] for x in out])
    return {**{x: y.detach() for x, y in out.items()}, **{"d" + x: y for x, y in zip(names, grads)}}


def _own_append(st):
    case = st["case"]
    B, S, Hq, Hkv, D = (case[x] for x in ("B", "S", "Hq", "Hkv", "D"))
    x = st["qkv"].view(B, S, Hq + 2 * Hkv, D).transpose(1, 2)
    st["cache"].append(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], st["rotary"], q=x[:, :Hq], new_lens=st["new"], q_norm=st["q_norm"],
                       k_norm=st["k_norm"], eps=EPS, q_out=st["q_out"])
    return {x: st[x] for x in ("q_out", "k_cache", "v_cache", "k_scale", "v_scale")}


def run(st):
    op = st["case"]["op"]
    if own:
        return {"fwd": _own_fwd, "bwd": _own_bwd, "step": _own_step, "append": _own_append}[op](st)
    if op == "step":
        return {**_plain_fwd(st), **_plain_bwd(st)}
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "append": _plain_append}[op](st)


# ------------------------------------------------------------------ 64 bits
def _complex_turn(case, x, positions):
    """Rows [B, H, S, D] in float64 with each pair as a complex number times m exp(i a)."""
    rot, s = case["rot"], case["stretch"]
    rates, m = [], 1.0
    for i in range(rot // 2):
        f = math.exp(-2 * i / rot * math.log(10000.0))
        if s > 1:
            keep = min(1.0, max(0.0, (LENGTH * f / math.tau - 1) / 31))
            f, m = f * keep + f / s * (1 - keep), 1 + math.log(s) / 10
        rates.append(f)
    angle = positions.double()[:, None, :, None] * torch.tensor(rates, dtype=torch.float64, device="cuda")
    shape = (rot // 2, 2) if case["interleaved"] else (2, rot // 2)
    z = x[..., :rot].unflatten(-1, shape)
    z = torch.view_as_complex((z if case["interleaved"] else z.transpose(-1, -2)).contiguous())
    z = torch.view_as_real(z * torch.polar(torch.full_like(angle, m), angle))
    z = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
    return torch.cat((z, x[..., rot:]), -1)


def _exact_heads(case, rows, weights, positions):
    """Normed and rotated float64 rows; what is None stays so."""
    for x, w in zip(rows, weights):
        if x is not None and w is not None:
            x = x / torch.linalg.vector_norm(torch.cat((x, x.new_full((*x.shape[:-1], 1), math.sqrt(EPS * x.shape[-1]))), -1),
                                             dim=-1, keepdim=True) * math.sqrt(x.shape[-1]) * w
        yield None if x is None else _complex_turn(case, x, positions)


def exact(case, seed):
    st = prepare(case, seed)
    B, S, Hq, Hkv, D, op = (case[x] for x in ("B", "S", "Hq", "Hkv", "D", "op"))
    leaf = {x: st[x].detach().double().requires_grad_(op in ("bwd", "step")) for x in ("qkv", "q", "k", "q_norm", "k_norm")
            if st.get(x) is not None}
    if case["packed"]:
        parts = leaf["qkv"].split([Hq * D, Hkv * D, Hkv * D], -1)
        q, k, v = (x.unflatten(-1, (-1, D)).permute(0, 2, 1, 3) for x in parts)
    else:
        q, k, v = leaf["q"].permute(0, 2, 1, 3), leaf["k"].permute(0, 2, 1, 3), None
    if op == "append":
        return _exact_append(case, st, q, k, v, leaf)
    positions = st["positions"] if case["docs"] else torch.arange(case["first"], case["first"] + S, device="cuda")[None]
    y = dict(zip("qk", _exact_heads(case, (q, k), (leaf.get("q_norm"), leaf.get("k_norm")), positions)))
    if v is not None:
        y["v"] = v
    out = {x: t.detach() for x, t in y.items()} if op != "bwd" else {}
    if op != "fwd":
        grads = torch.autograd.grad(list(y.values()), list(leaf.values()), [st["d" + x].double() for x in y])
        out.update({"d" + x: t for x, t in zip(leaf, grads)})
    if op == "bwd":
        out = {"dq_norm": None, "dk_norm": None, **out}
    return out


def _exact_append(case, st, q, k, v, leaf):
    """Codes as the quotients x / s before their rounding."""
    lens, new = _lens(case)
    block, table = case["block"], st["table"].tolist()
    out = {"q_out": torch.zeros_like(st["q_out"], dtype=torch.float64), "k_scale": st["k_scale"].double(),
           "v_scale": st["v_scale"].double(), "k_cache": st["k_cache"].double(), "v_cache": st["v_cache"].double()}
    for b, (t, n) in enumerate(zip(lens, new)):
        if n == 0:
            continue
        at = torch.arange(t - n, t, device="cuda")[None]
        y = dict(zip("qk", _exact_heads(case, (q[b:b + 1, :, :n], k[b:b + 1, :, :n]), (leaf.get("q_norm"), leaf.get("k_norm")), at)))
        out["q_out"][b, :, :n] = y["q"][0]
        for name, x in (("k", y["k"][0]), ("v", v[b, :, :n])):
            code, scale = out[name + "_cache"], out[name + "_scale"]
            for column in range((t - n) // block, -(-t // block)):
                lo, hi, page = max(t - n, column * block), min(t, column * block + block), table[b][column]
                rows = x[:, lo - (t - n):hi - (t - n)]
                big = rows.abs().amax((1, 2)).clamp(min=2.0 ** -118)
                need = torch.exp2(torch.ceil(torch.log2(big / 448)))
                need = torch.where(big > 448 * need, 2 * need, torch.where(big <= 224 * need, need / 2, need))
                held = lo - column * block
                if held:
                    need = torch.maximum(need, scale[page])
                    code[page, :, :held] *= (scale[page] / need)[:, None, None]
                code[page, :, held:held + hi - lo] = rows / need[:, None, None]
                scale[page] = need
    return out
