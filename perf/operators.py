"""Cases that measure the 8-bit key/value cache: writing it, reading it back, and attention over it.

The cache is paged.  A page ("block") holds ``block`` tokens of every key/value head as E4M3 codes,
[num_blocks, Hkv, block, D], with one fp32 scale per block and head for K and one for V; a token's
value is code * scale.  ``table`` [B, max_blocks] names each sequence's pages in order, and
``lens`` [B] counts the tokens each sequence holds, those of the current call included: the n_b new
tokens (or queries) of sequence b sit at positions lens[b] - n_b .. lens[b] - 1.

* write: new tokens k, v (bf16 [B, Hkv, S, D]) into the cache.  The scale of a block and head is the
  smallest power of two s with max|x| <= 448 s over its tokens; a block that already holds tokens
  keeps its scale unless a new token needs a larger one, and its codes then move to that scale.
* read: positions first .. first + S - 1 back as bf16 [B, Hkv, S, D]; rows past a sequence's end stay.
* attend: O = softmax(scale q K^T) V and the rows' log-sum-exp, query head h reading key/value head
  h / (Hq / Hkv); a query at position p sees keys 0 .. p.  A row that sees no key gives O = 0 and
  LSE = -inf; rows past a sequence's own query count stay as they were.

``run`` computes each in elementary torch operations, or with ``own`` set calls the library."""
import math
import random

import numpy as np
import torch

own = False


def listed():
    def case(name, op, B, Hq, Hkv, D, block, S, ctx, ragged, first=0):
        return dict(name=name, op=op, B=B, Hq=Hq, Hkv=Hkv, D=D, block=block, S=S, ctx=ctx, ragged=ragged, first=first)

    return [
        # Two whole prompts of the grouped-query workload enter the cache after their forward pass.
        case("write_prompt_gqa", "write", 2, 32, 8, 128, 64, 4096, 4096, False),
        # One token for each sequence of a serving batch, in the middle of its block: latency counts.
        case("write_token_b64", "write", 64, 32, 8, 128, 64, 1, 2048, True),
        # Chunks of uneven prompts (padded batch), small pages, starting inside a block.
        case("write_chunk_d64", "write", 8, 16, 16, 64, 16, 700, 2500, True),
        # The grouped-query workload's cache read back whole, for a bf16 pass over it.
        case("read_prompt_gqa", "read", 2, 32, 8, 128, 64, 4096, 4096, False),
        # A short stretch in the middle of uneven sequences.
        case("read_stretch_d64", "read", 3, 4, 2, 64, 16, 500, 900, True, 100),
        # The smallest workload's heads, one token: launch and latency.
        case("attend_token_small", "attend", 1, 2, 2, 64, 16, 1, 256, False),
        # One token of the 7B layer (32 heads of their own) at its sequence length.
        case("attend_token_7b", "attend", 1, 32, 32, 128, 64, 1, 2048, False),
        # One token for each sequence of a serving batch, grouped heads, uneven lengths.
        case("attend_token_b64", "attend", 64, 32, 8, 128, 64, 1, 4096, True),
        # Few sequences with very long caches: the keys are split over the machine and joined.
        case("attend_token_long", "attend", 2, 32, 8, 128, 128, 1, 131072, False),
        # A few drafted tokens to verify in each sequence, uneven counts.
        case("attend_draft_b16", "attend", 16, 32, 8, 128, 32, 5, 8192, True),
        # A prompt's next chunk over what is cached: the long workload's length.
        case("attend_chunk", "attend", 2, 32, 8, 128, 64, 1024, 8192, False),
        # Odd chunk, odd lengths, heads of 64, small pages.
        case("attend_chunk_d64", "attend", 3, 12, 4, 64, 16, 333, 3001, True),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo .. hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("write", "read", "attend")}
    while True:
        op = rng.choice(["write", "read", "attend", "attend", "attend"])
        Hkv = rng.choice([1, 2, 3, 4, 8, 16, 32])
        group = rng.choice([1, 2, 3, 4, 5, 8]) if op == "attend" else 1
        ctx = _spread(rng, 17, 65536)
        S = 1 if op == "attend" and rng.random() < 0.5 else _spread(rng, 1, min(ctx, 1024 if op == "attend" else 4096))
        case = dict(op=op, B=_spread(rng, 1, 64), Hq=Hkv * group, Hkv=Hkv, D=rng.choice([64, 128]),
                    block=rng.choice([16, 32, 64, 128]), S=S, ctx=ctx, ragged=rng.random() < 0.6,
                    first=rng.randrange(ctx) if op == "read" else 0)
        cells = case["B"] * ctx * Hkv * case["D"]
        scores = case["B"] * case["Hq"] * S * ctx
        if cells <= 1 << 28 and scores <= 1 << 29 and _cost(case) <= top[op]:
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
    return lens, [min(n, t) if S > 1 else 1 for n, t in zip(new, lens)]


def _reads(case):
    lens, _ = _lens(case)
    return [max(0, min(t - case["first"], case["S"])) for t in lens]


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def work(case):
    lens, new = _lens(case)
    D, Hkv, Hq = case["D"], case["Hkv"], case["Hq"]
    pages = lambda a, n: -(-(a + n) // case["block"]) - a // case["block"] if n else 0  # noqa: E731
    if case["op"] == "write":
        new = [min(n, t) for n, t in zip(new, lens)]
        tokens = sum(new)
        scales = sum(pages(t - n, n) for n, t in zip(new, lens))
        return {"bytes": 2 * Hkv * (tokens * D * 3 + 4 * scales) + 8 * case["B"], "flops": 4 * tokens * Hkv * D}
    if case["op"] == "read":
        count = _reads(case)
        scales = sum(pages(case["first"], n) for n in count)
        return {"bytes": 2 * Hkv * (sum(count) * D * 3 + 4 * scales) + 4 * case["B"], "flops": 2 * sum(count) * Hkv * D}
    rows = sum(new)
    pairs = sum(n * t - n * (n - 1) // 2 for n, t in zip(new, lens) if t >= n)
    nbytes = 2 * Hkv * (sum(lens) * D + 4 * sum(pages(0, t) for t in lens)) + rows * Hq * (4 * D + 4)
    return {"bytes": nbytes + 8 * case["B"], "flops": 4 * pairs * Hq * D}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, Hkv, D, block, S = (case[x] for x in ("B", "Hkv", "D", "block", "S"))
    lens, new = _lens(case)
    per = -(-case["ctx"] // block)
    total = B * per + 3

    def codes(sigma):
        """Pages as an earlier write left them: heads of different size, a few strong channels."""
        x = torch.randn((total, Hkv, block, D), generator=g, device="cuda")
        x *= sigma * (0.5 + torch.rand((1, Hkv, 1, 1), generator=g, device="cuda"))
        x *= 1 + 2 * (torch.rand((1, Hkv, 1, D), generator=g, device="cuda") > 0.97)
        s = _scale_of(x.abs().amax((2, 3)))
        return (x / s[:, :, None, None]).to(torch.float8_e4m3fn), s

    st = dict(case=case, block=block, S=S, first=case["first"])
    st["k"], st["k_scale"] = codes(1.0)
    st["v"], st["v_scale"] = codes(0.7)
    st["table"] = torch.randperm(total, generator=g, device="cuda")[:B * per].view(B, per).to(torch.int32)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["new"] = torch.tensor(new, dtype=torch.int32, device="cuda") if new != [S] * B else None
    if case["op"] == "write":
        st["k_new"] = torch.randn((B, Hkv, S, D), generator=g, device="cuda").mul(1.2).to(torch.bfloat16)
        st["v_new"] = torch.randn((B, Hkv, S, D), generator=g, device="cuda").mul(0.8).to(torch.bfloat16)
    elif case["op"] == "read":
        st["k_out"] = torch.zeros((B, Hkv, S, D), dtype=torch.bfloat16, device="cuda")
        st["v_out"] = torch.zeros_like(st["k_out"])
    else:
        st["q"] = torch.randn((B, case["Hq"], S, D), generator=g, device="cuda").to(torch.bfloat16)
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros((B, case["Hq"], S), dtype=torch.float32, device="cuda")
    if own:  # the handle that a serving program keeps over its cache tensors
        from causal_scaled_dot_gb300.kv_cache import KVCache
        st["cache"] = KVCache(st["k"], st["v"], st["k_scale"], st["v_scale"], st["table"], st["lens"])
    return st


def _scale_of(amax):
    """The smallest power of two s (at least 2^-126) with amax <= 448 s."""
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.ldexp(torch.ones_like(amax), e.clamp(min=-126))


def _counts(st):
    B = st["lens"].numel()
    return st["lens"].long(), st["new"].long() if st["new"] is not None else st["lens"].new_full((B,), st["S"]).long()


def _plain_write(st):
    block, S = st["block"], st["S"]
    lens, new = _counts(st)
    step = torch.arange(S, device="cuda")
    pos = (lens - new)[:, None] + step
    b, s = torch.nonzero((step < new[:, None]) & (pos >= 0), as_tuple=True)
    page, slot = st["table"][b, pos[b, s] // block].long(), pos[b, s] % block
    begin = (lens - new).clamp(min=0)
    held = begin % block  # tokens that the first block holds already
    part = torch.nonzero((held > 0) & (lens > begin), as_tuple=True)[0]
    part_page, old = st["table"][part, begin[part] // block].long(), torch.arange(block, device="cuda") < held[part, None]

    def one(code, scale, x):
        x = x[b, :, s].float()
        amax = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")
        before = torch.zeros_like(scale)
        before[part_page] = scale[part_page]
        fresh = torch.maximum(_scale_of(amax), before)
        bits = code.view(torch.uint8)
        had = code.view(torch.uint8)[part_page].view(torch.float8_e4m3fn).float()
        moved = (had * (scale[part_page] / fresh[part_page])[:, :, None, None]).to(torch.float8_e4m3fn)
        bits[part_page] = torch.where(old[:, None, :, None], moved.view(torch.uint8), bits[part_page])
        bits[page, :, slot] = (x / fresh[page][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scale[page] = fresh[page]

    one(st["k"], st["k_scale"], st["k_new"])
    one(st["v"], st["v_scale"], st["v_new"])
    return {"k": st["k"], "v": st["v"], "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


def _plain_values(st, code, scale, pages):
    """fp32 values [B, Hkv, pages * block, D] of the given columns of the table."""
    at = st["table"][:, pages].long()
    x = code.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * scale[at][..., None, None]
    B, n, Hkv, block, D = x.shape
    return x.transpose(1, 2).reshape(B, Hkv, n * block, D)


def _plain_read(st):
    first, S, block = st["first"], st["S"], st["block"]
    columns = slice(first // block, min(st["table"].shape[1], -(-(first + S) // block)))
    n = min(S, st["table"].shape[1] * block - first)
    there = (first + torch.arange(n, device="cuda") < st["lens"][:, None])[:, None, :, None]
    for name in ("k", "v"):
        x = _plain_values(st, st[name], st[name + "_scale"], columns)[:, :, first % block:][:, :, :n]
        out = st[name + "_out"]
        out[:, :, :n] = torch.where(there, x.to(torch.bfloat16), out[:, :, :n])
    return {"k": st["k_out"], "v": st["v_out"]}


def _plain_attend(st):
    q, (lens, new) = st["q"], _counts(st)
    B, Hq, S, D = q.shape
    k, v = (_plain_values(st, st[x], st[x + "_scale"], slice(None)) for x in ("k", "v"))
    Hkv, L = k.shape[1:3]
    s = (q.float().view(B, Hkv, Hq // Hkv * S, D) @ k.transpose(2, 3)).view(B, Hkv, -1, S, L) * (1 / math.sqrt(D))
    pos = (lens - new)[:, None] + torch.arange(S, device="cuda")
    seen = torch.arange(L, device="cuda") <= pos[:, :, None]
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top.masked_fill(top == -math.inf, 0))
    total = p.sum(-1, keepdim=True)
    p = p / total.masked_fill(total == 0, 1)
    held = (torch.arange(L, device="cuda") < lens[:, None])[:, None, :, None]
    o = (p.view(B, Hkv, -1, L) @ v.masked_fill(~held, 0)).view(B, Hq, S, D)
    lse = (torch.log(total) + top).view(B, Hq, S)
    mine = torch.arange(S, device="cuda") < new[:, None, None]
    st["out"].copy_(torch.where(mine[..., None], o.to(torch.bfloat16), st["out"]))
    st["lse"].copy_(torch.where(mine, lse, st["lse"]))
    return {"out": st["out"], "lse": st["lse"]}


def run(st):
    op = st["case"]["op"]
    if own:
        cache = st["cache"]
        if op == "write":
            cache.write(st["k_new"], st["v_new"], new_lens=st["new"])
            return {"k": st["k"], "v": st["v"], "k_scale": st["k_scale"], "v_scale": st["v_scale"]}
        if op == "read":
            cache.read(st["S"], first=st["first"], k_out=st["k_out"], v_out=st["v_out"])
            return {"k": st["k_out"], "v": st["v_out"]}
        cache.attention(st["q"], q_lens=st["new"], out=st["out"], lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend}[op](st)


def _to_grid(x):
    """The nearest E4M3 value (ties to even) of each float64 of magnitude at most 448."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    lens, new = _lens(case)
    block, S, first, table = case["block"], case["S"], case["first"], st["table"].tolist()
    value = {x: st[x].double() for x in ("k", "v")} if case["op"] == "write" else None
    if case["op"] == "write":
        out = dict(value)
        for name in ("k", "v"):
            scale = st[name + "_scale"].double()
            for b, (t, n) in enumerate(zip(lens, new)):
                at = max(t - n, 0)
                while at < t:
                    to = min(t, at - at % block + block)
                    page, a, z = table[b][at // block], at % block, at % block + to - at
                    x = st[name + "_new"][b, :, at - (t - n):to - (t - n)].double()
                    big = x.abs().amax((1, 2)).cpu().numpy()
                    need = np.array([2.0 ** max(-126, math.ceil(math.log2(m / 448))) if m else 2.0 ** -126 for m in big])
                    need[big > 448 * need] *= 2
                    need[big <= 224 * need] /= 2
                    need = torch.tensor(need, device="cuda")
                    if a:
                        need = torch.maximum(need, scale[page])
                        out[name][page, :, :a] = _to_grid(out[name][page, :, :a] * (scale[page] / need)[:, None, None])
                    out[name][page, :, a:z] = _to_grid(x / need[:, None, None])
                    scale[page] = need
                    at = to
            out[name + "_scale"] = scale
        return out

    def values(name, b, a, z):
        """float64 values [Hkv, z - a, D] of positions a .. z - 1 of sequence b."""
        cols = range(a // block, -(-z // block))
        x = torch.cat([st[name][table[b][c]].double() * st[name + "_scale"][table[b][c]].double()[:, None, None] for c in cols], 1)
        return x[:, a % block:a % block + z - a]

    if case["op"] == "read":
        out = {x: torch.zeros(st[x + "_out"].shape, dtype=torch.float64, device="cuda") for x in ("k", "v")}
        for b, n in enumerate(_reads(case)):
            if n:
                for name in ("k", "v"):
                    out[name][b, :, :n] = values(name, b, first, first + n)
        return out
    q = st["q"].double()
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], dtype=torch.float64, device="cuda")
    group = case["Hq"] // case["Hkv"]
    for b, (t, n) in enumerate(zip(lens, new)):
        if t == 0:
            lse[b, :, :n] = -math.inf
            continue
        k, v = values("k", b, 0, t), values("v", b, 0, t)
        after = torch.arange(t, device="cuda") > torch.arange(t - n, t, device="cuda")[:, None]
        for h in range(case["Hq"]):
            s = (q[b, h, :n] @ k[h // group].T / math.sqrt(case["D"])).masked_fill(after, -math.inf)
            lse[b, h, :n] = torch.logsumexp(s, -1)
            o[b, h, :n] = torch.exp(s - lse[b, h, :n, None]) @ v[h // group]
    return {"out": o, "lse": lse}
