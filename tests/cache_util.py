"""The 8-bit cache's operators from their definitions, in float64 on the CPU, and
helpers that build caches for the tests.  Nothing here calls the library."""
from __future__ import annotations

import math

import numpy as np
import torch

SMALLEST = -126  # exponent of the smallest scale


def codes_of(x):
    """float64 values of magnitude <= 448 rounded to E4M3 (ties to even), NaN kept."""
    x = np.asarray(x, np.float64)
    mag = np.abs(np.nan_to_num(x))
    e = np.maximum(np.floor(np.log2(np.maximum(mag, 2.0 ** -40))), -6)
    e = np.where(2.0 ** (e + 1) <= mag, e + 1, e)  # log2's own rounding next to a power of two
    step = 2.0 ** (e - 3)
    return np.where(np.isnan(x), np.nan, np.round(x / step) * step)


def scale_of(x):
    """The smallest power of two s >= 2^-126 with |x| <= 448 s for every finite x."""
    x = np.abs(x[np.isfinite(x)])
    big = float(x.max()) if x.size else 0.0
    s = 2.0 ** SMALLEST
    if big > 0:
        s = 2.0 ** max(SMALLEST, math.ceil(math.log2(big)) - 10)
        while big > 448 * s:
            s *= 2
    return s


class PlainCache:
    """Decoded codes [num_blocks, Hkv, block, D] (float64) and scales, written token by token's blocks."""

    def __init__(self, num_blocks, Hkv, block, D):
        self.k, self.v = np.zeros((num_blocks, Hkv, block, D)), np.zeros((num_blocks, Hkv, block, D))
        self.k_scale, self.v_scale = np.ones((num_blocks, Hkv)), np.ones((num_blocks, Hkv))
        self.block = block

    def write(self, k, v, table, lens, new):
        """k, v float64 [B, Hkv, S, D]; lens count the new tokens."""
        for b, (t, n) in enumerate(zip(lens, new)):
            at = max(t - n, 0)
            while at < t:
                to = min(t, (at // self.block + 1) * self.block)
                page, a = table[b][at // self.block], at % self.block
                row = at - (t - n)
                for code, scale, x in ((self.k, self.k_scale, k), (self.v, self.v_scale, v)):
                    for h in range(code.shape[1]):
                        new_x = x[b, h, row:row + to - at]
                        s = scale_of(new_x)
                        if a:
                            s = max(s, scale[page, h])
                            code[page, h, :a] = codes_of(code[page, h, :a] * (scale[page, h] / s))
                        code[page, h, a:a + to - at] = codes_of(np.where(np.isfinite(new_x), new_x, np.nan) / s)
                        scale[page, h] = s
                at = to

    def values(self, which, table, length):
        """float64 [Hkv, length, D] of one sequence (its row of the table); pages outside the cache read as NaN."""
        code, scale = (self.k, self.k_scale) if which == "k" else (self.v, self.v_scale)
        pages = [code[p] * scale[p][:, None, None] if 0 <= p < code.shape[0] else np.full(code.shape[1:], np.nan)
                 for p in table[:-(-length // self.block)]]
        if not pages:
            return np.zeros((code.shape[1], 0, code.shape[3]))
        return np.concatenate(pages, 1)[:, :length]


def attention(q, k, v, scale, first, causal):
    """O, LSE and each output's tolerance for one sequence: q [Hq, n, D] at positions
    first .. first + n - 1 over k, v [Hkv, length, D] (float64).  Keys whose K holds a NaN in
    every element are invisible (a page outside the cache).

    The tolerance counts, against this exact result: q rounded to 2^-18 of its row's largest
    element (a score moves by at most scale * 2^-18 max|q| sum|k|, and 2^-20 of the sum of its
    products' magnitudes for the fp32 accumulation and exp2), the weights rounded to 2^-8 of
    themselves plus 2^-14 of the largest one (weights as they multiply V's codes, so weighted
    by V's scale: the bound takes the largest |v| in that key's row; half a step of the smallest
    codes is 2^-10, and a row's largest weight counts 2^4 at least), and O's rounding to bf16, 2^-8 |O|."""
    Hq, n, D = q.shape
    Hkv, length = k.shape[:2]
    group = Hq // Hkv
    o, lse = np.zeros((Hq, n, D)), np.full((Hq, n), -np.inf)
    tol, tol_lse = np.zeros((Hq, n, D)), np.zeros((Hq, n))
    there = ~np.isnan(k).all((0, 2)) if length else np.zeros(0, bool)
    for h in range(Hq):
        kk, vv = k[h // group], v[h // group]
        for i in range(n):
            see = there & ((np.arange(length) <= first + i) if causal else np.ones(length, bool))
            if not see.any():
                continue
            K, V = kk[see], vv[see]
            s = scale * (K @ q[h, i])
            m = s.max()
            p = np.exp(s - m)
            total = p.sum()
            o[h, i] = (p / total) @ V
            lse[h, i] = m + math.log(total)
            w = p / total
            ds = scale * (2.0 ** -18 * np.abs(q[h, i]).max() * np.abs(K).sum(1) + 2.0 ** -20 * (np.abs(K) @ np.abs(q[h, i])))
            ds = float(ds.max()) + 2.0 ** -20
            mag = np.abs(V)
            heavy = (w * mag.max(1)).max()
            # sum over keys of 2^-14 of the largest weight-times-V-scale, in units of each key's codes
            floor = 2.0 ** -14 * heavy * (mag / np.maximum(mag.max(1, keepdims=True), 1e-300)).sum(0) * 2
            tol[h, i] = (2.0 ** -8 + 2 * ds) * (w @ mag) + floor + 2.0 ** -8 * np.abs(o[h, i]) + 1e-30
            tol_lse[h, i] = ds + 2.0 ** -20 * (abs(lse[h, i]) + abs(m))
    return o, lse, tol, tol_lse


def to_f64(t):
    return t.detach().double().cpu().numpy()


def make(B, Hkv, D, block, max_tokens, seed, spare=3, device="cuda"):
    """A KVCache over shuffled blocks (some of them spare), filled with NaN codes so that anything
    read without being written shows, and its table as lists."""
    from causal_scaled_dot_gb300.kv_cache import KVCache
    per = -(-max_tokens // block)
    total = B * per + spare
    g = torch.Generator().manual_seed(seed)
    table = torch.randperm(total, generator=g)[:B * per].view(B, per).to(torch.int32)
    code = lambda: torch.full((total, Hkv, block, D), 0x7F, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)  # noqa: E731
    scale = lambda: torch.full((total, Hkv), float("nan"), dtype=torch.float32, device=device)  # noqa: E731
    cache = KVCache(code(), code(), scale(), scale(), table.to(device), torch.zeros(B, dtype=torch.int32, device=device))
    return cache, table.tolist()


def rows(shape, seed, sigma=1.0):
    """bf16 CPU tensor of seeded normals, a few channels and tokens larger than the rest."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * sigma
    x = x * (1 + 3 * (torch.rand(shape[-1], generator=g) > 0.95)) * (1 + 7 * (torch.rand(shape[:-1], generator=g) > 0.97))[..., None]
    return x.to(torch.bfloat16)
