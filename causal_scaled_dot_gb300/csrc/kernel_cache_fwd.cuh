// kernel_cache_fwd.cuh -- attention over the 8-bit cache, the plain form: one
// warp per query row walks the row's keys with the running maximum and sum of
// an online softmax.
#pragma once

#include <cuda_bf16.h>

#include "cache_index.h"
#include "common.cuh"
#include "kernel_cache_rw.cuh"
#include "ptx.cuh"

namespace attn {

struct CacheFwdParams {
    CacheView c;
    const __nv_bfloat16* q;
    long long q_stride[3];  // batch, head, token, in elements
    __nv_bfloat16* out;
    float* lse;             // may be null
    const int* q_lens;      // may be null: Sq each
    int Hq, Sq, group, causal;
    float scale_log2;       // scale * log2(e)
};

template <int D>
__global__ void __launch_bounds__(128) attn_cache_fwd_row_kernel(const CacheFwdParams p) {
    constexpr int E = D / 32;  // elements per lane: d = lane * E ..
    const CacheView& c = p.c;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= (long long)c.B * p.Hq * p.Sq) return;
    const int i = (int)(row % p.Sq), hq = (int)(row / p.Sq % p.Hq), b = (int)(row / p.Sq / p.Hq);
    const int h = hq / p.group;
    bool bad = false;
    const CacheSpan s = cache_span(c.seq_lens[b], p.q_lens ? p.q_lens[b] : p.Sq, c.max_blocks * c.block_size, p.Sq, &bad);
    if (i >= s.count) return;
    const int n = min(s.len, p.causal ? max(s.first + i + 1, 0) : s.len);
    const __nv_bfloat16* q = p.q + b * p.q_stride[0] + hq * p.q_stride[1] + i * p.q_stride[2] + lane * E;
    float qf[E], o[E];
    for (int e = 0; e < E; ++e) {
        qf[e] = __bfloat162float(q[e]);
        o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < n; ++j) {
        const int block = cache_block(c.block_table[(long long)b * c.max_blocks + (j >> c.block_shift)], c.num_blocks, &bad);
        if (block < 0) continue;
        const size_t at = cache_offset(block, h, j & (c.block_size - 1), c.Hkv, c.block_size, D) + lane * E;
        const float ks = c.k_scale[(long long)block * c.Hkv + h], vs = c.v_scale[(long long)block * c.Hkv + h];
        float dot = 0.f;
        for (int e = 0; e < E; ++e) dot += qf[e] * e4m3_unpair(c.k[at + e]).x;
        for (int w = 16; w > 0; w >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, w);
        const float x = dot * ks * p.scale_log2, top = fmaxf(m, x);
        const float keep = top == -INFINITY ? 1.f : ptx::ex2(m - top), w = top == -INFINITY ? (x == x ? 0.f : x) : ptx::ex2(x - top);
        l = l * keep + w;
        for (int e = 0; e < E; ++e) o[e] = o[e] * keep + w * vs * e4m3_unpair(c.v[at + e]).x;
        m = top;
    }
    if (bad && lane == 0) atomicOr(c.status, kStatusBadCache);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int e = 0; e < E; ++e) p.out[row * D + lane * E + e] = __float2bfloat16(o[e] * inv);
    if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + ptx::lg2(l)) * kLn2;
}

}  // namespace attn
