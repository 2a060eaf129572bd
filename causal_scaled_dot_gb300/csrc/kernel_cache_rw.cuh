// kernel_cache_rw.cuh -- the 8-bit cache as it is written and read back.
//
// Write: per block and head, s = 2^e the smallest power of two with
// max|x| <= 448 s (448 = 1.75 * 2^8 is E4M3's largest value), code = RNE(x / s).
// A power of two costs a floating format nothing but the place of its
// underflow, and makes the division and every later change of the scale exact.
// A unit is one (sequence, block, head, K or V): its tokens are read once into
// registers (at most 64 elements a thread), the maximum is reduced over the
// unit's threads, and the codes leave from the registers.  Bound by the bytes:
// 2 in and 1 out per element.
//
// Read: one 16-byte load of codes and two 16-byte stores of bf16 per step, flat
// over the requested rows; bound by the bytes (1 in, 2 out per element).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "cache_index.h"
#include "ptx.cuh"

namespace attn {

struct CacheWriteParams {
    CacheView c;
    const __nv_bfloat16 *k, *v;
    long long k_stride[3], v_stride[3];  // batch, head, token, in elements
    const int* new_lens;                 // or null: S each
    int S;
    int blocks_per_seq;                  // blocks that S tokens can touch
    long long num_units;                 // B * Hkv * 2 * blocks_per_seq
};

// The smallest power of two s >= 2^-126 with amax <= 448 s, for finite amax >= 0:
// amax = m 2^x with 1 <= m < 2 needs s = 2^(x-8), or 2^(x-7) when m > 1.75.
__device__ __forceinline__ float e4m3_pow2_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(e < 1 ? 1 : e) << 23);
}

// Two values already divided by the scale -> two codes; not finite -> NaN.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float2 e4m3_unpair(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// kThreads threads per unit, 256 / kThreads units per CTA; 8 vectors of 8
// elements per thread cover block_size * D <= 64 * kThreads elements.
template <int kThreads>
__global__ void __launch_bounds__(256) attn_cache_write_kernel(const CacheWriteParams p) {
    constexpr int kVec = 8;
    __shared__ float warp_max[8];
    const CacheView& c = p.c;
    const int t = threadIdx.x % kThreads;
    const long long unit = (long long)blockIdx.x * (256 / kThreads) + threadIdx.x / kThreads;
    bool active = unit < p.num_units, bad = false;
    int b = 0, h = 0, is_v = 0, slot0 = 0, rows = 0, row0 = 0, block = -1;
    if (active) {
        const int blk = (int)(unit % p.blocks_per_seq);
        const long long x = unit / p.blocks_per_seq;
        is_v = (int)(x & 1);
        h = (int)((x >> 1) % c.Hkv);
        b = (int)((x >> 1) / c.Hkv);
        const CacheSpan s = cache_span(c.seq_lens[b], p.new_lens ? p.new_lens[b] : p.S,
                                       c.max_blocks * c.block_size, p.S, &bad);
        const int begin = s.first < 0 ? 0 : s.first;     // first position written
        const int lb = (begin >> c.block_shift) + blk;   // this unit's block of the sequence
        const int pos0 = blk == 0 ? begin : lb << c.block_shift;
        const int end = min(s.len, (lb + 1) << c.block_shift);
        active = pos0 < end;
        if (active) {
            slot0 = pos0 & (c.block_size - 1);
            rows = end - pos0;
            row0 = pos0 - s.first;
            block = cache_block(c.block_table[(long long)b * c.max_blocks + lb], c.num_blocks, &bad);
            active = block >= 0;
        }
    }
    if (bad && t == 0) atomicOr(c.status, kStatusBadCache);
    if (kThreads == 32 && !active) return;  // whole warps: no barrier below

    const int vec_per_row = c.D / 8, n_vec = active ? rows * vec_per_row : 0;
    const long long* st = is_v ? p.v_stride : p.k_stride;
    const __nv_bfloat16* src = (is_v ? p.v : p.k) + b * st[0] + h * st[1] + (long long)row0 * st[2];
    float* scale_at = active ? (is_v ? c.v_scale : c.k_scale) + (long long)block * c.Hkv + h : nullptr;
    const float s_old = active && slot0 > 0 ? *scale_at : 0.f;

    uint4 x[kVec];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int v = t + i * kThreads;
        x[i] = make_uint4(0, 0, 0, 0);
        if (v < n_vec)
            x[i] = __ldcs(reinterpret_cast<const uint4*>(src + (long long)(v / vec_per_row) * st[2] +
                                                         (v % vec_per_row) * 8));
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float lo = fabsf(__uint_as_float(w[j] << 16)), hi = fabsf(__uint_as_float(w[j] & 0xffff0000u));
            amax = fmaxf(amax, lo < INFINITY ? lo : 0.f);  // false for NaN and infinity
            amax = fmaxf(amax, hi < INFINITY ? hi : 0.f);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (kThreads > 32) {
        if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
        __syncthreads();
        const int w0 = (threadIdx.x / kThreads) * (kThreads / 32);
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, warp_max[w0 + w]);
    }
    if (!active) return;

    const float s_new = fmaxf(e4m3_pow2_scale(amax), s_old);
    const float inv = 1.f / s_new;  // exact for the powers of two that this kernel stores (at most 2^120)
    unsigned char* dst = (is_v ? c.v : c.k) + cache_offset(block, h, slot0, c.Hkv, c.block_size, c.D);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int v = t + i * kThreads;
        if (v >= n_vec) break;
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t code[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xffff0000u);
            lo = fabsf(lo) < INFINITY ? lo * inv : NAN;
            hi = fabsf(hi) < INFINITY ? hi * inv : NAN;
            code[j] = e4m3_pair(lo, hi);
        }
        *reinterpret_cast<uint2*>(dst + (long long)v * 8) = make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
    }
    if (slot0 > 0 && s_new > s_old) {  // the block's earlier tokens move to the larger scale
        const float ratio = s_old * inv;
        uint2* had = reinterpret_cast<uint2*>((is_v ? c.v : c.k) + cache_offset(block, h, 0, c.Hkv, c.block_size, c.D));
        for (int v = t; v < slot0 * vec_per_row; v += kThreads) {
            const uint2 w = had[v];
            uint32_t code[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = e4m3_unpair((j < 2 ? w.x : w.y) >> (16 * (j & 1)) & 0xffffu);
                code[j] = e4m3_pair(f.x * ratio, f.y * ratio);
            }
            had[v] = make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
        }
    }
    if (t == 0) *scale_at = s_new;
}

struct CacheReadParams {
    CacheView c;
    __nv_bfloat16 *k, *v;  // [B, Hkv, S, D], either may be null
    int first, S;
    long long num_vec;     // 16-element vectors of one output
};

// blockIdx.y: 0 reads K, 1 reads V (or the one that is asked for).
__global__ void __launch_bounds__(256) attn_cache_read_kernel(const CacheReadParams p) {
    const CacheView& c = p.c;
    const bool is_v = blockIdx.y == 1 || p.k == nullptr;
    const unsigned char* code = is_v ? c.v : c.k;
    const float* scale = is_v ? c.v_scale : c.k_scale;
    __nv_bfloat16* out = is_v ? p.v : p.k;
    const int vec_per_row = c.D / 16;
    bool bad = false;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < p.num_vec; i += (long long)gridDim.x * 256) {
        const int d = (int)(i % vec_per_row) * 16;
        const long long row = i / vec_per_row;
        const int s = (int)(row % p.S);
        const long long bh = row / p.S;
        const int h = (int)(bh % c.Hkv), b = (int)(bh / c.Hkv);
        const int len = cache_clamp(c.seq_lens[b], c.max_blocks * c.block_size, &bad);
        const long long pos = (long long)p.first + s;
        if (pos >= len) continue;
        const int block = cache_block(c.block_table[(long long)b * c.max_blocks + (pos >> c.block_shift)],
                                      c.num_blocks, &bad);
        if (block < 0) continue;
        const uint4 w = __ldcs(reinterpret_cast<const uint4*>(
            code + cache_offset(block, h, (int)pos & (c.block_size - 1), c.Hkv, c.block_size, c.D) + d));
        const float f = scale[(long long)block * c.Hkv + h];
        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 e = e4m3_unpair(in[j >> 1] >> (16 * (j & 1)) & 0xffffu);
            o[j] = ptx::pack_bf16x2(e.x * f, e.y * f);
        }
        uint4* to = reinterpret_cast<uint4*>(out + i * 16);
        to[0] = make_uint4(o[0], o[1], o[2], o[3]);
        to[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
    if (bad) atomicOr(c.status, kStatusBadCache);
}

}  // namespace attn
