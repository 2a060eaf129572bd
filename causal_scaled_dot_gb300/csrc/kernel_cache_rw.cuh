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
// Read: the same units the other way; bound by the bytes (1 in, 2 out per element).
//
// Both are latency-bound per unit (length, then table and data, then the rest),
// so what counts is that a unit's loads leave together and that many units are
// resident: 64 elements a thread, four blocks of 256 threads an SM (the write: 12.0
// us with three, 12.8 with five, which spill).  16.8 M elements of D = 128 in blocks
// of 64, cold: write 11.0 us, read 9.8 (4.6 and 5.1 TB/s, launch included).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "cache_index.h"
#include "ptx.cuh"
#include "ptx_cache.cuh"

namespace attn {

struct CacheWriteParams {
    CacheView c;
    const __nv_bfloat16 *k, *v;
    long long k_stride[3], v_stride[3];  // batch, head, token, in elements
    const int* new_lens;                 // or null: S each
    int S;
    int blocks_per_seq;                  // blocks that S tokens can touch
    int num_units;                       // B * Hkv * 2 * blocks_per_seq
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
// Two codes (bits 0-15) as two f16, exact.
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return h;
}
__device__ __forceinline__ float2 e4m3_unpair(uint32_t two) {
    const uint32_t h = e4m3_to_f16x2(two);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// x / s so that rounding it to a code rounds x / s itself: the quotient's first 24 bits, the last of them set when
// more follow, which a halfway value cannot have.
__device__ __forceinline__ float e4m3_divided(float x, float s) {
    if (!(fabsf(x) < INFINITY)) return NAN;
    const float q = __fdiv_rz(x, s);
    return __fmaf_rn(-q, s, x) == 0.f ? q : __uint_as_float(__float_as_uint(q) | 1u);
}

// The codes of a unit's vectors t, t + threads ... under a scale that is not a power of two, from x once more.  Out of line:
// a prompt's write takes 11.0 us with it, 11.2 with it inlined, and 10.85 without.
__device__ __noinline__ void cache_write_divided(const __nv_bfloat16* src, long long stride, unsigned char* dst, int t, int threads,
                                                 int n_vec, int row_shift, float s) {
#pragma unroll 1
    for (int v = t; v < n_vec; v += threads) {
        const uint4 y = *(reinterpret_cast<const uint4*>(src + (v >> row_shift) * stride) + (v & ((1 << row_shift) - 1)));
        const uint32_t w[4] = {y.x, y.y, y.z, y.w};
        uint32_t code[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            code[j] = e4m3_pair(e4m3_divided(__uint_as_float(w[j] << 16), s), e4m3_divided(__uint_as_float(w[j] & 0xffff0000u), s));
        *reinterpret_cast<uint2*>(dst + (long long)v * 8) = make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
    }
}

// A unit's place: sequence, head, K or V, and which of the blocks that the call touches.
struct CacheRwUnit {
    int b, h, is_v, blk;
};
__device__ __forceinline__ CacheRwUnit cache_rw_unit(int unit, int blocks, int Hkv, int kinds) {
    CacheRwUnit u;
    const int x = unit / blocks;
    u.blk = unit - x * blocks;
    const int y = kinds == 2 ? x >> 1 : x;
    u.is_v = kinds == 2 ? x & 1 : 0;
    u.b = y / Hkv;
    u.h = y - u.b * Hkv;
    return u;
}

// kThreads threads per unit, 256 / kThreads units per CTA; 8 vectors of 8
// elements per thread cover block_size * D <= 64 * kThreads elements.
template <int kThreads>
__global__ void __launch_bounds__(256, 4) attn_cache_write_kernel(const __grid_constant__ CacheWriteParams p) {
    constexpr int kVec = 8;
    __shared__ uint32_t warp_max[8];
    ptx::launch_next();
    ptx::wait_previous();
    const CacheView& c = p.c;
    const int t = threadIdx.x % kThreads;
    const int unit = blockIdx.x * (256 / kThreads) + threadIdx.x / kThreads;
    bool active = unit < p.num_units, bad = false;
    const CacheRwUnit u = cache_rw_unit(active ? unit : 0, p.blocks_per_seq, c.Hkv, 2);
    const CacheSpan s = cache_span(c.seq_lens[u.b], p.new_lens ? p.new_lens[u.b] : p.S, c.max_blocks * c.block_size, p.S, &bad);
    const int begin = s.first < 0 ? 0 : s.first;       // first position written
    const int lb = (begin >> c.block_shift) + u.blk;   // this unit's block of the sequence
    const int pos0 = u.blk == 0 ? begin : lb << c.block_shift;
    const int end = min(s.len, (lb + 1) << c.block_shift);
    active = active && pos0 < end;
    const int slot0 = pos0 & (c.block_size - 1), rows = active ? end - pos0 : 0, row0 = pos0 - s.first;
    const int entry = active ? c.block_table[(long long)u.b * c.max_blocks + lb] : 0;

    const int row_shift = c.D == 128 ? 4 : 3, n_vec = rows << row_shift;  // D / 8 vectors a row
    const long long stride = u.is_v ? p.v_stride[2] : p.k_stride[2];
    const __nv_bfloat16* src = u.is_v ? p.v + u.b * p.v_stride[0] + u.h * p.v_stride[1]
                                      : p.k + u.b * p.k_stride[0] + u.h * p.k_stride[1];
    uint4 x[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int v = t + i * kThreads;
        x[i] = make_uint4(0, 0, 0, 0);
        if (v < n_vec)
            x[i] = __ldcs(reinterpret_cast<const uint4*>(src + (row0 + (v >> row_shift)) * stride) + (v & ((1 << row_shift) - 1)));
    }
    const int block = active ? cache_block(entry, c.num_blocks, &bad) : -1;
    active = block >= 0;
    if (bad && t == 0) atomicOr(c.status, kStatusBadCache);
    if (kThreads == 32 && !active) return;  // whole warps: no barrier below
    float* scale_at = active ? (u.is_v ? c.v_scale : c.k_scale) + (long long)block * c.Hkv + u.h : nullptr;
    const float s_old = active && slot0 > 0 ? *scale_at : 0.f;
    // The largest magnitude by bit pattern, two elements an instruction (a comparison per element for what is not
    // finite made these instructions the bound: 0.7 us of 12.7 for 16.8 M elements).
    uint32_t two = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        two = __vmaxu2(__vmaxu2(__vmaxu2(two, x[i].x & 0x7fff7fffu), __vmaxu2(x[i].y & 0x7fff7fffu, x[i].z & 0x7fff7fffu)),
                       x[i].w & 0x7fff7fffu);
    uint32_t amax = max(two & 0xffffu, two >> 16);
    const bool odd = amax >= 0x7f80u;  // this thread holds an infinity or NaN: those do not count
    if (odd) {
        amax = 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t m = w[j >> 1] >> (16 * (j & 1)) & 0x7fffu;
                amax = max(amax, m < 0x7f80u ? m : 0u);
            }
        }
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    if (kThreads > 32) {
        if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
        __syncthreads();
        const int w0 = (threadIdx.x / kThreads) * (kThreads / 32);
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) amax = max(amax, warp_max[w0 + w]);
    }
    if (!active) return;

    const float s_new = fmaxf(e4m3_pow2_scale(__uint_as_float(amax << 16)), s_old);
    const float inv = 1.f / s_new;  // exact for the powers of two that this kernel stores (at most 2^120); else below
    const uint64_t inv2 = ptx::f2(inv, inv);
    unsigned char* dst = (u.is_v ? c.v : c.k) + cache_offset(block, u.h, slot0, c.Hkv, c.block_size, c.D);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int v = t + i * kThreads;
        if (v >= n_vec) break;
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t code[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xffff0000u);
            if (odd) {  // NaN becomes NaN by itself, infinity does not
                lo = fabsf(lo) < INFINITY ? lo : NAN;
                hi = fabsf(hi) < INFINITY ? hi : NAN;
            }
            ptx::f2_split(ptx::mul2(ptx::f2(lo, hi), inv2), lo, hi);
            code[j] = e4m3_pair(lo, hi);
        }
        *reinterpret_cast<uint2*>(dst + (long long)v * 8) = make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
    }
    if (slot0 > 0 && (__float_as_uint(s_new) & 0x7fffffu) != 0)  // a caller's scale, which the block had
        cache_write_divided(src + row0 * stride, stride, dst, t, kThreads, n_vec, row_shift, s_new);
    if (slot0 > 0 && s_new > s_old) {  // the block's earlier tokens move to the larger scale
        const float ratio = s_old * inv;
        uint2* had = reinterpret_cast<uint2*>((u.is_v ? c.v : c.k) + cache_offset(block, u.h, 0, c.Hkv, c.block_size, c.D));
        for (int v = t; v < slot0 << row_shift; v += kThreads) {
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
    int blocks_per_seq;    // blocks that S positions from `first` on touch
    int num_units;         // B * Hkv * blocks_per_seq, twice when both are read
};

// Units and threads as above; 8 vectors of 8 codes per thread, so that a warp's stores are 512 bytes in a row
// (16 codes a vector: 12.4 us where this takes 10.4).
template <int kThreads>
__global__ void __launch_bounds__(256, 4) attn_cache_read_kernel(const __grid_constant__ CacheReadParams p) {
    constexpr int kVec = 8;
    ptx::launch_next();
    ptx::wait_previous();
    const CacheView& c = p.c;
    const int t = threadIdx.x % kThreads, unit = blockIdx.x * (256 / kThreads) + threadIdx.x / kThreads;
    if (unit >= p.num_units) return;
    const CacheRwUnit u = cache_rw_unit(unit, p.blocks_per_seq, c.Hkv, p.k && p.v ? 2 : 1);
    const bool is_v = u.is_v || !p.k;
    const int lb = (p.first >> c.block_shift) + u.blk;
    bool bad = false;
    const int len = cache_clamp(c.seq_lens[u.b], c.max_blocks * c.block_size, &bad);
    const int pos0 = max(p.first, lb << c.block_shift), end = min(min(len, p.first + p.S), (lb + 1) << c.block_shift);
    if (bad && t == 0) atomicOr(c.status, kStatusBadCache);
    if (pos0 >= end) return;
    // only now: entries past a sequence's last token are not read
    const int block = cache_block(c.block_table[(long long)u.b * c.max_blocks + lb], c.num_blocks, &bad);
    if (block < 0) {
        if (t == 0) atomicOr(c.status, kStatusBadCache);
        return;
    }
    const uint2* code = reinterpret_cast<const uint2*>(
        (is_v ? c.v : c.k) + cache_offset(block, u.h, pos0 & (c.block_size - 1), c.Hkv, c.block_size, c.D));
    const float scale = (is_v ? c.v_scale : c.k_scale)[(long long)block * c.Hkv + u.h];
    uint4* out = reinterpret_cast<uint4*>((is_v ? p.v : p.k) +
                                          (((long long)u.b * c.Hkv + u.h) * p.S + (pos0 - p.first)) * c.D);
    const int n_vec = (end - pos0) * c.D / 8;
    uint2 x[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        if (t + i * kThreads < n_vec) x[i] = __ldcs(code + t + i * kThreads);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        if (t + i * kThreads >= n_vec) break;
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 e = e4m3_unpair((j < 2 ? x[i].x : x[i].y) >> (16 * (j & 1)) & 0xffffu);
            o[j] = ptx::pack_bf16x2(e.x * scale, e.y * scale);
        }
        out[t + i * kThreads] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

}  // namespace attn
