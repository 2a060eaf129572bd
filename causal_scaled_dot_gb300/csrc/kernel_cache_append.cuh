// kernel_cache_append.cuh -- a step's heads on their way into the 8-bit cache: K normed, rotated and quantised in one
// pass, V quantised, and q normed and rotated for the attention that follows, in one launch.
//
// Units of K and V are those of the write (kernel_cache_rw.cuh): one (sequence, block, head, K or V), whose values stay in
// registers, here as fp32, until their largest magnitude gives the scale; K is rounded once, from the rotated fp32 value
// to its code.  A thread holds up to four shares of rows, each both elements of its pairs (rope.cuh).  The blocks after
// theirs take q by the rotation's plan.  Bound by the bytes: 2 in and 1 out per element of K and V, 2 and 2 of q.
#pragma once

#include "cache_index.h"
#include "kernel_cache_rw.cuh"
#include "rope.cuh"

namespace attn {

struct CacheAppendParams {
    CacheView c;
    RopeParams r;
    RopeRows in, out;   // q, k, v of the step; q rotated
    const int* new_lens;
    int S;
    int blocks_per_seq, num_units, write_blocks;
    RopePlan plan;      // of q
};

// The place of a query row: its token's in the cache.  Bad lengths are reported by the units that write.
struct AppendPlace {
    const CacheAppendParams& p;
    __device__ bool operator()(long long b, long long s, long long* position) const {
        bool bad = false;
        const CacheView& c = p.c;
        const CacheSpan span = cache_span(c.seq_lens[b], p.new_lens ? p.new_lens[b] : p.S, c.max_blocks * c.block_size, p.S, &bad);
        const bool there = s < span.count;
        *position = !there ? 0 : p.r.positions ? rope_position(p.r, b, s) : p.r.first + span.first + s;
        return there;
    }
};

// kThreads threads per unit, kBlock / kThreads units per block; up to 4 shares of 16 elements a thread.  Blocks that write
// (much to compute) and blocks of q (much to load) alternate evenly, so that an SM has both at any time.
template <int kThreads>
constexpr int kAppendBlock = kThreads > 128 ? kThreads : 128;
template <int D, bool kInter, int kThreads>
__global__ void __launch_bounds__(kAppendBlock<kThreads>, 512 / kAppendBlock<kThreads>)
    attn_cache_append_kernel(const __grid_constant__ CacheAppendParams p) {
    constexpr int kLanes = D / 16, kItems = 4, kBlock = kAppendBlock<kThreads>;
    static_assert(kItems == kRopeDepth, "one ring serves both kinds of blocks");
    __shared__ uint32_t warp_max[kBlock / 32];
    __shared__ __align__(16) unsigned char smem[RopeRing<2, kRopeDepth, kBlock>::kBytes];
    ptx::launch_next();
    ptx::wait_previous();
    // of the first i + 1 blocks (i + 1) W / N write
    const unsigned int before = (unsigned int)((unsigned long long)blockIdx.x * p.write_blocks / gridDim.x);
    if ((unsigned int)((blockIdx.x + 1ull) * p.write_blocks / gridDim.x) == before) {
        const unsigned int unit = blockIdx.x - before;
        if (p.r.weight[0])
            rope_forward<D, kInter, true, kBlock>(p.r, p.plan, unit, p.S, p.in, p.out, AppendPlace{p}, smem);
        else
            rope_forward<D, kInter, false, kBlock>(p.r, p.plan, unit, p.S, p.in, p.out, AppendPlace{p}, smem);
        return;
    }
    const CacheView& c = p.c;
    const int t = threadIdx.x % kThreads;
    const int unit = before * (kBlock / kThreads) + threadIdx.x / kThreads;
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

    const int lane = t % kLanes, kind = u.is_v ? 2 : 1;
    const RopeLane l = rope_lane(lane, D, p.r.rot, kInter);
    const __nv_bfloat16* src = p.in.p[kind] + u.b * p.in.stride[kind][0] + u.h * p.in.stride[kind][1];
    const RopeRing<2, kItems, kBlock> ring(smem);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int row = (t + i * kThreads) / kLanes;
        const uint4* x = reinterpret_cast<const uint4*>(row < rows ? src + (row0 + row) * p.in.stride[kind][2] : p.in.p[kind]);
        ring.fill(i, 0, x + l.a, row < rows);
        ring.fill(i, 1, x + l.b, row < rows);
        ptx::cp_async_commit();
    }
    const int block = active ? cache_block(entry, c.num_blocks, &bad) : -1;
    active = block >= 0;
    if (bad && t == 0) atomicOr(c.status, kStatusBadCache);
    if (kThreads == 32 && !active) {  // whole warps: no barrier below
        ptx::cp_async_wait<0>();
        return;
    }
    float* scale_at = active ? (u.is_v ? c.v_scale : c.k_scale) + (long long)block * c.Hkv + u.h : nullptr;
    const float s_old = active && slot0 > 0 ? *scale_at : 0.f;
    // A warp's threads may be of one unit only (kThreads >= 32): what follows is the same for all of them.
    uint64_t x[kItems][8];
    float amax = 0.f;
    bool odd = false;  // this thread holds an infinity or NaN: those do not count
    const void* weight = u.is_v ? nullptr : p.r.weight[1];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        switch (i) {  // the copies of the items so far
            case 0: ptx::cp_async_wait<3>(); break;
            case 1: ptx::cp_async_wait<2>(); break;
            case 2: ptx::cp_async_wait<1>(); break;
            default: ptx::cp_async_wait<0>();
        }
        if (i * kThreads >= rows * kLanes) continue;
        const int row = (t + i * kThreads) / kLanes;
        rope_unpack(ring.at(i, 0), ring.at(i, 1), x[i]);
        if (!u.is_v) {
            const int at = row < rows ? row0 + row : row0;
            RopeTurn<kInter> turn;
            turn.template set<false>(p.r, l, lane, p.r.positions ? rope_position(p.r, u.b, at) : p.r.first + s.first + at);
            if (weight) {
                float down;
                uint64_t w[8];
                rope_weights(weight, p.r.weight_f32, l, w);
                turn.weigh(w);
                const float r = rope_norm<kLanes>(x[i], p.r.eps, &down);
                turn.template turn<true>(x[i]);
                rope_scale(x[i], r);
            } else {
                turn.template turn<false>(x[i]);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float lo, hi;
            ptx::f2_split(x[i][j], lo, hi);
            lo = fabsf(lo);
            hi = fabsf(hi);
            odd = odd || !(lo < INFINITY) || !(hi < INFINITY);
            amax = fmaxf(amax, fmaxf(lo < INFINITY ? lo : 0.f, hi < INFINITY ? hi : 0.f));
        }
    }
    uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
    if (kThreads > 32) {
        if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = top;
        __syncthreads();
        const int w0 = (threadIdx.x / kThreads) * (kThreads / 32);
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k) top = max(top, warp_max[w0 + k]);
    }
    if (!active) return;

    const float s_new = fmaxf(e4m3_pow2_scale(__uint_as_float(top)), s_old);
    const float inv = 1.f / s_new;  // exact for the powers of two that this kernel stores
    const bool divide = slot0 > 0 && (__float_as_uint(s_new) & 0x7fffffu) != 0;  // a caller's scale, which the block had
    unsigned char* dst = (u.is_v ? c.v : c.k) + cache_offset(block, u.h, slot0, c.Hkv, c.block_size, D);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const int row = (t + i * kThreads) / kLanes;
        if (row >= rows) break;
        uint32_t code[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float lo, hi;
            ptx::f2_split(x[i][j], lo, hi);
            if (divide) {
                lo = e4m3_divided(lo, s_new);
                hi = e4m3_divided(hi, s_new);
            } else {
                if (odd) {  // NaN becomes NaN by itself, infinity does not
                    lo = fabsf(lo) < INFINITY ? lo : NAN;
                    hi = fabsf(hi) < INFINITY ? hi : NAN;
                }
                lo *= inv;
                hi *= inv;
            }
            code[j] = e4m3_pair(lo, hi);
        }
        unsigned char* to = dst + (long long)row * D;
        *reinterpret_cast<uint2*>(to + 8 * l.a) = make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
        *reinterpret_cast<uint2*>(to + 8 * l.b) = make_uint2(code[4] | code[5] << 16, code[6] | code[7] << 16);
    }
    if (slot0 > 0 && s_new > s_old) {  // the block's earlier tokens move to the larger scale
        const float ratio = s_old * inv;
        uint2* had = reinterpret_cast<uint2*>((u.is_v ? c.v : c.k) + cache_offset(block, u.h, 0, c.Hkv, c.block_size, D));
        for (int v = t; v < slot0 * (D / 8); v += kThreads) {
            const uint2 y = had[v];
            uint32_t code[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = e4m3_unpair((j < 2 ? y.x : y.y) >> (16 * (j & 1)) & 0xffffu);
                code[j] = e4m3_pair(f.x * ratio, f.y * ratio);
            }
            had[v] = make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
        }
    }
    if (t == 0) *scale_at = s_new;
}

}  // namespace attn
