// kernel_cache_append.cuh -- a step's heads on their way into the 8-bit cache: K normed, rotated and quantised in one
// pass, V quantised, and q normed and rotated for the attention that follows, in one launch.
//
// Units of K and V are those of the write (kernel_cache_rw.cuh): one (sequence, block, head, K or V).  K is rounded once,
// from the rotated fp32 value to its code, so a unit's values wait in shared memory as fp32 until their largest magnitude
// gives the scale.  A thread holds its own shares of rows there (both elements of each of its pairs, rope.cuh), first as
// they come in, and nobody else's.  In registers they would have to be named one by one: the code, four times as long,
// missed the instruction cache for a quarter of the time (62 us for what takes 43 so, both before what follows).  Blocks of q,
// by the rotation's plan, have much to load, those of K much to compute: they alternate evenly, and V's, which are quick,
// come last, so that the launch ends evenly (37.8 us with K and V in one order with q, 35.1 so).
// Bound by the bytes, 2 in and 1 out per element of K and V, 2 and 2 of q, and for long prompts by the latency of K's units
// too: 20 warps an SM, issuing in 54 % of the cycles.  2 x 4096 tokens of 32 + 8 + 8 heads of 128 with norms, 185 MB: 34.4 us,
// 5.4 TB/s; one token of 64 sequences 4.0 us, of one 2.9, while the blocks' scales hold.  A step in which they rise passes
// over the blocks' earlier tokens, at the end of this kernel: for those 64 sequences up to 6 us more with blocks of 64, 16 with 128.
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
    int blocks_per_seq;
    int num_units;               // of K, and as many of V
    unsigned int first_v;        // the first of V's blocks
    unsigned long long k_share;  // append_share of K's and q's blocks
    int unit_shift;     // 2^unit_shift threads per unit: 32 .. kAppendThreads
    RopePlan plan;      // of q
};
constexpr int kAppendThreads = 128;
// Dynamic shared memory of a block whose threads hold up to `items` shares of 16 elements.
constexpr int append_smem(int items) {
    const int shares = items * 4 * kAppendThreads * 16, ring = RopeRing<2, kRopeDepth, kAppendThreads>::kBytes;
    return shares > ring ? shares : ring;
}

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

// A share's codes where one of its values may be infinite (NaN then), or the scale is a caller's and no power of two.
__device__ __forceinline__ void append_codes_slow(const uint64_t (&x)[8], float s, bool divide, uint32_t (&code)[4]) {
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
        const auto one = [&](float y) { return divide ? e4m3_divided(y, s) : fabsf(y) < INFINITY ? y / s : NAN; };
        float a, b, d, e;
        ptx::f2_split(j == 0 ? x[0] : j == 1 ? x[2] : j == 2 ? x[4] : x[6], a, b);
        ptx::f2_split(j == 0 ? x[1] : j == 1 ? x[3] : j == 2 ? x[5] : x[7], d, e);
        const uint32_t four = e4m3_pair(one(a), one(b)) | e4m3_pair(one(d), one(e)) << 16;
#pragma unroll
        for (int k = 0; k < 4; ++k) code[k] = k == j ? four : code[k];
    }
}
__device__ __forceinline__ float append_largest(const uint64_t (&x)[8]) {
    float m = 0.f, lo, hi;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        ptx::f2_split(x[i], lo, hi);
        m = ptx::max3(m, fabsf(lo), fabsf(hi));
    }
    return m;
}
__device__ __forceinline__ float append_largest_finite(const uint64_t (&x)[8]) {
    float m = 0.f, lo, hi;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        ptx::f2_split(x[i], lo, hi);
        m = ptx::max3(m, fabsf(lo) < INFINITY ? fabsf(lo) : 0.f, fabsf(hi) < INFINITY ? fabsf(hi) : 0.f);
    }
    return m;
}
// The largest finite magnitude of a thread's bf16 shares, as fp32 bits.
__device__ __noinline__ uint32_t append_finite(RopeRing<4, 1, kAppendThreads> mine, int count) {
    float m = 0.f;
    for (int i = 0; i < count; ++i) {
        uint64_t x[8];
        rope_unpack(mine.at(i, 0), mine.at(i, 1), x);
        m = fmaxf(m, append_largest_finite(x));
    }
    return __float_as_uint(m);
}

// Five blocks an SM: with 6 the prompt above takes 33.2 us, but one token of 64 sequences 4.4, and 512 of 2 9.4 where 5 take 8.7;
// with 4 (and twice the registers for the sines) it took 37.4 where 5 took 35.1.
template <int D, bool kInter>
__global__ void __launch_bounds__(kAppendThreads, 5) attn_cache_append_kernel(const __grid_constant__ CacheAppendParams p) {
    constexpr int kLanes = D / 16;
    __shared__ uint32_t warp_max[kAppendThreads / 32];
    __shared__ __align__(16) unsigned long long turns[64];
    extern __shared__ __align__(16) unsigned char smem[];
    ptx::launch_next();
    ptx::wait_previous();
    const bool is_v = blockIdx.x >= p.first_v;
    unsigned int index = blockIdx.x - p.first_v;
    if (!is_v && !append_is_k(p.k_share, blockIdx.x, &index)) {
        rope_forward<D, kInter, true, kAppendThreads>(p.r, p.plan, index, p.S, p.in, p.out, AppendPlace{p}, smem);
        return;
    }
    if (threadIdx.x < 64) turns[threadIdx.x] = p.r.turns[threadIdx.x];
    __syncthreads();
    const CacheView& c = p.c;
    const int threads = 1 << p.unit_shift, t = threadIdx.x & (threads - 1);
    const int unit = (int)(index * (kAppendThreads >> p.unit_shift) + (threadIdx.x >> p.unit_shift));
    bool active = unit < p.num_units, bad = false;
    CacheRwUnit u = cache_rw_unit(active ? unit : 0, p.blocks_per_seq, c.Hkv, 1);
    u.is_v = is_v;
    const CacheSpan s = cache_span(c.seq_lens[u.b], p.new_lens ? p.new_lens[u.b] : p.S, c.max_blocks * c.block_size, p.S, &bad);
    const int begin = s.first < 0 ? 0 : s.first;       // first position written
    const int lb = (begin >> c.block_shift) + u.blk;   // this unit's block of the sequence
    const int pos0 = u.blk == 0 ? begin : lb << c.block_shift;
    const int end = min(s.len, (lb + 1) << c.block_shift);
    active = active && pos0 < end;
    const int slot0 = pos0 & (c.block_size - 1), rows = active ? end - pos0 : 0, row0 = pos0 - s.first;

    const int lane = t % kLanes, kind = u.is_v ? 2 : 1;
    const RopeLane l = rope_lane(lane, D, p.r.rot, kInter);
    const long long stride = p.in.stride[kind][2];
    const __nv_bfloat16* src = p.in.p[kind] + (unsigned int)u.b * p.in.stride[kind][0] + (unsigned int)u.h * p.in.stride[kind][1] +
                               (unsigned int)(active ? row0 + t / kLanes : 0) * stride;
    // The shares of this thread: rows first, first + step ...
    const int first = t / kLanes, step_shift = p.unit_shift - (D == 128 ? 3 : 2), step = 1 << step_shift;
    const int count = active ? (rows - first + step - 1) >> step_shift : 0;
    const RopeRing<4, 1, kAppendThreads> mine(smem);
    for (int i = 0; i < count; ++i) {
        const uint4* x = reinterpret_cast<const uint4*>(src);
        mine.fill(i, 0, x + l.a, true);
        mine.fill(i, 1, x + l.b, true);
        src += stride << step_shift;
    }
    ptx::cp_async_commit();
    const int entry = active ? c.block_table[(unsigned int)u.b * (unsigned long long)(unsigned int)c.max_blocks + (unsigned int)lb] : 0;
    const int block = active ? cache_block(entry, c.num_blocks, &bad) : -1;
    active = block >= 0;
    if (bad && t == 0) atomicOr(c.status, kStatusBadCache);
    float* scale_at = active ? (u.is_v ? c.v_scale : c.k_scale) + (long long)block * c.Hkv + u.h : nullptr;
    const float s_old = active && slot0 > 0 ? *scale_at : 0.f;

    uint32_t top = 0;  // the largest magnitude, as bits
    bool odd = false;  // this thread holds an infinity: those do not count, nor do NaN
    if (u.is_v) {
        ptx::cp_async_wait<0>();
        uint32_t two = 0;  // two elements an instruction, by their bits
#pragma unroll 1
        for (int i = 0; i < count; ++i) {
            const uint4 a = mine.at(i, 0), b = mine.at(i, 1);
            two = __vmaxu2(__vmaxu2(two, a.x & 0x7fff7fffu), __vmaxu2(a.y & 0x7fff7fffu, a.z & 0x7fff7fffu));
            two = __vmaxu2(__vmaxu2(two, a.w & 0x7fff7fffu), __vmaxu2(b.x & 0x7fff7fffu, b.y & 0x7fff7fffu));
            two = __vmaxu2(__vmaxu2(two, b.z & 0x7fff7fffu), b.w & 0x7fff7fffu);
        }
        top = max(two & 0xffffu, two >> 16) << 16;
        if (top >= 0x7f800000u) {
            odd = true;
            top = append_finite(mine, count);
        }
    } else {
        const void* weight = p.r.weight[1];
        float amax = 0.f;
        // Whole warps stay together, as the sums over a row's lanes ask for: a warp is of one unit, a row of neighbouring lanes.
        const int most = active ? (rows + step - 1) >> step_shift : 0;
#pragma unroll 1
        for (int i = 0; i < most; ++i) {
            uint64_t x[8];
            const bool there = i < count;
            const int at = row0 + (there ? first + i * step : 0);
            RopeWaves<kInter> waves;
            waves.set(p.r, turns, l, lane, p.r.positions ? rope_position(p.r, u.b, at) : p.r.first + s.first + at);
            if (i == 0) ptx::cp_async_wait<0>();
            if (there) {
                rope_unpack(mine.at(i, 0), mine.at(i, 1), x);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = 0;
            }
            if (weight) {
                float down;
                uint64_t w[8];
                rope_weights(weight, p.r.weight_f32, l, w);
                const float r = rope_norm<kLanes>(x, p.r.eps, &down);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = ptx::mul2(x[j], w[j]);
                rope_scale(x, r);
            }
            waves.turn(l, x);
            float m = append_largest(x);
            if (m == INFINITY) {
                odd = true;
                m = append_largest_finite(x);
            }
            amax = fmaxf(amax, m);
            if (there) {
#pragma unroll
                for (int j = 0; j < 4; ++j) mine.put(i, j, x[2 * j], x[2 * j + 1]);
            }
        }
        top = __float_as_uint(amax);
    }
    ptx::cp_async_wait<0>();
    top = __reduce_max_sync(0xffffffffu, top);
    if (threads > 32) {
        if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = top;
        __syncthreads();
        const int w0 = threadIdx.x >> p.unit_shift << (p.unit_shift - 5);
        for (int k = 0; k < threads >> 5; ++k) top = max(top, warp_max[w0 + k]);
    }
    if (!active) return;

    const float s_new = fmaxf(e4m3_pow2_scale(__uint_as_float(top)), s_old);
    const float inv = 1.f / s_new;  // exact for the powers of two that this kernel stores
    const bool divide = slot0 > 0 && (__float_as_uint(s_new) & 0x7fffffu) != 0;  // a caller's scale, which the block had
    const uint64_t inv2 = rope_both(inv);
    unsigned char* dst = (u.is_v ? c.v : c.k) + cache_offset(block, u.h, slot0 + first, c.Hkv, c.block_size, D);
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
        uint32_t code[4];
        uint64_t x[8];
        if (u.is_v) {
            rope_unpack(mine.at(i, 0), mine.at(i, 1), x);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) mine.get(i, j, x[2 * j], x[2 * j + 1]);
        }
        if (divide || odd) {
            append_codes_slow(x, s_new, divide, code);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float a, b, d, e;
                ptx::f2_split(ptx::mul2(x[2 * j], inv2), a, b);
                ptx::f2_split(ptx::mul2(x[2 * j + 1], inv2), d, e);
                code[j] = e4m3_pair(a, b) | e4m3_pair(d, e) << 16;
            }
        }
        *reinterpret_cast<uint2*>(dst + 8 * l.a) = make_uint2(code[0], code[1]);
        *reinterpret_cast<uint2*>(dst + 8 * l.b) = make_uint2(code[2], code[3]);
        dst += D << step_shift;
    }
    if (slot0 > 0 && s_new > s_old) {  // the block's earlier tokens move to the larger scale, a round of memory latency a vector
        const float ratio = s_old * inv;
        uint2* had = reinterpret_cast<uint2*>((u.is_v ? c.v : c.k) + cache_offset(block, u.h, 0, c.Hkv, c.block_size, D));
        for (int v = t; v < slot0 * (D / 8); v += threads) {
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
