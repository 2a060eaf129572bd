// kernel_rope.cuh -- rotary positions and norms of heads, forward and backward (attn_rope, attn_rope_bwd).
//
// A row x is one head of one token at position p.  With a norm u = x w / sqrt(mean(x^2) + eps), else u = x; the pairs
// (a, b) that the layout names are turned by p f_i and scaled by m, y_a = m (u_a cos - u_b sin), y_b = m (u_b cos + u_a
// sin); what is not rotated stays u.  f_i comes as a fraction of a turn in 64 bits, so the angle p f_i is an integer
// product that drops whole turns by itself, right to |p| 2^-65 turns; its upper 32 bits are taken, and no table is read.
//
// Backward: g is the upstream gradient turned back, dw = sum over rows of g x r, and dx = r (g w - x r c) with r =
// 1 / sqrt(mean(x^2) + eps) and c = mean(g w x r); r is computed again from x, which has to be read in any case.
//
// Bound by the bytes: each element is read once and written once, from and to any layout of rows.  A lane holds both
// elements of each of its pairs, two vectors of 16 bytes, and keeps its token for all of its heads, so the sines are
// computed once for up to 8 rows.  What it took to come near the bytes was enough of them under way (RopeRing) and few
// instructions a row (two elements each).  4 x 4096 tokens of 48 heads of 128, 403 MB: 60.0 us, 6.7 TB/s, where the
// measured copy has 6.8; with norms 2 x 4096 of 32 + 8 + 8: forward 32.3 us for 201 MB, backward 45.7 for 285, and 52.0
// with the weights' gradients, which a second kernel adds up.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"
#include "ptx_stream.cuh"
#include "rope.cuh"
#include "rope_index.h"

namespace attn {

struct RopeFwdParams {
    RopeParams r;
    RopePlan plan;
    int S;
    RopeRows in, out;
};
struct RopeBwdParams {
    RopeParams r;
    RopePlan plan;
    int S;
    RopeRows up, in, out;     // upstream gradients; the forward's input (where normed); the input's gradient
    float* part[2];           // [units of q], [units of k][D]: the weights' gradients by unit; null: not wanted
};

struct RopePlace {
    const RopeFwdParams& p;
    __device__ bool operator()(long long b, long long s, long long* position) const {
        *position = rope_position(p.r, b, s);
        return true;
    }
};
// Blocks an SM: one more takes registers from what is kept (without norms 62.0 us where 7 take 60.3), and of the backward
// with norms, below, 5 take 69 us and 3 take 55 where 4 take 52.
template <int D, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads, kNorm ? 5 : 7) attn_rope_kernel(const __grid_constant__ RopeFwdParams p) {
    __shared__ __align__(16) unsigned char ring[RopeRing<2, kRopeDepth, kRopeThreads>::kBytes];
    ptx::launch_next();
    ptx::wait_previous();
    rope_forward<D, kInter, kNorm, kRopeThreads>(p.r, p.plan, blockIdx.x, p.S, p.in, p.out, RopePlace{p}, ring);
}

template <int D, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads, kNorm ? 4 : 6) attn_rope_bwd_kernel(const __grid_constant__ RopeBwdParams p) {
    constexpr int kLanes = D / 16, kWarps = kRopeThreads / 32;
    __shared__ __align__(16) unsigned char smem[RopeRing<kNorm ? 4 : 2, kRopeDepth, kRopeThreads>::kBytes];
    __shared__ float part[kNorm ? kWarps * D : 1];
    ptx::launch_next();
    ptx::wait_previous();
    RopeTask t;
    const bool there = rope_task<D>(p.plan, blockIdx.x, p.S, t);
    const int lane = threadIdx.x % kLanes, kind = t.kind;
    const RopeLane l = rope_lane(lane, D, p.r.rot, kInter);
    const bool copy = kind == 2;
    const void* weight = copy ? nullptr : p.r.weight[kind];
    const bool normed = kNorm && weight;
    const auto at = [&](const RopeRows& x) {
        return reinterpret_cast<uint4*>(x.p[kind] + t.b * x.stride[kind][0] + t.s * x.stride[kind][2] + (unsigned int)t.head * x.stride[kind][1]);
    };
    const uint4 *up = at(p.up), *in = normed ? at(p.in) : nullptr;
    uint4* out = p.out.p[kind] ? at(p.out) : nullptr;
    const long long up_step = p.plan.groups * p.up.stride[kind][1] / 8, in_step = p.plan.groups * p.in.stride[kind][1] / 8,
                    out_step = p.plan.groups * p.out.stride[kind][1] / 8;
    const int rows = there && t.head < t.end ? (t.end - t.head + p.plan.groups - 1) >> p.plan.group_shift : 0;  // of this thread
    const RopeRing<kNorm ? 4 : 2, kRopeDepth, kRopeThreads> ring(smem);
    int next = 0;  // the row whose copies leave next
    const auto fill = [&](int slot) {
        const bool mine = next < rows;
        const uint4* g = mine ? up : reinterpret_cast<const uint4*>(p.up.p[kind]);
        ring.fill(slot, 0, g + l.a, mine);
        ring.fill(slot, 1, g + l.b, mine);
        if (normed) {
            const uint4* x = mine ? in : reinterpret_cast<const uint4*>(p.in.p[kind]);
            ring.fill(slot, 2, x + l.a, mine);
            ring.fill(slot, 3, x + l.b, mine);
            in += in_step;
        }
        ptx::cp_async_commit();
        up += up_step;
        ++next;
    };
#pragma unroll
    for (int i = 0; i < kRopeDepth; ++i) fill(i);
    RopeTurn<kInter> turn;
    if (!copy) turn.template set<true>(p.r, p.r.turns, l, lane, rope_position(p.r, t.b, t.s));
    uint64_t w[8], dw[8];
    if (normed) rope_weights(weight, p.r.weight_f32, l, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = 0;
#pragma unroll 1
    for (int i = 0; i < t.most; ++i) {
        const int slot = i % kRopeDepth;
        ptx::cp_async_wait<kRopeDepth - 1>();
        uint4 a = ring.at(slot, 0), b = ring.at(slot, 1);
        if (!copy) {
            uint64_t g[8];
            rope_unpack(a, b, g);
            turn.template turn<false>(g);
            if (normed) {  // rows that are not there have g = 0
                uint64_t x[8];
                float down;
                rope_unpack(ring.at(slot, 2), ring.at(slot, 3), x);
                const float r = rope_norm<kLanes>(x, p.r.eps, &down);
                rope_scale(x, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dw[i] = ptx::fma2(g[i], x[i], dw[i]);
                    g[i] = ptx::mul2(g[i], w[i]);
                }
                const uint64_t c = rope_both(rope_row_sum<kLanes>(rope_dot(g, x)) * (-1.f / D));
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = ptx::fma2(x[i], c, g[i]);
                rope_scale(g, r * down);
            }
            rope_pack(g, a, b);
        }
        if (out) {
            if (i < rows) {
                out[l.a] = a;
                out[l.b] = b;
            }
            out += out_step;
        }
        fill(slot);  // once the slot's values are out of it
    }
    ptx::cp_async_wait<0>();
    if constexpr (kNorm) {
        if (!normed || !p.part[kind]) return;
        // The block's rows, in a fixed order: within a warp, then over the warps.
        float sums[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) ptx::f2_split(dw[i], sums[2 * i], sums[2 * i + 1]);
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int i = kLanes; i < 32; i *= 2) sums[j] += __shfl_xor_sync(0xffffffffu, sums[j], i);
        if (threadIdx.x % 32 < kLanes) {
            float* to = part + threadIdx.x / 32 * D;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                to[8 * l.a + j] = sums[j];
                to[8 * l.b + j] = sums[8 + j];
            }
        }
        __syncthreads();
        if (threadIdx.x < D) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) sum += part[i * D + threadIdx.x];
            const RopeUnit u = rope_unit(p.plan, blockIdx.x);
            p.part[kind][((long long)u.tile * p.plan.chunks[kind] + u.chunk) * D + threadIdx.x] = sum;
        }
    }
}

// The sum of the units' parts of a weight's gradient, in a fixed order: 8 columns a block, 256 rows side by side, so
// that those of 8192 tokens and 32 heads (2048 units) are all on their way at once.  With the units' own sums, the end of the
// kernel before it and its start it makes the weights' gradients 6 us of the backward above.
struct RopeSumParams {
    const float* part[2];
    long long rows[2];
    void* out[2];  // null: not wanted
    int D, f32;
};
constexpr int kRopeSumThreads = 512, kRopeSumColumns = 8;
__global__ void __launch_bounds__(kRopeSumThreads) attn_rope_sum_kernel(const __grid_constant__ RopeSumParams p) {
    constexpr int kLanes = kRopeSumColumns / 4, kSide = kRopeSumThreads / kLanes;  // four columns a thread
    __shared__ float4 part[kRopeSumThreads / 32][kLanes];
    ptx::launch_next();
    ptx::wait_previous();
    const int blocks = p.D / kRopeSumColumns, kind = blockIdx.x / blocks, base = (blockIdx.x - kind * blocks) * kRopeSumColumns;
    if (!p.out[kind]) return;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    const auto add = [&](const float4& x) {
        sum.x += x.x;
        sum.y += x.y;
        sum.z += x.z;
        sum.w += x.w;
    };
    const float* from = p.part[kind] + base + threadIdx.x % kLanes * 4;
#pragma unroll 8
    for (long long i = threadIdx.x / kLanes; i < p.rows[kind]; i += kSide) add(*reinterpret_cast<const float4*>(from + i * p.D));
#pragma unroll
    for (int i = kLanes; i < 32; i *= 2)
        add(make_float4(__shfl_xor_sync(0xffffffffu, sum.x, i), __shfl_xor_sync(0xffffffffu, sum.y, i), __shfl_xor_sync(0xffffffffu, sum.z, i),
                        __shfl_xor_sync(0xffffffffu, sum.w, i)));
    if (threadIdx.x % 32 < kLanes) part[threadIdx.x / 32][threadIdx.x % kLanes] = sum;
    __syncthreads();
    if (threadIdx.x >= kRopeSumColumns) return;
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < kRopeSumThreads / 32; ++i) total += reinterpret_cast<const float*>(part[i])[threadIdx.x];
    if (p.f32)
        static_cast<float*>(p.out[kind])[base + threadIdx.x] = total;
    else
        static_cast<__nv_bfloat16*>(p.out[kind])[base + threadIdx.x] = __float2bfloat16_rn(total);
}

}  // namespace attn
