// kernel_rope.cuh -- rotary positions and norms of heads, forward and backward (attn_rope, attn_rope_bwd).
//
// A row x is one head of one token at position p.  With a norm u = x w / sqrt(mean(x^2) + eps), else u = x; the pairs
// (a, b) that the layout names are turned by p f_i and scaled by m, y_a = m (u_a cos - u_b sin), y_b = m (u_b cos + u_a
// sin); what is not rotated stays u.  f_i comes as a fraction of a turn in 64 bits, so the angle p f_i is an integer
// product that drops whole turns by itself: exact to |p| 2^-65 turns at any position, and no table is read.
//
// Backward: g is the upstream gradient turned back, dw = sum over rows of g x r, and dx = r (g w - x r c) with r =
// 1 / sqrt(mean(x^2) + eps) and c = mean(g w x r); r is computed again from x, which has to be read in any case.
//
// Bound by the bytes: each element is read once and written once, from and to any layout of rows.  A lane holds both
// elements of each of its pairs, two vectors of 16 bytes, and keeps its token for all of its heads, so the sines are
// computed once for many rows.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"
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
template <int D, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads) attn_rope_kernel(const __grid_constant__ RopeFwdParams p) {
    ptx::launch_next();
    ptx::wait_previous();
    rope_forward<D, kInter, kNorm>(p.r, p.plan, blockIdx.x, p.S, p.in, p.out, RopePlace{p});
}

template <int D, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kRopeThreads) attn_rope_bwd_kernel(const __grid_constant__ RopeBwdParams p) {
    constexpr int kLanes = D / 16, kWarps = kRopeThreads / 32;
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
    const __nv_bfloat16* up = p.up.p[kind] + t.b * p.up.stride[kind][0] + t.s * p.up.stride[kind][2];
    const __nv_bfloat16* in = normed ? p.in.p[kind] + t.b * p.in.stride[kind][0] + t.s * p.in.stride[kind][2] : nullptr;
    __nv_bfloat16* out = p.out.p[kind] ? p.out.p[kind] + t.b * p.out.stride[kind][0] + t.s * p.out.stride[kind][2] : nullptr;
    RopeWaves<kInter> waves;
    if (!copy) waves.at(p.r, l, lane, rope_position(p.r, t.b, t.s));
    float w[16], dw[16];
    if (normed) rope_weights(weight, p.r.weight_f32, l, w);
#pragma unroll
    for (int j = 0; j < 16; ++j) dw[j] = 0.f;
    for (int i = 0; i < p.plan.per; ++i) {
        const int h = t.head + i * p.plan.groups;
        const bool mine = there && h < t.end;
        uint4 a = make_uint4(0, 0, 0, 0), b = a, xa = a, xb = a;
        if (mine) {
            const uint4* g = reinterpret_cast<const uint4*>(up + h * p.up.stride[kind][1]);
            a = g[l.a];
            b = g[l.b];
            if (normed) {
                const uint4* x = reinterpret_cast<const uint4*>(in + h * p.in.stride[kind][1]);
                xa = x[l.a];
                xb = x[l.b];
            }
        }
        if (!copy) {
            float g[16];
            rope_unpack(a, b, g);
            waves.template turn<true>(g);
            if (normed) {
                float x[16], down;
                rope_unpack(xa, xb, x);
                const float r = rope_norm<kLanes>(x, p.r.eps, &down);
                float dot = 0.f;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    x[j] *= r;
                    const float d = g[j] * x[j];
                    if (mine) dw[j] += d;
                    dot = fmaf(d, w[j], dot);
                }
                const float c = rope_row_sum<kLanes>(dot) * (1.f / D), rd = r * down;
#pragma unroll
                for (int j = 0; j < 16; ++j) g[j] = rd * fmaf(-x[j], c, g[j] * w[j]);
            }
            rope_pack(g, a, b);
        }
        if (mine && out) {
            uint4* y = reinterpret_cast<uint4*>(out + h * p.out.stride[kind][1]);
            y[l.a] = a;
            y[l.b] = b;
        }
    }
    if (!kNorm || !normed || !p.part[kind]) return;
    // The block's rows, in a fixed order: within a warp, then over the warps.
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int i = kLanes; i < 32; i *= 2) dw[j] += __shfl_xor_sync(0xffffffffu, dw[j], i);
    if (threadIdx.x % 32 < kLanes) {
        float* to = part + threadIdx.x / 32 * D;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            to[8 * l.a + j] = dw[j];
            to[8 * l.b + j] = dw[8 + j];
        }
    }
    __syncthreads();
    if (threadIdx.x < D) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) sum += part[i * D + threadIdx.x];
        const RopeUnit u = rope_unit(p.plan, blockIdx.x);
        p.part[kind][(u.tile * p.plan.chunks[kind] + u.chunk) * D + threadIdx.x] = sum;
    }
}

// The sum of the units' parts of a weight's gradient, in a fixed order: 16 columns a block, 64 rows side by side.
struct RopeSumParams {
    const float* part[2];
    long long rows[2];
    void* out[2];  // null: not wanted
    int D, f32;
};
constexpr int kRopeSumThreads = 1024;
__global__ void __launch_bounds__(kRopeSumThreads) attn_rope_sum_kernel(const __grid_constant__ RopeSumParams p) {
    __shared__ float part[kRopeSumThreads];
    ptx::launch_next();
    ptx::wait_previous();
    const int blocks = p.D / 16, kind = blockIdx.x / blocks, column = (blockIdx.x - kind * blocks) * 16 + threadIdx.x % 16;
    if (!p.out[kind]) return;
    float sum = 0.f;
#pragma unroll 8
    for (long long i = threadIdx.x / 16; i < p.rows[kind]; i += kRopeSumThreads / 16) sum += p.part[kind][i * p.D + column];
    part[threadIdx.x] = sum;
    __syncthreads();
    for (int n = kRopeSumThreads / 2; n >= 16; n /= 2) {
        if (threadIdx.x < n) part[threadIdx.x] += part[threadIdx.x + n];
        __syncthreads();
    }
    if (threadIdx.x >= 16) return;
    if (p.f32)
        static_cast<float*>(p.out[kind])[column] = part[threadIdx.x];
    else
        static_cast<__nv_bfloat16*>(p.out[kind])[column] = __float2bfloat16_rn(part[threadIdx.x]);
}

}  // namespace attn
