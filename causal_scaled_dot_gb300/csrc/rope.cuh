// rope.cuh -- a lane's share of a row that is normed and rotated: the arithmetic that the kernels of kernel_rope.cuh and
// the append to the cache have in common.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"
#include "rope_index.h"

namespace attn {

// What a call's rows have in common (attn_rope_t).
struct RopeParams {
    unsigned long long turns[64];
    int rot;
    float factor, eps;
    const void* weight[2];    // of q and k; null: no norm
    int weight_f32;
    const void* positions;    // or null: first + s
    int positions_64;
    long long position_stride, first;
};
// Rows [B, H, S, D] of q, k and v.
struct RopeRows {
    __nv_bfloat16* p[3];
    long long stride[3][3];   // batch, head, token, in elements
};

// m cos and m sin of position p and frequency F (2^-64 turns).  The product's upper half is the angle as a signed
// fraction of half a turn; what it drops is below 2^-31 of one.
__device__ __forceinline__ void rope_wave(long long p, unsigned long long F, float m, float& c, float& s) {
    const unsigned long long t = (unsigned long long)p * F;
    sincospif((float)(int)(t >> 32) * 4.656612873077393e-10f, &s, &c);
    c *= m;
    s *= m;
}
__device__ __forceinline__ long long rope_position(const RopeParams& r, long long b, long long s) {
    if (!r.positions) return r.first + s;
    const long long i = b * r.position_stride + s;
    return r.positions_64 ? static_cast<const long long*>(r.positions)[i] : static_cast<const int*>(r.positions)[i];
}

// A lane's share of a row in fp32: x[0..7] its vector a, x[8..15] its vector b.
__device__ __forceinline__ void rope_unpack(const uint4& a, const uint4& b, float (&x)[16]) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void rope_pack(const float (&x)[16], uint4& a, uint4& b) {
    a = make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]), ptx::pack_bf16x2(x[4], x[5]),
                   ptx::pack_bf16x2(x[6], x[7]));
    b = make_uint4(ptx::pack_bf16x2(x[8], x[9]), ptx::pack_bf16x2(x[10], x[11]), ptx::pack_bf16x2(x[12], x[13]),
                   ptx::pack_bf16x2(x[14], x[15]));
}

// The lane's 8 pairs: half layout (x[j], x[8 + j]); interleaved (x[2 j], x[2 j + 1]).
template <bool kInter>
struct RopeWaves {
    float c[8], s[8];
    bool turn_a, turn_b;
    __device__ __forceinline__ void at(const RopeParams& r, const RopeLane& l, int lane, long long p) {
        turn_a = l.turn_a;
        turn_b = l.turn_b;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            c[j] = 1.f;
            s[j] = 0.f;
            const bool turn = kInter && j >= 4 ? turn_b : turn_a;
            const int pair = kInter ? (j < 4 ? 4 * l.a + j : 4 * l.b + j - 4) : 8 * lane + j;
            if (turn) rope_wave(p, r.turns[pair], r.factor, c[j], s[j]);
        }
    }
    // Forward, or with `back` the transposed rotation.  Elements that are not rotated stay as they are, whatever they are.
    template <bool kBack>
    __device__ __forceinline__ void turn(float (&x)[16]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (!(kInter && j >= 4 ? turn_b : turn_a)) continue;
            const int i = kInter ? 2 * j : j, k = kInter ? 2 * j + 1 : 8 + j;
            const float sn = kBack ? -s[j] : s[j], u = x[i], v = x[k];
            x[i] = u * c[j] - v * sn;
            x[k] = v * c[j] + u * sn;
        }
    }
};

// The lane's weights of a norm.
__device__ __forceinline__ void rope_weights(const void* weight, int f32, const RopeLane& l, float (&w)[16]) {
    if (f32) {
        const float4* p = static_cast<const float4*>(weight);
        const float4 q[4] = {p[2 * l.a], p[2 * l.a + 1], p[2 * l.b], p[2 * l.b + 1]};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[4 * i] = q[i].x;
            w[4 * i + 1] = q[i].y;
            w[4 * i + 2] = q[i].z;
            w[4 * i + 3] = q[i].w;
        }
    } else {
        const uint4* p = static_cast<const uint4*>(weight);
        rope_unpack(p[l.a], p[l.b], w);
    }
}

// Sum over a row's lanes (neighbouring, kLanes a power of two).
template <int kLanes>
__device__ __forceinline__ float rope_row_sum(float x) {
#pragma unroll
    for (int i = 1; i < kLanes; i *= 2) x += __shfl_xor_sync(0xffffffffu, x, i);
    return x;
}
__device__ __forceinline__ float rope_squares(const float (&x)[16]) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        a = fmaf(x[i], x[i], a);
        b = fmaf(x[i + 1], x[i + 1], b);
    }
    return a + b;
}
// r of a row.  bf16's largest values have squares beyond fp32: such a row's x (not its infinities) is taken 2^-72 times
// smaller, where eps is nothing beside it, and *down is what r x is to be of x's own size.
template <int kLanes>
__device__ __forceinline__ float rope_norm(float (&x)[16], float eps, float* down) {
    constexpr float kInv = 1.f / (16 * kLanes);
    float ss = rope_row_sum<kLanes>(rope_squares(x));
    *down = 1.f;
    const bool big = ss == INFINITY;
    if (__any_sync(0xffffffffu, big)) {
        if (big) {
            *down = 2.117582368135751e-22f;  // 2^-72
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] *= 2.117582368135751e-22f;
        }
        const float again = rope_row_sum<kLanes>(rope_squares(x));
        if (big) return rsqrtf(again * kInv);
    }
    return rsqrtf(fmaf(ss, kInv, eps));
}

template <int kLanes>
__device__ __forceinline__ void rope_normed(float (&x)[16], const float (&w)[16], float eps) {
    float down;
    const float r = rope_norm<kLanes>(x, eps, &down);
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = x[j] * r * w[j];
}

// The rows of a unit that one lane group takes: its token, and heads first, first + groups ... below `end`.
struct RopeTask {
    long long b, s;
    int kind, head, end;
};
template <int D>
__device__ __forceinline__ bool rope_task(const RopePlan& p, unsigned int unit, int S, RopeTask& t) {
    const RopeUnit u = rope_unit(p, unit);
    const int row = threadIdx.x / (D / 16), side = p.tokens == 1 ? row : row / p.tokens;
    const long long token = u.tile * p.tokens + (row - side * p.tokens);
    t.kind = u.kind;
    t.head = u.chunk * p.groups * p.per + side;
    t.end = min(p.heads[u.kind], (u.chunk + 1) * p.groups * p.per);
    const bool there = token < p.total;
    t.b = there ? token / S : 0;
    t.s = there ? token - t.b * S : 0;
    return there;
}

// One unit of the forward.  `place(b, s, &position)`: where row s of sequence b stands, and whether it is one at all.  Every
// lane of a warp goes through the same steps (rows that are not there are computed from zeros and not stored), as the
// sums over a row's lanes ask for whole warps.
template <int D, bool kInter, bool kNorm, typename Place>
__device__ __forceinline__ void rope_forward(const RopeParams& r, const RopePlan& plan, unsigned int unit, int S, const RopeRows& from,
                                             const RopeRows& to, const Place& place) {
    constexpr int kLanes = D / 16;
    RopeTask t;
    bool there = rope_task<D>(plan, unit, S, t);
    const int lane = threadIdx.x % kLanes, kind = t.kind;
    const RopeLane l = rope_lane(lane, D, r.rot, kInter);
    long long position;
    there = place(t.b, t.s, &position) && there;
    const __nv_bfloat16* in = from.p[kind] + t.b * from.stride[kind][0] + t.s * from.stride[kind][2];
    __nv_bfloat16* out = to.p[kind] + t.b * to.stride[kind][0] + t.s * to.stride[kind][2];
    const bool copy = kind == 2;
    RopeWaves<kInter> waves;
    if (!copy) waves.at(r, l, lane, position);
    const void* weight = copy ? nullptr : r.weight[kind];
    float w[16];
    if (kNorm && weight) rope_weights(weight, r.weight_f32, l, w);
    for (int i = 0; i < plan.per; ++i) {
        const int h = t.head + i * plan.groups;
        const bool mine = there && h < t.end;
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (mine) {
            const uint4* x = reinterpret_cast<const uint4*>(in + h * from.stride[kind][1]);
            a = x[l.a];
            b = x[l.b];
        }
        if (!copy) {
            float x[16];
            rope_unpack(a, b, x);
            if (kNorm && weight) rope_normed<kLanes>(x, w, r.eps);
            waves.template turn<false>(x);
            rope_pack(x, a, b);
        }
        if (mine) {
            uint4* y = reinterpret_cast<uint4*>(out + h * to.stride[kind][1]);
            y[l.a] = a;
            y[l.b] = b;
        }
    }
}

}  // namespace attn
