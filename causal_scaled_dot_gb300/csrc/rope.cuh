// rope.cuh -- a lane's share of a row that is normed and rotated: the arithmetic that the kernels of kernel_rope.cuh and
// the append to the cache have in common.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"
#include "ptx_stream.cuh"
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

// cos and sin of position p and two frequencies (2^-64 turns), packed.  The product's upper half is the angle as a signed
// fraction of a turn (what it drops is below 2^-32 of one).  Twice that, as an integer, is the rest x in -1/2 .. 1/2 half
// turns, and both signs turn where its top bit differs from the angle's.  cos(pi x) = C(x^2) and sin(pi x) = x S(x^2) by
// the polynomials with the least largest error there (exchange algorithm of Remez): 7.7e-8 and 4.8e-8 with coefficients
// rounded to fp32, and with the other roundings 2.0e-7 and 1.7e-7 over two million angles, under 2^-22.
__device__ __forceinline__ void rope_wave2(long long p, unsigned long long F0, unsigned long long F1, uint64_t& c, uint64_t& s) {
    const uint32_t t0 = (uint32_t)((unsigned long long)p * F0 >> 32), t1 = (uint32_t)((unsigned long long)p * F1 >> 32);
    const auto both = [](float x) { return ptx::f2(x, x); };
    const uint64_t x = ptx::mul2(ptx::f2((float)(int)(t0 << 1), (float)(int)(t1 << 1)), both(2.3283064365386963e-10f));
    const uint64_t y = ptx::mul2(x, x);
    c = ptx::fma2(y, both(0.2200806587934494f), both(-1.3320938348770142f));
    c = ptx::fma2(y, c, both(4.058451175689697f));
    c = ptx::fma2(y, c, both(-4.934795379638672f));
    c = ptx::fma2(y, c, both(1.f));
    s = ptx::fma2(y, both(0.07722225040197372f), both(-0.5980464220046997f));
    s = ptx::fma2(y, s, both(2.5500316619873047f));
    s = ptx::fma2(y, s, both(-5.1677069664001465f));
    s = ptx::fma2(y, s, both(3.141592502593994f));
    s = ptx::mul2(s, x);
    const uint32_t f0 = (t0 ^ t0 << 1) & 0x80000000u, f1 = (t1 ^ t1 << 1) & 0x80000000u;
    const auto flip = [&](uint64_t v) {
        float lo, hi;
        ptx::f2_split(v, lo, hi);
        return ptx::f2(__uint_as_float(__float_as_uint(lo) ^ f0), __uint_as_float(__float_as_uint(hi) ^ f1));
    };
    c = flip(c);
    s = flip(s);
}
__device__ __forceinline__ long long rope_position(const RopeParams& r, long long b, long long s) {
    if (!r.positions) return r.first + s;
    const long long i = b * r.position_stride + s;
    return r.positions_64 ? static_cast<const long long*>(r.positions)[i] : static_cast<const int*>(r.positions)[i];
}

// A lane's share of a row in fp32, two elements a word: x[0..3] its vector a, x[4..7] its vector b.
__device__ __forceinline__ void rope_unpack(const uint4& a, const uint4& b, uint64_t (&x)[8]) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = ptx::f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ uint32_t rope_pack(uint64_t x) {
    float lo, hi;
    ptx::f2_split(x, lo, hi);
    return ptx::pack_bf16x2(lo, hi);
}
__device__ __forceinline__ void rope_pack(const uint64_t (&x)[8], uint4& a, uint4& b) {
    a = make_uint4(rope_pack(x[0]), rope_pack(x[1]), rope_pack(x[2]), rope_pack(x[3]));
    b = make_uint4(rope_pack(x[4]), rope_pack(x[5]), rope_pack(x[6]), rope_pack(x[7]));
}
__device__ __forceinline__ uint64_t rope_both(float x) { return ptx::f2(x, x); }
__device__ __forceinline__ uint64_t rope_swap(uint64_t x) {
    float lo, hi;
    ptx::f2_split(x, lo, hi);
    return ptx::f2(hi, lo);
}
__device__ __forceinline__ uint64_t rope_negate(uint64_t x) { return x ^ 0x8000000080000000ull; }

// The lane's weights of a norm, in the places of its elements.
__device__ __forceinline__ void rope_weights(const void* weight, int f32, const RopeLane& l, uint64_t (&w)[8]) {
    if (f32) {
        const float4* p = static_cast<const float4*>(weight);
        const float4 q[4] = {p[2 * l.a], p[2 * l.a + 1], p[2 * l.b], p[2 * l.b + 1]};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[2 * i] = ptx::f2(q[i].x, q[i].y);
            w[2 * i + 1] = ptx::f2(q[i].z, q[i].w);
        }
    } else {
        const uint4* p = static_cast<const uint4*>(weight);
        rope_unpack(p[l.a], p[l.b], w);
    }
}

// The rotation of a lane's elements as y = x p + z q, z their partners: the other vector in the half layout, the other of
// the two in the interleaved one.  Of elements that are not rotated p is 1 and q not used.
template <bool kInter>
struct RopeTurn {
    uint64_t p[8], q[8];
    bool turn_a, turn_b;

    // Position `at`; kBack: the transposed rotation.  `turns`: r.turns, or a copy of it where the lanes' reads, which a
    // constant bank serves one after the other, come more often.
    template <bool kBack>
    __device__ __forceinline__ void set(const RopeParams& r, const unsigned long long* turns, const RopeLane& l, int lane, long long at) {
        turn_a = l.turn_a;
        turn_b = l.turn_b;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[i] = rope_both(1.f);
            q[i] = 0;
        }
        if (kInter) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {  // pairs i and i + 1 of the lane, one in a word
                if (!(i < 4 ? turn_a : turn_b)) continue;
                const int pair = i < 4 ? 4 * l.a + i : 4 * l.b + i - 4;
                uint64_t c, s;
                rope_wave2(at, turns[pair], turns[pair + 1], c, s);
                float c0, c1, s0, s1;
                ptx::f2_split(c, c0, c1);
                ptx::f2_split(s, s0, s1);
                p[i] = rope_both(c0);
                p[i + 1] = rope_both(c1);
                q[i] = kBack ? ptx::f2(s0, -s0) : ptx::f2(-s0, s0);
                q[i + 1] = kBack ? ptx::f2(s1, -s1) : ptx::f2(-s1, s1);
            }
        } else if (turn_a) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint64_t c, s;
                rope_wave2(at, turns[8 * lane + 2 * i], turns[8 * lane + 2 * i + 1], c, s);
                p[i] = p[i + 4] = c;
                q[i] = kBack ? s : rope_negate(s);
                q[i + 4] = kBack ? rope_negate(s) : s;
            }
        }
        if (r.factor != 1.f) {
            const uint64_t m = rope_both(r.factor);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (!(i < 4 || !kInter ? turn_a : turn_b)) continue;
                p[i] = ptx::mul2(p[i], m);
                q[i] = ptx::mul2(q[i], m);
            }
        }
    }
    // With weights before the rotation: y = (x w) p + (z w') q.
    __device__ __forceinline__ void weigh(const uint64_t (&w)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[i] = ptx::mul2(p[i], w[i]);
            q[i] = ptx::mul2(q[i], kInter ? rope_swap(w[i]) : w[i ^ 4]);
        }
    }
    // y from x.  kWeighed: elements that are not rotated have weights too; else they stay as they are, whatever they are.
    template <bool kWeighed>
    __device__ __forceinline__ void turn(uint64_t (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i)  // half layout: words i and i + 4 together
            if (kInter) {
                if (i < 4 ? turn_a : turn_b)
                    x[i] = ptx::fma2(rope_swap(x[i]), q[i], ptx::mul2(x[i], p[i]));
                else if (kWeighed)
                    x[i] = ptx::mul2(x[i], p[i]);
            } else if (i < 4) {
                if (turn_a) {
                    const uint64_t u = x[i], v = x[i + 4];
                    x[i] = ptx::fma2(v, q[i], ptx::mul2(u, p[i]));
                    x[i + 4] = ptx::fma2(u, q[i + 4], ptx::mul2(v, p[i + 4]));
                } else if (kWeighed) {
                    x[i] = ptx::mul2(x[i], p[i]);
                    x[i + 4] = ptx::mul2(x[i + 4], p[i + 4]);
                }
            }
    }
};

// The sines of one row's pairs, two in a word, for a row that is the only one of its token: half of RopeTurn's registers.
template <bool kInter>
struct RopeWaves {
    uint64_t c[4], s[4];

    __device__ __forceinline__ void set(const RopeParams& r, const unsigned long long* turns, const RopeLane& l, int lane, long long at) {
        const uint64_t m = rope_both(r.factor);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!(kInter && i >= 2 ? l.turn_b : l.turn_a)) continue;
            const int pair = !kInter ? 8 * lane + 2 * i : i < 2 ? 4 * l.a + 2 * i : 4 * l.b + 2 * i - 4;
            rope_wave2(at, turns[pair], turns[pair + 1], c[i], s[i]);
            c[i] = ptx::mul2(c[i], m);
            s[i] = ptx::mul2(s[i], m);
        }
    }
    // The forward rotation; elements that are not rotated stay as they are.
    __device__ __forceinline__ void turn(const RopeLane& l, uint64_t (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!(kInter && i >= 2 ? l.turn_b : l.turn_a)) continue;
            if (kInter) {
                float c0, c1, s0, s1;
                ptx::f2_split(c[i], c0, c1);
                ptx::f2_split(s[i], s0, s1);
                x[2 * i] = ptx::fma2(rope_swap(x[2 * i]), ptx::f2(-s0, s0), ptx::mul2(x[2 * i], rope_both(c0)));
                x[2 * i + 1] = ptx::fma2(rope_swap(x[2 * i + 1]), ptx::f2(-s1, s1), ptx::mul2(x[2 * i + 1], rope_both(c1)));
            } else {
                const uint64_t u = x[i], v = x[i + 4];
                x[i] = ptx::fma2(v, rope_negate(s[i]), ptx::mul2(u, c[i]));
                x[i + 4] = ptx::fma2(u, s[i], ptx::mul2(v, c[i]));
            }
        }
    }
};

// Sum over a row's lanes (neighbouring, kLanes a power of two).
template <int kLanes>
__device__ __forceinline__ float rope_row_sum(float x) {
#pragma unroll
    for (int i = 1; i < kLanes; i *= 2) x += __shfl_xor_sync(0xffffffffu, x, i);
    return x;
}
// The sum of the products of a lane's elements.
__device__ __forceinline__ float rope_dot(const uint64_t (&x)[8], const uint64_t (&y)[8]) {
    uint64_t a = ptx::mul2(x[0], y[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) a = ptx::fma2(x[i], y[i], a);
    float lo, hi;
    ptx::f2_split(a, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ void rope_scale(uint64_t (&x)[8], float by) {
    const uint64_t b = rope_both(by);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = ptx::mul2(x[i], b);
}
// r of a row.  bf16's largest values have squares beyond fp32: where mean(x^2) + eps is infinite the row's x (not its
// infinities) is taken 2^-72 times smaller and eps 2^-144 times, and *down is what r x is to be of x's own size.
template <int kLanes>
__device__ __forceinline__ float rope_norm(uint64_t (&x)[8], float eps, float* down) {
    constexpr float kInv = 1.f / (16 * kLanes), kDown = 2.117582368135751e-22f;  // 2^-72
    const float mean = fmaf(rope_row_sum<kLanes>(rope_dot(x, x)), kInv, eps);
    *down = 1.f;
    const bool big = mean == INFINITY;
    if (__any_sync(0xffffffffu, big)) {
        if (big) {
            *down = kDown;
            rope_scale(x, kDown);
        }
        const float again = rope_row_sum<kLanes>(rope_dot(x, x));
        if (big) return rsqrtf(fmaf(again, kInv, eps * kDown * kDown));
    }
    return rsqrtf(mean);
}

// The rows of a unit that one lane group takes: its token, and heads first, first + groups ... below `end`.
struct RopeTask {
    unsigned int b, s;
    int kind, head, end;
    int most;  // rows of the thread that has most of them, the same for the block
};
template <int D>
__device__ __forceinline__ bool rope_task(const RopePlan& p, unsigned int unit, int S, RopeTask& t) {
    const RopeUnit u = rope_unit(p, unit);
    const int row = threadIdx.x / (D / 16), side = row >> p.token_shift;
    const unsigned int token = (u.tile << p.token_shift) + (row & (p.tokens - 1));
    t.kind = u.kind;
    const int most = p.per << p.group_shift, begin = u.chunk * most;
    t.head = begin + side;
    t.end = min(p.heads[u.kind], begin + most);
    t.most = (t.end - begin + p.groups - 1) >> p.group_shift;
    const bool there = token < p.total;
    t.b = there ? token / (unsigned int)S : 0;
    t.s = there ? token - t.b * (unsigned int)S : 0;
    return there;
}

// A thread's rows on their way: kVectors vectors of a row at a time, kDepth rows ahead, in shared memory that only this
// thread writes and reads, so nothing but its own copies is waited for.  Registers for as many rows would cost the warps
// that hide the latency: with one row ahead in registers the forward with norms took 44 us (2 x 4096 tokens of 32 + 8 + 8
// heads of 128), and 32 so.
template <int kVectors, int kDepth, int kThreads>
struct RopeRing {
    static constexpr int kBytes = kVectors * kDepth * kThreads * 16;
    uint32_t base;
    __device__ __forceinline__ explicit RopeRing(void* smem) : base(ptx::smem_addr(smem) + threadIdx.x * 16) {}
    __device__ __forceinline__ void fill(int slot, int vector, const void* src, bool there) const {
        ptx::cp_async_16(base + (slot * kVectors + vector) * kThreads * 16, src, there);
    }
    __device__ __forceinline__ uint4 at(int slot, int vector) const {
        uint4 x;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                     : "r"(base + (slot * kVectors + vector) * kThreads * 16)
                     : "memory");
        return x;
    }
    // Two words of fp32 pairs in a vector's place.
    __device__ __forceinline__ void put(int slot, int vector, uint64_t x, uint64_t y) const {
        asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(base + (slot * kVectors + vector) * kThreads * 16), "l"(x), "l"(y)
                     : "memory");
    }
    __device__ __forceinline__ void get(int slot, int vector, uint64_t& x, uint64_t& y) const {
        asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];"
                     : "=l"(x), "=l"(y)
                     : "r"(base + (slot * kVectors + vector) * kThreads * 16)
                     : "memory");
    }
};
// Rows ahead: with 2 the forward with norms takes 35.8 us where 4 take 32.4, with 6 its backward 55.9 and 52.4.
constexpr int kRopeDepth = 4;

// One unit of the forward.  `place(b, s, &position)`: where row s of sequence b stands, and whether it is one at all.  Every
// lane of a warp goes through the same steps (rows that are not there are computed from zeros and not stored), as the
// sums over a row's lanes ask for whole warps.
template <int D, bool kInter, bool kNorm, int kThreads, typename Place>
__device__ __forceinline__ void rope_forward(const RopeParams& r, const RopePlan& plan, unsigned int unit, int S, const RopeRows& from,
                                             const RopeRows& to, const Place& place, void* smem) {
    constexpr int kLanes = D / 16;
    const RopeRing<2, kRopeDepth, kThreads> ring(smem);
    RopeTask t;
    bool there = rope_task<D>(plan, unit, S, t);
    const int lane = threadIdx.x % kLanes, kind = t.kind;
    const RopeLane l = rope_lane(lane, D, r.rot, kInter);
    long long position;
    there = place(t.b, t.s, &position) && there;
    const __nv_bfloat16* base = from.p[kind] + t.b * from.stride[kind][0] + t.s * from.stride[kind][2];
    const uint4* in = reinterpret_cast<const uint4*>(base + (unsigned int)t.head * from.stride[kind][1]);
    uint4* out = reinterpret_cast<uint4*>(to.p[kind] + t.b * to.stride[kind][0] + t.s * to.stride[kind][2] + (unsigned int)t.head * to.stride[kind][1]);
    const long long in_step = plan.groups * from.stride[kind][1] / 8, out_step = plan.groups * to.stride[kind][1] / 8;
    const int rows = there && t.head < t.end ? (t.end - t.head + plan.groups - 1) >> plan.group_shift : 0;  // of this thread
    int next = 0;  // the row whose copy leaves next
    const auto fill = [&](int slot) {
        const bool mine = next < rows;
        const uint4* x = mine ? in : reinterpret_cast<const uint4*>(from.p[kind]);
        ring.fill(slot, 0, x + l.a, mine);
        ring.fill(slot, 1, x + l.b, mine);
        ptx::cp_async_commit();
        in += in_step;
        ++next;
    };
#pragma unroll
    for (int i = 0; i < kRopeDepth; ++i) fill(i);
    const bool copy = kind == 2;
    RopeTurn<kInter> turn;
    const void* weight = copy ? nullptr : r.weight[kind];
    const bool normed = kNorm && weight;
    if (!copy) {
        uint64_t w[8];
        if (normed) rope_weights(weight, r.weight_f32, l, w);
        turn.template set<false>(r, r.turns, l, lane, position);
        if (normed) turn.weigh(w);
    }
#pragma unroll 1
    for (int i = 0; i < t.most; ++i) {
        const int slot = i % kRopeDepth;
        ptx::cp_async_wait<kRopeDepth - 1>();
        uint4 a = ring.at(slot, 0), b = ring.at(slot, 1);
        if (!copy) {
            uint64_t x[8];
            rope_unpack(a, b, x);
            if (normed) {
                float down;
                const float rr = rope_norm<kLanes>(x, r.eps, &down);
                turn.template turn<true>(x);
                rope_scale(x, rr);
            } else {
                turn.template turn<false>(x);
            }
            rope_pack(x, a, b);
        }
        if (i < rows) {
            out[l.a] = a;
            out[l.b] = b;
        }
        out += out_step;
        fill(slot);  // once the slot's values are out of it
    }
    ptx::cp_async_wait<0>();
}

}  // namespace attn
