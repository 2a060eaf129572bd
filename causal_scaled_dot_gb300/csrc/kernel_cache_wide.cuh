// kernel_cache_wide.cuh -- attention over the 8-bit cache for many query rows:
// the rows are the tensor core's M.
//
// With more than a few rows a tile's exponentials come before its bytes, and the
// row-per-column form of kernel_cache_fwd.cuh, where 128 threads vote on a
// maximum for every few scores, is bound by the latency of its steps.  Here a
// thread owns a query row of a tile of 128 and sees all its scores:
//     S [128 rows x 128 keys]  = Qhi K^T + Qlo K^T     (E4M3, both pieces into the same columns)
//     O [128 rows x D]        += P V                   (f16, P as an operand in tensor memory)
// so the running maximum, the sum and the rescaling of O are the thread's own,
// without a barrier between warps.  V's scale within the weight, the plan and the join are as there.
//
// The weights are f16: two E4M3 pieces into the same columns would stand on one grid of
// 2^-9, and weights below it would be lost, which thousands of keys together are not;
// f16 reaches to 2^-24 under a largest weight of 2^6 .. 2^15, with 11 bits.  V's codes
// are widened for it, exactly, a half at a time: its rows of K are free once its S is
// there, so the first 64 columns of V go there and the others back to where V came from.
//
// A CTA is one warpgroup of softmax, a warp that copies pages and a warp that
// issues products; two CTAs share an SM.  A step is 64 keys, half a tile: the
// products of one half run while the other half's weights are worked out.
// Tensor memory of a CTA: S of two halves [0, 64), [64, 128), O [128, 256); the
// weights, two a column, replace the scores they came from (a half's first 32 columns).
//
// 2 x 1024 tokens at the end of 8192, 32 heads over 8, D = 128: 269 us, 956 TFLOP/s.  Two threads a row (half
// of a step's keys each) double what is around the weights, and a step of 128 keys leaves no tensor memory for a second
// buffer of S.  The wait for the O of two halves ago before each S costs 1.6 % of that: products of different kinds are
// not counted on to end in the order they were issued.
#pragma once

#include <type_traits>

#include "kernel_cache_fwd.cuh"

namespace attn {

struct CacheWideLayout {
    static constexpr int kR = 128;                 // query rows of a unit
    static constexpr bool kWide = true;
    static constexpr int kThreads = 192;           // warps 0-3 softmax, 4 pages, 5 products
    static constexpr int kCtas = 2;                // per SM
    static constexpr int kJoin = 8;                // pieces that one CTA joins
    static constexpr int kStages = 2;
    static constexpr uint32_t kTileBytes = 128 * 128;
    static constexpr uint32_t kStageBytes = 2 * kTileBytes;
    static constexpr uint32_t kQ = kStages * kStageBytes;             // hi, lo: 128 rows x 128 bytes each
    static constexpr uint32_t kInfo = kQ + 2 * kTileBytes;
    static constexpr uint32_t kInfoBytes = 112;
    static constexpr uint32_t kNanAt = kInfo + kStages * kInfoBytes;  // 2 x [128] first key with NaN in V's column
    static constexpr uint32_t kScan = kNanAt + 1024;                  // 20 int + 4 int
    static constexpr uint32_t kShared = kScan + 96;                   // 2 x CacheShared
    static constexpr uint32_t kBars = kShared + 128;
    static constexpr int kKFull = 0, kVFull = 0, kEmpty = kStages, kQFull = 2 * kStages, kSFull = kQFull + 1,
                         kPFull = kSFull + 2, kPvDone = kPFull + 2, kOFull = kPvDone + 1, kDrain = kOFull + 1, kNumBars = kDrain + 1;
    static constexpr uint32_t kTmemSlot = kBars + kNumBars * 8;
    static constexpr uint32_t kAbort = kTmemSlot + 4;
    static constexpr uint32_t kNanSeen = kAbort + 4;  // [2]
    static constexpr uint32_t kDynamicSmem = kNanSeen + 8 + 1024;
    static_assert(kInfo % 16 == 0 && kScan % 16 == 0 && kShared % 8 == 0 && kBars % 8 == 0, "alignment");
    static_assert(kCtas * (kDynamicSmem + 1024) <= 228 * 1024, "shared memory budget");
    static constexpr uint32_t kTmemCols = 256, kS = 0, kO = 128;
};

// No weight may pass 2^15 (f16's largest is almost 2^16), and where a half's largest is below 2^-8, a row's maximum
// falls to it: the weights lost in a half, less than 2^-25 each, are less than 2^-11 of its largest.  Rows of the same warp
// that are below 2^-2 then fall too: left to fall one by one, 32 rows under a key that is 12 nats above the rest look for
// their maxima that much more often (2 x 512 tokens over 4096: 108 us, and 95 together).
constexpr CacheRange kCacheWideRange{6.f, -2.f, 15.f};
constexpr float kCacheWideLow = 0x1p-8f, kCacheWideTop = 0x1p15f;

// The halves of a unit's key tile t that have a key some row sees (one at least).
__device__ __forceinline__ int cache_halves(const CacheUnit& u, int t) { return t * kCacheTile + 64 < u.keys ? 2 : 1; }

__device__ void cache_wide_mma_role(const CacheFwdParams& p, CacheCursor cur, uint32_t base, uint32_t tmem,
                                    volatile int* abort_flag) {
    using L = CacheWideLayout;
    constexpr uint32_t kIdescS = ptx::idesc_e4m3_f32(128, 64, false);
    const uint64_t lim = p.wait_limit_ns;
    const bool wide = p.c.D == 128, leader = ptx::elect_one();
    const uint32_t idesc_o = wide ? ptx::idesc_f16_f32(128, 128, true) : ptx::idesc_f16_f32(128, 64, true);
    bool ok = true;
    auto wait = [&](int bar, uint32_t par) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_call(cache_bar<L>(base, bar), par, abort_flag, p.c.status, lim));
        return ok;
    };
    const uint64_t q_hi = ptx::sdesc_rows<128>(base + L::kQ), q_lo = ptx::sdesc_rows<128>(base + L::kQ + L::kTileBytes);
    int stage = 0;            // of the half whose S is next
    uint32_t phase = 0;
    uint32_t step = 0;        // number of that half
    // The half before, whose O is still to come: its stage, half, and what it ends.
    int prev_stage = -1, prev_half = 0;
    bool prev_first = false, prev_ends_tile = false, prev_ends_unit = false;
    auto issue_pv = [&]() -> bool {
        const uint32_t sb = (step - 1) & 1;
        if (!wait(L::kPFull + (int)sb, ((step - 1) >> 1) & 1)) return false;
        ptx::tc_fence_after();
        if (leader) {
            // 64 keys = 64 rows of 128 bytes in each block of 64 columns.
            const uint64_t vd = ptx::sdesc_sw128(base + (uint32_t)prev_stage * L::kStageBytes + (uint32_t)prev_half * 8192u,
                                                 L::kTileBytes, 1024);
            ptx::mma_ts_k64(tmem + L::kO, tmem + L::kS + sb * 64, vd, idesc_o, prev_first ? 0u : 1u);
            ptx::mma_commit(cache_bar<L>(base, L::kPvDone));
            if (prev_ends_tile) ptx::mma_commit(cache_bar<L>(base, L::kEmpty + prev_stage));
            if (prev_ends_unit) ptx::mma_commit(cache_bar<L>(base, L::kOFull));
        }
        prev_stage = -1;
        return true;
    };
    CacheUnit u;
    for (int unit = 0; ok && cursor_next(p.plan, cur, u); ++unit) {
        const int n = __shfl_sync(0xffffffffu, u.n, 0);
        if (!wait(L::kQFull, unit & 1)) break;
        for (int k = 0; ok && k < n; ++k) {
            const int halves = __shfl_sync(0xffffffffu, cache_halves(u, u.t + k), 0);
            for (int h = 0; h < halves; ++h, ++step) {
                // The O of two halves ago, the last one issued here, has read its weights out of the columns of this S.
                // (At a unit's start all of the unit before is done, or its O would not have left.)
                if ((k > 0 || h > 0) && !wait(L::kPvDone, step & 1)) break;
                // Where the tile's pages are still on their way, the last half's O goes first.
                if (h == 0 && !__any_sync(0xffffffffu, ptx::mbar_test_wait(cache_bar<L>(base, L::kKFull + stage), phase))) {
                    if (prev_stage >= 0 && !issue_pv()) break;
                    if (!wait(L::kKFull + stage, phase)) break;
                }
                ptx::tc_fence_after();
                if (leader) {
                    const uint64_t kd = ptx::sdesc_rows<128>(base + (uint32_t)stage * L::kStageBytes + (uint32_t)h * 8192u);
                    const uint32_t st = tmem + L::kS + (step & 1) * 64;
                    if (wide) {
                        ptx::mma_ss_f8_x4<2, 2>(st, q_hi, kd, kIdescS, 0u);
                        ptx::mma_ss_f8_x4<2, 2>(st, q_lo, kd, kIdescS, 1u);
                    } else {  // D = 64: the other half of the rows is zero in K
                        ptx::mma_ss_f8(st, q_hi, kd, kIdescS, 0u);
                        ptx::mma_ss_f8(st, q_hi + 2, kd + 2, kIdescS, 1u);
                        ptx::mma_ss_f8(st, q_lo, kd, kIdescS, 1u);
                        ptx::mma_ss_f8(st, q_lo + 2, kd + 2, kIdescS, 1u);
                    }
                    ptx::mma_commit(cache_bar<L>(base, L::kSFull + (int)(step & 1)));
                }
                if (prev_stage >= 0 && !issue_pv()) break;
                prev_stage = stage;
                prev_half = h;
                prev_first = k == 0 && h == 0;
                prev_ends_tile = h == halves - 1;
                prev_ends_unit = prev_ends_tile && k == n - 1;
            }
            if (++stage == L::kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        // The next unit's q comes after this one's O.
        if (ok && prev_stage >= 0) issue_pv();
    }
    if (leader) {
        ptx::mma_commit(cache_bar<L>(base, L::kDrain));
        ptx::drain_wait(cache_bar<L>(base, L::kDrain), 0u, lim);
    }
}

// Widens V's codes of a half's 64 keys, rows `row0` on of a tile, to f16, MN-major in rows of 64 columns: columns 0-63 to
// the key's row of K's place (the products that read it are done) and 64-127 to its own.  Two lanes of a warp share a key.
// A weight of 0 times NaN is NaN: a key that nobody sees becomes 0, and NaN that only some rows see is taken out and
// noted by the first position that has it.
__device__ __forceinline__ void cache_widen_half(uint32_t at_stage, int row0, int key0, int D, int keys, int keys_all, int* nan_at,
                                                 volatile int* nan_seen) {
    using L = CacheWideLayout;
    const int lane = threadIdx.x & 31, part = lane >> 4, i = (threadIdx.x >> 5) * 16 + (lane & 15), row = row0 + i, key = key0 + i;
    const uint32_t k_row = at_stage + (uint32_t)row * 128u, v_row = k_row + L::kTileBytes;
    const bool gone = key >= keys;
    if (key0 + 64 > keys_all) {
        if (part == 0 && !gone && key >= keys_all && cache_take_nan(v_row, row, key, nan_at)) *nan_seen = 1;
        __syncwarp();
    }
    uint4 x[4];
    auto load = [&](int first, int n) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (c >= n) break;
            x[c] = ptx::ld_shared_v4(v_row + (uint32_t)(((first + c) ^ (row & 7)) << 4));
            if (gone) x[c] = make_uint4(0, 0, 0, 0);
        }
    };
    auto store = [&](uint32_t to, int first, int n) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (c >= n) break;
            const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
            for (int y = 0; y < 2; ++y)
                ptx::st_shared_v4(to + (uint32_t)((((first + c) * 2 + y) ^ (row & 7)) << 4), e4m3_to_f16x2(w[2 * y]),
                                  e4m3_to_f16x2(w[2 * y] >> 16), e4m3_to_f16x2(w[2 * y + 1]), e4m3_to_f16x2(w[2 * y + 1] >> 16));
        }
    };
    if (D == 128) {
        load(4 * part, 4);
        __syncwarp();  // both halves of a key's codes are read before its row is written
        store(part ? v_row : k_row, 0, 4);
    } else {
        load(2 * part, 2);
        store(k_row, 2 * part, 2);
    }
}

__device__ void cache_wide_softmax_role(const CacheFwdParams& p, CacheCursor cur, int total, int ctas,
                                        uint32_t base, uint8_t* smem, uint32_t tmem, volatile int* abort_flag) {
    using L = CacheWideLayout;
    const int r = threadIdx.x, lane = r & 31;  // this thread's row of a unit, and its lane of S and O
    const uint32_t my_tmem = tmem + ((uint32_t)(r & ~31) << 16);
    const int D = p.c.D, shift = p.c.block_shift;
    // A wait that ran out leaves this false: the lane goes on without waiting and without writing results.  No
    // warp waits for another here but through the bounded barriers.
    bool alive = true;
    auto wait = [&](int which, uint32_t par) {
        if (alive) alive = ptx::mbar_wait_call(cache_bar<L>(base, which), par, abort_flag, p.c.status, p.wait_limit_ns);
        __syncwarp();
    };
    auto arrive = [&](int which) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(cache_bar<L>(base, which));
    };
    int stage = 0;
    uint32_t phase = 0, step = 0;
    CacheUnit u;
    for (int unit = 0; cursor_next(p.plan, cur, u); ++unit) {
        int* nan_at = reinterpret_cast<int*>(smem + L::kNanAt) + (unit & 1) * 128;
        volatile int* nan_seen = reinterpret_cast<volatile int*>(smem + L::kNanSeen) + (unit & 1);
        // ---- q in two pieces, a row per thread: all its loads leave together
        int qi, hq;
        const bool used = cache_row(p, u, r, &qi, &hq);
        const long long at = used ? ((long long)u.b * p.Hq + hq) * p.Sq + qi : -1;
        const int keys = !used ? 0 : p.plan.causal ? max(u.s.first + qi + 1, 0) : u.s.len;
        const int keys_all = p.plan.causal ? max(u.s.first + u.qt * p.plan.qper + 1, 0) : u.s.len;
        float factor;  // of the row's scores
        bool finite;
        {
            uint4 x[16];
            const __nv_bfloat16* from = p.q + u.b * p.q_stride[0] + hq * p.q_stride[1] + qi * p.q_stride[2];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = used && i < D / 8 ? reinterpret_cast<const uint4*>(from)[i] : make_uint4(0, 0, 0, 0);
            // the largest magnitude, by bit pattern; not finite: the whole row is NaN
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                         __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
            m = max(m & 0xffffu, m >> 16);
            const float scale = e4m3_pow2_scale(__uint_as_float(m << 16));
            finite = m < 0x7f80u;
            const float inv = finite ? __uint_as_float((254u << 23) - __float_as_uint(scale)) : NAN;
            factor = scale * p.scale_log2;
            const uint32_t line = base + L::kQ + (uint32_t)r * 128u;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t v[8] = {x[2 * i].x,     x[2 * i].y,     x[2 * i].z,     x[2 * i].w,
                                       x[2 * i + 1].x, x[2 * i + 1].y, x[2 * i + 1].z, x[2 * i + 1].w};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float a0 = __uint_as_float(v[e] << 16) * inv, a1 = __uint_as_float(v[e] & 0xffff0000u) * inv;
                    const float a2 = __uint_as_float(v[e + 1] << 16) * inv, a3 = __uint_as_float(v[e + 1] & 0xffff0000u) * inv;
                    const uint32_t h0 = e4m3_pair(a0, a1), h1 = e4m3_pair(a2, a3);
                    const float2 f0 = e4m3_unpair(h0), f1 = e4m3_unpair(h1);
                    hi[e / 2] = h0 | h1 << 16;
                    lo[e / 2] = e4m3_pair(a0 - f0.x, a1 - f0.y) | (uint32_t)e4m3_pair(a2 - f1.x, a3 - f1.y) << 16;
                }
                const uint32_t to = line + (uint32_t)((i ^ (r & 7)) << 4);
                ptx::st_shared_v4(to, hi[0], hi[1], hi[2], hi[3]);
                ptx::st_shared_v4(to + L::kTileBytes, lo[0], lo[1], lo[2], lo[3]);
            }
        }
        if (!used) factor = 0.f;
        nan_at[r] = 0x7fffffff;
        if (r == 0) {
            *nan_seen = 0;
            if (u.n < u.tiles)
                cache_share(reinterpret_cast<CacheShared*>(smem + L::kShared) + (u.t > 0 ? 0 : 1), u, total, ctas);
        }
        ptx::fence_proxy_async_smem();
        arrive(L::kQFull);

        // of s + log2 vs, its largest so far, and the sum of w / vs; a row of NaN needs none, and is not to ask for one
        float row_max = used && !finite ? 0.f : -INFINITY, peak = row_max, l = 0.f;
        for (int k = 0; k < u.n; ++k) {
            const int halves = cache_halves(u, u.t + k);
            const float* info = reinterpret_cast<const float*>(smem + L::kInfo + stage * L::kInfoBytes);
            for (int h = 0; h < halves; ++h, ++step) {
                const int key0 = (u.t + k) * kCacheTile + h * 64;
                const uint32_t s_addr = my_tmem + L::kS + (step & 1) * 64;
                // S is there, the scales beside K too, and the O of two halves ago is done, which came before it.
                wait(L::kSFull + (int)(step & 1), (step >> 1) & 1);
                ptx::tc_fence_after();
                const int missing = reinterpret_cast<const int*>(info)[24];
                const bool full = key0 + 64 <= keys_all && missing == 0;
                // y = s + log2 vs + base of 16 keys, which share a block: s is the score times K's scale and the row's factor.
                const int seen = keys - key0;  // keys of the half that this row sees
                auto scores = [&](auto masked, int i, const uint32_t* s, float at0, float* y) {
                    const int page = (h * 64 + i * 16) >> shift;
                    const float f = info[page] * factor, c = info[8 + page] + at0;
                    const uint64_t f2 = ptx::f2(f, f), c2 = ptx::f2(c, c);
                    const int last = missing >> page & 1 ? 0 : seen - i * 16;
#pragma unroll
                    for (int x = 0; x < 16; x += 2) {
                        ptx::f2_split(ptx::fma2(ptx::f2(__uint_as_float(s[x]), __uint_as_float(s[x + 1])), f2, c2), y[x], y[x + 1]);
                        if (decltype(masked)::value) {
                            y[x] = x < last ? y[x] : -INFINITY;
                            y[x + 1] = x + 1 < last ? y[x + 1] : -INFINITY;
                        }
                    }
                };
                uint32_t code[32];  // two weights each
                float sum;
                // The weights against the row's maximum as it stands; returns the largest.
                auto pass = [&](auto masked) {
                    const float at0 = row_max == -INFINITY ? -INFINITY : kCacheWideRange.room - row_max;
                    float top = 0.f;
                    sum = 0.f;
                    uint32_t both[32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (i % 2 == 0) ptx::tmem_load<32>(s_addr + 16 * i, both);
                        const uint32_t* s = both + i % 2 * 16;
                        float y[16];
                        scores(masked, i, s, at0, y);
                        const float ivs = info[16 + ((h * 64 + i * 16) >> shift)];
                        uint64_t part = ptx::f2(0.f, 0.f);
#pragma unroll
                        for (int x = 0; x < 16; x += 4) {
                            float w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) w[e] = ptx::ex2(y[x + e]);
                            top = ptx::max3(top, w[0], w[1]);
                            top = ptx::max3(top, w[2], w[3]);
                            part = ptx::add2(part, ptx::add2(ptx::f2(w[0], w[1]), ptx::f2(w[2], w[3])));
                            code[i * 8 + x / 2] = ptx::pack_f16x2(w[0], w[1]);
                            code[i * 8 + x / 2 + 1] = ptx::pack_f16x2(w[2], w[3]);
                        }
                        float a, b;
                        ptx::f2_split(part, a, b);
                        sum = fmaf(a + b, ivs, sum);
                    }
                    return top;
                };
                // First as it stands; once more when some row's maximum has to rise or fall, or only so while one has none.
                for (bool move = __any_sync(0xffffffffu, row_max == -INFINITY && seen > 0);;) {
                    if (move) {
                        // Every row of the warp takes the maximum that it should have.
                        float m = -INFINITY;
#pragma unroll 1
                        for (int i = 0; i < 4; ++i) {
                            uint32_t s[16];
                            ptx::tmem_load<16>(s_addr + 16 * i, s);
                            float y[16];
                            scores(std::true_type(), i, s, 0.f, y);
#pragma unroll
                            for (int x = 0; x < 16; x += 2) m = ptx::max3(m, y[x], y[x + 1]);
                        }
                        bool moves;
                        m = cache_new_max(kCacheWideRange, row_max, peak, used ? m : -INFINITY, &moves);
                        const float f = row_max == -INFINITY ? 0.f : ptx::ex2(row_max - m);
                        row_max = m;
                        peak = fmaxf(peak, m);
                        l *= f;
                        if (k > 0 || h > 0) {
                            // The half before has its weights against the old maximum: its product has to be in O.
                            wait(L::kPvDone, (step - 1) & 1);
                            ptx::tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t s[32];
                                ptx::tmem_load<32>(my_tmem + L::kO + c, s);
#pragma unroll
                                for (int x = 0; x < 32; ++x) s[x] = __float_as_uint(__uint_as_float(s[x]) * f);
                                ptx::tmem_store<32>(my_tmem + L::kO + c, s);
                            }
                        }
                    }
                    const float top = full ? pass(std::false_type()) : pass(std::true_type());
                    const bool low = top < kCacheWideLow && top > 0.f && row_max > peak - kCacheFall;
                    if (move || !__any_sync(0xffffffffu, top > kCacheWideTop || low)) break;
                    move = true;
                }
                l += sum;
                ptx::tmem_st32(s_addr, code);
                if (h == 0) wait(L::kVFull + stage, phase);
                if (__all_sync(0xffffffffu, alive))
                    cache_widen_half(base + (uint32_t)stage * L::kStageBytes, h * 64, key0, D, u.keys, keys_all, nan_at, nan_seen);
                ptx::fence_proxy_async_smem();
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                arrive(L::kPFull + (int)(step & 1));
            }
            if (++stage == L::kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }

        // ---- the row leaves
        wait(L::kOFull, unit & 1);
        ptx::tc_fence_after();
        const bool whole = u.n == u.tiles, nan = *nan_seen != 0;
        const long long slot = (long long)blockIdx.x * 2 + (u.t > 0 ? 0 : 1);
        const float f = !whole ? 1.f : l == 0.f ? 0.f : ptx::rcp(l);
        if (alive && whole && at >= 0 && p.lse != nullptr)
            p.lse[at] = l == 0.f ? -INFINITY : (row_max - kCacheWideRange.room + ptx::lg2(l)) * kLn2;
        if (alive && !whole && used) p.part_ml[slot * L::kR + r] = make_float2(row_max - kCacheWideRange.room, l);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
            uint32_t s[32];
            ptx::tmem_load<32>(my_tmem + L::kO + c, s);
#pragma unroll
            for (int x = 0; x < 32; ++x) s[x] = __float_as_uint(__uint_as_float(s[x]) * f);
            if (nan) {
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    if (nan_at[c + x] < keys) s[x] = 0x7fffffffu;
            }
            if (alive && used) {
                if (!whole) {  // four columns of all rows side by side: [32][128] float4
                    uint4* to = reinterpret_cast<uint4*>(p.part_o) + (slot * 32 + c / 4) * L::kR + r;
#pragma unroll
                    for (int x = 0; x < 8; ++x) to[x * L::kR] = make_uint4(s[4 * x], s[4 * x + 1], s[4 * x + 2], s[4 * x + 3]);
                } else {
                    uint4* to = reinterpret_cast<uint4*>(p.out + at * D + c);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = ptx::pack_bf16x2(__uint_as_float(s[8 * x + 2 * e]), __uint_as_float(s[8 * x + 2 * e + 1]));
                        to[x] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
        }
        ptx::tc_fence_before();
    }
}

// Joins a shared unit, a row per thread of warps 0-3; 32 columns of two pieces are under way at once.
__device__ void cache_wide_join(const CacheFwdParams& p, const CacheJoin& join) {
    using L = CacheWideLayout;
    const int r = threadIdx.x, n = join.n;
    const CacheUnit& u = join.shared.u;
    int qi, hq;
    if (r >= L::kR || !cache_row(p, u, r, &qi, &hq)) return;
    const long long at = ((long long)u.b * p.Hq + hq) * p.Sq + qi;
    auto slot = [&](int x) { return join.slot(x); };
    float m = -INFINITY, l = 0.f;
#pragma unroll 4
    for (int x = 0; x < n; ++x) {
        const float2 ml = __ldcg(p.part_ml + slot(x) * L::kR + r);
        const float top = fmaxf(m, ml.x), ref = top == -INFINITY ? 0.f : top;
        l = l * ptx::ex2(m - ref) + ptx::ex2(ml.x - ref) * ml.y;
        m = top;
    }
    const float inv = l == 0.f ? 0.f : ptx::rcp(l), ref = m == -INFINITY ? 0.f : m;
    if (join.final && p.lse != nullptr) p.lse[at] = l == 0.f ? -INFINITY : (m + ptx::lg2(l)) * kLn2;
    for (int c = 0; c < p.c.D / 4; c += 8) {
        float4 o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int x = 0; x < n; ++x) {
            float4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __ldcg(reinterpret_cast<const float4*>(p.part_o) + (slot(x) * 32 + c + i) * L::kR + r);
            const float f = ptx::ex2(__ldcg(p.part_ml + slot(x) * L::kR + r).x - ref);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[i] = make_float4(o[i].x + f * v[i].x, o[i].y + f * v[i].y, o[i].z + f * v[i].z, o[i].w + f * v[i].w);
        }
        if (!join.final) {  // where this thread alone has read
#pragma unroll
            for (int i = 0; i < 8; ++i) reinterpret_cast<float4*>(p.part_o)[(slot(0) * 32 + c + i) * L::kR + r] = o[i];
            continue;
        }
        uint4* to = reinterpret_cast<uint4*>(p.out + at * p.c.D + c * 4);
#pragma unroll
        for (int i = 0; i < 8; i += 2)
            to[i / 2] = make_uint4(ptx::pack_bf16x2(o[i].x * inv, o[i].y * inv), ptx::pack_bf16x2(o[i].z * inv, o[i].w * inv),
                                   ptx::pack_bf16x2(o[i + 1].x * inv, o[i + 1].y * inv),
                                   ptx::pack_bf16x2(o[i + 1].z * inv, o[i + 1].w * inv));
    }
    if (!join.final) p.part_ml[slot(0) * L::kR + r] = make_float2(m, l);
}

__global__ void __launch_bounds__(CacheWideLayout::kThreads, CacheWideLayout::kCtas)
    attn_cache_fwd_wide_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                               const __grid_constant__ CacheFwdParams p) {
    using L = CacheWideLayout;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmemSlot);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);

    if (threadIdx.x == 160) {
        for (int s = 0; s < L::kStages; ++s) {
            ptx::mbar_init(cache_bar<L>(base, L::kKFull + s), 2);  // K and V
            ptx::mbar_init(cache_bar<L>(base, L::kEmpty + s), 1);
        }
        ptx::mbar_init(cache_bar<L>(base, L::kQFull), 4);  // the softmax warps
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(cache_bar<L>(base, L::kSFull + i), 1);
            ptx::mbar_init(cache_bar<L>(base, L::kPFull + i), 4);
        }
        ptx::mbar_init(cache_bar<L>(base, L::kPvDone), 1);
        ptx::mbar_init(cache_bar<L>(base, L::kOFull), 1);
        ptx::mbar_init(cache_bar<L>(base, L::kDrain), 1);
        *abort_flag = 0;
        for (int x = 0; x < 2; ++x) reinterpret_cast<CacheShared*>(smem + L::kShared)[x].pieces = 0;
        ptx::fence_barrier_init();
        ptx::prefetch_tensormap(&tm_k);
        ptx::prefetch_tensormap(&tm_v);
    }
    if (warp == 4) {
        ptx::tmem_alloc(ptx::smem_addr(tmem_slot), L::kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    int begin, end, total;
    CachePlace place;
    const int ctas = cache_locate<L::kThreads>(p.plan, reinterpret_cast<int*>(smem + L::kScan), p.c.status, &begin, &end,
                                               &total, &place);  // barriers of the block within
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

    if (begin == end) {
        // no tile for this CTA
    } else if (warp == 4) {
        cache_load_role<L>(&tm_k, &tm_v, p, cursor_at(p.plan, place, begin, end - begin), total, ctas, base, smem, abort_flag);
    } else if (warp == 5) {
        cache_wide_mma_role(p, cursor_at(p.plan, place, begin, end - begin), base, tmem, abort_flag);
    } else {
        cache_wide_softmax_role(p, cursor_at(p.plan, place, begin, end - begin), total, ctas, base, smem, tmem, abort_flag);
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, L::kTmemCols);
    }
    cache_join<L>(p, reinterpret_cast<const int*>(smem + L::kScan), reinterpret_cast<CacheShared*>(smem + L::kShared),
                  *abort_flag != 0, [&](const CacheJoin& x) { cache_wide_join(p, x); });
}

}  // namespace attn
