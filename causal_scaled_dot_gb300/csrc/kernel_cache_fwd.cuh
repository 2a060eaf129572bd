// kernel_cache_fwd.cuh -- attention over the 8-bit cache on sm_103a.
//
// The codes go from the cache to the tensor cores as they are: TMA copies whole
// pages into shared memory and tcgen05.mma kind::f8f6f4 multiplies E4M3 by
// E4M3, so no byte of K or V is ever widened.  What must not be rounded to
// E4M3's 4 significant bits, q and the softmax weights, enters as two E4M3
// pieces, x = hi + lo with hi the nearest code and lo the nearest code to the
// rest: 8 significant bits, which is all of a bf16 q (down to 2^-18 of its row's
// largest element, where lo underflows) and bf16's precision for the weights,
// whose lo stands 2^4 times larger, in columns of its own.
//
// Both products are computed transposed, so that the few query rows of a
// decoding step are the narrow N side of the instruction and not its M = 128:
//     S^T [128 keys x 2R] = K [128 x D] * Qp^T,   Qp = R rows hi, R rows lo
//     O^T [D x 2R]       += V^T [D x 128 keys] * Pp^T
// with R = 8, 16 or 32 query rows (the queries of a tile times the query heads
// of one key/value head); kernel_cache_wide.cuh takes more.  A product of K = 32 takes 64 cycles for any N up
// to 128 (the 128 rows of the cache's operand have to be read), so the pieces
// are columns of one product rather than two products into the same columns.
// In S^T a thread owns one key, so a block's scales are one factor per thread.  V's scale vs joins the weight:
//     w_j = 2^(s_j + log2 vs_j - M + 4),   M = max_j (s_j + log2 vs_j),
//     O = (sum_j w_j code_j) / (sum_j w_j / vs_j),
// so that a row's largest w is near 2^4 whatever the scales and lo's underflow
// (2^-14) is 2^-18 of it.  M rises only when some w passes 448 (E4M3's largest), and
// falls where no weight of a tile reaches 1, since what the others then lose to the
// underflow may be all that a long sequence consists of: the weights lost in a tile are
// less than 2^-7 of its largest one.  Then the warpgroup finds the tile's maxima and
// rescales O^T in tensor memory, which costs twice a tile's time; otherwise a tile needs
// one vote of the warpgroup, with the rows that reached 1 beside it, and no reduction.
// The sum of w / vs is kept per thread (per key) and reduced at the end.
//
// Roles: warp 0 copies pages (lane i takes page i of a tile) with
// the tables and scales of the pages ahead already in registers; warp 1
// issues the products; warps 2-3 split the next unit's q rows into pieces;
// the rest are two (R = 8, 16) or four softmax warpgroups, each with its part of
// the R rows: four interleave better, since a vote makes the warps of one wait
// for its slowest.
// CTAs take equal runs of key tiles of all units (cache_index.h); a unit that
// crosses into the next CTA leaves partial (O, M, l), and whichever CTA is the
// last to leave its piece joins them, in the order of the pieces.
//
// What bounds it: one token over a long cache moves 2 bytes per (key, d) pair
// and is bound by HBM; with R = 32 the latency of a tile's steps (products, vote,
// weights, fences) is longer than its bytes take.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "cache_index.h"
#include "cache_tickets.h"
#include "common.cuh"
#include "kernel_cache_rw.cuh"
#include "ptx.cuh"
#include "ptx_cache.cuh"

namespace attn {

struct CacheFwdParams {
    CacheView c;
    CachePlan plan;
    const __nv_bfloat16* q;
    long long q_stride[3];  // batch, head, token, in elements
    __nv_bfloat16* out;
    float* lse;             // may be null
    int Hq, Sq, group;
    int hper;               // query heads of a unit
    int hper_inv;           // ceil(2^16 / hper): r / hper = r * hper_inv >> 16 for r < 128
    int hgroups;            // units that share a key/value head: ceil(group / hper)
    float scale_log2;       // scale * log2(e)
    float* part_o;          // [G][2][R][128] partial sums of w code
    float2* part_ml;        // [G][2][R] their M - 4 and sum of w / vs
    unsigned long long* tickets;  // [2][G], cache_tickets.h, and this launch's number
    unsigned long long ticket;
    unsigned long long wait_limit_ns;
};

template <int R>
struct CacheLayout {
    static constexpr bool kWide = false;
    static constexpr int kWgs = R >= 32 ? 4 : 2;   // softmax warpgroups
    static constexpr int kThreads = 128 + 128 * kWgs;
    static constexpr int kH = R / kWgs;            // rows of one softmax warpgroup
    static constexpr int kCtas = R == 8 ? 2 : 1;   // per SM
    static constexpr int kJoin = 24;               // pieces that one CTA joins
    static constexpr int kStages = R == 8 ? 3 : R == 16 ? 6 : 5;
    static constexpr int kN = 2 * R;               // rows of Qp and Pp: hi and lo pieces
    static constexpr int kWidth = 2 * kH;          // columns of one softmax warpgroup: its rows' hi, then lo pieces
    // Row r's hi piece in Qp, S^T and O^T; the lo piece is kH further.
    __host__ __device__ static constexpr int hi_row(int r) { return r / kH * 2 * kH + r % kH; }
    static constexpr uint32_t kTileBytes = 128 * 128;       // 128 keys x 128 bytes
    static constexpr uint32_t kStageBytes = 2 * kTileBytes; // K, V
    static constexpr uint32_t kQ = kStages * kStageBytes;   // 2 x [2R x 128 bytes]
    static constexpr uint32_t kP = kQ + 2 * kN * 128;       // 2 x [2R x 128 keys]
    static constexpr uint32_t kInfo = kP + 2 * kN * 128;  // per stage and page: K's scale, log2 of V's, 1 / V's; bad pages
    static constexpr uint32_t kInfoBytes = 112;
    static constexpr uint32_t kRows = kInfo + kStages * kInfoBytes;  // 2 x [R] CacheRow
    static constexpr uint32_t kUnit = kRows + 2 * R * 16;            // 2 x CacheWork
    static constexpr uint32_t kTab = kUnit + 2 * 48;                 // [R / 2] float4 {two rows' factors, their 4 - M}
    static constexpr uint32_t kFac = kTab + R * 8;                   // [R] float: what l and O are multiplied by
    static constexpr uint32_t kRed = kFac + R * 4;                   // [R][4 warps] float
    static constexpr uint32_t kNanAt = kRed + R * 16;                // 2 x [128] first key with NaN in V's column
    static constexpr uint32_t kScan = kNanAt + 1024;                 // 20 int + 4 int
    static constexpr uint32_t kBars = kScan + 96;
    static constexpr int kKFull = 0, kVFull = kStages, kEmpty = 2 * kStages, kQFull = 3 * kStages, kQEmpty = kQFull + 2,
                         kSFull = kQEmpty + 2, kPFull = kSFull + 2, kOFull = kPFull + 2, kOFree = kOFull + 2, kNan = kOFree + 2, kDrain = kNan + 2,
                         kNumBars = kDrain + 1;
    static constexpr uint32_t kTmemSlot = kBars + kNumBars * 8;
    static constexpr uint32_t kAbort = kTmemSlot + 4;
    static constexpr uint32_t kNanSeen = kAbort + 4;  // [2]
    static constexpr uint32_t kReach = (kNanSeen + 8 + 15) & ~15u;   // 2 x [kWgs][4 warps]: rows with a weight of 1
    static constexpr uint32_t kShared = kReach + 2 * kWgs * 16;      // 2 x CacheShared
    static constexpr uint32_t kDynamicSmem = kShared + 2 * 64 + 1024;
    static_assert(kInfo % 16 == 0 && kRows % 16 == 0 && kUnit % 16 == 0 && kTab % 16 == 0 && kScan % 8 == 0 && kBars % 8 == 0,
                  "alignment");
    static_assert(kCtas * (kDynamicSmem + 1024) <= 228 * 1024, "shared memory budget");
    static constexpr uint32_t kS = 0, kO = 2 * kN;  // S^T of two tiles, O^T of two units
    static constexpr uint32_t kTmemCols = kO + 2 * kN;
    static_assert(kTmemCols >= 32 && (kTmemCols & (kTmemCols - 1)) == 0 && kCtas * kTmemCols <= 512, "tensor memory budget");
    // Pp^T: R = 8 keeps a row per column (K-major, 128 keys = 128 bytes); else a row per key (MN-major,
    // 2R bytes), where a thread writes its key's codes 16 at a time.
    static constexpr bool kPerKey = R > 8;
};

// A query row of a unit in shared memory: the factor of its scores, the keys it
// sees, and its place in out and lse (-1: padding).
struct CacheRow {
    float factor;
    int keys;
    long long at;
};
// A unit in shared memory, for the roles that follow the query warps.
struct CacheWork {
    int t, n;        // key tiles t .. t + n - 1; n = 0: no more units
    int keys;        // keys that some row sees
    int keys_all;    // keys that every row of the unit sees
    int slot;        // -1: the whole unit; else the partial slot (0: begun elsewhere, 1: begun here)
    int rows;        // rows in use
    int pad[6];
};
// A unit that this CTA shares with others, for the join: slot 0 begun elsewhere, 1 begun here.
struct CacheShared {
    CacheUnit u;
    int first, pieces;  // the CTA where it begins, and the CTAs that share it (0: no such unit)
    int last;           // CacheLast: whether this CTA was the last of its group to leave its piece, then of all groups
};
static_assert(sizeof(CacheRow) == 16 && sizeof(CacheWork) == 48 && sizeof(CacheShared) <= 64, "shared memory layout");

template <typename L>
__device__ __forceinline__ uint32_t cache_bar(uint32_t base, int i) {
    return base + L::kBars + 8u * (uint32_t)i;
}

// Sums the plan over the block and finds this CTA's run of tiles; every thread
// of the block calls it, `scan` is shared memory (20 int, then an int4).
// Returns the CTAs that share the tiles.
template <int kThreads>
__device__ int cache_locate(const CachePlan& p, int* scan, unsigned int* status, int* begin, int* end, int* total,
                            CachePlace* place) {
    const int cta = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // A later launch's block on this SM waits for this one and may hold tensor memory meanwhile.  It takes none that this
    // one needs: shared memory admits two R = 8 blocks (64 columns each) or one beside a wide one (256), and no other pair.
    ptx::launch_next();
    ptx::wait_previous();
    const int pairs = p.B * p.q_tiles, per = (pairs + kThreads - 1) / kThreads;
    const int first = min(tid * per, pairs), last = min(first + per, pairs);
    bool bad = false;
    const int mine = plan_chunk(p, first, last, &bad);
    if (bad && cta == 0) atomicOr(status, kStatusBadCache);
    int sum = mine;
    const int steps = pairs < 32 ? pairs : 32;  // lanes of a warp that have something
    for (int o = 1; o < steps; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
    }
    if (lane == steps - 1) scan[warp] = sum;
    __syncthreads();
    int before = sum - mine, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        const int x = scan[w];
        if (w < warp) before += x;
        all += x;
    }
    *total = all;
    const int ctas = plan_ctas(p, all, gridDim.x);
    *begin = plan_begin(all, cta, ctas);
    *end = plan_begin(all, cta + 1, ctas);
    const int want = *begin;
    if (want >= before && want < before + mine)
        *reinterpret_cast<CachePlace*>(scan + 20) = plan_find(p, first, want - before);
    __syncthreads();
    *place = want < all ? *reinterpret_cast<const CachePlace*>(scan + 20) : CachePlace{p.B, 0, 0, 0};
    if (tid == 0) {  // for cache_shared_again
        scan[0] = *begin;
        scan[1] = *end;
        scan[2] = all;
        scan[3] = ctas;
    }
    return ctas;
}

// Row r of a unit: its query, head, and whether it is in use.
__device__ __forceinline__ bool cache_row(const CacheFwdParams& p, const CacheUnit& u, int r, int* i, int* hq) {
    const int iq = r * p.hper_inv >> 16;
    const int hk = p.hgroups == 1 ? u.h : u.h / p.hgroups, g = (u.h - hk * p.hgroups) * p.hper + (r - iq * p.hper);
    *i = u.qt * p.plan.qper + iq;
    *hq = hk * p.group + g;
    return iq < p.plan.qper && *i < u.s.count && g < p.group;
}

// Notes a unit that CTAs share.
__device__ __forceinline__ void cache_share(CacheShared* shared, const CacheUnit& u, int total, int ctas) {
    shared->u = u;
    shared->first = plan_cta(total, u.at, ctas);
    shared->pieces = plan_cta(total, u.at + u.tiles - 1, ctas) - shared->first + 1;
}
struct CacheTicketMemory {
    static __device__ __forceinline__ unsigned long long load(unsigned long long* at) { return __ldcg(at); }
    static __device__ __forceinline__ void compare_exchange(unsigned long long* at, unsigned long long had, unsigned long long to) {
        atomicCAS(at, had, to);
    }
    static __device__ __forceinline__ unsigned long long add(unsigned long long* at, unsigned long long n) { return atomicAdd(at, n); }
    static __device__ __forceinline__ void set(unsigned long long* at, unsigned long long bits) { atomicOr(at, bits); }
    static __device__ __forceinline__ void clear(unsigned long long* at) { atomicExch(at, 0ull); }
};
__device__ __noinline__ void cache_open_tickets(const CacheFwdParams& p, int begin, int tiles, int total, int ctas, int most) {
    const int first = plan_cta(total, begin, ctas), pieces = plan_cta(total, begin + tiles - 1, ctas) - first + 1;
    tickets_open<CacheTicketMemory>(p.tickets, gridDim.x, p.ticket, first, pieces, blockIdx.x - first, most);
}

// Where a row's weights stand, as log2: its largest one when its maximum M is new, the one that some weight of a tile has to
// reach for M to stay, and the one that none may pass.
struct CacheRange {
    float room, low, top;
};
// Room: the weights of the tiles after may be up to 448 / 2^4 = 28 times the largest before M has to rise, which scores of
// unit variance hardly ever ask for (with 2^6 and 7 times, drafted tokens took 5 % more).
// Low: where no weight of a tile reaches 1, M falls to the tile's maximum.  One key far above the rest (a first token that
// every row attends to) would else leave the rest of a long sequence to lo's underflow.  Scores that vary more make M
// move more often: drafted tokens over 5000 keys take 48 us with scores of deviation 1 and 60 with 2; with 2^-2 instead of
// 1 that would be 55, and four times as much could be lost in a tile.
constexpr CacheRange kCacheRange{4.f, 0.f, 8.8f};  // 2^8.8 < 448
constexpr float kCacheTop = 448.f;                 // E4M3's largest value
constexpr uint32_t kCacheReach = 0x38;             // the code of 1
// M does not fall further than this below the largest M that the row has had: what is left out then is 2^-38 of that
// key's weight, and no sum passes 2^126 (a weight of 448 over a V scale of 2^-80, 2^17 times, 20 bits up).
constexpr float kCacheFall = 20.f;

// The maximum that a row with M = had and the largest M so far `peak` takes at a tile whose maximum is `tile`;
// *moves: it has to.
__device__ __forceinline__ float cache_new_max(CacheRange range, float had, float peak, float tile, bool* moves) {
    const bool falls = tile > -INFINITY && tile < had + (range.low - range.room) && had > peak - kCacheFall;
    *moves = falls || tile > had + (range.top - range.room);
    return falls ? fmaxf(tile, peak - kCacheFall) : fmaxf(had, tile);
}

// log2 of the least scale of V that a weight is computed for (values below 4e-22).
constexpr float kCacheLeastScale = -80.f;

// ---------------------------------------------------------------- warp 0: pages
template <typename L>
__device__ void cache_load_role(const CUtensorMap* tm_k, const CUtensorMap* tm_v, const CacheFwdParams& p, CacheCursor cur,
                                int total, int ctas, uint32_t base, uint8_t* smem, volatile int* abort_flag) {
    const CacheView& c = p.c;
    const int lane = threadIdx.x & 31;
    const bool leader = ptx::elect_one();
    const int pages = kCacheTile >> c.block_shift;  // of one tile
    const uint64_t lim = p.wait_limit_ns;
    int stage = 0;
    uint32_t phase = 0, pend = 0, pend_par = 0;
    bool bad = false;
    // One sequence's table as far as some row of the unit sees.
    struct Pages {
        const int* table;
        int last, hk;
    };
    auto pages_of = [&](const CacheUnit& u) {
        return Pages{c.block_table + (long long)u.b * c.max_blocks, (u.keys + c.block_size - 1) >> c.block_shift,
                     p.hgroups == 1 ? u.h : u.h / p.hgroups};
    };
    // Ordinary loads: a write that this launch overlapped (launch()) may have changed scales since it started, which the
    // non-coherent path would not have to see.
    auto entry = [&](const Pages& g, int page) { return page < g.last ? g.table[page] : -1; };
    auto block_of = [&](const Pages& g, int page, int e) { return page < g.last ? cache_block(e, c.num_blocks, &bad) : -1; };
    auto scales = [&](const Pages& g, int block) {
        const long long at = (long long)block * c.Hkv + g.hk;
        return block < 0 ? make_float2(0.f, 0.f) : make_float2(c.k_scale[at], c.v_scale[at]);
    };
    // This lane's page of a window of 32: its block (-1: none) and scales.  What comes after it is under way
    // meanwhile: of a long unit the next window's blocks and scales and the table entries of the one after
    // that, and at a unit's start the first window of the next unit.
    CacheUnit u, u2;
    bool more = cursor_next(p.plan, cur, u);
    Pages g = pages_of(u);
    const int e = more ? entry(g, u.t * pages + lane) : -1;
    int block = more ? block_of(g, u.t * pages + lane, e) : -1;
    float2 sc = scales(g, block);
    while (more) {
        const bool more2 = cursor_next(p.plan, cur, u2);
        const Pages g2 = pages_of(u2);
        const int e2 = more2 ? entry(g2, u2.t * pages + lane) : -1;
        int block2 = -1;
        float2 sc2 = make_float2(0.f, 0.f);
        int window = u.t * pages + lane;
        const bool wide = u.n * pages > 32;
        int next = wide ? block_of(g, window + 32, entry(g, window + 32)) : -1;
        float2 next_sc = scales(g, next);
        int ahead = wide ? entry(g, window + 64) : -1;
        int at = 0;  // the tile's first page in the window
        for (int t = u.t; t < u.t + u.n; ++t) {
            if (at == 32) {
                at = 0;
                window += 32;
                block = next;
                sc = next_sc;
                next = block_of(g, window + 32, ahead);
                next_sc = scales(g, next);
                ahead = entry(g, window + 64);
            }
            bool ok = ptx::mbar_wait_call(cache_bar<L>(base, L::kEmpty + stage), phase ^ 1u, abort_flag, p.c.status, lim);
            if (!__all_sync(0xffffffffu, ok)) goto drain;
            const int i = lane - at;
            const bool mine = i >= 0 && i < pages;
            // A page that is not there is read past the last block, where TMA fills zeros.  Each page's row goes
            // to the whole warp, and one lane issues all copies: their operands have to be uniform.
            const int row = block < 0 ? c.num_blocks * c.Hkv : block * c.Hkv + g.hk;
            uint32_t dst = base + (uint32_t)stage * L::kStageBytes;
            for (int x = 0; x < pages; ++x, dst += 128u << c.block_shift) {
                const int r = __shfl_sync(0xffffffffu, row, at + x);
                if (leader) {
                    ptx::tma_load_3d(dst, tm_k, cache_bar<L>(base, L::kKFull + stage), 0, 0, r);
                    ptx::tma_load_3d(dst + L::kTileBytes, tm_v, cache_bar<L>(base, L::kVFull + stage), 0, 0, r);
                }
            }
            if (t == u.t) {
                block2 = more2 ? block_of(g2, u2.t * pages + lane, e2) : -1;
                sc2 = scales(g2, block2);
                if (leader && u.n < u.tiles) cache_open_tickets(p, u.at, u.tiles, total, ctas, L::kJoin);
                __syncwarp();
            }
            // pages that some row should see but that the table places outside the cache
            const uint32_t missing = __ballot_sync(0xffffffffu, mine && block < 0 && window < g.last) >> at;
            float* info = reinterpret_cast<float*>(smem + L::kInfo + stage * L::kInfoBytes);
            if (mine) {
                const float lvs = fmaxf(ptx::lg2(sc.y), kCacheLeastScale);
                info[i] = sc.x;
                info[8 + i] = lvs;
                info[16 + i] = ptx::ex2(-lvs);
            }
            if (leader) reinterpret_cast<int*>(info)[24] = (int)missing;
            __syncwarp();
            // The copies' bytes may come in before they are announced: the phase ends with this arrival at the earliest.
            if (leader) {
                ptx::mbar_arrive_expect_tx(cache_bar<L>(base, L::kKFull + stage), L::kTileBytes);
                ptx::mbar_arrive_expect_tx(cache_bar<L>(base, L::kVFull + stage), L::kTileBytes);
            }
            pend |= 1u << stage;
            pend_par = (pend_par & ~(1u << stage)) | (phase << stage);
            at += pages;
            if (++stage == L::kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        more = more2;
        u = u2;
        g = g2;
        block = block2;
        sc = sc2;
    }
    if (bad) atomicOr(p.c.status, kStatusBadCache);
    return;
drain:
    for (int s = 0; s < L::kStages; ++s)
        if (pend & (1u << s)) {
            ptx::drain_wait(cache_bar<L>(base, L::kKFull + s), (pend_par >> s) & 1u, lim);
            ptx::drain_wait(cache_bar<L>(base, L::kVFull + s), (pend_par >> s) & 1u, lim);
        }
}

// Whether barrier a's phase ends before barrier b's, looked at in turn; false: b's has ended.  After 64 looks: true, for
// the caller to wait for a.  (With one look, 128 short sequences of 16 heads take 52.6 us instead of 49.3.)
__device__ __forceinline__ bool cache_comes_first(uint32_t a, uint32_t a_phase, uint32_t b, uint32_t b_phase) {
    for (int i = 0; i < 64; ++i) {
        if (__any_sync(0xffffffffu, ptx::mbar_test_wait(b, b_phase))) return false;
        if (__any_sync(0xffffffffu, ptx::mbar_test_wait(a, a_phase))) return true;
    }
    return true;
}

// ---------------------------------------------------------------- warp 1: products
template <int R>
__device__ void cache_mma_role(const CacheFwdParams& p, uint32_t base, uint8_t* smem, uint32_t tmem,
                               volatile int* abort_flag) {
    using L = CacheLayout<R>;
    constexpr uint32_t kIdescS = ptx::idesc_e4m3(128, L::kN, false, false);
    constexpr uint32_t kIdescO = ptx::idesc_e4m3(128, L::kN, true, L::kPerKey);
    const uint64_t lim = p.wait_limit_ns;
    const bool wide = p.c.D == 128;
    // The whole warp waits and counts, so that what it hands to the tensor core sits in uniform registers
    // (a register apiece moved there costs more than the product's issue); one lane issues.
    const bool leader = ptx::elect_one();
    bool ok = true;
    auto wait = [&](int bar, uint32_t par) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_call(cache_bar<L>(base, bar), par, abort_flag, p.c.status, lim));
        return ok;
    };
    struct Ring {  // a stage and its phase
        int stage;
        uint32_t phase;
        __device__ void next() {
            if (++stage == L::kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
    };
    Ring ring{0, 0u}, prev{0, 0u};  // of the tile whose S^T is next, and of the one before
    int g = 0;                      // number of that tile
    int prev_unit = -1;             // unit of the tile whose O^T is still to come
    bool prev_first = false, prev_last = false;
    auto issue_pv = [&]() -> bool {  // of tile g - 1
        const int ub = prev_unit & 1;
        if (prev_first && !wait(L::kOFree + ub, ((prev_unit >> 1) & 1) ^ 1)) return false;
        if (!wait(L::kPFull + ((g - 1) & 1), ((g - 1) >> 1) & 1)) return false;
        if (!wait(L::kVFull + prev.stage, prev.phase)) return false;
        ptx::tc_fence_after();
        const uint32_t o = tmem + L::kO + (uint32_t)(ub * L::kN);
        const uint32_t pp = base + L::kP + (uint32_t)((g - 1) & 1) * (L::kN * 128);
        const uint32_t accumulate = prev_first ? 0u : 1u;
        // V: 32 keys = 32 rows of 128 bytes further per product.  Pp: 32 bytes, or 32 rows.
        const uint64_t v = ptx::sdesc_rows<128>(base + (uint32_t)prev.stage * L::kStageBytes + L::kTileBytes);
        if (leader) {
            if constexpr (L::kPerKey)
                ptx::mma_ss_f8_x4<256, 2 * L::kN>(o, v, ptx::sdesc_rows<L::kN>(pp), kIdescO, accumulate);
            else
                ptx::mma_ss_f8_x4<256, 2>(o, v, ptx::sdesc_rows<128>(pp), kIdescO, accumulate);
            ptx::mma_commit(cache_bar<L>(base, L::kEmpty + prev.stage));
            if (prev_last) ptx::mma_commit(cache_bar<L>(base, L::kOFull + ub));
        }
        prev_unit = -1;
        return true;
    };
    for (int unit = 0; ok; ++unit) {
        const int ub = unit & 1;
        if (!wait(L::kQFull + ub, (unit >> 1) & 1)) break;
        const int n = __shfl_sync(0xffffffffu, reinterpret_cast<const CacheWork*>(smem + L::kUnit)[ub].n, 0);
        if (n == 0) break;
        const uint64_t b = ptx::sdesc_rows<128>(base + L::kQ + (uint32_t)ub * L::kN * 128);
        for (int k = 0; k < n; ++k, ++g) {
            const int sb = g & 1;
            // The last tile's O^T goes first when its weights are there before this tile's K.  (A look at a barrier takes
            // 200 cycles here, so K is not waited for when it has been seen.)
            bool k_there = false;
            if (prev_unit >= 0) {
                k_there = !cache_comes_first(cache_bar<L>(base, L::kPFull + ((g - 1) & 1)), ((g - 1) >> 1) & 1,
                                             cache_bar<L>(base, L::kKFull + ring.stage), ring.phase);
                if (!k_there && !issue_pv()) break;
            }
            // The buffer of S^T is free: every warp has written the weights of tile g - 2, whose O^T is issued.
            if (!k_there && !wait(L::kKFull + ring.stage, ring.phase)) break;
            ptx::tc_fence_after();
            const uint64_t a = ptx::sdesc_rows<128>(base + (uint32_t)ring.stage * L::kStageBytes);
            const uint32_t st = tmem + L::kS + (uint32_t)(sb * L::kN);
            if (leader) {
                if (wide) {
                    ptx::mma_ss_f8_x4<2, 2>(st, a, b, kIdescS, 0u);
                } else {  // D = 64: the other half of the rows is zero in K
                    ptx::mma_ss_f8(st, a, b, kIdescS, 0u);
                    ptx::mma_ss_f8(st, a + 2, b + 2, kIdescS, 1u);
                }
                ptx::mma_commit(cache_bar<L>(base, L::kSFull + sb));
                if (k + 1 == n) ptx::mma_commit(cache_bar<L>(base, L::kQEmpty + ub));
            }
            if (prev_unit >= 0 && !issue_pv()) break;
            prev = ring;
            ring.next();
            prev_unit = unit;
            prev_first = k == 0;
            prev_last = k + 1 == n;
        }
    }
    if (ok && prev_unit >= 0) issue_pv();
    if (leader) {
        ptx::mma_commit(cache_bar<L>(base, L::kDrain));
        ptx::drain_wait(cache_bar<L>(base, L::kDrain), 0u, lim);
    }
}

// ---------------------------------------------------------------- warps 2-3: query rows
template <int R>
__device__ void cache_query_role(const CacheFwdParams& p, CacheCursor cur, int total, int ctas, uint32_t base,
                                 uint8_t* smem, volatile int* abort_flag) {
    using L = CacheLayout<R>;
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - 2;
    // A lane takes 8 elements of a row: D / 8 lanes a row, 2 or 4 rows a step; warp w takes every other step.
    const int lanes = p.c.D / 8, part = lane & (lanes - 1), per = 32 / lanes;
    const int row0 = w * per + lane / lanes;
    constexpr int kBatch = R >= 32 ? 4 : R / 4 < 2 ? 1 : 2;  // steps under way at once
    uint4 x[kBatch];
    long long at[kBatch];
    int seen[kBatch];
    auto load = [&](const CacheUnit& u, int r0) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            int i, hq;
            const int r = r0 + k * 2 * per;
            const bool used = r < R && cache_row(p, u, r, &i, &hq);
            at[k] = used ? ((long long)u.b * p.Hq + hq) * p.Sq + i : -1;
            seen[k] = !used ? 0 : p.plan.causal ? max(u.s.first + i + 1, 0) : u.s.len;
            x[k] = make_uint4(0, 0, 0, 0);
            if (used)
                x[k] = *reinterpret_cast<const uint4*>(p.q + u.b * p.q_stride[0] + hq * p.q_stride[1] + i * p.q_stride[2] +
                                                       part * 8);
        }
    };
    CacheUnit u;
    for (int unit = 0;; ++unit) {
        const int ub = unit & 1;
        const bool more = cursor_next(p.plan, cur, u);
        if (more) load(u, row0);
        const bool ok = ptx::mbar_wait_call(cache_bar<L>(base, L::kQEmpty + ub), ((unit >> 1) & 1) ^ 1, abort_flag, p.c.status,
                                       p.wait_limit_ns);
        if (!__all_sync(0xffffffffu, ok)) return;
        CacheWork* work = reinterpret_cast<CacheWork*>(smem + L::kUnit) + ub;
        if (more) {
            CacheRow* rows = reinterpret_cast<CacheRow*>(smem + L::kRows) + ub * R;
            const int used = min(p.plan.qper, u.s.count - u.qt * p.plan.qper) * p.hper;  // no row from here on is in use
#pragma unroll 1
            for (int r0 = row0; r0 - row0 < R; r0 += kBatch * 2 * per) {
                if (r0 != row0) load(u, r0);
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int r = r0 + k * 2 * per;
                    if (r - lane / lanes >= used) {  // the step's rows; what stands in Qp for them only meets factors of 0
                        if (r < R && part == 0) rows[r] = CacheRow{0.f, 0, -1};
                        continue;
                    }
                    const uint32_t v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
                    // the largest magnitude, by bit pattern; not finite: the whole row is NaN
                    uint32_t m = __vmaxu2(__vmaxu2(v[0] & 0x7fff7fffu, v[1] & 0x7fff7fffu),
                                          __vmaxu2(v[2] & 0x7fff7fffu, v[3] & 0x7fff7fffu));
                    m = max(m & 0xffffu, m >> 16);
                    for (int o = 1; o < lanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                    const float scale = e4m3_pow2_scale(__uint_as_float(m << 16));
                    // 1 / scale, by its exponent: scale is a power of two of at most 2^120
                    const float inv = m >= 0x7f80u ? NAN : __uint_as_float((254u << 23) - __float_as_uint(scale));
                    uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float a = __uint_as_float(v[e] << 16) * inv, b = __uint_as_float(v[e] & 0xffff0000u) * inv;
                        const uint32_t h = e4m3_pair(a, b);
                        const float2 hf = e4m3_unpair(h);
                        hi[e >> 1] |= h << (16 * (e & 1));
                        lo[e >> 1] |= e4m3_pair(a - hf.x, b - hf.y) << (16 * (e & 1));
                    }
                    if (r < R) {
                        const int n = L::hi_row(r);
                        uint8_t* q8 = smem + L::kQ + ub * L::kN * 128;
                        auto put = [&](int row, const uint32_t* c) {
                            *reinterpret_cast<uint2*>(q8 + row * 128 + (((part >> 1) ^ (row & 7)) << 4) + (part & 1) * 8) =
                                make_uint2(c[0], c[1]);
                        };
                        put(n, hi);
                        put(n + L::kH, lo);
                        if (part == 0) rows[r] = CacheRow{at[k] >= 0 ? scale * p.scale_log2 : 0.f, seen[k], at[k]};
                    }
                }
            }
            if (w == 0 && lane == 0) {
                const int q0 = u.qt * p.plan.qper;
                work->t = u.t;
                work->n = u.n;
                work->keys = u.keys;
                work->keys_all = p.plan.causal ? max(u.s.first + q0 + 1, 0) : u.s.len;
                work->slot = u.n == u.tiles ? -1 : u.t > 0 ? 0 : 1;
                work->rows = used;
                if (u.n < u.tiles) cache_share(reinterpret_cast<CacheShared*>(smem + L::kShared) + work->slot, u, total, ctas);
            }
        } else if (w == 0 && lane == 0) {
            work->n = 0;
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(cache_bar<L>(base, L::kQFull + ub));
        if (!more) return;
    }
}

// ---------------------------------------------------------------- warps 4 on: softmax
// Takes NaN codes out of a key's 128 bytes of V (at `line`, row `row` of a tile)
// and lowers at[d] to the key for each; true if there were any.
__device__ __noinline__ bool cache_take_nan(uint32_t line, int row, int key, int* at) {
    bool found = false;
#pragma unroll 1
    for (int x = 0; x < 8; ++x) {
        const uint4 v = ptx::ld_shared_v4(line + 16 * x);
        uint32_t word[4] = {v.x, v.y, v.z, v.w};
        bool here = false;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            // 0x7f in a byte's low bits: adding 1 to them carries into its top bit
            uint32_t hit = ((word[y] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
            if (hit) here = true;
            while (hit) {
                const int b = (__ffs(hit) - 1) >> 3;
                hit &= hit - 1;
                word[y] &= ~(0xffu << (8 * b));
                atomicMin(at + (x ^ (row & 7)) * 16 + y * 4 + b, key);
            }
        }
        if (here) ptx::st_shared_v4(line + 16 * x, word[0], word[1], word[2], word[3]);
        found |= here;
    }
    return found;
}

// Adds each of a warp's H rows over its lanes; lane i returns the sum of row
// i / (32 / H).  Half of the rows change hands in the first step, a quarter in the next.
template <int H>
__device__ __forceinline__ float cache_sum_rows(float* l) {
    const int lane = threadIdx.x & 31;
    int o = 16;
#pragma unroll
    for (int n = H; n > 1; n /= 2, o /= 2) {
        const bool upper = lane & o;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float give = upper ? l[i] : l[i + n / 2], keep = upper ? l[i + n / 2] : l[i];
            l[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    float x = l[0];
    for (; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Eight rows' bits, row r's from bit r to bit 8 (r mod 4) + r / 4.
__device__ __forceinline__ uint32_t cache_row_bits(uint32_t x) {
    return ((x & 15u) * 0x00204081u & 0x01010101u) | ((x >> 4 & 15u) * 0x00204081u & 0x01010101u) << 1;
}

template <int R>
__device__ void cache_softmax_role(const CacheFwdParams& p, uint32_t base, uint8_t* smem, uint32_t tmem,
                                   volatile int* abort_flag) {
    using L = CacheLayout<R>;
    constexpr int H = L::kH, W = L::kWidth;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wg = (warp - 4) >> 2, wq = warp & 3;
    const int j = wq * 32 + lane;  // this thread's key of a tile (lane of S^T) and its d (lane of O^T)
    const uint32_t my_tmem = tmem + ((uint32_t)(wq * 32) << 16) + (uint32_t)(wg * W);
    const uint64_t lim = p.wait_limit_ns;
    float4* tab = reinterpret_cast<float4*>(smem + L::kTab) + wg * (H / 2);
    float* fac = reinterpret_cast<float*>(smem + L::kFac) + wg * H;
    float* red = reinterpret_cast<float*>(smem + L::kRed) + wg * 4 * H;  // [H][4 warps]
    const int bar = 1 + wg;  // the warpgroup's barrier
    // A wait that ran out leaves this false: the lane goes on without waiting and without writing
    // results, so that it meets its warpgroup at every barrier and nobody is left there.
    bool alive = true;
    auto wait = [&](int which, uint32_t par) {
        if (alive) alive = ptx::mbar_wait_call(cache_bar<L>(base, which), par, abort_flag, p.c.status, lim);
        __syncwarp();
    };
    auto arrive = [&](int which) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(cache_bar<L>(base, which));
    };
    const int page = j >> p.c.block_shift;  // of a tile
    int g = 0, stage = 0;   // number and stage of the current tile
    uint32_t phase = 0, nan_phase = 0;  // nan_phase, bit ub: phase of barrier kNan + ub
    float l[H];  // this thread's keys' part of the rows' sums of w / vs
    for (int unit = 0;; ++unit) {
        const int ub = unit & 1;
        int* nan_at = reinterpret_cast<int*>(smem + L::kNanAt) + ub * 128;
        volatile int* nan_seen = reinterpret_cast<volatile int*>(smem + L::kNanSeen) + ub;
        wait(L::kQFull + ub, (unit >> 1) & 1);
        const CacheWork work = reinterpret_cast<const CacheWork*>(smem + L::kUnit)[ub];
        const CacheRow* rows = reinterpret_cast<const CacheRow*>(smem + L::kRows) + ub * R + wg * H;
        // Some tile of the share holds keys that not every row sees.  Like all that decides about
        // barriers, it follows from `work` alone, which every warp has read the same.
        const bool borders = (work.t + work.n) * kCacheTile > work.keys_all;
        if (borders && wg == 0) {
            nan_at[j] = 0x7fffffff;
            if (j == 0) *nan_seen = 0;
        }
        float row_max = -INFINITY;  // of row `lane`, the same in the four warps
        if (j < H) {
            float* t = reinterpret_cast<float*>(tab + j / 2) + (j & 1);
            t[0] = rows[j].factor;
            t[2] = -INFINITY;
        }
        if (ptx::bar_any(bar, 128, !alive) || work.n == 0) break;  // the four warps go on together or not at all
        const bool idle = work.rows <= wg * H;
#pragma unroll
        for (int r = 0; r < H; ++r) l[r] = 0.f;
        bool todo = true;  // some row that sees keys has no maximum yet
        float peak = -INFINITY;       // the largest maximum that row `lane` has had
        // Rows whose maximum may fall, row r as bit 8 (r mod 4) + r / 4, where its code in Pp has its byte.
        uint32_t can_fall = 0;

        for (int k = 0; k < work.n; ++k, ++g) {
            const int sb = g & 1;
            // S^T is there; so are the scales beside K, which were written before it, and the O^T of tile g - 2
            // is done, which came before it: its buffer of Pp is free.
            wait(L::kSFull + sb, (g >> 1) & 1);
            ptx::tc_fence_after();
            const float* info = reinterpret_cast<const float*>(smem + L::kInfo + stage * L::kInfoBytes);
            const int missing = reinterpret_cast<const int*>(info)[24];
            const int key = (work.t + k) * kCacheTile + j;
            const float ks = info[page], lvs = info[8 + page], ivs = info[16 + page];
            const bool some = (work.t + k + 1) * kCacheTile > work.keys_all;  // some row does not see some key
            const bool full = !some && missing == 0, here = key < work.keys && !((missing >> page) & 1);
            if (some && wg == 0) {
                // A weight of 0 times NaN is NaN: keys that nobody sees become 0 in V, and NaN that only
                // some rows see is taken out and noted by the first position that has it.
                wait(L::kVFull + stage, phase);
                const uint32_t line = base + (uint32_t)stage * L::kStageBytes + L::kTileBytes + (uint32_t)j * 128u;
                if (alive && key >= work.keys) {
#pragma unroll
                    for (int y = 0; y < 8; ++y) ptx::st_shared_v4(line + 16 * y, 0, 0, 0, 0);
                } else if (alive && key >= work.keys_all) {
                    if (cache_take_nan(line, j, key, nan_at)) *nan_seen = 1;
                }
            }
            if (!idle) {
                const uint32_t s_addr = my_tmem + L::kS + (uint32_t)(sb * L::kN);
                const uint32_t p_tile = base + L::kP + (uint32_t)sb * (L::kN * 128);
                // The weights of this thread's key for every row, into Pp, and `sum`, the rows' sums with them; returns the
                // largest.  The sums count once the weights do: one that is too large, over V's least scale, may be past
                // what a float holds.
                float sum[H];
                uint32_t reach = 0;  // rows whose weight reached 1 here, as in can_fall
                auto pass = [&](auto masked) {
                    constexpr bool kMasked = decltype(masked)::value;
                    float top = 0.f;
                    uint32_t s[W];
                    ptx::tmem_load<W>(s_addr, s);
                    const uint64_t ks2 = ptx::f2(ks, ks), ivs2 = ptx::f2(ivs, ivs), lvs2 = ptx::f2(lvs, lvs);
                    uint32_t hi[H / 2], lo[H / 2];
#pragma unroll
                    for (int r = 0; r < H; r += 2) {
                        const float4 f = tab[r / 2];
                        uint64_t z = ptx::f2(__uint_as_float(s[r]), __uint_as_float(s[r + 1]));
                        z = ptx::add2(z, ptx::f2(__uint_as_float(s[H + r]), __uint_as_float(s[H + r + 1])));
                        // K's scale and the row's factor first: with K near its type's limit and a small q, the sum of
                        // products times K's scale alone is past a float's.
                        z = ptx::fma2(z, ptx::mul2(ptx::f2(f.x, f.y), ks2), ptx::add2(ptx::f2(f.z, f.w), lvs2));
                        float y0, y1;
                        ptx::f2_split(z, y0, y1);
                        if constexpr (kMasked) {
                            y0 = here && key < rows[r].keys ? y0 : -INFINITY;
                            y1 = here && key < rows[r + 1].keys ? y1 : -INFINITY;
                        }
                        const float w0 = ptx::ex2(y0), w1 = ptx::ex2(y1);
                        top = ptx::max3(top, w0, w1);
                        const uint64_t w = ptx::f2(w0, w1);
                        ptx::f2_split(ptx::fma2(w, ivs2, ptx::f2(l[r], l[r + 1])), sum[r], sum[r + 1]);
                        // hi: the nearest code; lo: the nearest code to 2^4 times what hi leaves
                        hi[r / 2] = e4m3_pair(w0, w1);
                        const float2 h = e4m3_unpair(hi[r / 2]);
                        float r0, r1;
                        ptx::f2_split(ptx::fma2(ptx::f2(h.x, h.y), ptx::f2(-16.f, -16.f), ptx::mul2(w, ptx::f2(16.f, 16.f))), r0, r1);
                        lo[r / 2] = e4m3_pair(r0, r1);
                    }
                    auto four = [](const uint32_t* v) { return __byte_perm(v[0], v[1], 0x5410); };
                    constexpr uint32_t kCarry = (0x80u - kCacheReach) * 0x01010101u;  // into a byte's top bit from 1 on
                    reach = (four(hi) + kCarry) >> 7 & 0x01010101u;
                    if constexpr (H == 8) reach |= (four(hi + 2) + kCarry) >> 6 & 0x02020202u;
                    if constexpr (L::kPerKey) {
                        constexpr uint32_t kTurn = L::kN == 64 ? 1 : 2;  // key bits that swizzle
                        const uint32_t turn = ((uint32_t)j >> kTurn) & (L::kN / 16 - 1);
                        ptx::st_shared_v4(p_tile + (uint32_t)j * L::kN + (((uint32_t)wg ^ turn) << 4), four(hi), four(hi + 2),
                                          four(lo), four(lo + 2));
                    } else {
                        auto put = [&](int n, uint32_t code) {  // n: row of the warpgroup's eight
                            ptx::st_shared_u8(p_tile + (uint32_t)(wg * 2 * H + n) * 128u + (((uint32_t)(j >> 4) ^ (uint32_t)(n & 7)) << 4) +
                                                  (uint32_t)(j & 15),
                                              code);
                        };
#pragma unroll
                        for (int r = 0; r < H; r += 2) {
                            put(r, hi[r / 2]);
                            put(r + 1, hi[r / 2] >> 8);
                            put(H + r, lo[r / 2]);
                            put(H + r + 1, lo[r / 2] >> 8);
                        }
                    }
                    return top;
                };
                // First as it stands; once more when a maximum has to rise or fall.  The maxima come first while a row
                // has none.
                for (bool look = todo;;) {
                    if (look) {
                        // The rows' maxima of s + log2 vs over the tile, through the order of the bit patterns.
                        uint32_t s[W];
                        ptx::tmem_load<W>(s_addr, s);
#pragma unroll
                        for (int r = 0; r < H; ++r) {
                            const float z = fmaf(__uint_as_float(s[r]) + __uint_as_float(s[H + r]), rows[r].factor * ks, lvs);
                            const float y = fmaxf(full || (here && key < rows[r].keys) ? z : -INFINITY, -INFINITY);
                            const int b = __float_as_int(y), m = __reduce_max_sync(0xffffffffu, b ^ (b >> 31 & 0x7fffffff));
                            if (lane == r) red[r * 4 + wq] = __int_as_float(m ^ (m >> 31 & 0x7fffffff));
                        }
                        ptx::bar_sync(bar, 128);
                        // Every warp works out the same new maxima, a row per lane.
                        bool open = false, moves = false;
                        float m = -INFINITY;
                        if (lane < H) {
                            const float4 x = reinterpret_cast<const float4*>(red)[lane];
                            const bool used = rows[lane].at >= 0;
                            m = cache_new_max(kCacheRange, row_max, peak, used ? fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)) : -INFINITY, &moves);
                            open = m == -INFINITY && used && rows[lane].keys > 0;
                        }
                        todo = __any_sync(0xffffffffu, open);
                        const bool moved = __any_sync(0xffffffffu, moves);
                        if (moved) {
                            const float f = row_max == -INFINITY ? 0.f : ptx::ex2(row_max - m);
                            row_max = m;
                            peak = fmaxf(peak, m);
                            const uint32_t can = __ballot_sync(0xffffffffu, m > -INFINITY && m > peak - kCacheFall);
                            can_fall = cache_row_bits(can);
                            if (wq == 0 && lane < H) {
                                fac[lane] = f;
                                reinterpret_cast<float*>(tab + lane / 2)[2 + (lane & 1)] = m == -INFINITY ? -INFINITY : kCacheRange.room - m;
                            }
                        }
                        ptx::bar_sync(bar, 128);  // `red` may be written again, and the new factors read
                        if (moved) {
#pragma unroll
                            for (int r = 0; r < H; ++r) l[r] *= fac[r];
                            if (k > 0) {
                                // the tile before is through the tensor core once its stage is empty
                                wait(L::kEmpty + (stage == 0 ? L::kStages : stage) - 1, stage == 0 ? phase ^ 1u : phase);
                                ptx::tc_fence_after();
                                const uint32_t o_addr = my_tmem + L::kO + (uint32_t)(ub * L::kN);
                                ptx::tmem_load<W>(o_addr, s);
#pragma unroll
                                for (int i = 0; i < W; ++i) s[i] = __float_as_uint(__uint_as_float(s[i]) * fac[i % H]);
                                ptx::tmem_store<W>(o_addr, s);
                            }
                        }
                    }
                    const float top = full ? pass(std::false_type()) : pass(std::true_type());
                    if (look) break;
                    // All four warps decide by what each has written, two tiles' words in turn, and by the unit: alike after an
                    // abort too.  Nobody falls where a page is missing.
                    uint32_t* reached = reinterpret_cast<uint32_t*>(smem + L::kReach) + (sb * L::kWgs + wg) * 4;
                    reach = __reduce_or_sync(0xffffffffu, missing == 0 ? reach : ~0u);
                    if (lane == 0) reached[wq] = reach;
                    look = ptx::bar_any(bar, 128, top > kCacheTop);
                    const uint4 x = *reinterpret_cast<const uint4*>(reached);
                    uint32_t low = can_fall & ~(x.x | x.y | x.z | x.w);
                    if (some) low &= cache_row_bits(__ballot_sync(0xffffffffu, lane < H && rows[lane].keys > key - j));
                    if (!look && low == 0) break;
                    look = true;
                }
#pragma unroll
                for (int r = 0; r < H; ++r) l[r] = sum[r];
                ptx::tc_fence_before();
            }
            ptx::fence_proxy_async_smem();
            arrive(L::kPFull + sb);
            if (++stage == L::kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }

        // ---- the unit's rows leave
        bool nan = false;
        if (borders) {
            // Warpgroup 0 has noted the NaN that it took out; the others wait for that.
            if (wg == 0)
                arrive(L::kNan + ub);
            else
                wait(L::kNan + ub, nan_phase >> ub & 1u);
            nan_phase ^= 1u << ub;
        }
        if (!idle) {
            const float sum = cache_sum_rows<H>(l);
            if (lane % (32 / H) == 0) red[lane / (32 / H) * 4 + wq] = sum;
        }
        ptx::bar_sync(bar, 128);
        if (borders) nan = *nan_seen != 0;
        const long long slot = (long long)blockIdx.x * 2 + work.slot;
        if (!idle && j < H) {
            const float4 x = reinterpret_cast<const float4*>(red)[j];
            const float sum = x.x + x.y + (x.z + x.w), m = row_max - kCacheRange.room;
            float f = 1.f;
            if (work.slot < 0) {
                f = sum == 0.f ? 0.f : ptx::rcp(sum);
                if (alive && p.lse != nullptr && rows[j].at >= 0)
                    p.lse[rows[j].at] = sum == 0.f ? -INFINITY : (m + ptx::lg2(sum)) * kLn2;
            } else if (alive) {
                p.part_ml[slot * R + wg * H + j] = make_float2(m, sum);
            }
            fac[j] = f;
        }
        ptx::bar_sync(bar, 128);
        wait(L::kOFull + ub, (unit >> 1) & 1);
        ptx::tc_fence_after();
        if (!idle) {
            const int first_nan = nan ? nan_at[j] : 0x7fffffff;
            uint32_t s[W];
            ptx::tmem_load<W>(my_tmem + L::kO + (uint32_t)(ub * L::kN), s);
            if (alive && j < p.c.D) {
#pragma unroll
                for (int r = 0; r < H; ++r) {
                    const CacheRow row = rows[r];
                    float o = fmaf(__uint_as_float(s[H + r]), 0.0625f, __uint_as_float(s[r])) * fac[r];
                    if (first_nan < row.keys) o = NAN;
                    if (work.slot >= 0)
                        p.part_o[(slot * R + wg * H + r) * 128 + j] = o;
                    else if (row.at >= 0)
                        p.out[row.at * p.c.D + j] = __float2bfloat16(o);
                }
            }
        }
        ptx::tc_fence_before();
        arrive(L::kOFree + ub);
        arrive(L::kQEmpty + ub);
    }
}

// Pieces x0, x0 + step, ... (`n` of them) of a shared unit.  Each is slot 1 of the CTA where the unit begins or slot 0 of
// a following one.  `final`: the joined rows go to out and lse, else to the place of piece x0.
struct CacheJoin {
    const CacheShared& shared;
    int x0, n, step;
    bool final;
    __device__ long long slot(int x) const {
        const int piece = x0 + x * step;
        return (long long)(shared.first + piece) * 2 + (piece == 0 ? 1 : 0);
    }
};
// Joins rows r .. r + kRows - 1 of a shared unit, a warp for all:
// O = sum 2^(M_i - M) O_i / sum 2^(M_i - M) l_i over the pieces, R rows each.  A lane takes every 32nd piece's (M, l), and 4 columns of every piece's O, of which
// 8 are under way at once.
template <int kRows>
__device__ void cache_join_rows(const CacheFwdParams& p, const CacheJoin& join, int R, int r) {
    const int lane = threadIdx.x & 31, n = join.n;
    const bool mine = lane * 4 < p.c.D;
    auto slot = [&](int x) { return join.slot(x) * R + r; };
    auto piece = [&](int x, int y) { return x < n ? __ldcg(p.part_ml + slot(x) + y) : make_float2(-INFINITY, 0.f); };
    float m[kRows], l[kRows];  // of the lane's pieces, then of all
#pragma unroll
    for (int y = 0; y < kRows; ++y) {
        m[y] = -INFINITY;
        l[y] = 0.f;
    }
    float2 near[kRows];  // of piece `lane`
    constexpr int kAhead = 8 / kRows;
    float4 v[kAhead][kRows];
    auto load = [&](int x0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int y = 0; y < kRows; ++y)
                v[i][y] = mine && x0 + i < n ? __ldcg(reinterpret_cast<const float4*>(p.part_o + (slot(x0 + i) + y) * 128) + lane)
                                             : make_float4(0.f, 0.f, 0.f, 0.f);
    };
#pragma unroll
    for (int y = 0; y < kRows; ++y) near[y] = piece(lane, y);
    load(0);
    for (int x0 = 0; x0 < n; x0 += 32) {
#pragma unroll
        for (int y = 0; y < kRows; ++y) {
            const float2 ml = x0 == 0 ? near[y] : piece(x0 + lane, y);
            const float top = fmaxf(m[y], ml.x), ref = top == -INFINITY ? 0.f : top;
            l[y] = l[y] * ptx::ex2(m[y] - ref) + ptx::ex2(ml.x - ref) * ml.y;
            m[y] = top;
        }
    }
    float ref[kRows];
    float4 o[kRows];
#pragma unroll
    for (int y = 0; y < kRows; ++y) {
        float top = m[y];
        for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        ref[y] = top == -INFINITY ? 0.f : top;
        l[y] *= ptx::ex2(m[y] - ref[y]);
        m[y] = top;
        for (int x = 16; x > 0; x >>= 1) l[y] += __shfl_xor_sync(0xffffffffu, l[y], x);
        o[y] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int x0 = 0; x0 < n; x0 += 32) {
        float f[kRows];  // of the lane's piece
#pragma unroll
        for (int y = 0; y < kRows; ++y) f[y] = ptx::ex2((x0 == 0 ? near[y] : piece(x0 + lane, y)).x - ref[y]);
        for (int x = x0; x < min(n, x0 + 32); x += kAhead) {
            if (x > 0) load(x);
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
#pragma unroll
                for (int y = 0; y < kRows; ++y) {
                    const float g = __shfl_sync(0xffffffffu, f[y], (x + i) & 31);
                    o[y] = make_float4(o[y].x + g * v[i][y].x, o[y].y + g * v[i][y].y, o[y].z + g * v[i][y].z, o[y].w + g * v[i][y].w);
                }
        }
    }
#pragma unroll
    for (int y = 0; y < kRows; ++y) {
        if (!join.final) {  // where this warp alone has read
            if (mine) *(reinterpret_cast<float4*>(p.part_o + (slot(0) + y) * 128) + lane) = o[y];
            __syncwarp();
            if (lane == 0) p.part_ml[slot(0) + y] = make_float2(m[y], l[y]);
            continue;
        }
        int qi, hq;
        if (!cache_row(p, join.shared.u, r + y, &qi, &hq)) continue;
        const long long at = ((long long)join.shared.u.b * p.Hq + hq) * p.Sq + qi;
        const float inv = l[y] == 0.f ? 0.f : ptx::rcp(l[y]);
        if (mine)
            *reinterpret_cast<uint2*>(p.out + at * p.c.D + lane * 4) =
                make_uint2(ptx::pack_bf16x2(o[y].x * inv, o[y].y * inv), ptx::pack_bf16x2(o[y].z * inv, o[y].w * inv));
        if (lane == 0 && p.lse != nullptr) p.lse[at] = l[y] == 0.f ? -INFINITY : (m[y] + ptx::lg2(l[y])) * kLn2;
    }
}

// After a wait has run out: the units that this CTA shares, looked up again and opened, since the roles may have ended
// before they came to them.  `scan` is as cache_locate left it.
template <typename L>
__device__ __noinline__ void cache_shared_again(const CacheFwdParams& p, const int* scan, CacheShared* shared) {
    const int begin = scan[0], end = scan[1], total = scan[2], ctas = scan[3];
    shared[0].pieces = shared[1].pieces = 0;
    if (begin == end) return;
    CacheCursor cur = cursor_at(p.plan, *reinterpret_cast<const CachePlace*>(scan + 20), begin, end - begin);
    CacheUnit u;
    while (cursor_next(p.plan, cur, u))
        if (u.n < u.tiles) {
            cache_share(shared + (u.t > 0 ? 0 : 1), u, total, ctas);
            cache_open_tickets(p, u.at, u.tiles, total, ctas, L::kJoin);
        }
}

// The end of a CTA, by all its threads, once every piece is left: of each unit that it shares, whoever counts last in
// its group joins the group's pieces, and whoever is the last of those joins the groups.
template <typename L, typename F>
__device__ void cache_join(const CacheFwdParams& p, const int* scan, CacheShared* shared, bool aborted, F join) {
    if (aborted) {
        if (threadIdx.x == 0) cache_shared_again<L>(p, scan, shared);
        __syncthreads();
    }
    if (shared[0].pieces == 0 && shared[1].pieces == 0) return;
    if (threadIdx.x < 2) {
        CacheShared& x = shared[threadIdx.x];
        __threadfence();
        x.last = kMoreToCome;
        if (x.pieces > 0)
            x.last = tickets_leave<CacheTicketMemory>(p.tickets, x.first, x.pieces, blockIdx.x - x.first, L::kJoin, aborted);
        __threadfence();
    }
    __syncthreads();
    for (int i = 0; i < 2; ++i) {
        CacheShared& x = shared[i];
        if (x.pieces == 0 || x.last == kMoreToCome) continue;
        const int group = cache_group(x.pieces, L::kJoin);
        const bool whole = x.last == kWasLast;  // every piece of the group was left
        if (group == x.pieces) {
            if (whole) join(CacheJoin{x, 0, group, 1, true});
            continue;
        }
        const CacheGroup g = cache_group_of(x.pieces, group, blockIdx.x - x.first);
        if (g.n > 1 && whole) join(CacheJoin{x, g.begin, g.n, 1, false});
        __syncthreads();
        if (threadIdx.x == 0) {
            __threadfence();
            x.last = tickets_joined<CacheTicketMemory>(p.tickets, gridDim.x, x.first, x.pieces, L::kJoin, !whole);
            __threadfence();
        }
        __syncthreads();
        if (x.last == kWasLast) join(CacheJoin{x, 0, (x.pieces + group - 1) / group, group, true});
    }
}

template <int R>
__global__ void __launch_bounds__(CacheLayout<R>::kThreads, CacheLayout<R>::kCtas)
    attn_cache_fwd_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                          const __grid_constant__ CacheFwdParams p) {
    using L = CacheLayout<R>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kTmemSlot);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);  // uniform, also to the compiler

    // not by warp 0, whose loads of the lengths come first
    if (threadIdx.x == 96) {
        for (int s = 0; s < L::kStages; ++s) {
            ptx::mbar_init(cache_bar<L>(base, L::kKFull + s), 1);
            ptx::mbar_init(cache_bar<L>(base, L::kVFull + s), 1);
            ptx::mbar_init(cache_bar<L>(base, L::kEmpty + s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(cache_bar<L>(base, L::kQFull + i), 2);    // the query warps
            ptx::mbar_init(cache_bar<L>(base, L::kQEmpty + i), 4 * L::kWgs + 1);  // the softmax warps and the last S^T product
            ptx::mbar_init(cache_bar<L>(base, L::kSFull + i), 1);
            ptx::mbar_init(cache_bar<L>(base, L::kPFull + i), 4 * L::kWgs);
            ptx::mbar_init(cache_bar<L>(base, L::kOFull + i), 1);
            ptx::mbar_init(cache_bar<L>(base, L::kOFree + i), 4 * L::kWgs);
            ptx::mbar_init(cache_bar<L>(base, L::kNan + i), 4);      // softmax warpgroup 0
        }
        ptx::mbar_init(cache_bar<L>(base, L::kDrain), 1);
        *abort_flag = 0;
        for (int x = 0; x < 2; ++x) reinterpret_cast<CacheShared*>(smem + L::kShared)[x].pieces = 0;
        ptx::fence_barrier_init();
        ptx::prefetch_tensormap(&tm_k);
        ptx::prefetch_tensormap(&tm_v);
    }
    if (warp == 1) {
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
    } else if (warp == 0) {
        cache_load_role<L>(&tm_k, &tm_v, p, cursor_at(p.plan, place, begin, end - begin), total, ctas, base, smem, abort_flag);
    } else if (warp == 1) {
        cache_mma_role<R>(p, base, smem, tmem, abort_flag);
    } else if (warp < 4) {
        cache_query_role<R>(p, cursor_at(p.plan, place, begin, end - begin), total, ctas, base, smem, abort_flag);
    } else {
        cache_softmax_role<R>(p, base, smem, tmem, abort_flag);
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, L::kTmemCols);
    }
    cache_join<L>(p, reinterpret_cast<const int*>(smem + L::kScan), reinterpret_cast<CacheShared*>(smem + L::kShared),
                  *abort_flag != 0, [&](const CacheJoin& x) {
        constexpr int kWarps = L::kThreads / 32, kRows = (R + kWarps - 1) / kWarps;
        static_assert(R % kRows == 0, "rows of a warp");
        if (warp * kRows < R) cache_join_rows<kRows>(p, x, R, warp * kRows);
    });
}

}  // namespace attn
