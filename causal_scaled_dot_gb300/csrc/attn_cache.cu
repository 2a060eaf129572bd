// attn_cache.cu -- the entry points of the 8-bit key/value cache
// (include/attn.h): argument checks, TMA descriptors, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/attn.h"
#include "cache_index.h"
#include "common.cuh"
#include "host.h"
#include "kernel_cache_append.cuh"
#include "kernel_cache_fwd.cuh"
#include "kernel_cache_rw.cuh"
#include "kernel_cache_wide.cuh"
#include "launch.h"
#include "rope_check.h"

namespace attn {
namespace {

size_t cache_bytes(const attn_cache_t* c) { return (size_t)c->num_blocks * c->Hkv * c->block_size * c->D; }

int check_cache(const attn_cache_t* c) {
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !c->block_table || !c->seq_lens)
        return ATTN_ERR_INVALID_ARG;
    if (c->num_blocks < 1 || c->max_blocks < 1 || c->B < 1 || c->Hkv < 1) return ATTN_ERR_INVALID_ARG;
    if (c->D != 64 && c->D != 128) return ATTN_ERR_UNSUPPORTED;
    const int bs = c->block_size;
    if (bs != 16 && bs != 32 && bs != 64 && bs != 128) return ATTN_ERR_UNSUPPORTED;
    // Positions (and the sum of two) are 32-bit, and so are the TMA coordinates of (block, head).
    if ((long long)c->max_blocks * bs > (1ll << 29) || (long long)c->num_blocks * c->Hkv > (1ll << 30) ||
        (long long)c->B * c->Hkv > (1ll << 30))
        return ATTN_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) & 15u) return ATTN_ERR_MISALIGNED;
    if ((reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale) |
         reinterpret_cast<uintptr_t>(c->block_table) | reinterpret_cast<uintptr_t>(c->seq_lens)) & 3u)
        return ATTN_ERR_MISALIGNED;
    return ATTN_OK;
}

// Whether [a, a + na) meets the cache's codes or scales; with `index` its table and lengths too.
bool meets_cache(const attn_cache_t* c, const void* a, size_t na, bool index) {
    const size_t n = cache_bytes(c), ns = (size_t)c->num_blocks * c->Hkv * 4;
    return host::ranges_overlap(a, na, c->k, n) || host::ranges_overlap(a, na, c->v, n) ||
           host::ranges_overlap(a, na, c->k_scale, ns) || host::ranges_overlap(a, na, c->v_scale, ns) ||
           (index && (host::ranges_overlap(a, na, c->block_table, (size_t)c->B * c->max_blocks * 4) ||
                      host::ranges_overlap(a, na, c->seq_lens, (size_t)c->B * 4)));
}

// Whether codes or scales, which a write changes, meet each other, the table or the lengths.
bool meets_itself(const attn_cache_t* c) {
    const size_t n = cache_bytes(c), ns = (size_t)c->num_blocks * c->Hkv * 4;
    const struct { const void* p; size_t n; } part[6] = {{c->k, n}, {c->v, n}, {c->k_scale, ns}, {c->v_scale, ns},
                                                         {c->block_table, (size_t)c->B * c->max_blocks * 4}, {c->seq_lens, (size_t)c->B * 4}};
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 6; ++j)
            if (host::ranges_overlap(part[i].p, part[i].n, part[j].p, part[j].n)) return true;
    return false;
}

// {batch, head, token} strides of rows [B, H, S, D] into `out`; *bytes
// receives the bytes from the first element to past the last.
int row_strides(const long long* strides, long long B, long long H, long long S, int D, long long out[3], size_t* bytes) {
    const long long dense[3] = {H * S * D, S * D, D};
    const long long* st = strides ? strides : dense;
    const long long n[3] = {B, H, S};
    size_t last = 0;
    for (int i = 0; i < 3; ++i) {
        if (st[i] < 0) return ATTN_ERR_INVALID_ARG;
        if (st[i] % 8) return ATTN_ERR_MISALIGNED;
        if (st[i] > (1ll << 40)) return ATTN_ERR_UNSUPPORTED;
        out[i] = st[i];
        last += (size_t)(n[i] - 1) * (size_t)st[i];
    }
    *bytes = (last + D) * 2;
    return ATTN_OK;
}

CacheView view_of(const attn_cache_t* c, unsigned int* status) {
    CacheView v{};
    v.k = static_cast<unsigned char*>(c->k);
    v.v = static_cast<unsigned char*>(c->v);
    v.k_scale = c->k_scale;
    v.v_scale = c->v_scale;
    v.block_table = c->block_table;
    v.seq_lens = c->seq_lens;
    v.num_blocks = c->num_blocks;
    v.block_size = c->block_size;
    v.block_shift = c->block_size == 16 ? 4 : c->block_size == 32 ? 5 : c->block_size == 64 ? 6 : 7;
    v.max_blocks = c->max_blocks;
    v.B = c->B;
    v.Hkv = c->Hkv;
    v.D = c->D;
    v.status = status;
    return v;
}

// Query rows of a unit: the least form that takes them all, and 128 from 33 rows on.  Up to 8192 keys, 8 key/value heads:
// 16 x 5 tokens of 4 query heads each (20 rows) take 48 us with 32 rows a unit and 63 with 128; 32 x 8 of 8 (64 rows) 109
// with 128, and 153 as two units of 32.
int rows_per_unit(long long group, long long Sq) {
    const long long rows = group * Sq;
    return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 128;
}
int ctas_per_sm(int R) { return R == 128 ? CacheWideLayout::kCtas : R == 8 ? CacheLayout<8>::kCtas : 1; }

// Key tiles that a unit may have, by the cache's capacity, where units are not split: up to 8 (1024 tokens) joining the
// pieces takes longer than the tiles in one CTA do.  4 x 200 tokens of 32 heads over 8 and up to 1000 keys 28 us, and 40
// with 4; 15 x 80 heads of their own over 967 keys 54 and 58; one token of 8 heads over 1000 keys 11.3 and 10.5.  With 11,
// 2 x 32 heads over 1400 keys 14.9 instead of 13.5.
constexpr int kWholeTiles = 8;
// What changing to a unit costs a CTA, in key tiles: q, the first maximum, the row's leaving.  Counted as nothing (0),
// CTAs with many short units end last: 32 sequences of up to 2060 tokens and one empty slot, 16 heads of 64, take 46 us,
// and 33 with 3; 16 x 5 drafted tokens 51 and 48; 4 x 64 tokens over up to 2000 keys 34 and 31.
constexpr int kStart = 3;
// Places that a CTA of the wide kernel takes at least: 1 joins more pieces, 6 leaves SMs without work.  4 x 64 tokens over
// up to 2000 keys, 32 heads over 8: 31.0 us with 4, 30.8 with 1, 31.5 with 6.
constexpr int kWideLeast = 4;
// CTAs that a unit keeps busy at most when there are few, and those that few units keep busy at least.  131072 keys, one
// unit of 8 / 16 / 32 / 128 rows: 23 / 25 / 31 / 55 us with 128 CTAs, 28 / 28 / 35 / 60 with 64; two units of 128 rows:
// 60 with 128, 67 with 256.
constexpr int kMostPieces = 64, kFewBlocks = 128;
long long tiles_of(const attn_cache_t* c) {
    return ((long long)c->max_blocks * c->block_size + kCacheTile - 1) / kCacheTile;
}
bool splits(const attn_cache_t* c) { return tiles_of(c) > kWholeTiles; }

struct Workspace {  // offsets of its parts, and its size
    unsigned long long ml, tickets, bytes;
};
Workspace workspace_of(const attn_cache_t* c, int R, int sms) {
    // two partial units per CTA: R rows of 128 sums, and (M, l); two tickets per CTA
    const unsigned long long ctas = (unsigned long long)sms * ctas_per_sm(R);
    Workspace w{};
    if (!splits(c)) return w;
    w.ml = ctas * 2 * R * 128 * 4;
    w.tickets = w.ml + ctas * 2 * R * 8;
    w.bytes = w.tickets + ctas * 16;
    return w;
}

// A number that no other launch of this process has, in the upper 48 bits, and
// never 0: the low bits count pieces.
unsigned long long next_ticket() {
    static std::atomic<unsigned long long> count{1};
    return (count.fetch_add(1, std::memory_order_relaxed) * 0x9E3779B97F4Bull + 1) << 16;
}

constexpr int kMaxDevices = 64;
std::mutex g_cache_mutex;
int g_cache_ready[kMaxDevices];  // 0 not yet, 1 ready, else an ATTN_ERR code

template <int R>
bool allow_smem() {
    return cudaFuncSetAttribute(attn_cache_fwd_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)CacheLayout<R>::kDynamicSmem) == cudaSuccess;
}
bool allow_append() {
    // a unit of 128 tokens of 128 elements in kAppendThreads threads
    const auto allow = [](auto kernel) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, append_smem(128 * 128 / 16 / kAppendThreads)) ==
               cudaSuccess;
    };
    return allow(attn_cache_append_kernel<64, false>) && allow(attn_cache_append_kernel<64, true>) &&
           allow(attn_cache_append_kernel<128, false>) && allow(attn_cache_append_kernel<128, true>);
}
int setup_cache_kernels(int dev) {
    if (dev < 0 || dev >= kMaxDevices) return ATTN_ERR_DEVICE;
    std::lock_guard<std::mutex> lock(g_cache_mutex);
    if (g_cache_ready[dev] == 0)
        g_cache_ready[dev] = allow_smem<8>() && allow_smem<16>() && allow_smem<32>() && allow_append() &&
                                     cudaFuncSetAttribute(attn_cache_fwd_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                          (int)CacheWideLayout::kDynamicSmem) == cudaSuccess
                                 ? 1
                                 : ATTN_ERR_DEVICE;
    return g_cache_ready[dev] == 1 ? ATTN_OK : g_cache_ready[dev];
}

template <typename L, typename K>
int launch_fwd(K kernel, const CUtensorMap& tk, const CUtensorMap& tv, const CacheFwdParams& p, int sms, long long tiles,
               cudaStream_t st) {
    const long long units = (long long)p.plan.B * p.plan.q_tiles * p.plan.heads, most = (long long)sms * L::kCtas;
    if (units > 0x7fffffffll / (tiles + p.plan.start)) return ATTN_ERR_UNSUPPORTED;
    const long long work = p.plan.whole ? units : units * tiles;  // CTAs that would get something
    const long long use = p.plan.whole || units * kMostPieces > kFewBlocks ? units * kMostPieces : kFewBlocks;
    const long long grid = std::min(std::min(work, use), most);
    return launch(kernel, (int)grid, L::kThreads, L::kDynamicSmem, !L::kWide, st, tk, tv, p);
}

// Launches a write or read kernel with the threads per unit that hold the
// largest unit's elements at 64 a thread.
template <typename P, typename K>
int launch_rw(K kernel, int threads, const P& p, cudaStream_t st) {
    const int per = 256 / threads;
    return launch(kernel, (p.num_units + per - 1) / per, 256, 0, true, st, p);
}

// q's heads a thread at most, and the units that their number comes down for (rope_plan).  2 x 4096 tokens of 32 + 8 + 8 heads
// of 128 with norms: 37.4 us with 8, 35.1 with 16 and with 32.  8 x 64 tokens of them 7.3 us with 152 units, 6.7 with 304, 8.7 with
// 608; 256 single tokens 6.1, 6.9 and 6.9.
constexpr int kAppendPer = 16;
constexpr long long kAppendUnits = 304;
// Shares of 16 elements that a thread of a unit holds at most, before the unit gets twice the threads: 2 x 4096 tokens as
// above 35.2 us with 2, 35.1 with 4, 41.7 with 8.
constexpr int kAppendItems = 4;
template <int D, bool kInter>
int launch_append(CacheAppendParams& p, int rows, long long q_units, cudaStream_t st) {
    const int shares = rows * (D / 16);
    p.unit_shift = 5;
    while (1 << p.unit_shift < kAppendThreads && shares > kAppendItems << p.unit_shift) ++p.unit_shift;
    const int per = kAppendThreads >> p.unit_shift, items = (shares + (1 << p.unit_shift) - 1) >> p.unit_shift;
    const long long writes = ((long long)p.num_units + per - 1) / per, blocks = 2 * writes + q_units;
    if (blocks > 0x7fffffffll) return ATTN_ERR_UNSUPPORTED;
    p.first_v = (unsigned int)(writes + q_units);
    p.k_share = append_share((unsigned int)writes, (unsigned int)q_units);
    return launch(attn_cache_append_kernel<D, kInter>, (int)blocks, kAppendThreads, append_smem(items), true, st, p);
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" int attn_cache_write(const attn_cache_t* cache, const void* k, const long long* k_strides, const void* v,
                                const long long* v_strides, const int* new_lens, int S, void* stream) {
    int rc = check_cache(cache);
    if (rc != ATTN_OK) return rc;
    if (!k || !v || S < 1) return ATTN_ERR_INVALID_ARG;
    if (S > (1 << 29)) return ATTN_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15u ||
        reinterpret_cast<uintptr_t>(new_lens) & 3u)
        return ATTN_ERR_MISALIGNED;
    CacheWriteParams p{};
    size_t kb = 0, vb = 0;
    if ((rc = row_strides(k_strides, cache->B, cache->Hkv, S, cache->D, p.k_stride, &kb)) != ATTN_OK) return rc;
    if ((rc = row_strides(v_strides, cache->B, cache->Hkv, S, cache->D, p.v_stride, &vb)) != ATTN_OK) return rc;
    if (meets_itself(cache) || meets_cache(cache, k, kb, false) || meets_cache(cache, v, vb, false) ||
        (new_lens && meets_cache(cache, new_lens, (size_t)cache->B * 4, false)))
        return ATTN_ERR_INVALID_ARG;
    int sms = 0, device = -1;
    unsigned int* status = nullptr;
    if ((rc = host::current_device(&sms, &status, &device)) != ATTN_OK) return rc;
    p.c = view_of(cache, status);
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.new_lens = new_lens;
    p.S = S;
    const int bs = cache->block_size;
    // S tokens from any slot touch at most this many blocks (and no more than there are).
    const long long touched = ((long long)S + bs - 2) / bs + 1;
    p.blocks_per_seq = (int)(touched < cache->max_blocks ? touched : cache->max_blocks);
    const long long units = (long long)cache->B * cache->Hkv * 2 * p.blocks_per_seq;
    if (units > 0x7fffff00ll) return ATTN_ERR_UNSUPPORTED;
    p.num_units = (int)units;
    const int elements = (S < bs ? S : bs) * cache->D;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (elements <= 64 * 32) return launch_rw(attn_cache_write_kernel<32>, 32, p, st);
    if (elements <= 64 * 64) return launch_rw(attn_cache_write_kernel<64>, 64, p, st);
    if (elements <= 64 * 128) return launch_rw(attn_cache_write_kernel<128>, 128, p, st);
    return launch_rw(attn_cache_write_kernel<256>, 256, p, st);
}

extern "C" int attn_cache_append(const attn_cache_t* cache, const attn_rope_t* rope, const attn_heads_t* in, void* q_out,
                                 const int* new_lens, int Hq, int S, void* stream) {
    int rc = check_cache(cache);
    if (rc != ATTN_OK) return rc;
    const int B = cache->B, Hkv = cache->Hkv, D = cache->D;
    if ((rc = host::check_rope(rope, D)) != ATTN_OK) return rc;
    if (!in || !in->k || !in->v || S < 1 || !in->q != !q_out || (in->q && Hq < 1)) return ATTN_ERR_INVALID_ARG;
    if (S > (1 << 29) || (in->q && Hq > (1 << 20)) || (long long)B * S > (1ll << 31) - 64) return ATTN_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(in->q) | reinterpret_cast<uintptr_t>(in->k) | reinterpret_cast<uintptr_t>(in->v) |
         reinterpret_cast<uintptr_t>(q_out)) & 15u || reinterpret_cast<uintptr_t>(new_lens) & 3u)
        return ATTN_ERR_MISALIGNED;
    CacheAppendParams p{};
    const void* from[3] = {in->q, in->k, in->v};
    const long long* strides[3] = {in->q_strides, in->k_strides, in->v_strides};
    size_t bytes[3] = {0, 0, 0};
    const size_t nl = new_lens ? (size_t)B * 4 : 0;
    for (int i = 0; i < 3; ++i) {
        if (!from[i]) continue;
        const int H = i == 0 ? Hq : Hkv;
        const long long* x = strides[i];
        const long long used[3] = {B > 1 ? x[0] : 0, H > 1 ? x[1] : 0, S > 1 ? x[2] : 0};
        if ((rc = row_strides(used, B, H, S, D, p.in.stride[i], &bytes[i])) != ATTN_OK) return rc;
        p.in.p[i] = static_cast<__nv_bfloat16*>(const_cast<void*>(from[i]));
        if (meets_cache(cache, from[i], bytes[i], false)) return ATTN_ERR_INVALID_ARG;
    }
    const size_t n = (size_t)cache_bytes(cache), ns = (size_t)cache->num_blocks * Hkv * 4;
    if (meets_itself(cache) || (nl && meets_cache(cache, new_lens, nl, false)) || host::rope_meets(rope, cache->k, n, B, S, D) ||
        host::rope_meets(rope, cache->v, n, B, S, D) || host::rope_meets(rope, cache->k_scale, ns, B, S, D) ||
        host::rope_meets(rope, cache->v_scale, ns, B, S, D))
        return ATTN_ERR_INVALID_ARG;
    const int bs = cache->block_size;
    long long q_units = 0;
    if (q_out) {
        const size_t qb = (size_t)B * Hq * S * D * 2;
        if (meets_cache(cache, q_out, qb, true) || (nl && host::ranges_overlap(q_out, qb, new_lens, nl)) ||
            host::rope_meets(rope, q_out, qb, B, S, D))
            return ATTN_ERR_INVALID_ARG;
        for (int i = 0; i < 3; ++i)
            if (host::ranges_overlap(q_out, qb, from[i], bytes[i])) return ATTN_ERR_INVALID_ARG;
        p.out.p[0] = static_cast<__nv_bfloat16*>(q_out);
        p.out.stride[0][0] = (long long)Hq * S * D;
        p.out.stride[0][1] = (long long)S * D;
        p.out.stride[0][2] = D;
        p.plan = rope_plan((long long)B * S, Hq, 0, 0, D, kAppendThreads, kAppendPer, kAppendUnits);
        q_units = rope_tiles(p.plan) * rope_chunks(p.plan);
    }
    int sms = 0, device = -1;
    unsigned int* status = nullptr;
    if ((rc = host::current_device(&sms, &status, &device)) != ATTN_OK) return rc;
    if ((rc = setup_cache_kernels(device)) != ATTN_OK) return rc;
    p.c = view_of(cache, status);
    host::fill_rope(rope, &p.r);
    p.new_lens = new_lens;
    p.S = S;
    // as in attn_cache_write
    const long long touched = ((long long)S + bs - 2) / bs + 1;
    p.blocks_per_seq = (int)(touched < cache->max_blocks ? touched : cache->max_blocks);
    const long long units = (long long)B * Hkv * p.blocks_per_seq;
    if (units > 0x3fffff00ll) return ATTN_ERR_UNSUPPORTED;
    p.num_units = (int)units;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int rows = S < bs ? S : bs;  // of the largest unit
    if (D == 64) return rope->interleaved ? launch_append<64, true>(p, rows, q_units, st) : launch_append<64, false>(p, rows, q_units, st);
    return rope->interleaved ? launch_append<128, true>(p, rows, q_units, st) : launch_append<128, false>(p, rows, q_units, st);
}

extern "C" int attn_cache_read(const attn_cache_t* cache, void* k, void* v, int first, int S, void* stream) {
    int rc = check_cache(cache);
    if (rc != ATTN_OK) return rc;
    if ((!k && !v) || S < 1 || first < 0) return ATTN_ERR_INVALID_ARG;
    if (S > (1 << 29) || first > (1 << 29)) return ATTN_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15u) return ATTN_ERR_MISALIGNED;
    const size_t n = (size_t)cache->B * cache->Hkv * S * cache->D;
    if ((k && meets_cache(cache, k, n * 2, true)) || (v && meets_cache(cache, v, n * 2, true)) ||
        (k && v && host::ranges_overlap(k, n * 2, v, n * 2)))
        return ATTN_ERR_INVALID_ARG;
    int sms = 0, device = -1;
    unsigned int* status = nullptr;
    if ((rc = host::current_device(&sms, &status, &device)) != ATTN_OK) return rc;
    CacheReadParams p{};
    p.c = view_of(cache, status);
    p.k = static_cast<__nv_bfloat16*>(k);
    p.v = static_cast<__nv_bfloat16*>(v);
    p.first = first;
    p.S = S;
    // Blocks from first's on, no further than the cache's capacity.
    const int bs = cache->block_size, from = first / bs;
    const long long to = ((long long)first + S + bs - 1) / bs, blocks = (to < cache->max_blocks ? to : cache->max_blocks) - from;
    if (blocks < 1) return ATTN_OK;  // past every sequence's end
    const long long units = (long long)cache->B * cache->Hkv * (k && v ? 2 : 1) * blocks;
    if (units > 0x7fffff00ll) return ATTN_ERR_UNSUPPORTED;
    p.blocks_per_seq = (int)blocks;
    p.num_units = (int)units;
    const int elements = (S < bs ? S : bs) * cache->D;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (elements <= 64 * 32) return launch_rw(attn_cache_read_kernel<32>, 32, p, st);
    if (elements <= 64 * 64) return launch_rw(attn_cache_read_kernel<64>, 64, p, st);
    if (elements <= 64 * 128) return launch_rw(attn_cache_read_kernel<128>, 128, p, st);
    return launch_rw(attn_cache_read_kernel<256>, 256, p, st);
}

extern "C" int attn_cache_workspace(const attn_cache_t* cache, int Hq, int Sq, unsigned long long* bytes) {
    int rc = check_cache(cache);
    if (rc != ATTN_OK) return rc;
    if (!bytes || Hq < 1 || Sq < 1 || Hq % cache->Hkv) return ATTN_ERR_INVALID_ARG;
    *bytes = 0;
    if (!splits(cache)) return ATTN_OK;
    int sms = 0, device = -1;
    unsigned int* status = nullptr;
    if ((rc = host::current_device(&sms, &status, &device)) != ATTN_OK) return rc;
    *bytes = workspace_of(cache, rows_per_unit(Hq / cache->Hkv, Sq), sms).bytes;
    return ATTN_OK;
}

extern "C" int attn_cache_fwd(const attn_cache_t* cache, const void* q, const long long* q_strides, void* out, float* lse,
                              const int* q_lens, int Hq, int Sq, float scale, int causal, void* workspace,
                              unsigned long long workspace_bytes, void* stream) {
    int rc = check_cache(cache);
    if (rc != ATTN_OK) return rc;
    if (!q || !out || Hq < 1 || Sq < 1 || Hq % cache->Hkv || (!workspace && splits(cache))) return ATTN_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
    if ((long long)cache->B * Hq > (1ll << 30) || (long long)Sq * (Hq / cache->Hkv) > (1ll << 30)) return ATTN_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(workspace)) & 15u ||
        (reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(q_lens)) & 3u)
        return ATTN_ERR_MISALIGNED;
    CacheFwdParams p{};
    size_t qb = 0;
    if ((rc = row_strides(q_strides, cache->B, Hq, Sq, cache->D, p.q_stride, &qb)) != ATTN_OK) return rc;
    const size_t rows = (size_t)cache->B * Hq * Sq, ob = rows * cache->D * 2, lb = rows * 4;
    const size_t nl = q_lens ? (size_t)cache->B * 4 : 0, wb = (size_t)workspace_bytes;
    struct { const void* p; size_t n; } written[3] = {{out, ob}, {lse, lse ? lb : 0}, {workspace, workspace ? wb : 0}};
    for (int i = 0; i < 3; ++i) {
        if (written[i].n == 0) continue;
        if (meets_cache(cache, written[i].p, written[i].n, true) || host::ranges_overlap(written[i].p, written[i].n, q, qb) ||
            (nl && host::ranges_overlap(written[i].p, written[i].n, q_lens, nl)))
            return ATTN_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (written[j].n && host::ranges_overlap(written[i].p, written[i].n, written[j].p, written[j].n))
                return ATTN_ERR_INVALID_ARG;
    }
    int sms = 0, device = -1;
    unsigned int* status = nullptr;
    if ((rc = host::current_device(&sms, &status, &device)) != ATTN_OK) return rc;
    if ((rc = setup_cache_kernels(device)) != ATTN_OK) return rc;
    const int group = Hq / cache->Hkv, R = rows_per_unit(group, Sq);
    const Workspace ws = workspace_of(cache, R, sms);
    if (workspace_bytes < ws.bytes) return ATTN_ERR_INVALID_ARG;
    if (ws.bytes > 0) {
        char* at = static_cast<char*>(workspace);
        p.part_o = reinterpret_cast<float*>(at);
        p.part_ml = reinterpret_cast<float2*>(at + ws.ml);
        p.tickets = reinterpret_cast<unsigned long long*>(at + ws.tickets);
        p.ticket = next_ticket();
    }
    alignas(64) CUtensorMap tk, tv;
    const long long outer = (long long)cache->num_blocks * cache->Hkv;
    if (host::encode_byte_box(&tk, device, cache->k, cache->D, cache->block_size, outer, cache->block_size) != ATTN_OK ||
        host::encode_byte_box(&tv, device, cache->v, cache->D, cache->block_size, outer, cache->block_size) != ATTN_OK)
        return ATTN_ERR_INVALID_ARG;
    p.c = view_of(cache, status);
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.Hq = Hq;
    p.Sq = Sq;
    p.group = group;
    p.hper = group < R ? group : R;
    p.hper_inv = (65536 + p.hper - 1) / p.hper;
    p.hgroups = (group + p.hper - 1) / p.hper;
    p.scale_log2 = scale * kLog2e;
    p.wait_limit_ns = host::wait_limit_ns();
    p.plan.seq_lens = cache->seq_lens;
    p.plan.q_lens = q_lens;
    p.plan.B = cache->B;
    p.plan.Sq = Sq;
    p.plan.capacity = cache->max_blocks * cache->block_size;
    p.plan.causal = causal ? 1 : 0;
    p.plan.qper = R / p.hper;
    p.plan.q_tiles = (Sq + p.plan.qper - 1) / p.plan.qper;
    if ((long long)cache->B * p.plan.q_tiles > (1ll << 30)) return ATTN_ERR_UNSUPPORTED;
    p.plan.heads = cache->Hkv * p.hgroups;
    const long long units = (long long)cache->B * p.plan.q_tiles * p.plan.heads;
    p.plan.whole = splits(cache) ? 0 : units <= (long long)sms * ctas_per_sm(R) ? 1 : 2;
    p.plan.least = R == 128 && !p.plan.whole ? kWideLeast : 1;
    p.plan.start = p.plan.whole == 1 ? 0 : kStart;
    const long long tiles = tiles_of(cache);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (R) {
        case 8: return launch_fwd<CacheLayout<8>>(attn_cache_fwd_kernel<8>, tk, tv, p, sms, tiles, st);
        case 16: return launch_fwd<CacheLayout<16>>(attn_cache_fwd_kernel<16>, tk, tv, p, sms, tiles, st);
        case 32: return launch_fwd<CacheLayout<32>>(attn_cache_fwd_kernel<32>, tk, tv, p, sms, tiles, st);
        default: return launch_fwd<CacheWideLayout>(attn_cache_fwd_wide_kernel, tk, tv, p, sms, tiles, st);
    }
}
