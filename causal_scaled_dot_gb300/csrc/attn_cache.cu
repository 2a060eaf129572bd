// attn_cache.cu -- the entry points of the 8-bit key/value cache
// (include/attn.h): argument checks, TMA descriptors, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/attn.h"
#include "cache_index.h"
#include "common.cuh"
#include "host.h"
#include "kernel_cache_fwd.cuh"
#include "kernel_cache_rw.cuh"

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

int launched() { return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH; }

template <int kThreads>
int launch_write(const CacheWriteParams& p, cudaStream_t st) {
    const long long per = 256 / kThreads, grid = (p.num_units + per - 1) / per;
    if (grid > (1ll << 31) - 1) return ATTN_ERR_UNSUPPORTED;
    attn_cache_write_kernel<kThreads><<<(unsigned)grid, 256, 0, st>>>(p);
    return launched();
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
    if (meets_cache(cache, k, kb, false) || meets_cache(cache, v, vb, false) ||
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
    p.num_units = (long long)cache->B * cache->Hkv * 2 * p.blocks_per_seq;
    const int elements = (S < bs ? S : bs) * cache->D;  // of the largest unit
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (elements <= 64 * 32) return launch_write<32>(p, st);
    if (elements <= 64 * 64) return launch_write<64>(p, st);
    if (elements <= 64 * 128) return launch_write<128>(p, st);
    return launch_write<256>(p, st);
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
    p.num_vec = (long long)(n / 16);
    const long long want = (p.num_vec + 255) / 256, most = (long long)sms * 8;
    const dim3 grid((unsigned)(want < most ? want : most), k && v ? 2 : 1);
    attn_cache_read_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return launched();
}

extern "C" int attn_cache_workspace(int Hq, int Hkv, int Sq, int D, unsigned long long* bytes) {
    if (!bytes || Hq < 1 || Hkv < 1 || Sq < 1 || Hq % Hkv) return ATTN_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    *bytes = 16;
    return ATTN_OK;
}

extern "C" int attn_cache_fwd(const attn_cache_t* cache, const void* q, const long long* q_strides, void* out, float* lse,
                              const int* q_lens, int Hq, int Sq, float scale, int causal, void* workspace,
                              unsigned long long workspace_bytes, void* stream) {
    int rc = check_cache(cache);
    if (rc != ATTN_OK) return rc;
    if (!q || !out || !workspace || Hq < 1 || Sq < 1 || Hq % cache->Hkv) return ATTN_ERR_INVALID_ARG;
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
    struct { const void* p; size_t n; } written[3] = {{out, ob}, {lse, lse ? lb : 0}, {workspace, wb}};
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
    p.c = view_of(cache, status);
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.q_lens = q_lens;
    p.Hq = Hq;
    p.Sq = Sq;
    p.group = Hq / cache->Hkv;
    p.causal = causal ? 1 : 0;
    p.scale_log2 = scale * kLog2e;
    const long long grid = ((long long)rows + 3) / 4;
    if (grid > (1ll << 31) - 1) return ATTN_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cache->D == 64)
        attn_cache_fwd_row_kernel<64><<<(unsigned)grid, 128, 0, st>>>(p);
    else
        attn_cache_fwd_row_kernel<128><<<(unsigned)grid, 128, 0, st>>>(p);
    return launched();
}
