// cache_index.h -- where a cache token lives: the checked index arithmetic of
// the paged 8-bit cache (attn_cache_t in include/attn.h).  Lengths and block
// numbers are device data that the host never sees, so every kernel goes
// through these functions, which turn a bad value into a safe one and report
// it.  Plain C++ without CUDA calls: host tests compile it by itself.
#pragma once

#ifdef __CUDACC__
#define ATTN_HD __host__ __device__ __forceinline__
#else
#define ATTN_HD inline
#endif

namespace attn {

// Status word bit: a block number or a length lay outside the cache.
enum : unsigned int { kStatusBadCache = 2u };

// The cache as kernels take it (attn_cache_t plus the device status word).
struct CacheView {
    unsigned char *k, *v;
    float *k_scale, *v_scale;
    const int* block_table;  // [B, max_blocks]
    const int* seq_lens;     // [B]
    int num_blocks, block_size, block_shift, max_blocks, B, Hkv, D;
    unsigned int* status;
};

// `value` moved into 0 .. cap; *bad is set when it lay outside.
ATTN_HD int cache_clamp(int value, int cap, bool* bad) {
    if (value < 0) {
        *bad = true;
        return 0;
    }
    if (value > cap) {
        *bad = true;
        return cap;
    }
    return value;
}

// What one sequence brings to a call: `len` tokens held, of which the `count`
// rows of this call are the last, row i at position first + i.  first < 0 when
// there are more rows than tokens: those rows stand for no token.
struct CacheSpan {
    int len, count, first;
};
ATTN_HD CacheSpan cache_span(int seq_len, int count, int capacity, int rows, bool* bad) {
    CacheSpan s;
    s.len = cache_clamp(seq_len, capacity, bad);
    s.count = cache_clamp(count, rows, bad);
    s.first = s.len - s.count;
    return s;
}

// A table entry as a block number: itself, or -1 (and *bad) outside the cache.
ATTN_HD int cache_block(int entry, int num_blocks, bool* bad) {
    if (entry < 0 || entry >= num_blocks) {
        *bad = true;
        return -1;
    }
    return entry;
}

// Element offset of a block's token `slot` for a head.
ATTN_HD unsigned long long cache_offset(int block, int head, int slot, int Hkv, int block_size, int D) {
    return (((unsigned long long)block * Hkv + head) * block_size + slot) * D;
}

}  // namespace attn
