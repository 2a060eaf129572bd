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

// ---------------------------------------------------------------- work of the attention
// A unit is one sequence, one tile of query rows and one group of query heads
// that share a key/value head; it takes the key tiles (128 keys) 0 .. tiles-1.
// All units' tiles stand in one row, by sequence, query tile, head, key tile,
// with `start` empty places before each unit's (what changing to it costs, in
// tiles), and CTA c of G takes places [c T / G, (c + 1) T / G) of it, so CTAs get
// equal work whatever the lengths; the pieces of a unit that crosses a border are
// joined by the CTA that finishes last.  Where every unit is short (`whole`),
// CTAs take whole units instead: one place each (1), for no more units than CTAs,
// or by the CTA where its first place falls (2).
// Lengths are device data, so this runs on the device.  The host makes sure
// that T fits in 31 bits.
constexpr int kCacheTile = 128;  // keys per tile

struct CachePlan {
    const int *seq_lens, *q_lens;  // q_lens may be null: Sq each
    int B, Sq, capacity, causal;
    int qper;     // queries per query tile
    int q_tiles;  // query tiles of Sq queries
    int heads;    // head groups per sequence and query tile
    int whole;    // 1, 2: units are not split
    int least;    // places that a CTA takes at least (but for the total's remainder), 1 or more
    int start;    // places before a unit's tiles
};

ATTN_HD CacheSpan plan_span(const CachePlan& p, int b, bool* bad) {
    return cache_span(p.seq_lens[b], p.q_lens ? p.q_lens[b] : p.Sq, p.capacity, p.Sq, bad);
}
ATTN_HD int plan_q_tiles(const CachePlan& p, const CacheSpan& s) { return (s.count + p.qper - 1) / p.qper; }
// Keys that some row of the query tile sees, and its key tiles: at least one,
// so that rows without a key have an owner too.
ATTN_HD int plan_keys(const CachePlan& p, const CacheSpan& s, int qt) {
    const int last = (qt + 1) * p.qper < s.count ? (qt + 1) * p.qper : s.count;
    const int n = p.causal ? s.first + last : s.len;
    return n < 0 ? 0 : n;
}
ATTN_HD int plan_tiles(const CachePlan& p, const CacheSpan& s, int qt) {
    const int n = plan_keys(p, s, qt);
    return n <= kCacheTile ? 1 : (n + kCacheTile - 1) / kCacheTile;
}

// Places of a unit of `tiles` key tiles.
ATTN_HD int plan_cost(const CachePlan& p, int tiles) { return p.whole == 1 ? 1 : p.start + tiles; }

// Places of the (sequence, query tile) pairs first .. last - 1, pair = b * q_tiles + qt.
ATTN_HD int plan_chunk(const CachePlan& p, int first, int last, bool* bad) {
    if (first >= last) return 0;
    int sum = 0;
    int b = p.q_tiles == 1 ? first : first / p.q_tiles, qt = first - b * p.q_tiles;
    CacheSpan s = plan_span(p, b, bad);
    for (int i = first; i < last; ++i) {
        if (qt == p.q_tiles) {
            qt = 0;
            s = plan_span(p, ++b, bad);
        }
        if (qt < plan_q_tiles(p, s)) sum += plan_cost(p, plan_tiles(p, s, qt)) * p.heads;
        ++qt;
    }
    return sum;
}

struct CachePlace {
    int b, qt, h, s;  // the s-th of a unit's places
};
// The place `offset` places after the start of pair `first` (offset < the places of the pairs from there on).
ATTN_HD CachePlace plan_find(const CachePlan& p, int first, int offset) {
    bool bad = false;
    const int b = p.q_tiles == 1 ? first : first / p.q_tiles;
    CachePlace x{b, first - b * p.q_tiles, 0, 0};
    CacheSpan s = plan_span(p, x.b, &bad);
    for (;;) {
        if (x.qt == p.q_tiles) {
            x.qt = 0;
            if (++x.b >= p.B) return CachePlace{p.B, 0, 0, 0};
            s = plan_span(p, x.b, &bad);
        }
        if (x.qt < plan_q_tiles(p, s)) {
            const int tiles = plan_cost(p, plan_tiles(p, s, x.qt));
            if (offset < tiles * p.heads) {
                x.h = offset / tiles;
                x.s = offset - x.h * tiles;
                return x;
            }
            offset -= tiles * p.heads;
        }
        ++x.qt;
    }
}

// The CTAs that share `total` places: all, or as many as leave each `least`, and so none without a tile between the
// first and the last piece of a unit.
ATTN_HD int plan_ctas(const CachePlan& p, int total, int ctas) {
    const int most = (total + p.least - 1) / p.least;
    return most < ctas ? most : ctas;
}
// First place of CTA `cta` of plan_ctas() many (the total for those past them):
// total * cta / ctas, for fewer than 2^15 CTAs.
ATTN_HD int plan_begin(int total, int cta, int ctas) {
    if (cta >= ctas) return total;
    const int q = total / ctas, r = total - q * ctas;
    return q * cta + (r * cta) / ctas;
}
// The CTA of plan_ctas() many that takes a place: the largest with plan_begin() <= place.
ATTN_HD int plan_cta(int total, int place, int ctas) {
    if (total < 1 << 22 && ctas < 1 << 10) return (int)((((unsigned)place + 1) * (unsigned)ctas - 1) / (unsigned)total);
    return (int)((((long long)place + 1) * ctas - 1) / total);
}

// A CTA's share of one unit: key tiles t .. t + n - 1 of its `tiles`.
struct CacheUnit {
    int b, qt, h, t, n, tiles, keys;
    int at;  // place of its tile 0 in the row of all
    CacheSpan s;
};
// Walks the units of a run of `left` places, the first of which is place `pos` of the row.
struct CacheCursor {
    CachePlace at;
    int pos, left;
    CacheSpan s;
    int tiles;
};
// To the next unit, `places` further.
ATTN_HD void cursor_step(const CachePlan& p, CacheCursor& c, int places) {
    c.left -= places;
    c.pos += places;
    c.at.s = 0;
    if (++c.at.h < p.heads) return;
    c.at.h = 0;
    bool bad = false;
    if (++c.at.qt >= plan_q_tiles(p, c.s)) {
        c.at.qt = 0;
        do {
            if (++c.at.b >= p.B) {
                c.left = 0;
                return;
            }
            c.s = plan_span(p, c.at.b, &bad);
        } while (c.s.count == 0);
    }
    c.tiles = plan_tiles(p, c.s, c.at.qt);
}
ATTN_HD CacheCursor cursor_at(const CachePlan& p, const CachePlace& at, int pos, int left) {
    bool bad = false;
    CacheCursor c{at, pos, at.b < p.B ? left : 0, {}, 0};
    if (c.left > 0) {
        c.s = plan_span(p, at.b, &bad);
        c.tiles = plan_tiles(p, c.s, at.qt);
        if (p.whole && at.s > 0) cursor_step(p, c, plan_cost(p, c.tiles) - at.s);  // the CTA before has it
    }
    return c;
}
ATTN_HD bool cursor_next(const CachePlan& p, CacheCursor& c, CacheUnit& u) {
    if (c.left <= 0) return false;
    u.b = c.at.b;
    u.qt = c.at.qt;
    u.h = c.at.h;
    u.tiles = c.tiles;
    const int rest = plan_cost(p, c.tiles) - c.at.s, places = p.whole || rest < c.left ? rest : c.left;
    const int start = p.whole == 1 ? 0 : p.start;
    u.t = c.at.s > start ? c.at.s - start : 0;
    u.n = (p.whole ? c.tiles : c.at.s + places - start) - u.t;
    u.at = c.pos - c.at.s + start;
    u.s = c.s;
    u.keys = plan_keys(p, c.s, c.at.qt);
    if (u.n <= 0) {  // the run ends before the unit's tiles
        c.left = 0;
        return false;
    }
    cursor_step(p, c, places);
    return true;
}

}  // namespace attn
