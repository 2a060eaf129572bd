// rope_index.h -- how the rotation's work is laid out (attn_rope and attn_rope_bwd in include/attn.h): which elements
// of a head a lane holds, and which rows a block takes.  Plain C++ without CUDA calls: host tests compile it by itself.
#pragma once

#ifdef __CUDACC__
#define ROPE_HD __host__ __device__ __forceinline__
#else
#define ROPE_HD inline
#endif

namespace attn {

// A row (one head of one token) is held by D / 16 lanes, two vectors of 8 elements each, so that both elements of every
// pair are in one lane.  Blocks of 256 threads leave more of the last wave empty: 1 x 2048 tokens of 32 + 32 + 32 heads with
// norms 19.7 us, with 128 18.0.
constexpr int kRopeThreads = 128;

// The vectors of lane `l` and whether they are rotated.  Half layout: rotated lanes hold vector l and the one rot / 2
// elements further, element j of the one paired with element j of the other (pair 8 l + j); the rest of the head goes to
// the other lanes so that neighbouring lanes hold neighbouring vectors (two in a row a lane took 29 us where this takes 19,
// for 33.5 M elements: half sectors).  Interleaved: vectors l and l + D / 16, four pairs each (pairs 4 * vector + 0 .. 3).
struct RopeLane {
    int a, b;        // vectors, in units of 8 elements
    int turn_a, turn_b;
};
ROPE_HD RopeLane rope_lane(int l, int D, int rot, int interleaved) {
    RopeLane x;
    if (interleaved) {
        x.a = l;
        x.b = l + D / 16;
        x.turn_a = x.a * 8 < rot;
        x.turn_b = x.b * 8 < rot;
    } else {
        const int n = rot / 16;
        x.turn_a = x.turn_b = l < n;
        x.a = l < n ? l : l + n;
        x.b = l < n ? l + n : l + D / 16;
    }
    return x;
}

// A block's rows: `tokens` (a power of two) by threads / (D / 16) / tokens heads side by side, and up to `per` such
// groups of heads one after the other, all of one kind (q, k or v).  The units of a tile of tokens stand side by side.
struct RopePlan {
    unsigned int total;  // tokens, B * S < 2^31
    int tokens, groups;  // tokens and heads side by side, powers of two
    int token_shift, group_shift;
    int per;             // heads of a thread, at most
    int heads[3];        // of q, k and v; 0: absent
    int chunks[3];       // units of each kind in a tile of tokens
};
ROPE_HD int rope_chunks(const RopePlan& p) { return p.chunks[0] + p.chunks[1] + p.chunks[2]; }
ROPE_HD long long rope_tiles(const RopePlan& p) { return ((long long)p.total + p.tokens - 1) / p.tokens; }

struct RopeUnit {
    unsigned int tile;
    int kind, chunk;
};
ROPE_HD RopeUnit rope_unit(const RopePlan& p, unsigned int unit) {
    const unsigned int all = (unsigned int)rope_chunks(p);
    RopeUnit u;
    u.tile = unit / all;
    u.chunk = (int)(unit - u.tile * all);
    u.kind = 0;
    while (u.chunk >= p.chunks[u.kind]) u.chunk -= p.chunks[u.kind++];
    return u;
}

// The plan for `total` tokens, these heads and blocks of `threads`: as many tokens side by side as there are and fit, and as many heads a
// thread as still give `units` units, `per` at most.
ROPE_HD RopePlan rope_plan(long long total, int Hq, int Hk, int Hv, int D, int threads, int per, long long units) {
    RopePlan p;
    const int rows = threads / (D / 16);
    p.total = (unsigned int)total;
    p.tokens = 1;
    p.token_shift = 0;
    while (p.tokens < rows && p.tokens < total) {
        p.tokens *= 2;
        ++p.token_shift;
    }
    p.groups = rows / p.tokens;
    p.group_shift = 0;
    while (1 << p.group_shift < p.groups) ++p.group_shift;
    p.heads[0] = Hq;
    p.heads[1] = Hk;
    p.heads[2] = Hv;
    for (p.per = per;; p.per = (p.per + 1) / 2) {
        for (int i = 0; i < 3; ++i) p.chunks[i] = (p.heads[i] + p.groups * p.per - 1) / (p.groups * p.per);
        if (p.per == 1 || rope_tiles(p) * rope_chunks(p) >= units) return p;
    }
}

// The first blocks of an append: `ks` that write K among `qs` of q, evenly.  Of the first i of them i share / 2^32 write K.
ROPE_HD unsigned long long append_share(unsigned int ks, unsigned int qs) {
    const unsigned long long all = (unsigned long long)ks + qs;
    return (((unsigned long long)ks << 32) + all - 1) / all;
}
// Whether block i is one that writes K, and which of its kind it is.
ROPE_HD bool append_is_k(unsigned long long share, unsigned int i, unsigned int* index) {
    const unsigned int before = (unsigned int)(i * share >> 32);
    const bool k = (unsigned int)((i + 1ull) * share >> 32) != before;
    *index = k ? before : i - before;
    return k;
}

}  // namespace attn
