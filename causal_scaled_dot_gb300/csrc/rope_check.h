// rope_check.h -- attn_rope_t as the entry points that take one check it and hand it to their kernels.
#pragma once

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "../../include/attn.h"
#include "host.h"
#include "rope.cuh"

namespace attn {
namespace host {

inline int check_rope(const attn_rope_t* r, int D) {
    if (!r) return ATTN_ERR_INVALID_ARG;
    if (r->rotary_dim < 0 || r->rotary_dim > D) return ATTN_ERR_INVALID_ARG;
    if (r->rotary_dim % (r->interleaved ? 8 : 16)) return ATTN_ERR_UNSUPPORTED;
    if (!std::isfinite(r->factor)) return ATTN_ERR_INVALID_ARG;
    if (r->q_weight || r->k_weight) {
        if (r->weight_format != ATTN_WEIGHT_BF16 && r->weight_format != ATTN_WEIGHT_F32) return ATTN_ERR_INVALID_ARG;
        // below, squares that fp32 loses would count beside it
        if (!std::isfinite(r->eps) || !(r->eps >= 0x1p-100f)) return ATTN_ERR_INVALID_ARG;
        if ((reinterpret_cast<uintptr_t>(r->q_weight) | reinterpret_cast<uintptr_t>(r->k_weight)) & 15u) return ATTN_ERR_MISALIGNED;
    }
    if (r->positions) {
        if (r->position_stride < 0) return ATTN_ERR_INVALID_ARG;
        if (r->position_stride > (1ll << 40)) return ATTN_ERR_UNSUPPORTED;
        if (reinterpret_cast<uintptr_t>(r->positions) & (r->positions_64 ? 7u : 3u)) return ATTN_ERR_MISALIGNED;
    }
    return ATTN_OK;
}

// Whether [a, a + n) meets the weights or the positions.
inline bool rope_meets(const attn_rope_t* r, const void* a, size_t n, int B, int S, int D) {
    const size_t w = (size_t)D * (r->weight_format == ATTN_WEIGHT_F32 ? 4 : 2);
    const size_t at = (size_t)((B - 1) * r->position_stride + S) * (r->positions_64 ? 8 : 4);
    return (r->q_weight && ranges_overlap(a, n, r->q_weight, w)) || (r->k_weight && ranges_overlap(a, n, r->k_weight, w)) ||
           (r->positions && ranges_overlap(a, n, r->positions, at));
}

inline void fill_rope(const attn_rope_t* r, RopeParams* p) {
    for (int i = 0; i < 64; ++i) p->turns[i] = i < r->rotary_dim / 2 ? r->turns[i] : 0;
    p->rot = r->rotary_dim;
    p->factor = r->factor;
    p->eps = r->eps;
    p->weight[0] = r->q_weight;
    p->weight[1] = r->k_weight;
    p->weight_f32 = r->weight_format == ATTN_WEIGHT_F32;
    p->positions = r->positions;
    p->positions_64 = r->positions_64;
    p->position_stride = r->position_stride;
    p->first = r->first;
}

}  // namespace host
}  // namespace attn
