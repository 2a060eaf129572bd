// attn_rope.cu -- the entry points of rotary positions and norms of heads (include/attn.h): argument checks, plans,
// launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/attn.h"
#include "host.h"
#include "kernel_rope.cuh"
#include "launch.h"
#include "rope_check.h"
#include "rows.h"

namespace attn {
namespace {

using host::RowsBox;

// Heads of a thread at most: 4 compute the sines twice as often (2 x 4096 tokens of 32 + 8 + 8 heads with norms, forward
// and backward: 35.3 and 64 us, with 8 32.4 and 52.4, with 16 33.5 and 51.6), 16 leave less to go round (1 x 2048 tokens of 32
// + 32 + 32: 18.0 and 19.7).
// And the units (blocks) that this comes down for, forward / backward with norms: 300 tokens of 32 + 8 + 8 heads of 128 take 5.1
// / 8.4 us with 152, 4.4 / 7.6 with 304, 5.3 / 9.5 with 608; 3 x 1237 of 12 + 4 + 4 heads of 64 6.5 / 10.9, 6.5 / 10.9 and 5.8 /
// 10.9.
constexpr int kPer = 8;
constexpr long long kUnits = 304;

int check_sizes(int B, int Hq, int Hkv, int S, int D) {
    if (B < 1 || Hq < 1 || Hkv < 1 || S < 1) return ATTN_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
    if (Hq > (1 << 20) || Hkv > (1 << 20) || (long long)B * S > (1ll << 31) - 64) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

// The plan of a call: the split follows the sizes alone, not which of q, k and v are present.
int plan_of(int B, int Hq, int Hkv, int S, int D, const bool (&present)[3], RopePlan* plan) {
    *plan = rope_plan((long long)B * S, Hq, Hkv, Hkv, D, kRopeThreads, kPer, kUnits);
    if (rope_tiles(*plan) * rope_chunks(*plan) > 0x7fffffffll) return ATTN_ERR_UNSUPPORTED;
    for (int i = 0; i < 3; ++i)
        if (!present[i]) plan->heads[i] = plan->chunks[i] = 0;
    return ATTN_OK;
}

// One of a call's tensors; `box` gets its rows, dimensions of one element with a stride of 0.
int rows_of(const attn_heads_t* x, int kind, int B, int H, int S, int D, RowsBox* box) {
    void* const p = kind == 0 ? x->q : kind == 1 ? x->k : x->v;
    const long long* st = kind == 0 ? x->q_strides : kind == 1 ? x->k_strides : x->v_strides;
    *box = RowsBox{p, {B, H, S}, {0, 0, 0}, D};
    if (!p) return ATTN_OK;
    if (reinterpret_cast<uintptr_t>(p) & 15u) return ATTN_ERR_MISALIGNED;
    for (int i = 0; i < 3; ++i) {
        if (box->n[i] == 1) continue;
        if (st[i] < 0) return ATTN_ERR_INVALID_ARG;
        if (st[i] % 8) return ATTN_ERR_MISALIGNED;
        if (st[i] > (1ll << 46) / (box->n[i] - 1)) return ATTN_ERR_UNSUPPORTED;  // 2^47 bytes from the first to the last
        box->stride[i] = st[i];
    }
    return ATTN_OK;
}
int all_rows_of(const attn_heads_t* x, int B, int Hq, int Hkv, int S, int D, RowsBox (&box)[3]) {
    for (int i = 0; i < 3; ++i) {
        const int rc = rows_of(x, i, B, i == 0 ? Hq : Hkv, S, D, &box[i]);
        if (rc != ATTN_OK) return rc;
    }
    return ATTN_OK;
}
void take(RopeRows* to, const RowsBox (&box)[3]) {
    for (int i = 0; i < 3; ++i) {
        to->p[i] = static_cast<__nv_bfloat16*>(const_cast<void*>(box[i].p));
        for (int j = 0; j < 3; ++j) to->stride[i][j] = box[i].stride[j];
    }
}

// Whether the outputs keep apart from each other and from what is read, but for rows written where they were read.
bool outputs_fit(const RowsBox (&out)[3], const RowsBox* const* read, int reads, const attn_rope_t* r, int B, int S, int D) {
    for (int i = 0; i < 3; ++i) {
        if (!out[i].p) continue;
        if (!rows_distinct(out[i])) return false;
        for (int j = 0; j < i; ++j)
            if (out[j].p && !rows_apart(out[i], out[j])) return false;
        for (int k = 0; k < reads; ++k)
            for (int j = 0; j < 3; ++j)
                if (read[k][j].p && !(i == j && rows_same(out[i], read[k][j])) && !rows_apart(out[i], read[k][j])) return false;
        if (host::rope_meets(r, out[i].p, 2 * (size_t)rows_extent(out[i]), B, S, D)) return false;
    }
    return true;
}

bool any_weight(const attn_rope_t* r) { return r->q_weight || r->k_weight; }

template <template <int, bool, bool> class Launch, typename P>
int dispatch(const P& p, int D, bool inter, bool norm, cudaStream_t st) {
    const int grid = (int)(rope_tiles(p.plan) * rope_chunks(p.plan));
    if (D == 64) {
        if (inter) return norm ? Launch<64, true, true>::go(p, grid, st) : Launch<64, true, false>::go(p, grid, st);
        return norm ? Launch<64, false, true>::go(p, grid, st) : Launch<64, false, false>::go(p, grid, st);
    }
    if (inter) return norm ? Launch<128, true, true>::go(p, grid, st) : Launch<128, true, false>::go(p, grid, st);
    return norm ? Launch<128, false, true>::go(p, grid, st) : Launch<128, false, false>::go(p, grid, st);
}
template <int D, bool kInter, bool kNorm>
struct Forward {
    static int go(const RopeFwdParams& p, int grid, cudaStream_t st) {
        return launch(attn_rope_kernel<D, kInter, kNorm>, grid, kRopeThreads, 0, true, st, p);
    }
};
template <int D, bool kInter, bool kNorm>
struct Backward {
    static int go(const RopeBwdParams& p, int grid, cudaStream_t st) {
        return launch(attn_rope_bwd_kernel<D, kInter, kNorm>, grid, kRopeThreads, 0, true, st, p);
    }
};

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" int attn_rope(const attn_rope_t* rope, const attn_heads_t* in, const attn_heads_t* out, int B, int Hq, int Hkv, int S,
                         int D, void* stream) {
    int rc = check_sizes(B, Hq, Hkv, S, D);
    if (rc != ATTN_OK) return rc;
    if ((rc = host::check_rope(rope, D)) != ATTN_OK) return rc;
    if (!in || !out) return ATTN_ERR_INVALID_ARG;
    RowsBox from[3], to[3];
    if ((rc = all_rows_of(in, B, Hq, Hkv, S, D, from)) != ATTN_OK || (rc = all_rows_of(out, B, Hq, Hkv, S, D, to)) != ATTN_OK) return rc;
    const bool present[3] = {to[0].p != nullptr, to[1].p != nullptr, to[2].p != nullptr};
    for (int i = 0; i < 3; ++i)
        if (present[i] != (from[i].p != nullptr)) return ATTN_ERR_INVALID_ARG;
    if (!present[0] && !present[1] && !present[2]) return ATTN_ERR_INVALID_ARG;
    const RowsBox* read[1] = {from};
    if (!outputs_fit(to, read, 1, rope, B, S, D)) return ATTN_ERR_INVALID_ARG;
    RopeFwdParams p{};
    if ((rc = plan_of(B, Hq, Hkv, S, D, present, &p.plan)) != ATTN_OK) return rc;
    int sms = 0, device = -1;
    unsigned int* status = nullptr;
    if ((rc = host::current_device(&sms, &status, &device)) != ATTN_OK) return rc;
    host::fill_rope(rope, &p.r);
    p.S = S;
    take(&p.in, from);
    take(&p.out, to);
    return dispatch<Forward>(p, D, rope->interleaved != 0, any_weight(rope), static_cast<cudaStream_t>(stream));
}

extern "C" int attn_rope_workspace(const attn_rope_t* rope, int B, int Hq, int Hkv, int S, int D, unsigned long long* bytes) {
    int rc = check_sizes(B, Hq, Hkv, S, D);
    if (rc != ATTN_OK) return rc;
    if ((rc = host::check_rope(rope, D)) != ATTN_OK) return rc;
    if (!bytes) return ATTN_ERR_INVALID_ARG;
    const bool present[3] = {rope->q_weight != nullptr, rope->k_weight != nullptr, false};
    RopePlan plan;
    if ((rc = plan_of(B, Hq, Hkv, S, D, present, &plan)) != ATTN_OK) return rc;
    *bytes = (unsigned long long)rope_tiles(plan) * rope_chunks(plan) * D * 4;
    return ATTN_OK;
}

extern "C" int attn_rope_bwd(const attn_rope_t* rope, const attn_heads_t* grad, const attn_heads_t* in, const attn_heads_t* out,
                             void* dq_weight, void* dk_weight, int B, int Hq, int Hkv, int S, int D, void* workspace,
                             unsigned long long workspace_bytes, void* stream) {
    int rc = check_sizes(B, Hq, Hkv, S, D);
    if (rc != ATTN_OK) return rc;
    if ((rc = host::check_rope(rope, D)) != ATTN_OK) return rc;
    if (!grad || !out || (!in && any_weight(rope))) return ATTN_ERR_INVALID_ARG;
    RowsBox up[3], from[3] = {}, to[3];
    if ((rc = all_rows_of(grad, B, Hq, Hkv, S, D, up)) != ATTN_OK || (rc = all_rows_of(out, B, Hq, Hkv, S, D, to)) != ATTN_OK) return rc;
    void* const dw[2] = {dq_weight, dk_weight};
    const void* const weight[2] = {rope->q_weight, rope->k_weight};
    bool present[3];
    for (int i = 0; i < 3; ++i) {
        const bool wants = i < 2 && dw[i];
        if (wants && !weight[i]) return ATTN_ERR_INVALID_ARG;
        present[i] = up[i].p != nullptr;
        if (present[i] != (to[i].p || wants)) return ATTN_ERR_INVALID_ARG;
        if (present[i] && i < 2 && weight[i]) {  // the norm's input is read again
            if ((rc = rows_of(in, i, B, i == 0 ? Hq : Hkv, S, D, &from[i])) != ATTN_OK) return rc;
            if (!from[i].p) return ATTN_ERR_INVALID_ARG;
        }
    }
    if (!present[0] && !present[1] && !present[2]) return ATTN_ERR_INVALID_ARG;
    const size_t wide = rope->weight_format == ATTN_WEIGHT_F32 ? 4 : 2;
    RopeBwdParams p{};
    if ((rc = plan_of(B, Hq, Hkv, S, D, present, &p.plan)) != ATTN_OK) return rc;
    size_t rows[2], need = 0;
    for (int i = 0; i < 2; ++i) {
        rows[i] = dw[i] ? (size_t)rope_tiles(p.plan) * p.plan.chunks[i] : 0;
        need += rows[i] * D * 4;
    }
    if (need && (!workspace || workspace_bytes < need)) return ATTN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(need ? workspace : nullptr) | reinterpret_cast<uintptr_t>(dq_weight) |
         reinterpret_cast<uintptr_t>(dk_weight)) & 15u)
        return ATTN_ERR_MISALIGNED;
    const RowsBox* read[2] = {up, from};
    if (!outputs_fit(to, read, 2, rope, B, S, D)) return ATTN_ERR_INVALID_ARG;
    // The weights' gradients and the workspace keep apart from all else.
    struct { const void* p; size_t n; } flat[3] = {{dq_weight, dq_weight ? D * wide : 0}, {dk_weight, dk_weight ? D * wide : 0},
                                                   {workspace, need}};
    for (int i = 0; i < 3; ++i) {
        if (flat[i].n == 0) continue;
        for (int j = 0; j < i; ++j)
            if (flat[j].n && host::ranges_overlap(flat[i].p, flat[i].n, flat[j].p, flat[j].n)) return ATTN_ERR_INVALID_ARG;
        if (host::rope_meets(rope, flat[i].p, flat[i].n, B, S, D)) return ATTN_ERR_INVALID_ARG;
        for (const RowsBox* boxes : {up, from, to})
            for (int j = 0; j < 3; ++j)
                if (boxes[j].p && host::ranges_overlap(flat[i].p, flat[i].n, boxes[j].p, 2 * (size_t)rows_extent(boxes[j])))
                    return ATTN_ERR_INVALID_ARG;
    }
    int sms = 0, device = -1;
    unsigned int* status = nullptr;
    if ((rc = host::current_device(&sms, &status, &device)) != ATTN_OK) return rc;
    host::fill_rope(rope, &p.r);
    p.S = S;
    take(&p.up, up);
    take(&p.in, from);
    take(&p.out, to);
    RopeSumParams sum{};
    float* at = static_cast<float*>(workspace);
    for (int i = 0; i < 2; ++i) {
        p.part[i] = dw[i] ? at : nullptr;
        sum.part[i] = p.part[i];
        sum.rows[i] = (long long)rows[i];
        sum.out[i] = dw[i];
        at += rows[i] * D;
    }
    sum.D = D;
    sum.f32 = rope->weight_format == ATTN_WEIGHT_F32;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((rc = dispatch<Backward>(p, D, rope->interleaved != 0, any_weight(rope), st)) != ATTN_OK || need == 0) return rc;
    return launch(attn_rope_sum_kernel, 2 * D / kRopeSumColumns, kRopeSumThreads, 0, true, st, sum);
}
