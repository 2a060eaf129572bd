// rows.h -- rows of heads [B, H, S, D] at any strides in memory, as the host checks them: whether two such tensors share
// an element, or one of them holds an element twice.  Views of one packed tensor interleave without sharing any, so
// address ranges alone do not tell.  Plain C++ without CUDA calls.
#pragma once

#include <cstddef>
#include <cstdint>

namespace attn {
namespace host {

// Rows of D elements of 2 bytes at p + 2 (b stride[0] + h stride[1] + s stride[2]).
struct RowsBox {
    const void* p;
    long long n[3], stride[3];
    int D;
};

inline long long rows_extent(const RowsBox& x) {  // elements from the first to past the last
    long long e = x.D;
    for (int i = 0; i < 3; ++i) e += (x.n[i] - 1) * x.stride[i];
    return e;
}

// Whether every element has a place of its own, shown by each stride passing what lies below it.
inline bool rows_distinct(const RowsBox& x) {
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (x.stride[order[j]] < x.stride[order[i]]) {
                const int t = order[i];
                order[i] = order[j];
                order[j] = t;
            }
    long long e = x.D;
    for (int k : order) {
        if (x.n[k] == 1) continue;
        if (x.stride[k] < e) return false;
        e += (x.n[k] - 1) * x.stride[k];
    }
    return true;
}

// Whether two tensors share no element: their ranges are apart, or there is a period (one of their strides) that every
// other stride either is a multiple of or stays within, and within it they are.
inline bool rows_apart(const RowsBox& x, const RowsBox& y) {
    const intptr_t a = reinterpret_cast<intptr_t>(x.p), b = reinterpret_cast<intptr_t>(y.p);
    if (a + 2 * rows_extent(x) <= b || b + 2 * rows_extent(y) <= a) return true;
    for (int i = 0; i < 6; ++i) {
        const long long period = i < 3 ? x.stride[i] : y.stride[i - 3];
        if (period <= 0) continue;
        long long width[2];
        const RowsBox* box[2] = {&x, &y};
        for (int k = 0; k < 2; ++k) {
            width[k] = box[k]->D;
            for (int d = 0; d < 3; ++d)
                if (box[k]->stride[d] % period) width[k] += (box[k]->n[d] - 1) * box[k]->stride[d];
        }
        long long at = ((b - a) / 2) % period;
        if (at < 0) at += period;
        if (width[0] <= at && at + width[1] <= period) return true;
    }
    return false;
}

inline bool rows_same(const RowsBox& x, const RowsBox& y) {
    for (int i = 0; i < 3; ++i)
        if (x.n[i] != y.n[i] || x.stride[i] != y.stride[i]) return false;
    return x.p == y.p && x.D == y.D;
}

}  // namespace host
}  // namespace attn
