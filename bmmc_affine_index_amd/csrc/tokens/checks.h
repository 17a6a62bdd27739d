// checks.h -- argument checks that the entry points on token rows share: types,
// strides, the bytes an array touches and what two arrays have in common.
#pragma once

#include <algorithm>

#include "../../../include/bmmc_tokens.h"

namespace bmmc {
namespace {

constexpr int64_t kMaxIndex = (int64_t(1) << 31) - 1;
// A stride or a width past this is no address on any card; below it the
// products below stay in 64 bits.
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxHeads = 65536;

int element_bytes(int type) { return type == BMMC_F32 ? 4 : type == BMMC_E4M3 ? 1 : 2; }

bool data_type(int type) { return type == BMMC_F32 || type == BMMC_F16 || type == BMMC_BF16; }

bool index_type_ok(int type) { return type == BMMC_I32 || type == BMMC_I64; }

bool aligned(const void *p, size_t bytes) { return (uintptr_t)p % bytes == 0; }

bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }

// The bytes [lo, hi) that a strided array touches.
struct Extent {
    uintptr_t lo, hi;
};

Extent extent(const void *p, int bytes, int64_t inner, const int64_t *sizes,
              const int64_t *strides, int dims) {
    unsigned __int128 last = (unsigned __int128)inner;
    for (int i = 0; i < dims; ++i) {
        if (sizes[i] <= 0) return Extent{(uintptr_t)p, (uintptr_t)p};
        last += (unsigned __int128)(sizes[i] - 1) * (unsigned __int128)strides[i];
    }
    const unsigned __int128 hi = (unsigned __int128)(uintptr_t)p + last * (unsigned)bytes;
    return Extent{(uintptr_t)p, hi > UINTPTR_MAX ? UINTPTR_MAX : (uintptr_t)hi};
}

bool meet(const Extent &a, const Extent &b) { return a.lo < b.hi && b.lo < a.hi; }

// No two elements of a written array share an address: taken by rising
// stride, each dimension steps past all that the ones before it cover.
bool apart(int64_t inner, const int64_t *sizes, const int64_t *strides, int dims) {
    int order[3] = {0, 1, 2};
    std::sort(order, order + dims, [&](int x, int y) { return strides[x] < strides[y]; });
    __int128 covered = inner;
    for (int i = 0; i < dims; ++i) {
        const int d = order[i];
        if (sizes[d] <= 1) continue;
        if (strides[d] < covered) return false;
        covered += (__int128)(sizes[d] - 1) * strides[d];
    }
    return true;
}

// An array's steps, widest first: without those that lead nowhere.
struct Steps {
    int64_t inner;  // adjacent elements at each step
    int dims = 0;
    int64_t sizes[3], strides[3];

    Steps(int64_t elements, const int64_t *n, const int64_t *s, int count) : inner(elements) {
        for (int i = 0; i < count; ++i) {
            if (n[i] <= 1 || s[i] == 0) continue;
            int at = dims++;
            for (; at > 0 && strides[at - 1] < s[i]; --at) {
                sizes[at] = sizes[at - 1];
                strides[at] = strides[at - 1];
            }
            sizes[at] = n[i];
            strides[at] = s[i];
        }
    }
    // Elements from the first to past the last of one step of the first `from`.
    __int128 reach(int from) const {
        __int128 r = inner;
        for (int i = from; i < dims; ++i) r += (__int128)(sizes[i] - 1) * strides[i];
        return r;
    }
};

__int128 floor_div(__int128 a, int64_t b) { return a / b - (a % b < 0); }

// Whether b, `off` elements from a, has an element that a has too.  Without
// their i and j widest steps the two are compared for each difference of the
// next step that brings their stretches together, which is one or none for
// arrays in step; after `looks` comparisons the answer is yes.
bool shared(const Steps &a, int i, const Steps &b, int j, __int128 off, int *looks) {
    if (off >= a.reach(i) || -off >= b.reach(j)) return false;
    if (i == a.dims && j == b.dims) return true;
    if (--*looks < 0) return true;
    const int64_t sa = i < a.dims ? a.strides[i] : 0, sb = j < b.dims ? b.strides[j] : 0;
    const int64_t step = std::max(sa, sb);
    const int64_t na = sa == step ? a.sizes[i] : 1, nb = sb == step ? b.sizes[j] : 1;
    i += sa == step;
    j += sb == step;
    const __int128 lo = std::max<__int128>(1 - na, floor_div(-b.reach(j) - off, step) + 1);
    const __int128 hi = std::min<__int128>(nb - 1, floor_div(a.reach(i) - off - 1, step));
    for (__int128 k = lo; k <= hi; ++k)
        if (shared(a, i, b, j, off + k * step, looks)) return true;
    return false;
}

bool share(const void *p, const Steps &a, const void *q, const Steps &b, int bytes) {
    int looks = 256;
    const __int128 off = ((__int128)(uintptr_t)q - (__int128)(uintptr_t)p) / bytes;
    return shared(a, 0, b, 0, off, &looks);
}

Extent matrix(const void *p, int type, int64_t rows, int64_t stride, int64_t dim) {
    return extent(p, element_bytes(type), dim, &rows, &stride, 1);
}

int check_rotation(const bmmc_rotation &r, int head_dim) {
    if (r.pairs < 1 || 2 * (int64_t)r.pairs > head_dim || r.axes < 1 || r.axes > BMMC_MAX_AXES ||
        !stride_ok(r.axis_stride) || !index_type_ok(r.position_type) || !r.freqs)
        return BMMC_ERR_INVALID_ARG;
    if (!aligned(r.freqs, r.freqs_are_64 ? 8 : 4) || !aligned(r.axis_of_pair, 4) ||
        !aligned(r.positions, r.position_type == BMMC_I64 ? 8 : 4))
        return BMMC_ERR_INVALID_ARG;
    return BMMC_OK;
}

struct HeadsExtent {
    Extent in, out;
};

// The heads' strides and pointers; `writes`: they have an out.
int check_heads(const bmmc_heads &x, int64_t batch, int64_t tokens, int dim, int type,
                bool writes, HeadsExtent *e) {
    const int bytes = element_bytes(type);
    if (x.heads < 1 || x.heads > kMaxHeads || !x.in || !aligned(x.in, bytes) ||
        !stride_ok(x.in_batch) || !stride_ok(x.in_token) || !stride_ok(x.in_head))
        return BMMC_ERR_INVALID_ARG;
    const int64_t sizes[3] = {batch, tokens, x.heads};
    const int64_t is[3] = {x.in_batch, x.in_token, x.in_head};
    e->in = extent(x.in, bytes, dim, sizes, is, 3);
    if (!writes) return BMMC_OK;
    if (!x.out || !aligned(x.out, bytes) || !stride_ok(x.out_batch) || !stride_ok(x.out_token) ||
        !stride_ok(x.out_head))
        return BMMC_ERR_INVALID_ARG;
    const int64_t os[3] = {x.out_batch, x.out_token, x.out_head};
    if (!apart(dim, sizes, os, 3)) return BMMC_ERR_ALIAS;
    e->out = extent(x.out, bytes, dim, sizes, os, 3);
    bool same = x.in == x.out;
    for (int i = 0; i < 3; ++i) same &= sizes[i] <= 1 || is[i] == os[i];
    if (!same && meet(e->in, e->out)) return BMMC_ERR_ALIAS;
    return BMMC_OK;
}

Steps steps_in(const bmmc_heads &x, int64_t batch, int64_t tokens, int dim) {
    const int64_t sizes[3] = {batch, tokens, x.heads};
    const int64_t strides[3] = {x.in_batch, x.in_token, x.in_head};
    return Steps(dim, sizes, strides, 3);
}

Steps steps_out(const bmmc_heads &x, int64_t batch, int64_t tokens, int dim) {
    const int64_t sizes[3] = {batch, tokens, x.heads};
    const int64_t strides[3] = {x.out_batch, x.out_token, x.out_head};
    return Steps(dim, sizes, strides, 3);
}

}  // namespace
}  // namespace bmmc
