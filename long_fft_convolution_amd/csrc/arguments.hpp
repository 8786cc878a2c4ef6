// arguments.hpp -- host helpers that the sequence operators' entry points
// share: status reporting, tensor arguments as views and their checks.
#pragma once
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>

#include "../../include/fftconv.h"
#include "fftconv_internal.hpp"

namespace fftconv {

constexpr int64_t kCus = 256;
constexpr int64_t kMaxGroups = (int64_t(1) << 24) - 1;   // workgroups of 256 threads: a launch has fewer than 2^32 threads
constexpr int64_t kMaxHeadDim = 256;

inline fftconv_status_t fail(fftconv_status_t st, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return st;
}
inline fftconv_status_t ok() {
    set_last_error("");
    return FFTCONV_OK;
}
inline fftconv_status_t hip_status(const char *what, hipError_t e) {
    return e == hipSuccess ? ok() : fail(FFTCONV_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

inline bool dtype_ok(int dt) { return dt == FFTCONV_F32 || dt == FFTCONV_F16 || dt == FFTCONV_BF16; }
inline int64_t elem_bytes(int dt) { return dt == FFTCONV_F32 ? 4 : 2; }
inline bool aligned(const void *p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)n == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// A tensor argument: `dims` sizes and strides (elements) above a contiguous row of `row` values.
struct View {
    const char *name;
    const void *p;
    int dims;
    int64_t size[3], stride[3], row;
    int64_t bytes_per;

    // A dimension of one element has no use for its stride, whatever the caller's view carries there: kernels and
    // checks see 0 (the walks from a sequence's end start at a row some strides before its first).
    View &settle() {
        for (int i = 0; i < dims; ++i)
            if (size[i] <= 1) stride[i] = 0;
        return *this;
    }
    bool empty() const {
        for (int i = 0; i < dims; ++i)
            if (size[i] == 0) return true;
        return row == 0;
    }
    // bytes from p to the end of the last row
    int64_t span() const {
        if (empty()) return 0;
        int64_t last = row;
        for (int i = 0; i < dims; ++i) last += (size[i] - 1) * stride[i];
        return last * bytes_per;
    }
    // bytes from p that the view's elements stay within modulo a period: dimensions that step by whole periods
    // add nothing
    int64_t extent(int64_t period) const {
        int64_t last = row;
        for (int i = 0; i < dims; ++i)
            if (stride[i] * bytes_per % period) last += (size[i] - 1) * stride[i];
        return last * bytes_per;
    }
    // Whether the views may share memory.  Spans that meet belong to tensors of one buffer (column blocks of a matrix,
    // heads side by side): those are apart where for some stride as a period their extents are arcs of its
    // circle that do not touch.  What no stride tells apart counts as shared.
    bool overlaps(const View &o) const {
        if (!p || !o.p || empty() || o.empty()) return false;
        const auto a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
        if (a >= b + (uintptr_t)o.span() || b >= a + (uintptr_t)span()) return false;
        for (const View *v : {this, &o})
            for (int i = 0; i < v->dims; ++i) {
                const int64_t period = v->stride[i] * v->bytes_per;
                if (period <= 0) continue;
                const int64_t mine = extent(period), its = o.extent(period), way = (int64_t)(b - a) % period;
                const int64_t ahead = way < 0 ? way + period : way;      // from this view's start round to o's
                if (mine <= ahead && ahead + its <= period) return false;
            }
        return true;
    }
    // every element at a place of its own: each stride reaches past what the smaller ones span
    bool distinct() const {
        int order[3] = {0, 1, 2};
        std::sort(order, order + dims, [&](int x, int y) { return stride[x] < stride[y]; });
        int64_t reach = row;
        for (int i = 0; i < dims; ++i) {
            const int d = order[i];
            if (size[d] <= 1) continue;
            if (stride[d] < reach) return false;
            reach += (size[d] - 1) * stride[d];
        }
        return true;
    }
    // rows may be met 16 bytes at a time
    bool vec16() const {
        const int64_t e = 16 / bytes_per;
        if (!aligned(p, 16)) return false;
        for (int i = 0; i < dims; ++i)
            if (size[i] > 1 && stride[i] % e) return false;
        return true;
    }
};

// The checks that every tensor argument passes; outputs also hold each element once.
inline fftconv_status_t check_view(const View &v, bool required, bool output) {
    if (!v.p) {
        if (!required || v.empty()) return FFTCONV_OK;
        return fail(FFTCONV_ERR_INVALID_ARGUMENT, "%s must be non-null", v.name);
    }
    if (!aligned(v.p, v.bytes_per))
        return fail(FFTCONV_ERR_INVALID_ARGUMENT, "%s must be aligned to its %d-byte elements", v.name, (int)v.bytes_per);
    for (int i = 0; i < v.dims; ++i) {
        if (v.size[i] <= 1) continue;
        if (v.stride[i] < 0) return fail(FFTCONV_ERR_INVALID_ARGUMENT, "%s has a negative stride", v.name);
        if (v.stride[i] > (int64_t(1) << 40) / v.size[i])
            return fail(FFTCONV_ERR_INVALID_ARGUMENT, "%s has a stride of %lld elements", v.name, (long long)v.stride[i]);
    }
    if (output && !v.distinct())
        return fail(FFTCONV_ERR_INVALID_ARGUMENT, "%s: strides let its elements share memory", v.name);
    return FFTCONV_OK;
}

inline fftconv_status_t check_workspace(const void *ws, size_t have, size_t need) {
    if (need == 0) return FFTCONV_OK;
    if (!ws || have < need) return fail(FFTCONV_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws ? have : (size_t)0, need);
    if (!aligned(ws, 16)) return fail(FFTCONV_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
    return FFTCONV_OK;
}

inline View raw_view(const char *name, const void *p, int64_t bytes) { return View{name, p, 1, {1, 1, 1}, {0, 0, 0}, bytes, 1}; }

inline fftconv_status_t check_apart(const View *outs, int nout, const View *ins, int nin) {
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (outs[i].overlaps(ins[j]))
                return fail(FFTCONV_ERR_INVALID_ARGUMENT, "%s overlaps %s", outs[i].name, ins[j].name);
        for (int j = 0; j < i; ++j)
            if (outs[i].overlaps(outs[j]))
                return fail(FFTCONV_ERR_INVALID_ARGUMENT, "%s overlaps %s", outs[i].name, outs[j].name);
    }
    return FFTCONV_OK;
}

// whole 16-byte pieces along rows
inline bool chunk_vec(const View &v) { return v.vec16() && v.row % (16 / v.bytes_per) == 0; }

}  // namespace fftconv
