// sequence_ops.cpp -- host side of the decay-attention and linear-product
// entry points of include/fftconv.h: argument checks, the rules that choose a
// kernel variant and split the work, workspace layout, launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "../../include/fftconv.h"
#include "fftconv_internal.hpp"
#include "sequence_ops.hpp"

using namespace fftconv;

namespace {

fftconv_status_t fail(fftconv_status_t st, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return st;
}
fftconv_status_t ok() {
    set_last_error("");
    return FFTCONV_OK;
}
fftconv_status_t hip_status(const char *what, hipError_t e) {
    return e == hipSuccess ? ok() : fail(FFTCONV_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool dtype_ok(int dt) { return dt == FFTCONV_F32 || dt == FFTCONV_F16 || dt == FFTCONV_BF16; }
int64_t elem_bytes(int dt) { return dt == FFTCONV_F32 ? 4 : 2; }
bool aligned(const void *p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)n == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

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
fftconv_status_t check_view(const View &v, bool required, bool output) {
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

// ---- decay attention --------------------------------------------------------
constexpr int64_t kMaxHeadDim = 256;
constexpr int64_t kSegStep = 64;          // parts of a segment are whole chunks
constexpr int64_t kMinSegment = 256;      // below this the second read of y, z costs more than it spreads
constexpr int64_t kCus = 256;
constexpr int64_t kMaxGroups = (int64_t(1) << 24) - 1;   // workgroups of 256 threads: a launch has fewer than 2^32 threads

int64_t z_tiles(int64_t dx, int64_t dz) { return ceil_div(dz, decay_z_tile(dx, dz)); }

struct DecayShape {
    int64_t B, N, H, Hk, Dk, Dv;
    int dt;
    bool packed;
    int64_t T() const { return packed ? N : B * N; }
};

// How sequences are cut.  A walk is serial, so the chip fills only when the walks (kinds of walk x
// sequences x heads x z tiles) number two (rows wider than 64) or three a CU; fewer are cut into segments, at
// the price of reading y and z twice (a pass of its own sums each segment first).  That pass reads half as
// much per token and is cut finer where segments are few: a segment is `seglen / sublen` parts.
// Measured in bf16, B x N tokens x heads of D x D:
//     walks a CU 1, 2, 4:        4 x 4096 x 20 of 128: 136, 126, 151 us; 1 x 32768 x 12 of 64 at 1, 3, 4: 90, 73, 79 us
//     shortest segment 128, 256, 512:  1 x 2048 x 20 of 128: 48, 47, 56 us; 1 x 8192: 80, 81, 93 us
//     two segments against none:  12 x 4096 x 20 of 128: 332 against 245 us; its gradients at 4 x 4096: 259 against
//         234 us; three or more against none: gradients of 5 x 2048 x 12 of 64: 58 against 72 us
//     parts against whole segments in the sums:  1 x 512 x 20 of 128: 38 against 42 us; gradients of
//         4 x 4096 cut in two: 259 against 287 us
// Packed sequences have lengths that only the device knows: they are cut by the mean load (two walks a CU
// against one: 148 against 168 us for 12 sequences of 0 to 6001 tokens, 136 against 107 for 12 of 1386).
struct DecayCut {
    int64_t seglen, sublen, segments, parts;   // tokens; how many there are at most
    bool cut;                                  // more than one segment a sequence
};
DecayCut decay_cut(const DecayShape &s, int64_t walks_per_token, int64_t sums_per_token, bool wide) {
    const int64_t slots = kCus * (wide ? 2 : 3), T = s.T();
    DecayCut c{};
    int64_t len;
    if (s.packed) {
        len = std::max(kMinSegment, ceil_div(T * walks_per_token, slots));
    } else {
        // equal sequences: as many equal segments as all walk at once
        const int64_t most = std::max<int64_t>(1, slots / std::max<int64_t>(1, s.B * walks_per_token));
        len = std::max(std::min(kMinSegment, std::max<int64_t>(s.N, 1)), ceil_div(s.N, most));
    }
    len = round_up(len, kSegStep);
    // two segments: the sums cost more than they spread
    if (!s.packed && ceil_div(s.N, len) < 3) len = round_up(std::max<int64_t>(s.N, 1), kSegStep);
    c.cut = (s.packed ? T : s.N) > len;
    // parts: two sums a CU, of at least four chunks
    const int64_t segs = std::max<int64_t>(1, s.packed ? T / len : s.B * (ceil_div(s.N, len) - 1));
    int64_t parts = !c.cut ? 1 : std::max<int64_t>(1, 2 * kCus / std::max<int64_t>(1, segs * sums_per_token));
    parts = std::min(parts, std::max<int64_t>(1, len / 128));
    c.sublen = round_up(ceil_div(len, parts), kSegStep);
    c.seglen = c.sublen * parts;
    auto count = [&](int64_t l) { return s.packed ? T / l + s.B : s.B * std::max<int64_t>(1, ceil_div(s.N, l)); };
    c.segments = count(c.seglen), c.parts = count(c.sublen);
    c.cut = (s.packed ? T : s.N) > c.seglen;
    return c;
}
bool wide_walks(int64_t Dk, int64_t Dv) { return Dk > 64 || Dv > 64; }
DecayCut fwd_cut(const DecayShape &s) {
    const int64_t walks = s.H * z_tiles(s.Dk, s.Dv);
    return decay_cut(s, walks, walks, wide_walks(s.Dk, s.Dv));
}
// dq, dk (Dv x Dk) and dv (Dk x Dv); sums of both states as Dv x Dk
DecayCut bwd_cut(const DecayShape &s) {
    const int64_t sums = 2 * s.H * z_tiles(s.Dv, s.Dk);
    return decay_cut(s, sums + s.H * z_tiles(s.Dk, s.Dv), sums, wide_walks(s.Dk, s.Dv));
}
size_t cut_bytes(const DecayShape &s, const DecayCut &c) {
    return c.cut ? align_up((size_t)c.parts * s.H * s.Dk * s.Dv * sizeof(float), 256) : 0;
}
// Workspace sizes are asked for by the number of tokens: the most of B equal sequences and of a packed
// call, whose sequences may have any lengths.
size_t most_bytes(DecayCut (*cut)(const DecayShape &), int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv) {
    const DecayShape equal{B, ceil_div(T, std::max<int64_t>(B, 1)), H, H, Dk, Dv, 0, false}, packed{B, T, H, H, Dk, Dv, 0, true};
    return std::max(cut_bytes(equal, cut(equal)), cut_bytes(packed, cut(packed)));
}

hipError_t launch_sums(int dt, const DecaySet &a, hipStream_t s) {
    return dt == FFTCONV_F32   ? launch_decay_sums_f32(a, s)
           : dt == FFTCONV_F16 ? launch_decay_sums_f16(a, s)
                               : launch_decay_sums_bf16(a, s);
}
hipError_t launch_walks(int dt, const DecaySet &a, hipStream_t s) {
    return dt == FFTCONV_F32   ? launch_decay_walks_f32(a, s)
           : dt == FFTCONV_F16 ? launch_decay_walks_f16(a, s)
                               : launch_decay_walks_bf16(a, s);
}

// heads: H or Hk; strides (batch, token, head) at st
View heads_view(const char *name, const void *p, const DecayShape &s, int64_t heads, int64_t row, const int64_t *st) {
    View v{name, p, 3, {s.packed ? 1 : s.B, s.N, heads}, {0, 0, 0}, row, elem_bytes(s.dt)};
    if (st) {
        for (int i = 0; i < 3; ++i) v.stride[i] = st[i];
        if (s.packed) v.stride[0] = 0;
    } else {
        v.stride[0] = s.N * heads * row;
        v.stride[1] = heads * row;
        v.stride[2] = row;
    }
    return v.settle();
}

fftconv_status_t check_shape(const DecayShape &s, float scale) {
    if (!dtype_ok(s.dt)) return fail(FFTCONV_ERR_UNSUPPORTED, "dtype %d is not supported", s.dt);
    if (s.B < 0 || s.N < 0 || s.H < 0 || s.Hk < 0)
        return fail(FFTCONV_ERR_INVALID_ARGUMENT, "B=%lld, N=%lld, H=%lld and Hk=%lld must be >= 0", (long long)s.B,
                    (long long)s.N, (long long)s.H, (long long)s.Hk);
    if (s.Dk < 1 || s.Dk > kMaxHeadDim || s.Dv < 1 || s.Dv > kMaxHeadDim)
        return fail(FFTCONV_ERR_UNSUPPORTED, "head widths Dk=%lld and Dv=%lld must be in [1, %lld]", (long long)s.Dk,
                    (long long)s.Dv, (long long)kMaxHeadDim);
    if (s.H > 0 && (s.Hk < 1 || s.H % s.Hk))
        return fail(FFTCONV_ERR_INVALID_ARGUMENT, "H=%lld must be a multiple of Hk=%lld", (long long)s.H, (long long)s.Hk);
    if (s.H > 65535) return fail(FFTCONV_ERR_UNSUPPORTED, "H=%lld is above 65535", (long long)s.H);
    if (s.B >= (int64_t(1) << 31) || s.N >= (int64_t(1) << 31) || (s.B > 0 && s.N > (int64_t(1) << 40) / s.B) ||
        (s.H > 0 && s.B > kMaxGroups / s.H))
        return fail(FFTCONV_ERR_UNSUPPORTED, "B=%lld, N=%lld, H=%lld: too many sequences or tokens", (long long)s.B,
                    (long long)s.N, (long long)s.H);
    if (!std::isfinite(scale)) return fail(FFTCONV_ERR_INVALID_ARGUMENT, "scale must be finite");
    return FFTCONV_OK;
}

fftconv_status_t check_workspace(const void *ws, size_t have, size_t need) {
    if (need == 0) return FFTCONV_OK;
    if (!ws || have < need) return fail(FFTCONV_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws ? have : (size_t)0, need);
    if (!aligned(ws, 16)) return fail(FFTCONV_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
    return FFTCONV_OK;
}

View state_view(const char *name, const void *p, int64_t count, const DecayShape &s) {
    return View{name, p, 1, {count, 1, 1}, {s.H * s.Dk * s.Dv, 0, 0}, s.H * s.Dk * s.Dv, 4};
}
View raw_view(const char *name, const void *p, int64_t bytes) { return View{name, p, 1, {1, 1, 1}, {0, 0, 0}, bytes, 1}; }

fftconv_status_t check_apart(const View *outs, int nout, const View *ins, int nin) {
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
bool chunk_vec(const View &v) { return v.vec16() && v.row % (16 / v.bytes_per) == 0; }
// The walks reach a chunk's rows by 31-bit offsets.
fftconv_status_t check_reach(const View &v) {
    if (v.size[1] > 1 && v.stride[1] * v.bytes_per >= (int64_t(1) << 25))
        return fail(FFTCONV_ERR_UNSUPPORTED, "%s has a token stride of %lld elements, above 32 MiB", v.name, (long long)v.stride[1]);
    return FFTCONV_OK;
}
void set_x(DecayWalk &w, const View &v, int64_t H) {
    w.x = v.p, w.xb = v.stride[0], w.xt = v.stride[1], w.xh = v.stride[2], w.gx = (int)(H / v.size[2]);
    w.DX = (int)v.row;
    w.vec_x = chunk_vec(v);
}
void set_y(DecayWalk &w, const View &v, int64_t H) {
    w.y = v.p, w.yb = v.stride[0], w.yt = v.stride[1], w.yh = v.stride[2], w.gy = (int)(H / v.size[2]);
    w.vec_y = chunk_vec(v);
}
void set_z(DecayWalk &w, const View &v, int64_t H) {
    w.z = v.p, w.zb = v.stride[0], w.zt = v.stride[1], w.zh = v.stride[2], w.gz = (int)(H / v.size[2]);
    w.DZ = (int)v.row;
    w.vec_z = chunk_vec(v);
}
void set_out(DecayWalk &w, const View &v, int64_t H) {
    w.out = const_cast<void *>(v.p), w.ob = v.stride[0], w.ot = v.stride[1], w.oh = v.stride[2];
    w.go = (int)(H / v.size[2]);
    w.vec_o = v.vec16();
}
void set_cut(DecayWalk &w, const DecayCut &c) {
    w.seglen = c.seglen, w.sublen = c.sublen, w.parts = (int)(c.seglen / c.sublen), w.nblk = c.segments;
}
// the same walks over the parts that have sums of their own
DecaySet parts_of(DecaySet set, const DecayCut &c) {
    for (int i = 0; i < set.kinds; ++i) set.w[i].seglen = c.sublen, set.w[i].nblk = c.parts;
    return set;
}
DecaySet make_set(std::initializer_list<const DecayWalk *> walks, int64_t group) {
    DecaySet set{};
    for (const DecayWalk *w : walks)
        if (w) {
            set.w[set.kinds++] = *w;
            set.w[set.kinds - 1].ztile = decay_z_tile(w->DX, w->DZ);
            set.ztiles = std::max(set.ztiles, (int)z_tiles(w->DX, w->DZ));
        }
    // neighbours share tensors: the walks of a head, its z tiles, and the heads of a group
    set.share = (int)std::min<int64_t>(16, set.kinds * set.ztiles * group);
    return set;
}
// the padded widths that a launch's walks must have in common
bool same_class(const DecayWalk &a, const DecayWalk &b) {
    auto width = [](int dx) { return dx <= 64 ? 64 : dx <= 128 ? 128 : 256; };
    return width(a.DX) == width(b.DX) && decay_z_tile(a.DX, a.DZ) == decay_z_tile(b.DX, b.DZ);
}
// items of a launch, as a check that they fit a grid
bool too_many(const DecaySet &s) {
    return (double)s.w[0].nblk * s.w[0].H * s.ztiles * s.kinds + 8 * 16 > (double)kMaxGroups;
}

}  // namespace

size_t fftconv_decay_fwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv,
                                         fftconv_dtype_t dtype) {
    if (!dtype_ok(dtype) || B < 1 || T < 1 || H < 1 || Dk < 1 || Dv < 1 || Dk > kMaxHeadDim || Dv > kMaxHeadDim) return 0;
    return most_bytes(fwd_cut, B, T, H, Dk, Dv);
}

fftconv_status_t fftconv_decay_fwd(const void *q, const void *k, const void *v, const float *log_decay, void *out,
                                   const int64_t *strides, const float *state_in, float *state_out,
                                   const int32_t *state_slots, int64_t n_slots, const int32_t *cu_seqlens, int64_t B,
                                   int64_t N, int64_t H, int64_t Hk, int64_t Dk, int64_t Dv, float scale,
                                   fftconv_dtype_t dtype, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const DecayShape s{B, N, H, Hk, Dk, Dv, (int)dtype, cu_seqlens != nullptr};
    fftconv_status_t st = check_shape(s, scale);
    if (st != FFTCONV_OK) return st;
    if (n_slots < 0) return fail(FFTCONV_ERR_INVALID_ARGUMENT, "n_slots=%lld must be >= 0", (long long)n_slots);
    if (B == 0 || H == 0) return ok();
    const View vq = heads_view("q", q, s, H, Dk, strides), vk = heads_view("k", k, s, Hk, Dk, strides ? strides + 3 : nullptr),
               vv = heads_view("v", v, s, Hk, Dv, strides ? strides + 6 : nullptr),
               vo = heads_view("out", out, s, H, Dv, strides ? strides + 9 : nullptr);
    for (const View *x : {&vq, &vk, &vv})
        if ((st = check_view(*x, true, false)) != FFTCONV_OK) return st;
    if ((st = check_view(vo, true, true)) != FFTCONV_OK) return st;
    for (const View *x : {&vq, &vk, &vv, &vo})
        if ((st = check_reach(*x)) != FFTCONV_OK) return st;
    if (!log_decay) return fail(FFTCONV_ERR_INVALID_ARGUMENT, "log_decay must be non-null");
    const int64_t states = state_slots ? n_slots : B;
    const View si = state_view("state_in", state_in, states, s), so = state_view("state_out", state_out, states, s);
    for (const View *x : {&si, &so})
        if ((st = check_view(*x, false, false)) != FFTCONV_OK) return st;
    for (const void *p : {(const void *)log_decay, (const void *)state_slots, (const void *)cu_seqlens})
        if (!aligned(p, 4)) return fail(FFTCONV_ERR_INVALID_ARGUMENT, "log_decay, state_slots and cu_seqlens must be 4-byte aligned");
    const size_t need = fftconv_decay_fwd_workspace_bytes(B, s.T(), H, Dk, Dv, dtype);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != FFTCONV_OK) return st;
    const View ws = raw_view("workspace", need ? workspace : nullptr, (int64_t)need);
    const View ld = raw_view("log_decay", log_decay, H * 4), sl = raw_view("state_slots", state_slots, B * 4),
               cu = raw_view("cu_seqlens", cu_seqlens, (B + 1) * 4);
    // state_out may be state_in itself (the pool updated in place), nothing else
    if (state_out && state_in && state_out != state_in && si.overlaps(so))
        return fail(FFTCONV_ERR_INVALID_ARGUMENT, "state_out overlaps state_in without being it");
    const View outs[] = {vo, so, ws}, ins[] = {vq, vk, vv, ld, sl, cu};
    if ((st = check_apart(outs, 3, ins, 6)) != FFTCONV_OK) return st;
    const View apart[] = {vo, ws};
    if ((st = check_apart(apart, 2, &si, 1)) != FFTCONV_OK) return st;
    if (s.T() == 0 && !state_out) return ok();

    DecayWalk w{};
    set_x(w, vq, H);
    set_y(w, vk, H);
    set_z(w, vv, H);
    set_out(w, vo, H);
    w.log_decay = log_decay;
    w.state0 = state_in, w.state1 = state_out, w.keeps = 1;
    w.s0x = w.s1x = Dv, w.s0z = w.s1z = 1;
    w.slots = state_slots, w.n_slots = n_slots;
    w.cu = cu_seqlens;
    w.B = B, w.N = N, w.H = (int)H;
    w.p_scale = scale, w.u_scale = 1.0f, w.i_scale = scale;
    w.off = 1;
    const DecayCut cut = fwd_cut(s);
    set_cut(w, cut);
    w.seg = cut.cut ? static_cast<float *>(workspace) : nullptr;
    w.segx = 1, w.segz = Dk;
    const DecaySet set = make_set({&w}, H / Hk), sums = parts_of(set, cut);
    if (too_many(set) || too_many(sums))
        return fail(FFTCONV_ERR_UNSUPPORTED, "B=%lld, N=%lld, H=%lld: too many sequences or tokens", (long long)B,
                    (long long)N, (long long)H);
    hipError_t e = launch_sums(dtype, sums, stream);
    if (e == hipSuccess) e = launch_walks(dtype, set, stream);
    return hip_status("decay attention", e);
}

fftconv_status_t fftconv_decay_step(const void *q, const void *k, const void *v, const float *log_decay, float *state,
                                    void *out, const int64_t *strides, const int32_t *state_slots, int64_t n_slots,
                                    int64_t B, int64_t H, int64_t Hk, int64_t Dk, int64_t Dv, float scale,
                                    fftconv_dtype_t dtype, hipStream_t stream) {
    const DecayShape s{B, 1, H, Hk, Dk, Dv, (int)dtype, false};
    fftconv_status_t st = check_shape(s, scale);
    if (st != FFTCONV_OK) return st;
    if (n_slots < 0) return fail(FFTCONV_ERR_INVALID_ARGUMENT, "n_slots=%lld must be >= 0", (long long)n_slots);
    if (B == 0 || H == 0) return ok();
    int64_t full[12];
    if (strides)
        for (int i = 0; i < 4; ++i) full[3 * i] = strides[2 * i], full[3 * i + 1] = 0, full[3 * i + 2] = strides[2 * i + 1];
    const int64_t *f = strides ? full : nullptr;
    const View vq = heads_view("q", q, s, H, Dk, f), vk = heads_view("k", k, s, Hk, Dk, f ? f + 3 : nullptr),
               vv = heads_view("v", v, s, Hk, Dv, f ? f + 6 : nullptr), vo = heads_view("out", out, s, H, Dv, f ? f + 9 : nullptr);
    for (const View *x : {&vq, &vk, &vv})
        if ((st = check_view(*x, true, false)) != FFTCONV_OK) return st;
    if ((st = check_view(vo, true, true)) != FFTCONV_OK) return st;
    if (!log_decay || !state) return fail(FFTCONV_ERR_INVALID_ARGUMENT, "log_decay and state must be non-null");
    const View vs = state_view("state", state, state_slots ? n_slots : B, s);
    if ((st = check_view(vs, false, false)) != FFTCONV_OK) return st;
    for (const void *p : {(const void *)log_decay, (const void *)state_slots})
        if (!aligned(p, 4)) return fail(FFTCONV_ERR_INVALID_ARGUMENT, "log_decay and state_slots must be 4-byte aligned");
    const View outs[] = {vo, vs}, ins[] = {vq, vk, vv, raw_view("log_decay", log_decay, H * 4),
                                           raw_view("state_slots", state_slots, B * 4)};
    if ((st = check_apart(outs, 2, ins, 5)) != FFTCONV_OK) return st;

    DecayStep a{};
    a.q = q, a.k = k, a.v = v, a.out = out;
    a.qb = vq.stride[0], a.qh = vq.stride[2], a.kb = vk.stride[0], a.kh = vk.stride[2];
    a.vb = vv.stride[0], a.vh = vv.stride[2], a.ob = vo.stride[0], a.oh = vo.stride[2];
    a.log_decay = log_decay, a.state = state, a.slots = state_slots, a.n_slots = n_slots;
    a.B = B, a.H = (int)H, a.group = (int)(H / Hk), a.Dk = (int)Dk, a.Dv = (int)Dv, a.scale = scale;
    const bool vec = Dv % 4 == 0 && aligned(state, 16);
    const hipError_t e = dtype == FFTCONV_F32   ? launch_decay_step_f32(a, vec, stream)
                         : dtype == FFTCONV_F16 ? launch_decay_step_f16(a, vec, stream)
                                                : launch_decay_step_bf16(a, vec, stream);
    return hip_status("decay step", e);
}

// workspace of the backward call: the states and the states' gradients before each segment, then fp32
// gradients of the heads that share a key/value head
namespace {
struct DecayBwdLayout {
    size_t grads, dk, dv, total;
};
DecayBwdLayout decay_bwd_layout(int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t Dk, int64_t Dv) {
    DecayBwdLayout l{};
    l.grads = most_bytes(bwd_cut, B, T, H, Dk, Dv);
    l.dk = 2 * l.grads;
    l.dv = l.dk + (H == Hk ? 0 : align_up((size_t)T * H * Dk * sizeof(float), 256));
    l.total = l.dv + (H == Hk ? 0 : align_up((size_t)T * H * Dv * sizeof(float), 256));
    return l;
}
}  // namespace

size_t fftconv_decay_bwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t Dk, int64_t Dv,
                                         fftconv_dtype_t dtype) {
    if (!dtype_ok(dtype) || B < 1 || T < 1 || H < 1 || Hk < 1 || Dk < 1 || Dv < 1 || Dk > kMaxHeadDim || Dv > kMaxHeadDim)
        return 0;
    return decay_bwd_layout(B, T, H, Hk, Dk, Dv).total;
}

fftconv_status_t fftconv_decay_bwd(const void *dout, const void *q, const void *k, const void *v,
                                   const float *log_decay, void *dq, void *dk, void *dv, const int64_t *strides,
                                   const float *state_in, const float *dstate_out, float *dstate_in,
                                   const int32_t *cu_seqlens, int64_t B, int64_t N, int64_t H, int64_t Hk, int64_t Dk,
                                   int64_t Dv, float scale, fftconv_dtype_t dtype, void *workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
    const DecayShape s{B, N, H, Hk, Dk, Dv, (int)dtype, cu_seqlens != nullptr};
    fftconv_status_t st = check_shape(s, scale);
    if (st != FFTCONV_OK) return st;
    if (B == 0 || H == 0) return ok();
    auto at = [&](int i) { return strides ? strides + 3 * i : nullptr; };
    const View vd = heads_view("dout", dout, s, H, Dv, at(0)), vq = heads_view("q", q, s, H, Dk, at(1)),
               vk = heads_view("k", k, s, Hk, Dk, at(2)), vv = heads_view("v", v, s, Hk, Dv, at(3)),
               gq = heads_view("dq", dq, s, H, Dk, at(4)), gk = heads_view("dk", dk, s, Hk, Dk, at(5)),
               gv = heads_view("dv", dv, s, Hk, Dv, at(6));
    for (const View *x : {&vd, &vq, &vk, &vv})
        if ((st = check_view(*x, true, false)) != FFTCONV_OK) return st;
    for (const View *x : {&gq, &gk, &gv})
        if ((st = check_view(*x, false, true)) != FFTCONV_OK) return st;
    for (const View *x : {&vd, &vq, &vk, &vv, &gq, &gk, &gv})
        if (x->p && (st = check_reach(*x)) != FFTCONV_OK) return st;
    if (!log_decay) return fail(FFTCONV_ERR_INVALID_ARGUMENT, "log_decay must be non-null");
    const View si = state_view("state_in", state_in, B, s), dso = state_view("dstate_out", dstate_out, B, s),
               dsi = state_view("dstate_in", dstate_in, B, s);
    for (const View *x : {&si, &dso, &dsi})
        if ((st = check_view(*x, false, false)) != FFTCONV_OK) return st;
    for (const void *p : {(const void *)log_decay, (const void *)cu_seqlens})
        if (!aligned(p, 4)) return fail(FFTCONV_ERR_INVALID_ARGUMENT, "log_decay and cu_seqlens must be 4-byte aligned");
    const size_t need = fftconv_decay_bwd_workspace_bytes(B, s.T(), H, Hk, Dk, Dv, dtype);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != FFTCONV_OK) return st;
    const View ws = raw_view("workspace", need ? workspace : nullptr, (int64_t)need);
    const View outs[] = {gq, gk, gv, dsi, ws},
               ins[] = {vd, vq, vk, vv, si, dso, raw_view("log_decay", log_decay, H * 4),
                        raw_view("cu_seqlens", cu_seqlens, (B + 1) * 4)};
    if ((st = check_apart(outs, 5, ins, 8)) != FFTCONV_OK) return st;

    const DecayBwdLayout lay = decay_bwd_layout(B, s.T(), H, Hk, Dk, Dv);
    char *base = static_cast<char *>(workspace);
    const bool shared = H != Hk, tokens = s.T() > 0;
    DecayWalk w{};
    w.log_decay = log_decay;
    w.cu = cu_seqlens;
    w.B = B, w.N = N, w.H = (int)H;
    const DecayCut c = bwd_cut(s);
    const bool cut = c.cut;
    set_cut(w, c);
    // dq: x, y, z = dout, v, k forwards, state S^T (Dv x Dk)
    DecayWalk q_ = w;
    set_x(q_, vd, H);
    set_y(q_, vv, H);
    set_z(q_, vk, H);
    set_out(q_, gq, H);
    q_.state0 = state_in, q_.s0x = 1, q_.s0z = Dv;
    q_.p_scale = scale, q_.u_scale = 1.0f, q_.i_scale = scale;
    q_.off = 1;
    q_.seg = cut ? reinterpret_cast<float *>(base) : nullptr, q_.segx = 1, q_.segz = Dv;
    // dk: x, y, z = v, dout, q from each sequence's end, state G^T (Dv x Dk)
    auto set_grad = [&](DecayWalk &g, const View &grad, size_t part) {
        View o = grad;
        if (shared) o = heads_view("", grad.p ? base + part : nullptr, s, H, grad.row, nullptr), o.bytes_per = 4;
        set_out(g, o, H);
        g.out_f32 = shared;
        g.p_scale = scale, g.u_scale = scale, g.i_scale = 1.0f;
        g.reverse = 1;
        g.state0 = dstate_out;
        g.seg = cut ? reinterpret_cast<float *>(base + lay.grads) : nullptr;
    };
    DecayWalk k_ = w;
    set_x(k_, vv, H);
    set_y(k_, vd, H);
    set_z(k_, vq, H);
    set_grad(k_, gk, lay.dk);
    k_.s0x = 1, k_.s0z = Dv;
    k_.state1 = dstate_in, k_.s1x = 1, k_.s1z = Dv, k_.keeps = 1;
    k_.segx = 1, k_.segz = Dv;
    // dv: x, y, z = k, q, dout, state G (Dk x Dv): the same sums read the other way round
    DecayWalk v_ = w;
    set_x(v_, vk, H);
    set_y(v_, vq, H);
    set_z(v_, vd, H);
    set_grad(v_, gv, lay.dv);
    v_.s0x = Dv, v_.s0z = 1;
    v_.segx = Dv, v_.segz = 1;

    // the gradient of the carried state comes out of dk's walk
    const bool run_q = dq && tokens, run_k = (dk && tokens) || dstate_in, run_v = dv && tokens, sum_g = run_k || run_v;
    const DecaySet sums = make_set({run_q ? &q_ : nullptr, sum_g ? &k_ : nullptr}, H / Hk);
    const DecaySet all = make_set({&q_, &k_, &v_}, H / Hk);
    if (too_many(all) || too_many(parts_of(all, c)))
        return fail(FFTCONV_ERR_UNSUPPORTED, "B=%lld, N=%lld, H=%lld: too many sequences or tokens", (long long)B,
                    (long long)N, (long long)H);
    hipError_t e = hipSuccess;
    if (sums.kinds) e = launch_sums(dtype, parts_of(sums, c), stream);
    const bool together = same_class(k_, v_);
    const DecaySet first = make_set({run_k ? &k_ : nullptr, run_v && together ? &v_ : nullptr, run_q ? &q_ : nullptr}, H / Hk);
    if (e == hipSuccess && first.kinds) e = launch_walks(dtype, first, stream);
    if (e == hipSuccess && run_v && !together) e = launch_walks(dtype, make_set({&v_}, H / Hk), stream);
    if (e == hipSuccess && shared && tokens && (dk || dv)) {
        DecayGroupSum g{};
        const View *grads[] = {&gk, &gv};
        const size_t parts[] = {lay.dk, lay.dv};
        for (int i = 0; i < 2; ++i) {
            const View &o = *grads[i];
            g.src[i] = reinterpret_cast<const float *>(base + parts[i]);
            g.dst[i] = const_cast<void *>(o.p);
            g.D[i] = (int)o.row;
            g.db[i] = o.stride[0], g.dt[i] = o.stride[1], g.dh[i] = o.stride[2];
            g.vec[i] = o.row % 4 == 0 && aligned(o.p, 4 * o.bytes_per) && o.stride[0] % 4 == 0 && o.stride[1] % 4 == 0 &&
                       o.stride[2] % 4 == 0;
        }
        g.B = s.packed ? 1 : B, g.N = N, g.cu = cu_seqlens, g.seqs = B, g.Hk = (int)Hk, g.group = (int)(H / Hk);
        e = dtype == FFTCONV_F32   ? launch_decay_group_sum_f32(g, stream)
            : dtype == FFTCONV_F16 ? launch_decay_group_sum_f16(g, stream)
                                   : launch_decay_group_sum_bf16(g, stream);
    }
    return hip_status("decay attention gradients", e);
}

// ---- linear product -----------------------------------------------------------
namespace {

// Rows that the kernel for single tokens takes.  It against the tile kernel, bf16, 2560 -> 10240: 11.0 against
// 14.8 us for one row, 11.5 / 14.8 for two, 13.4 / 15.0 for four, where its sums and rows of x fill the registers;
// 768 -> 768: 8.8 / 12 us.
constexpr int64_t kVectorRows = 4;

struct GemmPlan {
    int tile, splits;
    int64_t tiles, full, kper;
};

// Tile and split of K for an M x N x K product: the least of a model's times.  A stage (128 bytes of K)
// of one tile takes a CU `alone` microseconds, and `each` where several tiles share the CU (measured
// with bf16 and fp32 at M = 300 .. 8192, N = 768 .. 10240, K = 768 .. 10240; the 256 tile fills a CU).
// The fullest of 256 CUs decides.  Tiles beyond a multiple of 256 may be split along K: their parts
// then pass through memory and a second kernel.  Measured, us by tile (bf16; M x N x K), the plan's choice
// first: 16384 x 10240 x 2560: 256 692, 128 837, 64 1242; 512 x 10240 x 2560: 128 37, 64 44, 256 46;
// 1000 x 2304 x 768 fp32: 64 37, 128 50; without splits the first three take 708, 40 and 42, and 300 x 768 x 10240
// 46 where the split takes 18.
GemmPlan plan_gemm(int64_t M, int64_t N, int64_t K, int dt, bool vec) {
    struct Kind {
        int tile;
        double alone16, each16, alone32, each32;
    };
    static const Kind kinds[] = {{256, 1.45, 1.45, 0.0, 0.0}, {128, 0.60, 0.47, 2.2, 2.05}, {64, 0.28, 0.22, 0.60, 0.52}};
    constexpr double kStart = 4.0, kJoin = 2.0, kBytesPerUs = 6.0e6;
    constexpr int64_t kCus = 256;
    const int64_t bk = 128 / elem_bytes(dt), stages = std::max<int64_t>(1, ceil_div(K, bk));
    GemmPlan best{};
    double least = 1e300;
    for (const Kind &k : kinds) {
        if (vec ? (dt == FFTCONV_F32 && k.tile == 256) : k.tile != 128) continue;
        const int64_t tiles = ceil_div(M, k.tile) * ceil_div(N, k.tile);
        const double alone = dt == FFTCONV_F32 ? k.alone32 : k.alone16, each = dt == FFTCONV_F32 ? k.each32 : k.each16;
        for (int splits = 1; splits <= 16; ++splits) {
            if (splits > 1 && stages < 4 * splits) break;
            const int64_t per = ceil_div(stages, splits);
            if (ceil_div(stages, per) != splits) continue;
            const int64_t full = splits == 1 ? tiles : tiles / kCus * kCus, parts = (tiles - full) * splits;
            if (splits > 1 && parts == 0) break;
            const int64_t whole = ceil_div(full, kCus), part = ceil_div(parts, kCus);
            double us = kStart + (double)(whole * stages + part * per) * (whole + part <= 1 ? alone : each);
            if (splits > 1) us += kJoin + 2.0 * parts * k.tile * k.tile * 4 / kBytesPerUs;
            if (us < least) {
                least = us;
                best = GemmPlan{k.tile, splits, tiles, full, per * bk};
            }
        }
    }
    return best;
}
size_t plan_bytes(const GemmPlan &p) {
    return align_up((size_t)(p.tiles - p.full) * p.splits * p.tile * p.tile * sizeof(float), 256);
}
// the workspace covers a call with or without 16-byte access
size_t gemm_bytes(int64_t M, int64_t N, int64_t K, int dt) {
    return std::max(plan_bytes(plan_gemm(M, N, K, dt, true)), plan_bytes(plan_gemm(M, N, K, dt, false)));
}

hipError_t run_gemm(int dt, LinearGemm &g, int layout, bool vec, float *part, hipStream_t s) {
    const GemmPlan p = plan_gemm(g.M, g.N, g.K, dt, vec);
    const int64_t reach = (int64_t(1) << 22) / elem_bytes(dt);
    g.quads = g.N % 4 == 0 && g.vec_c && g.ldc < reach && (!g.bias || g.vec_b) && (!g.res || (g.vec_r && g.ldr < reach)) &&
              (!g.pre || (g.vec_p && g.ldp < reach));
    g.tiles = p.tiles, g.full = p.full, g.splits = p.splits, g.kper = p.kper, g.part = part;
    return dt == FFTCONV_F32   ? launch_linear_gemm_f32(g, layout, p.tile, vec, s)
           : dt == FFTCONV_F16 ? launch_linear_gemm_f16(g, layout, p.tile, vec, s)
                               : launch_linear_gemm_bf16(g, layout, p.tile, vec, s);
}

// a launch has fewer than 2^32 threads: 512 a tile; 256 for each 16 columns in the kernels that go over rows
constexpr int64_t kMaxColumns = (int64_t(1) << 28) - 16;
bool too_large(int64_t M, int64_t N, int64_t K, int dt) {
    for (bool vec : {true, false}) {
        const GemmPlan p = plan_gemm(M, N, K, dt, vec);
        if (p.full + (p.tiles - p.full) * p.splits >= int64_t(1) << 23) return true;
    }
    return N > kMaxColumns;
}
fftconv_status_t too_large_status(int64_t M, int64_t N, int64_t K) {
    return fail(FFTCONV_ERR_UNSUPPORTED, "M=%lld, N=%lld, K=%lld: too large a product", (long long)M, (long long)N, (long long)K);
}

fftconv_status_t check_linear(int64_t M, int64_t N, int64_t K, int act, int dt) {
    if (!dtype_ok(dt)) return fail(FFTCONV_ERR_UNSUPPORTED, "dtype %d is not supported", dt);
    if (act < 0 || act > 4) return fail(FFTCONV_ERR_UNSUPPORTED, "activation %d is not supported", act);
    for (int64_t n : {M, N, K})
        if (n < 0 || n >= (int64_t(1) << 31))
            return fail(FFTCONV_ERR_INVALID_ARGUMENT, "M=%lld, N=%lld, K=%lld must be in [0, 2^31)", (long long)M,
                        (long long)N, (long long)K);
    return FFTCONV_OK;
}
View matrix(const char *name, const void *p, int64_t rows, int64_t cols, int64_t ld, int dt) {
    return View{name, p, 1, {rows, 1, 1}, {ld, 0, 0}, cols, elem_bytes(dt)}.settle();
}
// four neighbouring values at a time
bool quad(const View &v) {
    return aligned(v.p, 4 * v.bytes_per) && (v.size[0] <= 1 || v.stride[0] % 4 == 0);
}
// whole 16-byte pieces along rows, and byte offsets of a tile of 256 rows within 31 bits
bool pieces(const View &v) {
    return v.vec16() && v.row % (16 / v.bytes_per) == 0 && v.stride[0] * v.bytes_per < (int64_t(1) << 22);
}

}  // namespace

size_t fftconv_linear_fwd_workspace_bytes(int64_t M, int64_t N, int64_t K, fftconv_dtype_t dtype) {
    if (!dtype_ok(dtype) || M < 1 || N < 1 || K < 1 || M <= kVectorRows) return 0;
    return gemm_bytes(M, N, K, dtype);
}

fftconv_status_t fftconv_linear_fwd(const void *x, const void *W, const void *bias, const void *residual, void *out,
                                    void *pre, const int64_t *strides, int64_t M, int64_t N, int64_t K,
                                    fftconv_activation_t activation, fftconv_dtype_t dtype, void *workspace,
                                    size_t workspace_bytes, hipStream_t stream) {
    fftconv_status_t st = check_linear(M, N, K, activation, dtype);
    if (st != FFTCONV_OK) return st;
    if (M == 0 || N == 0) return ok();
    if (too_large(M, N, K, dtype)) return too_large_status(M, N, K);
    auto ld = [&](int i, int64_t dense) { return strides ? strides[i] : dense; };
    const View vx = matrix("x", x, M, K, ld(0, K), dtype), vw = matrix("W", W, N, K, ld(1, K), dtype),
               vb = matrix("bias", bias, 1, N, N, dtype), vr = matrix("residual", residual, M, N, ld(2, N), dtype),
               vo = matrix("out", out, M, N, ld(3, N), dtype), vp = matrix("pre", pre, M, N, ld(4, N), dtype);
    for (const View *v : {&vx, &vw})
        if ((st = check_view(*v, true, false)) != FFTCONV_OK) return st;
    for (const View *v : {&vb, &vr})
        if ((st = check_view(*v, false, false)) != FFTCONV_OK) return st;
    if ((st = check_view(vo, true, true)) != FFTCONV_OK) return st;
    if ((st = check_view(vp, false, true)) != FFTCONV_OK) return st;
    const size_t need = fftconv_linear_fwd_workspace_bytes(M, N, K, dtype);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != FFTCONV_OK) return st;
    const View ws = raw_view("workspace", need ? workspace : nullptr, (int64_t)need);
    const View outs[] = {vo, vp, ws}, ins[] = {vx, vw, vb};
    if ((st = check_apart(outs, 3, ins, 3)) != FFTCONV_OK) return st;
    // out may be the residual itself: each value is read by the lane that then writes it
    const bool in_place = residual && residual == out && vr.stride[0] == vo.stride[0];
    const View touched[] = {vp, ws};
    if ((st = check_apart(touched, 2, &vr, 1)) != FFTCONV_OK) return st;
    if (!in_place && vo.overlaps(vr))
        return fail(FFTCONV_ERR_INVALID_ARGUMENT, "out overlaps residual without being it");

    LinearGemm g{};
    g.A = x, g.lda = vx.stride[0], g.B = W, g.ldb = vw.stride[0];
    g.M = M, g.N = N, g.K = K;
    g.C = out, g.ldc = vo.stride[0], g.vec_c = quad(vo);
    g.bias = bias, g.vec_b = quad(vb);
    g.res = residual, g.ldr = vr.stride[0], g.vec_r = quad(vr);
    g.pre = pre, g.ldp = vp.stride[0], g.vec_p = quad(vp);
    g.act = activation;
    const bool vec = pieces(vx) && pieces(vw);
    if (M <= kVectorRows) {
        const hipError_t e = dtype == FFTCONV_F32   ? launch_linear_vector_f32(g, vec, stream)
                             : dtype == FFTCONV_F16 ? launch_linear_vector_f16(g, vec, stream)
                                                    : launch_linear_vector_bf16(g, vec, stream);
        return hip_status("linear product", e);
    }
    return hip_status("linear product", run_gemm(dtype, g, LAYOUT_NT, vec, static_cast<float *>(workspace), stream));
}

// workspace of the backward call: dz (rows of whole 16-byte pieces), column sums of slabs of
// rows, then the partial sums of a split product
namespace {
struct LinearBwdLayout {
    int64_t ldz, rows, slabs;
    size_t dz, colsum, part, total;
};
LinearBwdLayout linear_bwd_layout(int64_t M, int64_t N, int64_t K, int dt) {
    LinearBwdLayout l{};
    l.ldz = round_up(N, 16 / elem_bytes(dt));
    // slabs of rows: enough workgroups (of 256 columns) to fill the chip eight times over, few enough
    // that their sums are cheap to join
    l.slabs = std::max<int64_t>(1, std::min<int64_t>(ceil_div(M, 32), ceil_div(2048, ceil_div(N, 256) + 1)));
    l.rows = round_up(std::max<int64_t>(1, ceil_div(M, l.slabs)), 8);
    l.slabs = std::max<int64_t>(1, ceil_div(M, l.rows));
    l.colsum = align_up((size_t)M * l.ldz * elem_bytes(dt), 256);
    l.part = l.colsum + align_up((size_t)l.slabs * N * sizeof(float), 256);
    l.total = l.part + std::max(gemm_bytes(M, K, N, dt), gemm_bytes(N, K, M, dt));
    return l;
}
}  // namespace

size_t fftconv_linear_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K, fftconv_dtype_t dtype) {
    if (!dtype_ok(dtype) || M < 0 || N < 0 || K < 0) return 0;
    return linear_bwd_layout(M, N, K, dtype).total;
}

fftconv_status_t fftconv_linear_bwd(const void *dout, const void *x, const void *W, const void *pre, void *dx, void *dW,
                                    void *dbias, const int64_t *strides, int64_t M, int64_t N, int64_t K,
                                    fftconv_activation_t activation, fftconv_dtype_t dtype, void *workspace,
                                    size_t workspace_bytes, hipStream_t stream) {
    fftconv_status_t st = check_linear(M, N, K, activation, dtype);
    if (st != FFTCONV_OK) return st;
    auto ld = [&](int i, int64_t dense) { return strides ? strides[i] : dense; };
    const View vd = matrix("dout", dout, M, N, ld(0, N), dtype), vx = matrix("x", x, M, K, ld(1, K), dtype),
               vw = matrix("W", W, N, K, ld(2, K), dtype), vp = matrix("pre", pre, M, N, ld(3, N), dtype),
               gx = matrix("dx", dx, M, K, ld(4, K), dtype), gw = matrix("dW", dW, N, K, ld(5, K), dtype),
               gb = matrix("dbias", dbias, 1, N, N, dtype);
    if (too_large(M, K, N, dtype) || too_large(N, K, M, dtype) || N > kMaxColumns) return too_large_status(M, N, K);
    const bool need_pre = activation != FFTCONV_ACT_NONE;
    if ((st = check_view(vd, true, false)) != FFTCONV_OK) return st;
    if ((st = check_view(vx, dW != nullptr, false)) != FFTCONV_OK) return st;
    if ((st = check_view(vw, dx != nullptr, false)) != FFTCONV_OK) return st;
    if ((st = check_view(vp, need_pre, false)) != FFTCONV_OK) return st;
    for (const View *v : {&gx, &gw, &gb})
        if ((st = check_view(*v, false, true)) != FFTCONV_OK) return st;
    const LinearBwdLayout l = linear_bwd_layout(M, N, K, dtype);
    if ((st = check_workspace(workspace, workspace_bytes, l.total)) != FFTCONV_OK) return st;
    const View ws = raw_view("workspace", workspace, (int64_t)l.total);
    const View outs[] = {gx, gw, gb, ws}, ins[] = {vd, vx, vw, vp};
    if ((st = check_apart(outs, 4, ins, 4)) != FFTCONV_OK) return st;

    char *base = static_cast<char *>(workspace);
    // without an activation dout itself is dz, unless its rows are not whole 16-byte pieces
    const bool own_dz = (dx || dW) && (need_pre || !pieces(vd));
    LinearDz z{};
    z.dout = dout, z.pre = pre, z.ldo = vd.stride[0], z.ldp = vp.stride[0], z.M = M, z.N = N, z.act = activation;
    z.dz = own_dz ? base : nullptr, z.ldz = l.ldz;
    z.colsum = dbias ? reinterpret_cast<float *>(base + l.colsum) : nullptr;
    z.rows = l.rows;
    z.vec = pieces(vd) && (!need_pre || pieces(vp));
    hipError_t e = hipSuccess;
    if ((own_dz && M > 0 && N > 0) || (dbias && N > 0)) {
        e = dtype == FFTCONV_F32   ? launch_linear_dz_f32(z, l.slabs, dbias, stream)
            : dtype == FFTCONV_F16 ? launch_linear_dz_f16(z, l.slabs, dbias, stream)
                                   : launch_linear_dz_bf16(z, l.slabs, dbias, stream);
        if (e != hipSuccess) return hip_status("dz", e);
    }
    const void *dz = own_dz ? base : dout;
    const int64_t ldz = own_dz ? l.ldz : vd.stride[0];
    const bool small_ldz = ldz * elem_bytes(dtype) < (int64_t(1) << 22);
    float *part = reinterpret_cast<float *>(base + l.part);
    if (dx && M > 0 && K > 0) {
        LinearGemm g{};
        g.A = dz, g.lda = ldz, g.B = W, g.ldb = vw.stride[0];
        g.M = M, g.N = K, g.K = N;
        g.C = dx, g.ldc = gx.stride[0], g.vec_c = quad(gx);
        e = run_gemm(dtype, g, LAYOUT_NN, small_ldz && pieces(vw), part, stream);
        if (e != hipSuccess) return hip_status("dx", e);
    }
    if (dW && N > 0 && K > 0) {
        LinearGemm g{};
        g.A = dz, g.lda = ldz, g.B = x, g.ldb = vx.stride[0];
        g.M = N, g.N = K, g.K = M;
        g.C = dW, g.ldc = gw.stride[0], g.vec_c = quad(gw);
        e = run_gemm(dtype, g, LAYOUT_TN, small_ldz && pieces(vx), part, stream);
        if (e != hipSuccess) return hip_status("dW", e);
    }
    return ok();
}
