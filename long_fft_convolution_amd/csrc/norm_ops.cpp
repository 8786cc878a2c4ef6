// norm_ops.cpp -- host side of the root-mean-square norm's entry points of
// include/fftconv.h: argument checks, how rows are dealt to threads, launches.
#include <cmath>

#include "arguments.hpp"
#include "norm_ops.hpp"

using namespace fftconv;

namespace {

constexpr int64_t kMaxWidth = int64_t(1) << 20;
// Partial sums of the weight's gradient.  bf16 with dsum, a call (both launches) on inputs that no cache holds: 512 are two
// workgroups a CU, as many as hold rows of 2560 at once (16384 rows: 103 us, 158 with 256, 116 with 1024); narrower ones
// leave room for four (65536 rows of 768: 116 us, 154 with 512, 139 with 2048).  Of the narrowest, a workgroup holds sixteen
// rows and more at once, and 512 do (131072 rows of 128: 50 us, 48 with 1024; on inputs in the caches 38 and 42).
int64_t slabs_of(int64_t rows, int64_t D) { return std::min<int64_t>(rows, D > 128 && D <= 1024 ? 1024 : 512); }
// Workgroups of a forward call; more rows are met in turn (65536 rows of 768: 79 us, 80 with 8192, 90 with 1024).
constexpr int64_t kMostGroups = 16384;

struct NormShape {
    int64_t M, G, D;
    int dt;
};

// rows (M, G) of D values of `bytes` bytes; strides (row, group) at st
View rows_view(const char *name, const void *p, const NormShape &s, int64_t bytes, const int64_t *st) {
    View v{name, p, 2, {s.M, s.G, 1}, {s.G * s.D, s.D, 0}, s.D, bytes};
    if (st) v.stride[0] = st[0], v.stride[1] = st[1];
    return v.settle();
}

fftconv_status_t check_shape(const NormShape &s, float eps) {
    if (!dtype_ok(s.dt)) return fail(FFTCONV_ERR_UNSUPPORTED, "dtype %d is not supported", s.dt);
    if (s.M < 0 || s.G < 0)
        return fail(FFTCONV_ERR_INVALID_ARGUMENT, "M=%lld and G=%lld must be >= 0", (long long)s.M, (long long)s.G);
    if (s.D < 1 || s.D > kMaxWidth)
        return fail(FFTCONV_ERR_UNSUPPORTED, "width D=%lld must be in [1, %lld]", (long long)s.D, (long long)kMaxWidth);
    if (s.G > 0 && s.M > ((int64_t(1) << 31) - 1) / s.G)
        return fail(FFTCONV_ERR_UNSUPPORTED, "M=%lld, G=%lld: 2^31 rows or more", (long long)s.M, (long long)s.G);
    if (!std::isfinite(eps) || eps < 0) return fail(FFTCONV_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
    return FFTCONV_OK;
}

bool same_place(const View &a, const View &b) {
    if (a.p != b.p) return false;
    for (int i = 0; i < a.dims; ++i)
        if (a.stride[i] != b.stride[i]) return false;
    return true;
}

// A part of a wave holds a row where one piece a lane does; else a wave where the rows are many and take at most
// `wave` pieces a lane; else a workgroup with up to eight pieces a lane; else the row is read again.  bf16, us by waves /
// by workgroups, a call in a captured graph on inputs that no cache holds:
//     forward, 768 wide: 64 rows 3.3 / 2.7, 2048 rows 6.0 / 5.0, 4096 rows 7.2 / 9.5, 16384 rows 22.4 / 28.8
//     forward, 16384 rows: 1536 wide 40.7 / 39.5, 2560 wide 72.7 / 64.9, 4096 wide 122 / 97
//     gradients, 2560 wide: 64 rows 12.5 / 8.3, 512 rows 17.2 / 21.2, 16384 rows 101 / 161
//     gradients, 4096 wide: 512 rows 25.6 / 22.9, 16384 rows 258 / 179
NormPlan plan_of(int64_t rows, int64_t D, int vec, int wave, int64_t few) {
    NormPlan p{};
    p.vec = vec;
    const int64_t pieces = ceil_div(D, vec);
    if (pieces <= 32) {
        p.lanes = pieces <= 8 ? 8 : pieces <= 16 ? 16 : 32, p.loads = 1;
    } else {
        p.lanes = pieces <= 64 || (pieces <= 64 * wave && rows > few) ? 64 : 256;
        p.loads = pieces <= 2048 ? (int)ceil_div(pieces, p.lanes) : 0;
    }
    p.groups = ceil_div(rows, 256 / p.lanes);
    return p;
}

}  // namespace

fftconv_status_t fftconv_norm_fwd(const void *x, const void *residual, const void *weight, void *out, void *sum,
                                  float *scales, const int64_t *strides, int64_t M, int64_t G, int64_t D, float eps,
                                  fftconv_dtype_t dtype, hipStream_t stream) {
    const NormShape s{M, G, D, (int)dtype};
    fftconv_status_t st = check_shape(s, eps);
    if (st != FFTCONV_OK) return st;
    if (M == 0 || G == 0) return ok();
    const int64_t e = elem_bytes(s.dt);
    auto at = [&](int i) { return strides ? strides + 2 * i : nullptr; };
    const View vx = rows_view("x", x, s, e, at(0)), vr = rows_view("residual", residual, s, e, at(1)),
               vo = rows_view("out", out, s, scales ? 1 : e, at(2)), vs = rows_view("sum", sum, s, e, at(3));
    const View vw{"weight", weight, 1, {1, 1, 1}, {0, 0, 0}, D, e}, vc{"scales", scales, 1, {1, 1, 1}, {0, 0, 0}, M * G, 4};
    if ((st = check_view(vx, true, false)) != FFTCONV_OK || (st = check_view(vr, false, false)) != FFTCONV_OK ||
        (st = check_view(vw, false, false)) != FFTCONV_OK || (st = check_view(vo, true, true)) != FFTCONV_OK ||
        (st = check_view(vs, false, true)) != FFTCONV_OK || (st = check_view(vc, false, true)) != FFTCONV_OK)
        return st;
    // sum may be the residual or x itself, each row of which is read before it is written
    const View outs[] = {vo, vc, vs}, ins[] = {vx, vr, vw}, sums[] = {vs};
    if ((st = check_apart(outs, 3, ins + 2, 1)) != FFTCONV_OK || (st = check_apart(outs, 2, ins, 2)) != FFTCONV_OK) return st;
    for (int i = 0; i < 2; ++i)
        if (!same_place(vs, ins[i]) && (st = check_apart(sums, 1, ins + i, 1)) != FFTCONV_OK) return st;

    NormFwd a{};
    a.x = x, a.res = residual, a.weight = weight, a.out = out, a.sum = sum, a.scales = scales;
    for (int i = 0; i < 2; ++i)
        a.xs[i] = vx.stride[i], a.rs[i] = vr.stride[i], a.os[i] = vo.stride[i], a.ss[i] = vs.stride[i];
    a.rows = (uint32_t)(M * G), a.G = (uint32_t)G, a.D = (int)D, a.eps = eps;
    const int v = (int)(16 / e);
    bool vec = chunk_vec(vx) && (!residual || chunk_vec(vr)) && (!sum || chunk_vec(vs)) && (!weight || chunk_vec(vw));
    if (scales) {       // pieces of v bytes
        vec = vec && aligned(out, v);
        for (int i = 0; i < 2; ++i) vec = vec && vo.stride[i] % v == 0;
    } else {
        vec = vec && chunk_vec(vo);
    }
    NormPlan p = plan_of(M * G, D, vec ? v : 1, kFwdWave, 2048);
    p.groups = std::min(p.groups, kMostGroups);
    return hip_status("norm", launch_norm_fwd(s.dt, a, p, stream));
}

size_t fftconv_norm_bwd_workspace_bytes(int64_t rows, int64_t D) {
    if (rows < 1 || rows >= (int64_t(1) << 31) || D < 1 || D > kMaxWidth) return 0;
    return align_up((size_t)slabs_of(rows, D) * D * 4, 256) + (size_t)rows * 8;
}

fftconv_status_t fftconv_norm_bwd(const void *dout, const void *x, const void *weight, const void *dsum, void *dx,
                                  void *dweight, const int64_t *strides, int64_t M, int64_t G, int64_t D, float eps,
                                  fftconv_dtype_t dtype, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const NormShape s{M, G, D, (int)dtype};
    fftconv_status_t st = check_shape(s, eps);
    if (st != FFTCONV_OK) return st;
    const int64_t e = elem_bytes(s.dt), rows = M * G;
    auto at = [&](int i) { return strides ? strides + 2 * i : nullptr; };
    const View vg = rows_view("dout", dout, s, e, at(0)), vx = rows_view("x", x, s, e, at(1)),
               vu = rows_view("dsum", dsum, s, e, at(2)), vd = rows_view("dx", dx, s, e, at(3));
    const View vw{"weight", weight, 1, {1, 1, 1}, {0, 0, 0}, D, e}, vdw{"dweight", dweight, 1, {1, 1, 1}, {0, 0, 0}, D, e};
    if ((st = check_view(vg, true, false)) != FFTCONV_OK || (st = check_view(vx, true, false)) != FFTCONV_OK ||
        (st = check_view(vw, false, false)) != FFTCONV_OK || (st = check_view(vu, false, false)) != FFTCONV_OK ||
        (st = check_view(vd, false, true)) != FFTCONV_OK || (st = check_view(vdw, false, true)) != FFTCONV_OK)
        return st;
    const size_t need = fftconv_norm_bwd_workspace_bytes(rows, D);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != FFTCONV_OK) return st;
    const View ws = raw_view("workspace", need ? workspace : nullptr, (int64_t)need);
    // dx may be dsum itself
    const View outs[] = {vd, vdw, ws}, ins[] = {vg, vx, vw}, rest[] = {vdw, ws};
    if ((st = check_apart(outs, 3, ins, 3)) != FFTCONV_OK || (st = check_apart(rest, 2, &vu, 1)) != FFTCONV_OK) return st;
    if (!same_place(vd, vu) && (st = check_apart(outs, 1, &vu, 1)) != FFTCONV_OK) return st;

    NormBwd a{};
    a.dout = dout, a.x = x, a.weight = weight, a.dsum = dsum, a.dx = dx;
    for (int i = 0; i < 2; ++i)
        a.gs[i] = vg.stride[i], a.xs[i] = vx.stride[i], a.us[i] = vu.stride[i], a.ds[i] = vd.stride[i];
    a.rows = (uint32_t)rows, a.G = (uint32_t)G, a.D = (int)D, a.eps = eps;
    const bool vec = chunk_vec(vg) && chunk_vec(vx) && (!weight || chunk_vec(vw)) && (!dsum || chunk_vec(vu)) && (!dx || chunk_vec(vd));
    NormPlan p = plan_of(rows, D, vec ? (int)(16 / e) : 1, kBwdWave, 256);
    p.slabs = p.loads ? std::min(p.groups, slabs_of(rows, D)) : slabs_of(rows, D);
    p.groups = p.loads ? p.slabs : std::min(rows, kMostGroups);
    a.part = dweight ? static_cast<float *>(workspace) : nullptr;
    a.stats = need ? reinterpret_cast<float *>(static_cast<char *>(workspace) + align_up((size_t)slabs_of(rows, D) * D * 4, 256)) : nullptr;
    return hip_status("norm backward", launch_norm_bwd(s.dt, a, p, dweight, stream));
}
