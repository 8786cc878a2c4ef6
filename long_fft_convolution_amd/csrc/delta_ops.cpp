// delta_ops.cpp -- host side of the gated delta rule's entry points of
// include/fftconv.h: argument checks, how sequences are cut, workspace
// layout, launches.
#include <cmath>
#include <initializer_list>

#include "arguments.hpp"
#include "delta_ops.hpp"

using namespace fftconv;

namespace {

struct DeltaShape {
    int64_t B, N, H, Hk, Dk, Dv;
    int dt;
    bool packed;
    int64_t T() const { return packed ? N : B * N; }
    // places of units of `length` tokens (see first_place of the kernels)
    int64_t places(int64_t length) const { return packed ? N / length + B : B * std::max<int64_t>(1, ceil_div(N, length)); }
};

size_t record_bytes(const DeltaShape &s) { return (size_t)delta_pieces(delta_terms((int)elem_bytes(s.dt))) * 1024; }

// How sequences are cut.  A walk is serial: 64 tokens take microseconds, whatever else the chip does.  With segments the
// walks' work is three times that of the walk alone (sums and maps, outputs) and the chain adds to it, so sequences are cut
// where at least four segments of each walk at once, and more than four where the walks of 128 columns fill the chip.
// bf16, us a call uncut / cut:
//     4096 tokens, heads of 128: 16 heads 241 / 133, 32 heads 249 / 187, 50 heads 272 / 274, 64 heads (four) 283 / 324
//     heads of 128, 2048 tokens: 8 heads 126 / 108, 20 heads 128 / 111; 1024 tokens, 20 heads (two) 76 / 103
//     4096 tokens, 64 heads of 64 (four): 206 / 156; 16384 tokens, 16 heads of 256: 1738 / 1085
// Packed sequences' lengths live on the device, so their mean stands for them: one of 100000 tokens beside 60 of 64 walks
// uncut (20 heads of 128: 7.4 ms, by itself 2.2).
// Walks of 128 columns read k, q and the records half as often as those of 64 and take longer a chunk, so an uncut call has
// them where those of 64 columns would be more than one a CU (1024 tokens, 128 columns, us by 64 / by 128: 120 heads 90 /
// 110, 129 heads 156 / 123, 400 heads 352 / 312), and a cut one always (16384 tokens, 20 heads: 479 / 442).
struct DeltaCut {
    int64_t seg_chunks, segs;
    bool cut, wide;
};
DeltaCut fwd_cut(const DeltaShape &s) {
    DeltaCut c{};
    const int64_t chunks = std::max<int64_t>(1, ceil_div(s.packed ? ceil_div(s.N, s.B) : s.N, kDeltaChunk));
    const int64_t wide = s.B * s.H * ceil_div(s.Dv, 128), narrow = s.B * s.H * ceil_div(s.Dv, 64);
    c.wide = s.Dk <= 128 && s.Dv > 64 && narrow > kCus;
    const int64_t most = kCus / std::max<int64_t>(1, s.Dv > 64 && s.Dk <= 128 ? wide : narrow);
    const int64_t segments = std::min<int64_t>(most, chunks / 8);
    if (segments >= 4 && (most > 4 || s.Dv <= 64 || s.Dk > 128)) {
        c.seg_chunks = ceil_div(chunks, segments);
        c.cut = true;
        c.wide = s.Dk <= 128 && s.Dv > 64;
    } else {
        c.seg_chunks = (int64_t(1) << 31) / kDeltaChunk;      // one segment, whatever the length
    }
    c.segs = s.places(c.seg_chunks * kDeltaChunk);
    return c;
}

struct DeltaFwdLayout {
    int64_t sum_ld, map_ld;
    size_t sums, maps, states, total;
};
int64_t padded_width(int64_t Dk) { return Dk <= 64 ? 64 : Dk <= 128 ? 128 : 256; }
DeltaFwdLayout fwd_layout(const DeltaShape &s, const DeltaCut &c) {
    DeltaFwdLayout l{};
    const int64_t tile = c.wide ? 128 : 64, rows = padded_width(s.Dk);
    l.sum_ld = round_up(s.Dv, tile), l.map_ld = std::max(rows, round_up(s.Dk, tile));
    const size_t matrices = c.cut ? (size_t)c.segs * s.H * rows * 4 : 0;
    l.sums = align_up((size_t)s.places(kDeltaChunk) * s.H * record_bytes(s), 256);
    l.maps = l.sums + matrices * l.sum_ld;
    l.states = l.maps + matrices * l.map_ld;
    l.total = l.states + matrices * l.sum_ld;
    return l;
}

fftconv_status_t check_shape(const DeltaShape &s, float scale) {
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
    // a launch has a workgroup for four (chunk, head) pairs and one for each walk and 64 of at most 512 columns
    if (s.B >= (int64_t(1) << 31) || s.N >= (int64_t(1) << 31) || (s.B > 0 && s.N > (int64_t(1) << 40) / s.B) ||
        (s.H > 0 && (s.B > kMaxGroups / 16 / s.H || s.places(kDeltaChunk) > kMaxGroups / s.H)))
        return fail(FFTCONV_ERR_UNSUPPORTED, "B=%lld, N=%lld, H=%lld: too many sequences or tokens", (long long)s.B,
                    (long long)s.N, (long long)s.H);
    if (!std::isfinite(scale)) return fail(FFTCONV_ERR_INVALID_ARGUMENT, "scale must be finite");
    return FFTCONV_OK;
}

// heads: H or Hk; strides (batch, token, head) at st
View heads_view(const char *name, const void *p, const DeltaShape &s, int64_t heads, int64_t row, const int64_t *st) {
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
View gate_view(const char *name, const void *p, const DeltaShape &s) {
    return View{name, p, 1, {s.T(), 1, 1}, {s.H, 0, 0}, s.H, 4}.settle();
}
View state_view(const char *name, const void *p, int64_t count, const DeltaShape &s) {
    return View{name, p, 1, {count, 1, 1}, {s.H * s.Dk * s.Dv, 0, 0}, s.H * s.Dk * s.Dv, 4}.settle();
}
// The walks reach a chunk's rows by 31-bit offsets.
fftconv_status_t check_reach(const View &v) {
    if (v.size[1] > 1 && v.stride[1] * v.bytes_per >= (int64_t(1) << 24))
        return fail(FFTCONV_ERR_UNSUPPORTED, "%s has a token stride of %lld elements, 16 MiB or more", v.name, (long long)v.stride[1]);
    return FFTCONV_OK;
}
fftconv_status_t check_ints(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (!aligned(p, 4)) return fail(FFTCONV_ERR_INVALID_ARGUMENT, "state_slots and cu_seqlens must be 4-byte aligned");
    return FFTCONV_OK;
}

hipError_t launch_prepare(int dt, const DeltaArgs &a, hipStream_t s) {
    return dt == FFTCONV_F32   ? launch_delta_prepare_f32(a, s)
           : dt == FFTCONV_F16 ? launch_delta_prepare_f16(a, s)
                               : launch_delta_prepare_bf16(a, s);
}
hipError_t launch_fwd(int dt, const DeltaArgs &a, hipStream_t s) {
    return dt == FFTCONV_F32   ? launch_delta_fwd_f32(a, s)
           : dt == FFTCONV_F16 ? launch_delta_fwd_f16(a, s)
                               : launch_delta_fwd_bf16(a, s);
}

// what every call over whole sequences hands to the kernels
DeltaArgs common_args(const DeltaShape &s, const View &q, const View &k, const View &v, const float *log_decay, const float *beta,
                      float scale, const int32_t *cu) {
    DeltaArgs a{};
    a.q = q.p, a.qb = q.stride[0], a.qt = q.stride[1], a.qh = q.stride[2];
    a.k = k.p, a.kb = k.stride[0], a.kt = k.stride[1], a.kh = k.stride[2];
    a.v = v.p, a.vb = v.stride[0], a.vt = v.stride[1], a.vh = v.stride[2];
    a.log_decay = log_decay, a.beta = beta, a.scale = scale, a.cu = cu;
    a.B = s.B, a.N = s.N, a.H = (int)s.H, a.group = (int)(s.H / s.Hk), a.Dk = (int)s.Dk, a.Dv = (int)s.Dv;
    a.chunks = s.places(kDeltaChunk);
    if (s.T() == 0) a.chunks = 0;
    return a;
}

}  // namespace

size_t fftconv_delta_fwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t Dk, int64_t Dv,
                                         fftconv_dtype_t dtype) {
    if (!dtype_ok(dtype) || B < 1 || T < 1 || H < 1 || Hk < 1 || Dk < 1 || Dv < 1 || Dk > kMaxHeadDim || Dv > kMaxHeadDim) return 0;
    // by the number of tokens: the most of B equal sequences and of a packed call
    const DeltaShape equal{B, ceil_div(T, B), H, Hk, Dk, Dv, dtype, false}, packed{B, T, H, Hk, Dk, Dv, dtype, true};
    return std::max(fwd_layout(equal, fwd_cut(equal)).total, fwd_layout(packed, fwd_cut(packed)).total);
}

fftconv_status_t fftconv_delta_fwd(const void *q, const void *k, const void *v, const float *log_decay, const float *beta,
                                   void *out, const int64_t *strides, const float *state_in, float *state_out,
                                   const int32_t *state_slots, int64_t n_slots, const int32_t *cu_seqlens, int64_t B,
                                   int64_t N, int64_t H, int64_t Hk, int64_t Dk, int64_t Dv, float scale,
                                   fftconv_dtype_t dtype, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const DeltaShape s{B, N, H, Hk, Dk, Dv, (int)dtype, cu_seqlens != nullptr};
    fftconv_status_t st = check_shape(s, scale);
    if (st != FFTCONV_OK) return st;
    if (n_slots < 0) return fail(FFTCONV_ERR_INVALID_ARGUMENT, "n_slots=%lld must be >= 0", (long long)n_slots);
    if (B == 0 || H == 0) return ok();
    auto at = [&](int i) { return strides ? strides + 3 * i : nullptr; };
    const View vq = heads_view("q", q, s, Hk, Dk, at(0)), vk = heads_view("k", k, s, Hk, Dk, at(1)),
               vv = heads_view("v", v, s, H, Dv, at(2)), vo = heads_view("out", out, s, H, Dv, at(3));
    const View vg = gate_view("log_decay", log_decay, s), vb = gate_view("beta", beta, s);
    for (const View *x : {&vq, &vk, &vv, &vg, &vb})
        if ((st = check_view(*x, true, false)) != FFTCONV_OK) return st;
    if ((st = check_view(vo, true, true)) != FFTCONV_OK) return st;
    for (const View *x : {&vq, &vk, &vv, &vo})
        if ((st = check_reach(*x)) != FFTCONV_OK) return st;
    const int64_t states = state_slots ? n_slots : B;
    const View si = state_view("state_in", state_in, states, s), so = state_view("state_out", state_out, states, s);
    for (const View *x : {&si, &so})
        if ((st = check_view(*x, false, false)) != FFTCONV_OK) return st;
    if ((st = check_ints({state_slots, cu_seqlens})) != FFTCONV_OK) return st;
    const size_t need = fftconv_delta_fwd_workspace_bytes(B, s.T(), H, Hk, Dk, Dv, dtype);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != FFTCONV_OK) return st;
    const View ws = raw_view("workspace", need ? workspace : nullptr, (int64_t)need);
    const View sl = raw_view("state_slots", state_slots, B * 4), cu = raw_view("cu_seqlens", cu_seqlens, (B + 1) * 4);
    // state_out may be state_in itself (the pool updated in place), nothing else
    if (state_out && state_in && state_out != state_in && si.overlaps(so))
        return fail(FFTCONV_ERR_INVALID_ARGUMENT, "state_out overlaps state_in without being it");
    const View outs[] = {vo, so, ws}, ins[] = {vq, vk, vv, vg, vb, sl, cu};
    if ((st = check_apart(outs, 3, ins, 7)) != FFTCONV_OK) return st;
    const View apart[] = {vo, ws};
    if ((st = check_apart(apart, 2, &si, 1)) != FFTCONV_OK) return st;
    if (s.T() == 0 && !state_out) return ok();

    DeltaArgs a = common_args(s, vq, vk, vv, log_decay, beta, scale, cu_seqlens);
    a.out = out, a.ob = vo.stride[0], a.ot = vo.stride[1], a.oh = vo.stride[2];
    a.state0 = state_in, a.state1 = state_out, a.slots = state_slots, a.n_slots = n_slots;
    a.vec = chunk_vec(vq) && chunk_vec(vk) && chunk_vec(vv) && chunk_vec(vo);
    const DeltaCut c = fwd_cut(s);
    const DeltaFwdLayout l = fwd_layout(s, c);
    a.seg_chunks = c.seg_chunks, a.segs = c.segs, a.wide = c.wide;
    a.rec = static_cast<char *>(workspace);
    a.rec_bytes = (int64_t)record_bytes(s);
    if (c.cut) {
        a.seg_sum = reinterpret_cast<float *>(a.rec + l.sums);
        a.seg_map = reinterpret_cast<float *>(a.rec + l.maps);
        a.seg_state = reinterpret_cast<float *>(a.rec + l.states);
        a.sum_ld = (int)l.sum_ld, a.map_ld = (int)l.map_ld;
    }
    hipError_t e = launch_prepare(dtype, a, stream);
    if (e == hipSuccess) e = launch_fwd(dtype, a, stream);
    return hip_status("delta rule", e);
}

fftconv_status_t fftconv_delta_step(const void *q, const void *k, const void *v, const float *log_decay,
                                    const float *beta, float *state, void *out, const int64_t *strides,
                                    const int32_t *state_slots, int64_t n_slots, int64_t B, int64_t H, int64_t Hk,
                                    int64_t Dk, int64_t Dv, float scale, fftconv_dtype_t dtype, hipStream_t stream) {
    const DeltaShape s{B, 1, H, Hk, Dk, Dv, (int)dtype, false};
    fftconv_status_t st = check_shape(s, scale);
    if (st != FFTCONV_OK) return st;
    if (n_slots < 0) return fail(FFTCONV_ERR_INVALID_ARGUMENT, "n_slots=%lld must be >= 0", (long long)n_slots);
    if (B == 0 || H == 0) return ok();
    int64_t full[12];
    if (strides)
        for (int i = 0; i < 4; ++i) full[3 * i] = strides[2 * i], full[3 * i + 1] = 0, full[3 * i + 2] = strides[2 * i + 1];
    auto at = [&](int i) { return strides ? full + 3 * i : nullptr; };
    const View vq = heads_view("q", q, s, Hk, Dk, at(0)), vk = heads_view("k", k, s, Hk, Dk, at(1)),
               vv = heads_view("v", v, s, H, Dv, at(2)), vo = heads_view("out", out, s, H, Dv, at(3));
    const View vg = gate_view("log_decay", log_decay, s), vb = gate_view("beta", beta, s);
    for (const View *x : {&vq, &vk, &vv, &vg, &vb})
        if ((st = check_view(*x, true, false)) != FFTCONV_OK) return st;
    if ((st = check_view(vo, true, true)) != FFTCONV_OK) return st;
    if (!state && !(state_slots && n_slots == 0)) return fail(FFTCONV_ERR_INVALID_ARGUMENT, "state must be non-null");
    const View vs = state_view("state", state, state_slots ? n_slots : B, s);
    if ((st = check_view(vs, false, false)) != FFTCONV_OK) return st;
    if ((st = check_ints({state_slots})) != FFTCONV_OK) return st;
    const View outs[] = {vo, vs}, ins[] = {vq, vk, vv, vg, vb, raw_view("state_slots", state_slots, B * 4)};
    if ((st = check_apart(outs, 2, ins, 6)) != FFTCONV_OK) return st;

    DeltaStep a{};
    a.q = q, a.k = k, a.v = v, a.out = out;
    a.qb = vq.stride[0], a.qh = vq.stride[2], a.kb = vk.stride[0], a.kh = vk.stride[2];
    a.vb = vv.stride[0], a.vh = vv.stride[2], a.ob = vo.stride[0], a.oh = vo.stride[2];
    a.log_decay = log_decay, a.beta = beta, a.state = state, a.slots = state_slots, a.n_slots = n_slots;
    a.B = B, a.H = (int)H, a.group = (int)(H / Hk), a.Dk = (int)Dk, a.Dv = (int)Dv, a.scale = scale;
    const bool vec = Dv % 4 == 0 && aligned(state, 16);
    const hipError_t e = dtype == FFTCONV_F32   ? launch_delta_step_f32(a, vec, stream)
                         : dtype == FFTCONV_F16 ? launch_delta_step_f16(a, vec, stream)
                                                : launch_delta_step_bf16(a, vec, stream);
    return hip_status("delta step", e);
}

// ---- gradients ----------------------------------------------------------------
namespace {
// Workspace of the backward call: the chunks' records, states, their gradients, w and y, and fp32 gradients of the heads
// that share a query/key head.
struct DeltaBwdLayout {
    bool wide;
    int64_t dkp, dvp;
    size_t states, grads, wrong, dright, dq, dk, total;
};
DeltaBwdLayout bwd_layout(const DeltaShape &s) {
    DeltaBwdLayout l{};
    // as for an uncut forward call, with two walks (1024 tokens, 128 columns, us by 64 / by 128: 60 heads 217 / 237, 65
    // heads 333 / 280, 80 heads 349 / 311)
    l.wide = s.Dk <= 128 && s.Dv > 64 && 2 * s.B * s.H * ceil_div(s.Dv, 64) > kCus;
    l.dkp = padded_width(s.Dk);
    l.dvp = round_up(s.Dv, l.wide ? 128 : 64);
    const size_t items = (size_t)s.places(kDeltaChunk) * s.H;
    l.states = items * kDeltaBackPieces * 1024;
    l.grads = l.states + items * l.dkp * l.dvp * 4;
    l.wrong = l.grads + items * l.dkp * l.dvp * 4;
    l.dright = l.wrong + items * kDeltaChunk * l.dvp * 4;
    l.dq = l.dright + items * kDeltaChunk * l.dvp * 4;
    const size_t part = s.H == s.Hk ? 0 : align_up((size_t)s.T() * s.H * s.Dk * 4, 256);
    l.dk = l.dq + part;
    l.total = l.dk + part;
    return l;
}
}  // namespace

size_t fftconv_delta_bwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Hk, int64_t Dk, int64_t Dv,
                                         fftconv_dtype_t dtype) {
    if (!dtype_ok(dtype) || B < 1 || T < 1 || H < 1 || Hk < 1 || Dk < 1 || Dv < 1 || Dk > kMaxHeadDim || Dv > kMaxHeadDim) return 0;
    const DeltaShape equal{B, ceil_div(T, B), H, Hk, Dk, Dv, dtype, false}, packed{B, T, H, Hk, Dk, Dv, dtype, true};
    return std::max(bwd_layout(equal).total, bwd_layout(packed).total);
}

fftconv_status_t fftconv_delta_bwd(const void *dout, const void *q, const void *k, const void *v, const float *log_decay,
                                   const float *beta, void *dq, void *dk, void *dv, float *dlog_decay, float *dbeta,
                                   const int64_t *strides, const float *state_in, const float *dstate_out,
                                   float *dstate_in, const int32_t *cu_seqlens, int64_t B, int64_t N, int64_t H,
                                   int64_t Hk, int64_t Dk, int64_t Dv, float scale, fftconv_dtype_t dtype,
                                   void *workspace, size_t workspace_bytes, hipStream_t stream) {
    const DeltaShape s{B, N, H, Hk, Dk, Dv, (int)dtype, cu_seqlens != nullptr};
    fftconv_status_t st = check_shape(s, scale);
    if (st != FFTCONV_OK) return st;
    if (B == 0 || H == 0) return ok();
    auto at = [&](int i) { return strides ? strides + 3 * i : nullptr; };
    const View vd = heads_view("dout", dout, s, H, Dv, at(0)), vq = heads_view("q", q, s, Hk, Dk, at(1)),
               vk = heads_view("k", k, s, Hk, Dk, at(2)), vv = heads_view("v", v, s, H, Dv, at(3)),
               gq = heads_view("dq", dq, s, Hk, Dk, at(4)), gk = heads_view("dk", dk, s, Hk, Dk, at(5)),
               gv = heads_view("dv", dv, s, H, Dv, at(6));
    const View vg = gate_view("log_decay", log_decay, s), vb = gate_view("beta", beta, s),
               gg = gate_view("dlog_decay", dlog_decay, s), gb = gate_view("dbeta", dbeta, s);
    for (const View *x : {&vd, &vq, &vk, &vv, &vg, &vb})
        if ((st = check_view(*x, true, false)) != FFTCONV_OK) return st;
    for (const View *x : {&gq, &gk, &gv, &gg, &gb})
        if ((st = check_view(*x, false, true)) != FFTCONV_OK) return st;
    for (const View *x : {&vd, &vq, &vk, &vv, &gq, &gk, &gv})
        if (x->p && (st = check_reach(*x)) != FFTCONV_OK) return st;
    const View si = state_view("state_in", state_in, B, s), dso = state_view("dstate_out", dstate_out, B, s),
               dsi = state_view("dstate_in", dstate_in, B, s);
    for (const View *x : {&si, &dso, &dsi})
        if ((st = check_view(*x, false, false)) != FFTCONV_OK) return st;
    if ((st = check_ints({cu_seqlens})) != FFTCONV_OK) return st;
    const size_t need = fftconv_delta_bwd_workspace_bytes(B, s.T(), H, Hk, Dk, Dv, dtype);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != FFTCONV_OK) return st;
    const View ws = raw_view("workspace", need ? workspace : nullptr, (int64_t)need);
    const View outs[] = {gq, gk, gv, gg, gb, dsi, ws},
               ins[] = {vd, vq, vk, vv, vg, vb, si, dso, raw_view("cu_seqlens", cu_seqlens, (B + 1) * 4)};
    if ((st = check_apart(outs, 7, ins, 9)) != FFTCONV_OK) return st;
    if (s.T() == 0 && !dstate_in) return ok();

    DeltaArgs a = common_args(s, vq, vk, vv, log_decay, beta, scale, cu_seqlens);
    const DeltaBwdLayout l = bwd_layout(s);
    char *base = static_cast<char *>(workspace);
    const bool shared = H != Hk;
    a.state0 = state_in, a.dstate1 = dstate_out, a.dstate0 = dstate_in;
    a.seg_chunks = (int64_t(1) << 31) / kDeltaChunk, a.segs = s.places(a.seg_chunks * kDeltaChunk);
    a.wide = l.wide, a.dkp = (int)l.dkp, a.dvp = (int)l.dvp;
    a.rec = base, a.rec_bytes = kDeltaBackPieces * 1024;
    a.states = reinterpret_cast<float *>(base + l.states), a.grads = reinterpret_cast<float *>(base + l.grads);
    a.wrong = reinterpret_cast<float *>(base + l.wrong), a.dright = reinterpret_cast<float *>(base + l.dright);
    a.dout = dout, a.gb = vd.stride[0], a.gt = vd.stride[1], a.gh = vd.stride[2];
    a.parts = shared;
    a.dq = shared && dq ? base + l.dq : dq, a.dk = shared && dk ? base + l.dk : dk, a.dv = dv;
    a.dqb = gq.stride[0], a.dqt = gq.stride[1], a.dqh = gq.stride[2];
    a.dkb = gk.stride[0], a.dkt = gk.stride[1], a.dkh = gk.stride[2];
    a.dvb = gv.stride[0], a.dvt = gv.stride[1], a.dvh = gv.stride[2];
    a.dlog_decay = dlog_decay, a.dbeta = dbeta;
    a.vec = chunk_vec(vq) && chunk_vec(vk) && chunk_vec(vv) && chunk_vec(vd);
    for (const View *x : {&gq, &gk, &gv}) a.vec = a.vec && (!x->p || chunk_vec(*x));
    hipError_t e = launch_prepare(dtype, a, stream);
    if (e == hipSuccess)
        e = dtype == FFTCONV_F32   ? launch_delta_bwd_f32(a, stream)
            : dtype == FFTCONV_F16 ? launch_delta_bwd_f16(a, stream)
                                   : launch_delta_bwd_bf16(a, stream);
    if (e == hipSuccess && shared && (dq || dk) && s.T() > 0) {
        DecayGroupSum g{};
        const View *grads[] = {&gq, &gk};
        const size_t parts[] = {l.dq, l.dk};
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
    return hip_status("delta rule gradients", e);
}
