// libselscan C ABI: the gated linear recurrence, the norms around a block and
// rotary positions. Every check runs before the first HIP call.
#include <stdint.h>

#include <initializer_list>

#include "../../include/selscan.h"
#include "api_util.hpp"
#include "launch.hpp"

using namespace selscan;

namespace {

bool known_dtype(int32_t d) { return d == SELSCAN_F32 || d == SELSCAN_BF16; }
DType dtype_of(int32_t d) { return d == SELSCAN_BF16 ? DType::BF16 : DType::F32; }
int64_t size_of(DType d) { return d == DType::BF16 ? 2 : 4; }

bool all_aligned(std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (!aligned16(p)) return false;
    return true;
}
bool bad_workspace(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) != 0; }

// a may be b itself, but must not overlap it otherwise
bool half_over(const Span& a, const Span& b) { return overlaps(a, b) && a.lo != b.lo; }

int done(hipError_t e) { return e == hipSuccess ? SELSCAN_OK : SELSCAN_ERR_LAUNCH; }

int check_gated(const selscan_gated_dims_t* d, bool step, GatedShape* s) {
    if (!d) return SELSCAN_ERR_NULL;
    const int64_t L = step ? 1 : d->seqlen;
    if (d->batch < 0 || d->dim < 0 || L < 0 || L >= (int64_t(1) << 27) || d->dim > (int64_t(1) << 20))
        return SELSCAN_ERR_DIMS;
    if (!known_dtype(d->dtype)) return SELSCAN_ERR_DTYPE;
    if (d->kind != SELSCAN_GATED_MIX && d->kind != SELSCAN_GATED_DECAY) return SELSCAN_ERR_CONFIG;
    int64_t t;
    // one workgroup or more for every 8 channels of an entry
    if (!mul_ok(d->batch, d->dim > 8 ? (d->dim + 7) / 8 : 1, &t) || t > (int64_t(1) << 22)) return SELSCAN_ERR_DIMS;
    if (!mul_ok(d->batch * d->dim, L, &t) || !mul_ok(t, 4, &t)) return SELSCAN_ERR_DIMS;
    *s = GatedShape{d->batch, L, d->dim, dtype_of(d->dtype), d->kind};
    return SELSCAN_OK;
}

// The arguments that belong to SELSCAN_GATED_DECAY alone: r, A and (backward) dr.
int check_kind(const GatedShape& s, bool values, const void* r, const void* A) {
    const bool decay = s.kind == SELSCAN_GATED_DECAY;
    if (!decay && (r || A)) return SELSCAN_ERR_CONFIG;
    if (decay && ((values && !r) || (s.dim > 0 && !A))) return SELSCAN_ERR_NULL;
    return SELSCAN_OK;
}

int gated_make_plan(const GatedShape& s, int32_t segments, bool backward, GatedPlan* p) {
    if (segments < 0 || segments > 65536) return SELSCAN_ERR_CONFIG;
    return gated_plan(s, segments, backward, p) ? SELSCAN_OK : SELSCAN_ERR_DIMS;
}

int check_addnorm(const selscan_addnorm_dims_t* d, const float* gate, bool forward, AddnormShape* s) {
    if (!d) return SELSCAN_ERR_NULL;
    if (d->rows < 0 || d->channels < 0 || d->rows >= (int64_t(1) << 31) || d->channels > 16384)
        return SELSCAN_ERR_DIMS;
    if (gate && (d->gate_rows < 1 || d->gate_rows >= (int64_t(1) << 31) || d->rows % d->gate_rows))
        return SELSCAN_ERR_DIMS;
    if (!known_dtype(d->dtype) || (d->res_dtype != SELSCAN_F32 && d->res_dtype != d->dtype)) return SELSCAN_ERR_DTYPE;
    for (const int32_t n : {d->post, d->pre})
        if (n < SELSCAN_NORM_NONE || n > SELSCAN_NORM_LAYER) return SELSCAN_ERR_CONFIG;
    if (!finite_f32(d->scale) || !finite_f32(d->res_scale)) return SELSCAN_ERR_CONFIG;
    if (forward && (!(d->eps >= 0.0f) || !finite_f32(d->eps))) return SELSCAN_ERR_CONFIG;
    *s = AddnormShape{d->rows, d->channels, gate ? d->gate_rows : 0, dtype_of(d->dtype), dtype_of(d->res_dtype),
                      d->post, d->pre, d->eps, d->scale, d->res_scale};
    return SELSCAN_OK;
}

// Parameters, and gradients of parameters, of a norm that is not there.
bool unused_params(const AddnormShape& s, const void* post_w, const void* post_b, const void* pre_w,
                   const void* pre_b) {
    return (s.post == SELSCAN_NORM_NONE && (post_w || post_b)) || (s.pre == SELSCAN_NORM_NONE && (pre_w || pre_b));
}

AddnormTensors addnorm_wanted(const selscan_addnorm_grads_t& g) {
    AddnormTensors t{};
    t.dpost_w = g.dpost_weight; t.dpost_b = g.dpost_bias;
    t.dpre_w = g.dpre_weight; t.dpre_b = g.dpre_bias; t.dgate = g.dgate;
    return t;
}

}  // namespace

extern "C" {

int selscan_gated_fwd_workspace_size(const selscan_gated_dims_t* dims, const selscan_gated_opts_t* opts,
                                     uint64_t* bytes) {
    if (!bytes) return SELSCAN_ERR_NULL;
    GatedShape s;
    int rc = check_gated(dims, false, &s);
    if (rc != SELSCAN_OK) return rc;
    GatedPlan p;
    rc = gated_make_plan(s, opts ? opts->segments : 0, false, &p);
    if (rc != SELSCAN_OK) return rc;
    *bytes = s.batch * s.dim * s.L > 0 ? gated_fwd_workspace_bytes(s, p) : 0;
    return SELSCAN_OK;
}

int selscan_gated_fwd(const void* x, const void* g, const void* r, const float* A, const void* z,
                      void* y, float* last_state, const selscan_gated_dims_t* dims,
                      const selscan_gated_opts_t* opts, void* stream) {
    GatedShape s;
    int rc = check_gated(dims, false, &s);
    if (rc != SELSCAN_OK) return rc;
    const selscan_gated_opts_t o = opts ? *opts : selscan_gated_opts_t{};
    GatedPlan plan;
    rc = gated_make_plan(s, o.segments, false, &plan);
    if (rc != SELSCAN_OK) return rc;
    const int64_t bd = s.batch * s.dim, n = bd * s.L, es = size_of(s.dtype);
    // A tensor with no elements may come with a null pointer (torch gives one).
    if (n > 0 && (!x || !g || !y)) return SELSCAN_ERR_NULL;
    rc = check_kind(s, n > 0, r, A);
    if (rc != SELSCAN_OK) return rc;
    if (!all_aligned({x, g, r, A, z, y, last_state, o.h0, o.lengths, o.ckpt})) return SELSCAN_ERR_ALIGN;
    const size_t ws_bytes = n > 0 ? gated_fwd_workspace_bytes(s, plan) : 0;
    if (bad_workspace(o.workspace) || (o.workspace && o.workspace_bytes < ws_bytes)) return SELSCAN_ERR_CONFIG;
    const int64_t kept = (s.L + SELSCAN_GATED_CKPT - 1) / SELSCAN_GATED_CKPT * bd * 4;
    const Span ins[] = {span(x, n * es), span(g, n * es), span(r, n * es), span(z, n * es), span(A, s.dim * 4),
                        span(o.lengths, s.batch * 4)};
    const Span oy = span(y, n * es), os = span(last_state, bd * 4), oc = span(o.ckpt, kept),
               w = span(o.workspace, int64_t(ws_bytes)), ih = span(o.h0, bd * 4);
    const Span outs[] = {oy, os, oc, w};
    // h0 may be last_state itself (read before it is written)
    if (any_alias(ins, outs) || overlaps(ih, oy) || overlaps(ih, oc) || overlaps(ih, w) || half_over(ih, os))
        return SELSCAN_ERR_ALIAS;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (bd == 0) return SELSCAN_OK;
    if (s.L == 0) return done(pass_state(last_state, o.h0, bd, st));
    GatedTensors t{};
    t.x = x; t.g = g; t.r = r; t.A = A; t.z = z;
    t.lengths = o.lengths; t.h0 = o.h0;
    t.y = y; t.last_state = last_state; t.ckpt = o.ckpt;
    Workspace ws;
    rc = ws.take(o.workspace, ws_bytes, st);
    if (rc != SELSCAN_OK) return rc;
    const hipError_t e = launch_gated_fwd(t, s, plan, ws.p, st);
    ws.give_back(st);
    return done(e);
}

int selscan_gated_step(float* state, const void* x, const void* g, const void* r, const float* A,
                       const void* z, void* y, const selscan_gated_dims_t* dims, void* stream) {
    GatedShape s;
    int rc = check_gated(dims, true, &s);
    if (rc != SELSCAN_OK) return rc;
    const int64_t n = s.batch * s.dim, es = size_of(s.dtype);
    if (n > 0 && (!state || !x || !g || !y)) return SELSCAN_ERR_NULL;
    rc = check_kind(s, n > 0, r, A);
    if (rc != SELSCAN_OK) return rc;
    if (!all_aligned({state, x, g, r, A, z, y})) return SELSCAN_ERR_ALIGN;
    const Span ins[] = {span(x, n * es), span(g, n * es), span(r, n * es), span(z, n * es), span(A, s.dim * 4)};
    const Span outs[] = {span(state, n * 4), span(y, n * es)};
    if (any_alias(ins, outs)) return SELSCAN_ERR_ALIAS;
    if (n == 0) return SELSCAN_OK;
    GatedTensors t{};
    t.x = x; t.g = g; t.r = r; t.A = A; t.z = z; t.y = y;
    return done(launch_gated_step(state, t, s, static_cast<hipStream_t>(stream)));
}

int selscan_gated_bwd_workspace_size(const selscan_gated_dims_t* dims, const selscan_gated_bwd_opts_t* opts,
                                     uint64_t* bytes) {
    if (!bytes) return SELSCAN_ERR_NULL;
    GatedShape s;
    int rc = check_gated(dims, false, &s);
    if (rc != SELSCAN_OK) return rc;
    GatedPlan p;
    rc = gated_make_plan(s, opts ? opts->segments : 0, true, &p);
    if (rc != SELSCAN_OK) return rc;
    *bytes = s.batch * s.dim * s.L > 0 ? gated_bwd_workspace_bytes(s, p, opts && opts->ckpt) : 0;
    return SELSCAN_OK;
}

int selscan_gated_bwd(const void* x, const void* g, const void* r, const float* A, const void* z,
                      const void* dy, void* dx, void* dg, void* dr, float* dA, void* dz,
                      const selscan_gated_dims_t* dims, const selscan_gated_bwd_opts_t* opts,
                      void* stream) {
    GatedShape s;
    int rc = check_gated(dims, false, &s);
    if (rc != SELSCAN_OK) return rc;
    const selscan_gated_bwd_opts_t o = opts ? *opts : selscan_gated_bwd_opts_t{};
    GatedPlan plan;
    rc = gated_make_plan(s, o.segments, true, &plan);
    if (rc != SELSCAN_OK) return rc;
    const int64_t bd = s.batch * s.dim, n = bd * s.L, es = size_of(s.dtype);
    if (n > 0 && (!x || !g || !dy || !dx || !dg)) return SELSCAN_ERR_NULL;
    rc = check_kind(s, n > 0, r, A);
    if (rc != SELSCAN_OK) return rc;
    const bool decay = s.kind == SELSCAN_GATED_DECAY;
    if (!decay && (dr || dA)) return SELSCAN_ERR_CONFIG;
    if (n > 0 && ((decay && !dr) || (z != nullptr) != (dz != nullptr))) return SELSCAN_ERR_NULL;
    if (!all_aligned({x, g, r, A, z, dy, dx, dg, dr, dA, dz, o.h0, o.lengths, o.dlast_state, o.dh0, o.ckpt}))
        return SELSCAN_ERR_ALIGN;
    const size_t ws_bytes = n > 0 ? gated_bwd_workspace_bytes(s, plan, o.ckpt != nullptr) : 0;
    if (bad_workspace(o.workspace) || (o.workspace && o.workspace_bytes < ws_bytes)) return SELSCAN_ERR_CONFIG;
    const int64_t kept = (s.L + SELSCAN_GATED_CKPT - 1) / SELSCAN_GATED_CKPT * bd * 4;
    const Span ins[] = {span(x, n * es), span(g, n * es), span(r, n * es), span(z, n * es), span(dy, n * es),
                        span(A, s.dim * 4), span(o.lengths, s.batch * 4), span(o.h0, bd * 4),
                        span(o.dlast_state, bd * 4), span(o.ckpt, kept)};
    const Span outs[] = {span(dx, n * es), span(dg, n * es), span(dr, n * es), span(dz, n * es),
                         span(dA, s.dim * 4), span(o.dh0, bd * 4), span(o.workspace, int64_t(ws_bytes))};
    if (any_alias(ins, outs)) return SELSCAN_ERR_ALIAS;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (n == 0) {  // no terms; the last state is h0 itself: its gradient passes straight through
        if (dA && s.dim > 0 && launch_fill_zero(dA, s.dim, st) != hipSuccess) return SELSCAN_ERR_LAUNCH;
        return done(pass_state(o.dh0, o.dlast_state, bd, st));
    }
    GatedTensors t{};
    t.x = x; t.g = g; t.r = r; t.A = A; t.z = z;
    t.lengths = o.lengths; t.h0 = o.h0;
    t.ckpt = const_cast<float*>(o.ckpt);
    t.dy = dy; t.dlast = o.dlast_state;
    t.dx = dx; t.dg = dg; t.dr = dr; t.dA = dA; t.dz = dz; t.dh0 = o.dh0;
    Workspace ws;
    rc = ws.take(o.workspace, ws_bytes, st);
    if (rc != SELSCAN_OK) return rc;
    const hipError_t e = launch_gated_bwd(t, s, plan, ws.p, st);
    ws.give_back(st);
    return done(e);
}

int selscan_addnorm(const void* x, const void* res, void* res_out, void* y, float* stats,
                    const selscan_addnorm_dims_t* dims, const selscan_addnorm_opts_t* opts,
                    void* stream) {
    const selscan_addnorm_opts_t o = opts ? *opts : selscan_addnorm_opts_t{};
    AddnormShape s;
    const int rc = check_addnorm(dims, o.gate, true, &s);
    if (rc != SELSCAN_OK) return rc;
    if (unused_params(s, o.post_weight, o.post_bias, o.pre_weight, o.pre_bias)) return SELSCAN_ERR_CONFIG;
    const bool pre = s.pre != SELSCAN_NORM_NONE;
    if (!pre && y) return SELSCAN_ERR_CONFIG;
    const int64_t n = s.R * s.C, es = size_of(s.dtype), er = size_of(s.res_dtype);
    if (n > 0 && (!x || (pre && !y) || (!pre && !res_out))) return SELSCAN_ERR_NULL;
    if (!all_aligned({x, res, res_out, y, stats, o.post_weight, o.post_bias, o.pre_weight, o.pre_bias, o.gate}))
        return SELSCAN_ERR_ALIGN;
    const int64_t c4 = s.C * 4;
    const Span ins[] = {span(x, n * es), span(o.post_weight, c4), span(o.post_bias, c4), span(o.pre_weight, c4),
                        span(o.pre_bias, c4), span(o.gate, s.G * c4)};
    const Span ir = span(res, n * er), os = span(res_out, n * er), oy = span(y, n * es), ot = span(stats, s.R * 16);
    const Span outs[] = {os, oy, ot};
    // res_out may be res itself (a row is read before it is written)
    if (any_alias(ins, outs) || half_over(ir, os) || overlaps(ir, oy) || overlaps(ir, ot)) return SELSCAN_ERR_ALIAS;
    if (n == 0) {  // rows without channels: the mean and the variance of nothing count as 0
        if (stats && s.R > 0) {
            const AddnormTensors t{nullptr, nullptr, nullptr, nullptr, stats};
            return done(launch_addnorm(t, s, static_cast<hipStream_t>(stream)));
        }
        return SELSCAN_OK;
    }
    AddnormTensors t{};
    t.x = x; t.res = res; t.sum = res_out; t.y = y; t.stats = stats;
    t.post_w = o.post_weight; t.post_b = o.post_bias; t.pre_w = o.pre_weight; t.pre_b = o.pre_bias; t.gate = o.gate;
    return done(launch_addnorm(t, s, static_cast<hipStream_t>(stream)));
}

int selscan_addnorm_bwd_workspace_size(const selscan_addnorm_dims_t* dims, const selscan_addnorm_opts_t* opts,
                                       const selscan_addnorm_grads_t* grads, uint64_t* bytes) {
    if (!bytes) return SELSCAN_ERR_NULL;
    AddnormShape s;
    const int rc = check_addnorm(dims, opts ? opts->gate : nullptr, false, &s);
    if (rc != SELSCAN_OK) return rc;
    *bytes = s.R * s.C > 0 && grads ? addnorm_bwd_workspace_bytes(s, addnorm_wanted(*grads)) : 0;
    return SELSCAN_OK;
}

int selscan_addnorm_bwd(const void* x, const void* sum, const float* stats, const void* dy,
                        const void* dres_out, void* dx, void* dres,
                        const selscan_addnorm_grads_t* grads, const selscan_addnorm_dims_t* dims,
                        const selscan_addnorm_opts_t* opts, void* stream) {
    const selscan_addnorm_opts_t o = opts ? *opts : selscan_addnorm_opts_t{};
    const selscan_addnorm_grads_t gr = grads ? *grads : selscan_addnorm_grads_t{};
    AddnormShape s;
    int rc = check_addnorm(dims, o.gate, false, &s);
    if (rc != SELSCAN_OK) return rc;
    if (unused_params(s, o.post_weight, o.post_bias, o.pre_weight, o.pre_bias) ||
        unused_params(s, gr.dpost_weight, gr.dpost_bias, gr.dpre_weight, gr.dpre_bias) || (!o.gate && gr.dgate))
        return SELSCAN_ERR_CONFIG;
    const bool pre = s.pre != SELSCAN_NORM_NONE, post = s.post != SELSCAN_NORM_NONE;
    if (!pre && (sum || dy)) return SELSCAN_ERR_CONFIG;
    const int64_t n = s.R * s.C, es = size_of(s.dtype), er = size_of(s.res_dtype);
    if (n > 0 && ((pre && (!sum || !dy)) || ((post || gr.dgate) && !x) || ((pre || post) && !stats) ||
                  (!dx && !dres)))
        return SELSCAN_ERR_NULL;
    if (!all_aligned({x, sum, stats, dy, dres_out, dx, dres, o.post_weight, o.post_bias, o.pre_weight, o.pre_bias,
                      o.gate, gr.dpost_weight, gr.dpost_bias, gr.dpre_weight, gr.dpre_bias, gr.dgate}))
        return SELSCAN_ERR_ALIGN;
    AddnormTensors t = addnorm_wanted(gr);
    const size_t ws_bytes = n > 0 ? addnorm_bwd_workspace_bytes(s, t) : 0;
    if (bad_workspace(o.workspace) || (o.workspace && o.workspace_bytes < ws_bytes)) return SELSCAN_ERR_CONFIG;
    const int64_t c4 = s.C * 4;
    const Span ins[] = {span(x, n * es), span(sum, n * er), span(stats, s.R * 16), span(dy, n * es),
                        span(o.post_weight, c4), span(o.post_bias, c4), span(o.pre_weight, c4),
                        span(o.pre_bias, c4), span(o.gate, s.G * c4)};
    const Span id = span(dres_out, n * er), od = span(dres, n * er);
    const Span outs[] = {span(dx, n * es), span(gr.dpost_weight, c4), span(gr.dpost_bias, c4),
                         span(gr.dpre_weight, c4), span(gr.dpre_bias, c4), span(gr.dgate, s.G * c4),
                         span(o.workspace, int64_t(ws_bytes)), od};
    if (any_alias(ins, outs) || half_over(id, od)) return SELSCAN_ERR_ALIAS;
    for (const Span& out : outs)
        if (&out != &outs[7] && overlaps(id, out)) return SELSCAN_ERR_ALIAS;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (n == 0) {  // no terms
        for (float* p : {gr.dpost_weight, gr.dpost_bias, gr.dpre_weight, gr.dpre_bias})
            if (p && s.C > 0 && launch_fill_zero(p, s.C, st) != hipSuccess) return SELSCAN_ERR_LAUNCH;
        return done(pass_state(gr.dgate, nullptr, s.G * s.C, st));
    }
    t.x = x; t.sum = const_cast<void*>(sum); t.stats = const_cast<float*>(stats);
    t.dy = dy; t.dsum = dres_out; t.dx = dx; t.dres = dres;
    t.post_w = o.post_weight; t.post_b = o.post_bias; t.pre_w = o.pre_weight; t.pre_b = o.pre_bias; t.gate = o.gate;
    Workspace ws;
    rc = ws.take(o.workspace, ws_bytes, st);
    if (rc != SELSCAN_OK) return rc;
    const hipError_t e = launch_addnorm_bwd(t, s, ws.p, st);
    ws.give_back(st);
    return done(e);
}

int selscan_rotary(const void* q, const void* k, const float* inv_freq, const int32_t* positions,
                   void* q_out, void* k_out, const selscan_rotary_dims_t* d, void* stream) {
    if (!d) return SELSCAN_ERR_NULL;
    if (d->batch < 0 || d->seqlen < 0 || d->heads < 0 || d->kv_heads < 0 || d->seqlen >= (int64_t(1) << 27))
        return SELSCAN_ERR_DIMS;
    if (!known_dtype(d->dtype)) return SELSCAN_ERR_DTYPE;
    if (d->rot < 1 || d->rot % 2 || d->rot > d->width || d->width > 4096) return SELSCAN_ERR_DSTATE;
    int64_t tokens, th;
    const int64_t most = int64_t(1) << 38;  // (heads up to 2^38 by a width up to 2^12 stay in 64 bits)
    if (d->heads >= most || d->kv_heads >= most || !mul_ok(d->batch, d->seqlen, &tokens) || tokens >= most ||
        !mul_ok(tokens, d->heads + d->kv_heads, &th) || th >= most)
        return SELSCAN_ERR_DIMS;
    if ((d->heads + d->kv_heads) * d->width > (int64_t(1) << 22)) return SELSCAN_ERR_DIMS;
    if (d->offset <= -(int64_t(1) << 31) || d->offset >= (int64_t(1) << 31)) return SELSCAN_ERR_DIMS;
    if ((d->layout != SELSCAN_ROTARY_HALF && d->layout != SELSCAN_ROTARY_INTERLEAVED) || !finite_f32(d->scale))
        return SELSCAN_ERR_CONFIG;
    const RotaryShape s{d->batch, d->seqlen, d->heads, d->kv_heads, d->width, d->rot, d->offset, dtype_of(d->dtype),
                        d->layout, d->inverse != 0, d->scale == 0.0f ? 1.0f : d->scale};
    const int64_t es = size_of(s.dtype), nq = tokens * s.heads * s.W, nk = tokens * s.kv_heads * s.W;
    if (!inv_freq || (nq > 0 && (!q || !q_out)) || (nk > 0 && (!k || !k_out))) return SELSCAN_ERR_NULL;
    if (!all_aligned({q, k, inv_freq, positions, q_out, k_out})) return SELSCAN_ERR_ALIGN;
    const Span iq = span(q, nq * es), ik = span(k, nk * es), oq = span(q_out, nq * es), ok = span(k_out, nk * es);
    const Span ins[] = {span(inv_freq, s.rot / 2 * 4), span(positions, tokens * 4)};
    const Span outs[] = {oq, ok};
    // in place, or elsewhere
    if (any_alias(ins, outs) || half_over(iq, oq) || half_over(ik, ok) || overlaps(iq, ok) || overlaps(ik, oq))
        return SELSCAN_ERR_ALIAS;
    if (th == 0) return SELSCAN_OK;
    return done(launch_rotary(q, k, inv_freq, positions, q_out, k_out, s, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
