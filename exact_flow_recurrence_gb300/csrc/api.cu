// api.cu -- the extern "C" boundary declared in include/efla.h: argument
// validation, workspace sizing, dispatch to the kernels, status reporting.
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <atomic>

#include <nvtx3/nvToolsExt.h>

#include "../../include/efla.h"
#include "gated.h"
#include "launch.h"

namespace {
// An NVTX range around an entry point's host-side work (argument checks, launches), for
// timeline tools; with no tool attached the calls do nothing.
struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};
}  // namespace

namespace {

thread_local char g_msg[512] = "";

// Whether this process has launched, or captured, kernels that keep a status word of their own.
std::atomic<bool> g_used_gated{false}, g_used_step{false}, g_used_norm{false};

efla_status fail(efla_status s, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_msg, sizeof g_msg, fmt, ap);
    va_end(ap);
    return s;
}

efla_status cuda_fail(cudaError_t e, const char* where) {
    return fail(EFLA_ERR_CUDA, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool dim_ok(int d) { return d >= 16 && d <= 128 && d % 16 == 0; }
bool dtype_ok(int t) { return t == EFLA_F32 || t == EFLA_BF16; }
size_t esize(efla_dtype t) { return t == EFLA_BF16 ? 2 : 4; }
bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

struct Span {
    const void* p;
    size_t n;
    const char* name;
};

bool overlap(const Span& a, const Span& b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.n && b0 < a0 + a.n;
}

// Common shape validation.  needs_chunk: fwd/bwd (chunk in {16,32,64}); step: L == 1.
efla_status check_shape(const efla_shape* s, bool step, efla::Dims* d) {
    if (!s) return fail(EFLA_ERR_INVALID_ARG, "shape is NULL");
    if (s->B < 0 || s->H < 0 || s->L < 0)
        return fail(EFLA_ERR_INVALID_ARG, "negative size (B=%d H=%d L=%d)", s->B, s->H, s->L);
    if (!dim_ok(s->dk) || !dim_ok(s->dv))
        return fail(EFLA_ERR_UNSUPPORTED, "dk=%d dv=%d: need multiples of 16 in [16,128]", s->dk, s->dv);
    if (!dtype_ok(s->dtype) || !dtype_ok(s->out_dtype))
        return fail(EFLA_ERR_UNSUPPORTED, "dtype=%d out_dtype=%d: need EFLA_F32 or EFLA_BF16",
                    (int)s->dtype, (int)s->out_dtype);
    if (s->mode != EFLA_EXACT && s->mode != EFLA_EULER)
        return fail(EFLA_ERR_UNSUPPORTED, "mode=%d: need EFLA_EXACT or EFLA_EULER", (int)s->mode);
    if (s->path != EFLA_PATH_AUTO && s->path != EFLA_PATH_SIMT && s->path != EFLA_PATH_TENSOR)
        return fail(EFLA_ERR_UNSUPPORTED, "path=%d: need EFLA_PATH_AUTO, _SIMT or _TENSOR", (int)s->path);
    const long long bh = (long long)s->B * s->H;
    if (bh > 0x7fffffffLL) return fail(EFLA_ERR_UNSUPPORTED, "B*H=%lld exceeds 2^31-1", bh);
    int C = 1;
    if (step) {
        if (s->L != 1) return fail(EFLA_ERR_INVALID_ARG, "efla_step needs L == 1 (got %d)", s->L);
    } else {
        C = s->chunk;
        if (C != 16 && C != 32 && C != 64)
            return fail(EFLA_ERR_UNSUPPORTED, "chunk=%d: need 16, 32 or 64", C);
    }
    const long long NC = ((long long)s->L + C - 1) / C;
    if (!step && NC > 65535)
        return fail(EFLA_ERR_UNSUPPORTED, "L=%d gives %lld chunks (> 65535)", s->L, NC);
    d->B = s->B; d->H = s->H; d->L = s->L; d->dk = s->dk; d->dv = s->dv;
    d->C = C; d->NC = (int)NC;
    d->in_bf16 = s->dtype == EFLA_BF16;
    d->out_bf16 = s->out_dtype == EFLA_BF16;
    d->euler = s->mode == EFLA_EULER;
    d->tensor = 0;
    return EFLA_OK;
}

// Forward path choice (after check_shape).
efla_status pick_fwd_path(const efla_shape* s, efla::Dims* d) {
    const bool ok = efla::fwd_tc_supported(*d);
    if (s->path == EFLA_PATH_TENSOR && !ok && d->L > 0)
        return fail(EFLA_ERR_UNSUPPORTED,
                    "EFLA_PATH_TENSOR needs bf16 inputs, dk = dv = 128 and chunk 64 "
                    "(got dtype=%d dk=%d dv=%d chunk=%d)", (int)s->dtype, s->dk, s->dv, s->chunk);
    d->tensor = ok && s->path != EFLA_PATH_SIMT;
    return EFLA_OK;
}

size_t fwd_ws_for(const efla::Dims& d) {
    return d.tensor ? efla::fwd_tc_ws_bytes(d) : efla::fwd_ws_bytes(d);
}

efla_status check_ptrs(const Span* req, int nreq, const Span* opt, int nopt) {
    for (int i = 0; i < nreq; ++i) {
        if (!req[i].p) return fail(EFLA_ERR_INVALID_ARG, "%s is NULL", req[i].name);
        if (!aligned16(req[i].p)) return fail(EFLA_ERR_ALIGNMENT, "%s is not 16-byte aligned", req[i].name);
    }
    for (int i = 0; i < nopt; ++i)
        if (opt[i].p && !aligned16(opt[i].p))
            return fail(EFLA_ERR_ALIGNMENT, "%s is not 16-byte aligned", opt[i].name);
    return EFLA_OK;
}

// every output must not overlap any input or another output
efla_status check_alias(const Span* outs, int nout, const Span* ins, int nin) {
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (overlap(outs[i], ins[j]))
                return fail(EFLA_ERR_INVALID_ARG, "%s overlaps input %s", outs[i].name, ins[j].name);
        for (int j = i + 1; j < nout; ++j)
            if (overlap(outs[i], outs[j]))
                return fail(EFLA_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, outs[j].name);
    }
    return EFLA_OK;
}

}  // namespace

void efla::set_last_error(const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_msg, sizeof g_msg, fmt, ap);
    va_end(ap);
}

extern "C" {

const char* efla_status_string(efla_status s) {
    switch (s) {
        case EFLA_OK: return "EFLA_OK";
        case EFLA_ERR_INVALID_ARG: return "EFLA_ERR_INVALID_ARG";
        case EFLA_ERR_UNSUPPORTED: return "EFLA_ERR_UNSUPPORTED";
        case EFLA_ERR_ALIGNMENT: return "EFLA_ERR_ALIGNMENT";
        case EFLA_ERR_WORKSPACE: return "EFLA_ERR_WORKSPACE";
        case EFLA_ERR_CUDA: return "EFLA_ERR_CUDA";
        case EFLA_ERR_TIMEOUT: return "EFLA_ERR_TIMEOUT";
        case EFLA_ERR_BOUNDS: return "EFLA_ERR_BOUNDS";
    }
    return "EFLA_ERR_UNKNOWN";
}

const char* efla_last_error(void) { return g_msg; }

size_t efla_fwd_workspace_size(const efla_shape* shape) {
    efla::Dims d;
    if (check_shape(shape, false, &d) != EFLA_OK) return 0;
    if (pick_fwd_path(shape, &d) != EFLA_OK) return 0;
    return fwd_ws_for(d);
}

size_t efla_bwd_workspace_size(const efla_shape* shape) {
    efla::Dims d;
    if (check_shape(shape, false, &d) != EFLA_OK) return 0;
    if (shape->path == EFLA_PATH_TENSOR) return 0;
    d.tensor = shape->path != EFLA_PATH_SIMT;
    return efla::bwd_ws_bytes(d);
}

}  // extern "C"

namespace {

// efla_fwd, and efla_fwd_save when `states` is not null.
efla_status fwd_common(const efla_shape* shape, const void* q, const void* k, const void* v,
                       const float* beta, const float* S0, void* o, float* S_final, float* states,
                       size_t states_bytes, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    g_msg[0] = 0;
    efla::Dims d;
    efla_status st = check_shape(shape, false, &d);
    if (st != EFLA_OK) return st;
    if ((st = pick_fwd_path(shape, &d)) != EFLA_OK) return st;
    if (d.BH() == 0) return EFLA_OK;
    const size_t rec_need = efla::states_bytes(d);
    if (states) {
        if (!aligned16(states)) return fail(EFLA_ERR_ALIGNMENT, "states is not 16-byte aligned");
        if (states_bytes < rec_need)
            return fail(EFLA_ERR_INVALID_ARG, "states %zu bytes < required %zu", states_bytes, rec_need);
    }
    const size_t ntok = (size_t)d.BH() * d.L;
    const size_t ein = esize(shape->dtype), eout = esize(shape->out_dtype);
    const size_t sbytes = (size_t)d.BH() * d.dk * d.dv * 4;
    const Span sq{q, ntok * d.dk * ein, "q"}, sk{k, ntok * d.dk * ein, "k"},
        sv{v, ntok * d.dv * ein, "v"}, sb{beta, ntok * 4, "beta"}, sS0{S0, sbytes, "S0"},
        so{o, ntok * d.dv * eout, "o"}, sSf{S_final, sbytes, "S_final"},
        sw{workspace, workspace_bytes, "workspace"};
    if (d.L > 0) {
        const Span req[] = {sq, sk, sv, sb, so};
        const Span opt[] = {sS0, sSf, sw};
        if ((st = check_ptrs(req, 5, opt, 3)) != EFLA_OK) return st;
    } else {
        const Span opt[] = {sS0, sSf};
        if ((st = check_ptrs(nullptr, 0, opt, 2)) != EFLA_OK) return st;
    }
    // S_final may alias S0 exactly; any other overlap is an error
    if (S_final && S0 && S_final != (float*)S0 && overlap(sSf, sS0))
        return fail(EFLA_ERR_INVALID_ARG, "S_final partially overlaps S0");
    {
        const Span outs[] = {so, sSf};
        const Span ins[] = {sq, sk, sv, sb};
        if ((st = check_alias(outs, 2, ins, 4)) != EFLA_OK) return st;
        if (overlap(so, sS0)) return fail(EFLA_ERR_INVALID_ARG, "o overlaps input S0");
        const Span all[] = {sq, sk, sv, sb, sS0, so, sSf};
        for (const Span& x : all)
            if (overlap(sw, x)) return fail(EFLA_ERR_INVALID_ARG, "workspace overlaps %s", x.name);
        const Span srec{states, rec_need, "states"};
        const Span all2[] = {sq, sk, sv, sb, sS0, so, sSf, sw};
        for (const Span& x : all2)
            if (overlap(srec, x)) return fail(EFLA_ERR_INVALID_ARG, "states overlaps %s", x.name);
    }
    if (d.L == 0) {
        if (!S_final || S_final == S0) return EFLA_OK;
        efla::prof_mark(nullptr, stream);
        cudaError_t e = efla::launch_state_copy((long long)d.BH() * d.dk * d.dv, S0, S_final, stream);
        return e == cudaSuccess ? EFLA_OK : cuda_fail(e, "efla_fwd(state copy)");
    }
    const size_t need = fwd_ws_for(d);
    if (!workspace || workspace_bytes < need)
        return fail(EFLA_ERR_WORKSPACE, "workspace %zu bytes < required %zu", workspace_bytes, need);
    efla::prof_mark(nullptr, stream);
    cudaError_t e;
    if (d.tensor) {
        e = efla::launch_fwd_tc(d, q, k, v, beta, S0, o, S_final, workspace, stream, states,
                                states ? efla::states_Up(d, states) : nullptr,
                                states ? efla::states_T(d, states) : nullptr,
                                states ? efla::states_alpha(d, states) : nullptr);
    } else {
        efla::FwdWs ws = efla::fwd_ws_carve(d, workspace);
        if (states) {   // the preparation and the scan write straight into the record
            ws.Sc = states;
            ws.Up = efla::states_Up(d, states);
            ws.T = efla::states_T(d, states);
            ws.alpha = efla::states_alpha(d, states);
        }
        e = efla::launch_fwd_simt(d, q, k, v, beta, S0, o, S_final, ws, stream);
    }
    return e == cudaSuccess ? EFLA_OK : cuda_fail(e, states ? "efla_fwd_save" : "efla_fwd");
}

// efla_bwd, and efla_bwd_saved when `states` is not null (S0 then comes from the record).
efla_status bwd_common(const efla_shape* shape, const void* q, const void* k, const void* v,
                       const float* beta, const float* S0, const float* states, size_t states_bytes,
                       const void* dO, const float* dS_final, void* dq, void* dk, void* dv, float* dbeta,
                       float* dS0, void* workspace, size_t workspace_bytes, cudaStream_t stream);

}  // namespace

extern "C" {

efla_status efla_fwd(const efla_shape* shape, const void* q, const void* k, const void* v,
                     const float* beta, const float* S0, void* o, float* S_final,
                     void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    NvtxRange nvtx_range("efla_fwd");
    return fwd_common(shape, q, k, v, beta, S0, o, S_final, nullptr, 0, workspace, workspace_bytes, stream);
}

efla_status efla_fwd_save(const efla_shape* shape, const void* q, const void* k, const void* v,
                          const float* beta, const float* S0, void* o, float* S_final, float* states,
                          size_t states_bytes, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    NvtxRange nvtx_range("efla_fwd_save");
    return fwd_common(shape, q, k, v, beta, S0, o, S_final, states, states_bytes, workspace, workspace_bytes,
                      stream);
}

size_t efla_fwd_states_size(const efla_shape* shape) {
    efla::Dims d;
    if (check_shape(shape, false, &d) != EFLA_OK) return 0;
    return efla::states_bytes(d);
}

size_t efla_bwd_saved_workspace_size(const efla_shape* shape) {
    efla::Dims d;
    if (check_shape(shape, false, &d) != EFLA_OK) return 0;
    if (shape->path == EFLA_PATH_TENSOR) return 0;
    d.tensor = shape->path != EFLA_PATH_SIMT;
    return efla::bwd_saved_ws_bytes(d);
}

int efla_bwd_plan(const efla_shape* shape, size_t free_bytes) {
    efla::Dims d;
    if (check_shape(shape, false, &d) != EFLA_OK || shape->path == EFLA_PATH_TENSOR) return -1;
    d.tensor = shape->path != EFLA_PATH_SIMT;
    const bool rec_fits = efla::states_bytes(d) + efla::bwd_saved_ws_bytes(d) <= free_bytes;
    const bool bwd_fits = efla::bwd_ws_bytes(d) <= free_bytes;
    if (efla::bwd_runs_recording_forward(d)) {   // efla_bwd is the faster form here
        if (bwd_fits) return 0;
        return rec_fits ? 1 : -1;
    }
    if (rec_fits) return 1;
    return bwd_fits ? 0 : -1;
}

efla_status efla_bwd_saved(const efla_shape* shape, const void* q, const void* k, const void* v,
                           const float* beta, const float* states, size_t states_bytes, const void* dO,
                           const float* dS_final, void* dq, void* dk, void* dv, float* dbeta, float* dS0,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    NvtxRange nvtx_range("efla_bwd_saved");
    if (!states) {
        g_msg[0] = 0;
        return fail(EFLA_ERR_INVALID_ARG, "efla_bwd_saved: states is NULL");
    }
    return bwd_common(shape, q, k, v, beta, nullptr, states, states_bytes, dO, dS_final, dq, dk, dv, dbeta,
                      dS0, workspace, workspace_bytes, stream);
}

efla_status efla_bwd(const efla_shape* shape, const void* q, const void* k, const void* v,
                     const float* beta, const float* S0, const void* dO, const float* dS_final,
                     void* dq, void* dk, void* dv, float* dbeta, float* dS0,
                     void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    NvtxRange nvtx_range("efla_bwd");
    return bwd_common(shape, q, k, v, beta, S0, nullptr, 0, dO, dS_final, dq, dk, dv, dbeta, dS0, workspace,
                      workspace_bytes, stream);
}

}  // extern "C"

namespace {

efla_status bwd_common(const efla_shape* shape, const void* q, const void* k, const void* v,
                       const float* beta, const float* S0, const float* states, size_t states_bytes,
                       const void* dO, const float* dS_final, void* dq, void* dk, void* dv, float* dbeta,
                       float* dS0, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    g_msg[0] = 0;
    efla::Dims d;
    efla_status st = check_shape(shape, false, &d);
    if (st != EFLA_OK) return st;
    if (shape->path == EFLA_PATH_TENSOR)
        return fail(EFLA_ERR_UNSUPPORTED,
                    "efla_bwd: path must be AUTO (tensor-pipe products where the shape allows) or SIMT");
    d.tensor = shape->path != EFLA_PATH_SIMT;   // allows the tensor-pipe kernels
    if (d.BH() == 0) return EFLA_OK;
    const size_t rec_need = efla::states_bytes(d);
    if (states) {
        if (!aligned16(states)) return fail(EFLA_ERR_ALIGNMENT, "states is not 16-byte aligned");
        if (states_bytes < rec_need)
            return fail(EFLA_ERR_INVALID_ARG, "states %zu bytes < required %zu", states_bytes, rec_need);
    }
    const size_t ntok = (size_t)d.BH() * d.L;
    const size_t ein = esize(shape->dtype), eout = esize(shape->out_dtype);
    const size_t sbytes = (size_t)d.BH() * d.dk * d.dv * 4;
    const Span sq{q, ntok * d.dk * ein, "q"}, sk{k, ntok * d.dk * ein, "k"},
        sv{v, ntok * d.dv * ein, "v"}, sb{beta, ntok * 4, "beta"}, sS0{S0, sbytes, "S0"},
        sdO{dO, ntok * d.dv * ein, "dO"}, sdSf{dS_final, sbytes, "dS_final"},
        sdq{dq, ntok * d.dk * eout, "dq"}, sdk{dk, ntok * d.dk * eout, "dk"},
        sdv{dv, ntok * d.dv * eout, "dv"}, sdb{dbeta, ntok * 4, "dbeta"},
        sdS0{dS0, sbytes, "dS0"}, sw{workspace, workspace_bytes, "workspace"};
    if (d.L > 0) {
        const Span req[] = {sq, sk, sv, sb, sdO, sdq, sdk, sdv, sdb};
        const Span opt[] = {sS0, sdSf, sdS0, sw};
        if ((st = check_ptrs(req, 9, opt, 4)) != EFLA_OK) return st;
    } else {
        const Span opt[] = {sdSf, sdS0};
        if ((st = check_ptrs(nullptr, 0, opt, 2)) != EFLA_OK) return st;
    }
    {
        const Span srec{states, rec_need, "states"};
        const Span outs[] = {sdq, sdk, sdv, sdb, sdS0};
        const Span ins[] = {sq, sk, sv, sb, sS0, sdO, sdSf, srec};
        if ((st = check_alias(outs, 5, ins, 8)) != EFLA_OK) return st;
        const Span all[] = {sq, sk, sv, sb, sS0, sdO, sdSf, sdq, sdk, sdv, sdb, sdS0, srec};
        for (const Span& x : all)
            if (overlap(sw, x)) return fail(EFLA_ERR_INVALID_ARG, "workspace overlaps %s", x.name);
    }
    const char* where = states ? "efla_bwd_saved" : "efla_bwd";
    if (d.L == 0) {
        // no tokens: dS0 = dS_final
        if (!dS0) return EFLA_OK;
        efla::prof_mark(nullptr, stream);
        cudaError_t e = efla::launch_state_copy((long long)d.BH() * d.dk * d.dv, dS_final, dS0, stream);
        return e == cudaSuccess ? EFLA_OK : cuda_fail(e, where);
    }
    const size_t need = states ? efla::bwd_saved_ws_bytes(d) : efla::bwd_ws_bytes(d);
    if (!workspace || workspace_bytes < need)
        return fail(EFLA_ERR_WORKSPACE, "workspace %zu bytes < required %zu", workspace_bytes, need);
    const efla::BwdWs ws = states ? efla::bwd_saved_ws_carve(d, workspace, states) : efla::bwd_ws_carve(d, workspace);
    efla::prof_mark(nullptr, stream);
    cudaError_t e = efla::launch_bwd_simt(d, q, k, v, beta, S0, dO, dS_final, dq, dk, dv, dbeta,
                                          dS0, ws, stream, states != nullptr);
    return e == cudaSuccess ? EFLA_OK : cuda_fail(e, where);
}

}  // namespace

extern "C" {

efla_status efla_step(const efla_shape* shape, const void* q, const void* k, const void* v,
                      const float* beta, float* S, void* o, cudaStream_t stream) {
    NvtxRange nvtx_range("efla_step");
    g_msg[0] = 0;
    efla::Dims d;
    efla_status st = check_shape(shape, true, &d);
    if (st != EFLA_OK) return st;
    if (shape->path == EFLA_PATH_TENSOR)
        return fail(EFLA_ERR_UNSUPPORTED, "efla_step runs on CUDA cores: path must be AUTO or SIMT");
    if (d.BH() == 0) return EFLA_OK;
    const size_t n = (size_t)d.BH();
    const size_t ein = esize(shape->dtype), eout = esize(shape->out_dtype);
    const Span sq{q, n * d.dk * ein, "q"}, sk{k, n * d.dk * ein, "k"}, sv{v, n * d.dv * ein, "v"},
        sb{beta, n * 4, "beta"}, sS{S, n * d.dk * d.dv * 4, "S"}, so{o, n * d.dv * eout, "o"};
    const Span req[] = {sq, sk, sv, sb, sS, so};
    if ((st = check_ptrs(req, 6, nullptr, 0)) != EFLA_OK) return st;
    const Span outs[] = {sS, so};
    const Span ins[] = {sq, sk, sv, sb};
    if ((st = check_alias(outs, 2, ins, 4)) != EFLA_OK) return st;
    efla::prof_mark(nullptr, stream);
    cudaError_t e = efla::launch_step(d, q, k, v, beta, S, o, stream);
    return e == cudaSuccess ? EFLA_OK : cuda_fail(e, "efla_step");
}

efla_status efla_mixer_proj(const efla_mixer_shape* s, const void* x, const void* w, void* q, void* k, void* v,
                            float* beta, cudaStream_t stream) {
    NvtxRange nvtx_range("efla_mixer_proj");
    g_msg[0] = 0;
    if (!s) return fail(EFLA_ERR_INVALID_ARG, "shape is NULL");
    if (s->B < 0 || s->L < 0 || s->D < 0 || s->H < 0)
        return fail(EFLA_ERR_INVALID_ARG, "negative size (B=%d L=%d D=%d H=%d)", s->B, s->L, s->D, s->H);
    if (s->dk != 128 || s->L % 128 || s->D % 64 || s->D < 64 || s->H < 2 || s->H > 32 || s->H % 2)
        return fail(EFLA_ERR_UNSUPPORTED,
                    "efla_mixer_proj needs dk = 128, L % 128 == 0, D % 64 == 0 (D >= 64), even H in [2, 32] "
                    "(got L=%d D=%d H=%d dk=%d)", s->L, s->D, s->H, s->dk);
    const long long M = (long long)s->B * s->L;
    if (M == 0) return EFLA_OK;
    if (M * s->H > 0x7fffffffLL || (long long)s->D * (3 * s->H * 128 + s->H) > 0x7fffffffLL)
        return fail(EFLA_ERR_UNSUPPORTED, "efla_mixer_proj: B L H = %lld rows exceed 2^31-1", M * s->H);
    const size_t nw = (size_t)(3 * s->H * 128 + s->H) * s->D, nqkv = (size_t)M * s->H * 128;
    const Span sx{x, (size_t)M * s->D * 2, "x"}, sw{w, nw * 2, "w"}, sq{q, nqkv * 2, "q"}, sk{k, nqkv * 2, "k"},
        sv{v, nqkv * 2, "v"}, sb{beta, (size_t)M * s->H * 4, "beta"};
    const Span req[] = {sx, sw, sq, sk, sv, sb};
    efla_status st = check_ptrs(req, 6, nullptr, 0);
    if (st != EFLA_OK) return st;
    const Span outs[] = {sq, sk, sv, sb};
    const Span ins[] = {sx, sw};
    if ((st = check_alias(outs, 4, ins, 2)) != EFLA_OK) return st;
    efla::prof_mark(nullptr, stream);
    cudaError_t e = efla::launch_mixer_proj(s->B, s->L, s->D, s->H, x, w, q, k, v, beta, stream);
    return e == cudaSuccess ? EFLA_OK : cuda_fail(e, "efla_mixer_proj");
}

efla_status efla_wait_selftest(int kind, int limit, cudaStream_t stream) {
    g_msg[0] = 0;
    if ((kind != 0 && kind != 1) || limit < 1 || limit > (1 << 20))
        return fail(EFLA_ERR_INVALID_ARG, "efla_wait_selftest: kind 0 or 1, limit 1..2^20 (got %d, %d)",
                    kind, limit);
    efla::prof_mark(nullptr, stream);
    cudaError_t e = efla::launch_wait_selftest(kind, (uint32_t)limit, stream);
    return e == cudaSuccess ? EFLA_OK : cuda_fail(e, "efla_wait_selftest");
}

efla_status efla_get_status(cudaStream_t stream) {
    NvtxRange nvtx_range("efla_get_status");
    g_msg[0] = 0;
    cudaError_t e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return cuda_fail(e, "efla_get_status(sync)");
    e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "efla_get_status");
    // A read is a copy of 9 us: the words of kernels that no call of this process has launched stay unread.
    const struct {
        bool used;
        cudaError_t (*read)(unsigned int*);
    } words[] = {{true, efla::tc_status_read_clear},     {true, efla::proj_status_read_clear},
                 {true, efla::bt_status_read_clear},     {true, efla::gt_status_read_clear},
                 {true, efla::sd_status_read_clear},     {g_used_gated, efla::gated_tc_status_read_clear},
                 {g_used_gated, efla::gated_bwd_tc_status_read_clear}, {g_used_step, efla::gated_step_status_read_clear},
                 {g_used_norm, efla::norm_status_read_clear}};
    unsigned int word = 0;
    for (const auto& w : words) {
        unsigned int one = 0;
        if (!w.used) continue;
        e = w.read(&one);
        if (e != cudaSuccess) return cuda_fail(e, "efla_get_status(status word)");
        word |= one;
    }
    if (word & efla::kStatusBounds)
        return fail(EFLA_ERR_BOUNDS, "a debug-build bounds check skipped a global write (status 0x%x)", word);
    if (word) return fail(EFLA_ERR_TIMEOUT, "a bounded device-side wait expired (status 0x%x)", word);
    return EFLA_OK;
}

efla_status efla_tc_selftest(int N, int K, int flags, const void* A, const void* B, const float* C,
                             float* D, cudaStream_t stream) {
    g_msg[0] = 0;
    if ((N != 64 && N != 128 && N != 192 && N != 256) || (K != 64 && K != 128) || (flags & ~7) ||
        ((flags & 5) == 5))
        return fail(EFLA_ERR_UNSUPPORTED, "efla_tc_selftest: N in {64, 128, 192, 256}, K in {64, 128}, flags in 0..7 without bits 0 and 2 together (got %d, %d, %d)",
                    N, K, flags);
    const Span req[] = {{A, 1, "A"}, {B, 1, "B"}, {C, 1, "C"}, {D, 1, "D"}};
    efla_status st = check_ptrs(req, 4, nullptr, 0);
    if (st != EFLA_OK) return st;
    efla::prof_mark(nullptr, stream);
    cudaError_t e = efla::launch_tc_selftest(N, K, flags, A, B, C, D, stream);
    return e == cudaSuccess ? EFLA_OK : cuda_fail(e, "efla_tc_selftest");
}

}  // extern "C"

// ------------------------------------------------------------------ gated delta rule, layer norm
namespace {

// A [rows][d] array reached through {batch, head, token} strides (elements).
struct Strided {
    const void* p;
    const char* name;
    int n[3], d, es;
    const long long* s;
    size_t bytes() const {
        if (!n[0] || !n[1] || !n[2]) return 0;
        long long e = d;
        for (int i = 0; i < 3; ++i) e += (n[i] - 1LL) * s[i];
        return (size_t)e * es;
    }
    Span span() const { return Span{p, bytes(), name}; }
    // whether vector copies and tensor maps can read it: 16-byte rows, no broadcast dimension
    bool wide() const {
        if (!aligned16(p)) return false;
        for (int i = 0; i < 3; ++i)
            if (n[i] > 1 && (s[i] <= 0 || (s[i] * es) % 16 != 0 || s[i] * es >= (1LL << 39))) return false;
        return true;
    }
    // no two rows share an element
    bool disjoint_rows() const {
        bool used[3] = {false, false, false};
        long long ext = d;
        for (int k = 0; k < 3; ++k) {   // dimensions by growing stride
            int m = -1;
            for (int i = 0; i < 3; ++i)
                if (!used[i] && n[i] > 1 && (m < 0 || s[i] < s[m])) m = i;
            if (m < 0) break;
            used[m] = true;
            if (s[m] < ext) return false;
            ext += (n[m] - 1LL) * s[m];
        }
        return true;
    }
};

// Two arrays whose spans overlap but whose elements do not: slices of the same token rows.
bool interleaved(const Strided& a, const Strided& b) {
    if (a.es != b.es || a.s[2] != b.s[2] || (a.n[0] > 1 && a.s[0] != b.s[0])) return false;
    const long long st = a.s[2], wa = a.d + (a.n[1] - 1LL) * a.s[1], wb = b.d + (b.n[1] - 1LL) * b.s[1];
    const long long bytes = (long long)((uintptr_t)b.p - (uintptr_t)a.p);
    if (st <= 0 || bytes % a.es || (a.n[0] > 1 && a.s[0] % st)) return false;
    const long long off = ((bytes / a.es) % st + st) % st;   // b's place in a's token row
    return off >= wa && off + wb <= st;
}

efla_status check_gated(const efla_gated_shape* s, bool step, efla::GDims* d) {
    if (!s) return fail(EFLA_ERR_INVALID_ARG, "shape is NULL");
    if (s->B < 0 || s->H < 0 || s->Hk < 0 || s->L < 0)
        return fail(EFLA_ERR_INVALID_ARG, "negative size (B=%d H=%d Hk=%d L=%d)", s->B, s->H, s->Hk, s->L);
    if (s->H > 0 && (s->Hk == 0 || s->H % s->Hk))
        return fail(EFLA_ERR_INVALID_ARG, "H=%d value heads are not a multiple of Hk=%d key heads", s->H, s->Hk);
    if (s->packed != 0 && s->packed != 1) return fail(EFLA_ERR_INVALID_ARG, "packed=%d: need 0 or 1", s->packed);
    if (step && (s->packed || s->L != 1))
        return fail(EFLA_ERR_INVALID_ARG, "efla_gated_step needs L == 1 and packed == 0 (got %d, %d)", s->L, s->packed);
    if (!dim_ok(s->dk) || !dim_ok(s->dv))
        return fail(EFLA_ERR_UNSUPPORTED, "dk=%d dv=%d: need multiples of 16 in [16,128]", s->dk, s->dv);
    if (!dtype_ok(s->dtype) || !dtype_ok(s->out_dtype))
        return fail(EFLA_ERR_UNSUPPORTED, "dtype=%d out_dtype=%d: need EFLA_F32 or EFLA_BF16", (int)s->dtype,
                    (int)s->out_dtype);
    if (s->mode != EFLA_EXACT && s->mode != EFLA_EULER)
        return fail(EFLA_ERR_UNSUPPORTED, "mode=%d: need EFLA_EXACT or EFLA_EULER", (int)s->mode);
    if (s->path != EFLA_PATH_AUTO && s->path != EFLA_PATH_SIMT && s->path != EFLA_PATH_TENSOR)
        return fail(EFLA_ERR_UNSUPPORTED, "path=%d: need EFLA_PATH_AUTO, _SIMT or _TENSOR", (int)s->path);
    if (s->H > 65535) return fail(EFLA_ERR_UNSUPPORTED, "H=%d exceeds 65535", s->H);
    if ((long long)s->B * s->H > 0x7fffffffLL || (s->packed ? 1LL : s->B) * (s->L / 16 + 1LL) + s->B > 0x7fffffffLL)
        return fail(EFLA_ERR_UNSUPPORTED, "B=%d H=%d L=%d: too many chunks for one launch", s->B, s->H, s->L);
    const long long(*all[10])[3] = {&s->q_stride, &s->k_stride, &s->v_stride, &s->g_stride, &s->beta_stride,
                                    &s->o_stride, &s->do_stride, &s->dq_stride, &s->dk_stride, &s->dv_stride};
    long long(*to[10])[3] = {&d->qs, &d->ks, &d->vs, &d->gs, &d->bs, &d->os, &d->dos, &d->dqs, &d->dks, &d->dvs};
    for (int i = 0; i < 10; ++i)
        for (int j = 0; j < 3; ++j) {
            if ((*all[i])[j] < 0) return fail(EFLA_ERR_INVALID_ARG, "negative stride");
            (*to[i])[j] = (*all[i])[j];
        }
    d->B = s->B; d->H = s->H; d->Hk = s->Hk; d->L = s->L; d->dk = s->dk; d->dv = s->dv;
    d->in_bf16 = s->dtype == EFLA_BF16;
    d->out_bf16 = s->out_dtype == EFLA_BF16;
    d->euler = s->mode == EFLA_EULER;
    d->packed = s->packed;
    d->tensor = 0;
    d->offsets = nullptr;
    return EFLA_OK;
}

struct GatedIo {
    Strided x[10];   // q, k, v, g, beta, o, dO, dq, dk, dv (those the call has)
};

GatedIo gated_io(const efla_gated_shape* s, const void* q, const void* k, const void* v, const void* g,
                 const void* beta, const void* o, const void* dO, const void* dq, const void* dk, const void* dv) {
    const int b = s->packed ? 1 : s->B, e = (int)esize(s->dtype), eo = (int)esize(s->out_dtype);
    return GatedIo{{{q, "q", {b, s->Hk, s->L}, s->dk, e, s->q_stride},
                    {k, "k", {b, s->Hk, s->L}, s->dk, e, s->k_stride},
                    {v, "v", {b, s->H, s->L}, s->dv, e, s->v_stride},
                    {g, "g", {b, s->H, s->L}, 1, 4, s->g_stride},
                    {beta, "beta", {b, s->H, s->L}, 1, 4, s->beta_stride},
                    {o, "o", {b, s->H, s->L}, s->dv, eo, s->o_stride},
                    {dO, "dO", {b, s->H, s->L}, s->dv, e, s->do_stride},
                    {dq, "dq", {b, s->Hk, s->L}, s->dk, eo, s->dq_stride},
                    {dk, "dk", {b, s->Hk, s->L}, s->dk, eo, s->dk_stride},
                    {dv, "dv", {b, s->H, s->L}, s->dv, eo, s->dv_stride}}};
}

// Required arrays: present, aligned to their element; outputs with rows apart from each other.
efla_status check_strided(const Strided* x, int n, int first_out) {
    for (int i = 0; i < n; ++i) {
        if (x[i].bytes() == 0) continue;
        if (!x[i].p) return fail(EFLA_ERR_INVALID_ARG, "%s is NULL", x[i].name);
        if ((uintptr_t)x[i].p % (unsigned)x[i].es)
            return fail(EFLA_ERR_ALIGNMENT, "%s is not aligned to its elements", x[i].name);
        if (i >= first_out && !x[i].disjoint_rows())
            return fail(EFLA_ERR_INVALID_ARG, "%s: strides make its rows overlap", x[i].name);
    }
    return EFLA_OK;
}

// The tensor-core kernels take bf16 tokens whose rows (of every token array: x[0..2] and the
// outputs x[5..]) can be copied 16 bytes at a time.
efla_status pick_gated_path(const efla_gated_shape* s, const Strided* x, int n, efla::GDims* d) {
    bool ok = efla::gated_tc_supported(*d);
    for (int i = 0; i < n; ++i)
        if (i != 3 && i != 4) ok = ok && x[i].wide();
    if (s->path == EFLA_PATH_TENSOR && !ok && d->L > 0)
        return fail(EFLA_ERR_UNSUPPORTED, "EFLA_PATH_TENSOR needs bf16 tokens in rows on 16-byte boundaries");
    d->tensor = ok && s->path != EFLA_PATH_SIMT;
    return EFLA_OK;
}

// Strided inputs and outputs, dense outputs, and the workspace: every output apart from
// every input, from the other outputs and from the workspace.
efla_status check_gated_alias(const Strided* x, int n, int first_out, const Span* ins, int nin, const Span* outs,
                              int nout, const Span& ws) {
    for (int i = first_out; i < n; ++i) {
        const Span o = x[i].span();
        for (int j = 0; j < first_out; ++j)
            if (overlap(o, x[j].span())) return fail(EFLA_ERR_INVALID_ARG, "%s overlaps input %s", o.name, x[j].name);
        for (int j = 0; j < nin; ++j)
            if (overlap(o, ins[j])) return fail(EFLA_ERR_INVALID_ARG, "%s overlaps input %s", o.name, ins[j].name);
        for (int j = 0; j < nout; ++j)
            if (overlap(o, outs[j])) return fail(EFLA_ERR_INVALID_ARG, "%s overlaps %s", o.name, outs[j].name);
        for (int j = i + 1; j < n; ++j)
            if (overlap(o, x[j].span()) && !interleaved(x[i], x[j]) && !interleaved(x[j], x[i]))
                return fail(EFLA_ERR_INVALID_ARG, "%s overlaps %s", o.name, x[j].name);
        if (overlap(o, ws)) return fail(EFLA_ERR_INVALID_ARG, "workspace overlaps %s", o.name);
    }
    for (int j = 0; j < first_out; ++j) {
        for (int i = 0; i < nout; ++i)
            if (overlap(outs[i], x[j].span()))
                return fail(EFLA_ERR_INVALID_ARG, "%s overlaps input %s", outs[i].name, x[j].name);
        if (overlap(ws, x[j].span())) return fail(EFLA_ERR_INVALID_ARG, "workspace overlaps %s", x[j].name);
    }
    for (int i = 0; i < nout; ++i) {
        for (int j = i + 1; j < nout; ++j)
            if (overlap(outs[i], outs[j])) return fail(EFLA_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, outs[j].name);
        if (overlap(ws, outs[i])) return fail(EFLA_ERR_INVALID_ARG, "workspace overlaps %s", outs[i].name);
    }
    for (int j = 0; j < nin; ++j)
        if (overlap(ws, ins[j])) return fail(EFLA_ERR_INVALID_ARG, "workspace overlaps %s", ins[j].name);
    return EFLA_OK;
}

}  // namespace

extern "C" {

// (of the larger path: which one runs also depends on the arrays' alignment)
size_t efla_gated_fwd_workspace_size(const efla_gated_shape* s) {
    efla::GDims d;
    if (check_gated(s, false, &d) != EFLA_OK) return 0;
    return s->path != EFLA_PATH_SIMT && d.in_bf16 ? efla::gated_tc_fwd_ws_bytes(d) : 0;   // (the fp32 kernel needs none)
}

size_t efla_gated_bwd_workspace_size(const efla_gated_shape* s) {
    efla::GDims d;
    if (check_gated(s, false, &d) != EFLA_OK) return 0;
    const size_t simt = efla::gated_simt_bwd_ws_bytes(d);
    const size_t tc = s->path != EFLA_PATH_SIMT && efla::gated_tc_supported(d) ? efla::gated_tc_bwd_ws_bytes(d) : 0;
    return tc > simt ? tc : simt;
}

efla_status efla_gated_fwd(const efla_gated_shape* s, const int* offsets, const void* q, const void* k, const void* v,
                           const float* g, const float* beta, const float* S0, void* o, float* S_final,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    NvtxRange nvtx_range("efla_gated_fwd");
    g_msg[0] = 0;
    efla::GDims d;
    efla_status st = check_gated(s, false, &d);
    if (st != EFLA_OK) return st;
    if (d.BH() == 0) return EFLA_OK;
    const GatedIo io = gated_io(s, q, k, v, g, beta, o, nullptr, nullptr, nullptr, nullptr);
    if ((st = check_strided(io.x, 6, 5)) != EFLA_OK) return st;
    if ((st = pick_gated_path(s, io.x, 6, &d)) != EFLA_OK) return st;
    const size_t sbytes = (size_t)d.BH() * d.dk * d.dv * 4;
    const Span sS0{S0, sbytes, "S0"}, sSf{S_final, sbytes, "S_final"}, sw{workspace, workspace_bytes, "workspace"},
        soff{offsets, ((size_t)d.B + 1) * 4, "offsets"};
    const Span opt[] = {sS0, sSf, sw};
    if ((st = check_ptrs(nullptr, 0, opt, 3)) != EFLA_OK) return st;
    if (d.packed && !offsets) return fail(EFLA_ERR_INVALID_ARG, "offsets is NULL (packed)");
    if (d.packed && (uintptr_t)offsets % 4) return fail(EFLA_ERR_ALIGNMENT, "offsets is not 4-byte aligned");
    d.offsets = d.packed ? offsets : nullptr;
    if (S_final && S0 && S_final != (float*)S0 && overlap(sSf, sS0))
        return fail(EFLA_ERR_INVALID_ARG, "S_final partially overlaps S0");
    {
        const Span ins[] = {sS0, d.packed ? soff : Span{nullptr, 0, ""}};
        const Span outs[] = {S_final == (float*)S0 ? Span{nullptr, 0, ""} : sSf};
        if ((st = check_gated_alias(io.x, 6, 5, ins, 2, outs, 1, sw)) != EFLA_OK) return st;
        if (overlap(sSf, ins[1])) return fail(EFLA_ERR_INVALID_ARG, "S_final overlaps input offsets");
    }
    const size_t need = d.tensor ? efla::gated_tc_fwd_ws_bytes(d) : 0;
    if (need && (!workspace || workspace_bytes < need))
        return fail(EFLA_ERR_WORKSPACE, "workspace %zu bytes < required %zu", workspace_bytes, need);
    if (s->path == EFLA_PATH_AUTO && efla::gated_fwd_short(d)) d.tensor = 0;   // (the workspace asked for is the shape's all the same)
    g_used_gated = true;
    efla::prof_mark(nullptr, stream);
    const cudaError_t e =
        d.tensor ? efla::launch_gated_fwd_tc(d, q, k, v, g, beta, S0, o, S_final, workspace, stream)
                 : efla::launch_gated_fwd_simt(d, q, k, v, g, beta, S0, o, S_final, stream);
    return e == cudaSuccess ? EFLA_OK : cuda_fail(e, "efla_gated_fwd");
}

efla_status efla_gated_bwd(const efla_gated_shape* s, const int* offsets, const void* q, const void* k, const void* v,
                           const float* g, const float* beta, const float* S0, const void* dO, const float* dS_final,
                           void* dq, void* dk, void* dv, float* dg, float* dbeta, float* dS0, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
    NvtxRange nvtx_range("efla_gated_bwd");
    g_msg[0] = 0;
    efla::GDims d;
    efla_status st = check_gated(s, false, &d);
    if (st != EFLA_OK) return st;
    if (d.BH() == 0) return EFLA_OK;
    GatedIo io = gated_io(s, q, k, v, g, beta, nullptr, dO, dq, dk, dv);
    io.x[5] = io.x[6];   // no o here: dO is the sixth input
    for (int i = 6; i < 9; ++i) io.x[i] = io.x[i + 1];
    if ((st = check_strided(io.x, 9, 6)) != EFLA_OK) return st;
    if ((st = pick_gated_path(s, io.x, 9, &d)) != EFLA_OK) return st;
    const size_t sbytes = (size_t)d.BH() * d.dk * d.dv * 4, gbytes = (d.packed ? 1 : (size_t)d.B) * d.H * d.L * 4;
    const Span sS0{S0, sbytes, "S0"}, sdS{dS_final, sbytes, "dS_final"}, sd0{dS0, sbytes, "dS0"},
        sdg{dg, gbytes, "dg"}, sdb{dbeta, gbytes, "dbeta"}, sw{workspace, workspace_bytes, "workspace"},
        soff{offsets, ((size_t)d.B + 1) * 4, "offsets"};
    const Span req[] = {sdg, sdb};
    const Span opt[] = {sS0, sdS, sd0, sw};
    if ((st = check_ptrs(req, gbytes ? 2 : 0, opt, 4)) != EFLA_OK) return st;
    if (d.packed && !offsets) return fail(EFLA_ERR_INVALID_ARG, "offsets is NULL (packed)");
    if (d.packed && (uintptr_t)offsets % 4) return fail(EFLA_ERR_ALIGNMENT, "offsets is not 4-byte aligned");
    d.offsets = d.packed ? offsets : nullptr;
    {
        const Span ins[] = {sS0, sdS, d.packed ? soff : Span{nullptr, 0, ""}};
        const Span outs[] = {sdg, sdb, sd0};
        if ((st = check_gated_alias(io.x, 9, 6, ins, 3, outs, 3, sw)) != EFLA_OK) return st;
        for (const Span& a : outs)
            for (const Span& b : ins)
                if (overlap(a, b)) return fail(EFLA_ERR_INVALID_ARG, "%s overlaps input %s", a.name, b.name);
    }
    const size_t need = d.tensor ? efla::gated_tc_bwd_ws_bytes(d) : efla::gated_simt_bwd_ws_bytes(d);
    if (need && (!workspace || workspace_bytes < need))
        return fail(EFLA_ERR_WORKSPACE, "workspace %zu bytes < required %zu", workspace_bytes, need);
    g_used_gated = true;
    efla::prof_mark(nullptr, stream);
    const auto launch = d.tensor ? efla::launch_gated_bwd_tc : efla::launch_gated_bwd_simt;
    const cudaError_t e = launch(d, q, k, v, g, beta, S0, dO, dS_final, dq, dk, dv, dg, dbeta, dS0, workspace, stream);
    return e == cudaSuccess ? EFLA_OK : cuda_fail(e, "efla_gated_bwd");
}

efla_status efla_gated_step(const efla_gated_shape* s, const void* q, const void* k, const void* v, const float* g,
                            const float* beta, float* S, const int* slots, int nslots, void* o, cudaStream_t stream) {
    NvtxRange nvtx_range("efla_gated_step");
    g_msg[0] = 0;
    efla::GDims d;
    efla_status st = check_gated(s, true, &d);
    if (st != EFLA_OK) return st;
    if (s->path == EFLA_PATH_TENSOR)
        return fail(EFLA_ERR_UNSUPPORTED, "efla_gated_step runs on CUDA cores: path must be AUTO or SIMT");
    if (nslots < 0 || (!slots && nslots < d.B))
        return fail(EFLA_ERR_INVALID_ARG, "nslots=%d: the cache holds fewer states than the B=%d sequences", nslots, d.B);
    if (d.BH() == 0) return EFLA_OK;
    const GatedIo io = gated_io(s, q, k, v, g, beta, o, nullptr, nullptr, nullptr, nullptr);
    if ((st = check_strided(io.x, 6, 5)) != EFLA_OK) return st;
    if (slots && (uintptr_t)slots % 4) return fail(EFLA_ERR_ALIGNMENT, "slots is not 4-byte aligned");
    const Span sS{S, (size_t)nslots * d.H * d.dk * d.dv * 4, "S"}, ssl{slots, (size_t)d.B * 4, "slots"};
    if ((st = check_ptrs(&sS, nslots ? 1 : 0, nullptr, 0)) != EFLA_OK) return st;
    if ((st = check_gated_alias(io.x, 6, 5, &ssl, 1, &sS, 1, Span{nullptr, 0, "workspace"})) != EFLA_OK) return st;
    if (overlap(sS, ssl)) return fail(EFLA_ERR_INVALID_ARG, "S overlaps input slots");
    g_used_step = true;
    efla::prof_mark(nullptr, stream);
    const cudaError_t e = efla::launch_gated_step(d, q, k, v, g, beta, S, slots, nslots, o, stream);
    return e == cudaSuccess ? EFLA_OK : cuda_fail(e, "efla_gated_step");
}

}  // extern "C"

namespace {

efla_status check_norm(const efla_norm_shape* s, efla::NormDims* d) {
    if (!s) return fail(EFLA_ERR_INVALID_ARG, "shape is NULL");
    if (s->rows < 0 || s->D < 0) return fail(EFLA_ERR_INVALID_ARG, "negative size (rows=%lld D=%d)", s->rows, s->D);
    if (s->D < 1 || s->D > 16384) return fail(EFLA_ERR_UNSUPPORTED, "D=%d: need 1 .. 16384", s->D);
    if (s->rows > 0x7fffffffLL) return fail(EFLA_ERR_UNSUPPORTED, "rows=%lld exceed 2^31-1", s->rows);
    if (!dtype_ok(s->dtype) || !dtype_ok(s->weight_dtype))
        return fail(EFLA_ERR_UNSUPPORTED, "dtype=%d weight_dtype=%d: need EFLA_F32 or EFLA_BF16", (int)s->dtype,
                    (int)s->weight_dtype);
    if (!(s->eps >= 0.f)) return fail(EFLA_ERR_INVALID_ARG, "eps=%g: need a non-negative number", (double)s->eps);
    if (s->rows > 1 && (s->x_stride < s->D || s->y_stride < s->D))
        return fail(EFLA_ERR_INVALID_ARG, "row strides %lld, %lld are below D=%d", s->x_stride, s->y_stride, s->D);
    *d = efla::NormDims{s->rows, s->rows > 1 ? s->x_stride : s->D, s->rows > 1 ? s->y_stride : s->D, s->D,
                        s->dtype == EFLA_BF16, s->weight_dtype == EFLA_BF16, s->eps};
    return EFLA_OK;
}

// alignment of the rows and weights to their elements (their vector copies ask for more where they are
// used) and of stats to its pairs, which are read and written as one
efla_status check_elems(const Span* x, const size_t* es, int n) {
    for (int i = 0; i < n; ++i)
        if (x[i].n && (uintptr_t)x[i].p % es[i])
            return fail(EFLA_ERR_ALIGNMENT, "%s is not aligned to %zu bytes", x[i].name, es[i]);
    return EFLA_OK;
}

size_t rows_bytes(const efla::NormDims& d, long long stride) {
    return d.rows ? ((size_t)(d.rows - 1) * stride + d.D) * (d.bf16 ? 2 : 4) : 0;
}

}  // namespace

extern "C" {

efla_status efla_norm_fwd(const efla_norm_shape* s, const void* x, const void* weight, const void* bias, void* y,
                          float* stats, cudaStream_t stream) {
    NvtxRange nvtx_range("efla_norm_fwd");
    g_msg[0] = 0;
    efla::NormDims d;
    efla_status st = check_norm(s, &d);
    if (st != EFLA_OK || d.rows == 0) return st;
    const size_t e = d.bf16 ? 2 : 4, we = d.w_bf16 ? 2 : 4;
    const Span in[] = {{x, rows_bytes(d, d.x_stride), "x"}, {weight, d.D * we, "weight"}, {bias, d.D * we, "bias"}};
    const Span out[] = {{y, rows_bytes(d, d.y_stride), "y"}, {stats, (size_t)d.rows * 8, "stats"}};
    if (!x || !weight || !y || !stats)
        return fail(EFLA_ERR_INVALID_ARG, "%s is NULL", !x ? "x" : !weight ? "weight" : !y ? "y" : "stats");
    const Span el[] = {in[0], in[1], in[2], out[0], out[1]};
    const size_t es[] = {e, we, we, e, 8};
    if ((st = check_elems(el, es, 5)) != EFLA_OK) return st;
    if ((st = check_alias(out, 2, in, 3)) != EFLA_OK) return st;
    g_used_norm = true;
    efla::prof_mark(nullptr, stream);
    const cudaError_t r = efla::launch_norm_fwd(d, x, weight, bias, y, stats, stream);
    return r == cudaSuccess ? EFLA_OK : cuda_fail(r, "efla_norm_fwd");
}

size_t efla_norm_bwd_workspace_size(const efla_norm_shape* s) {
    efla::NormDims d;
    return check_norm(s, &d) == EFLA_OK ? efla::norm_bwd_ws_bytes(d) : 0;
}

efla_status efla_norm_bwd(const efla_norm_shape* s, const void* x, const void* weight, const void* dy,
                          const float* stats, void* dx, void* dweight, void* dbias, void* workspace,
                          size_t workspace_bytes, cudaStream_t stream) {
    NvtxRange nvtx_range("efla_norm_bwd");
    g_msg[0] = 0;
    efla::NormDims d;
    efla_status st = check_norm(s, &d);
    if (st != EFLA_OK) return st;
    const size_t e = d.bf16 ? 2 : 4, we = d.w_bf16 ? 2 : 4;
    const Span in[] = {{x, rows_bytes(d, d.x_stride), "x"}, {weight, d.D * we, "weight"},
                       {dy, rows_bytes(d, d.y_stride), "dy"}, {stats, (size_t)d.rows * 8, "stats"}};
    const Span out[] = {{dx, rows_bytes(d, d.D), "dx"}, {dweight, d.D * we, "dweight"}, {dbias, d.D * we, "dbias"},
                        {workspace, workspace_bytes, "workspace"}};
    for (const Span& a : in)
        if (a.n && !a.p) return fail(EFLA_ERR_INVALID_ARG, "%s is NULL", a.name);
    if (out[0].n && !dx) return fail(EFLA_ERR_INVALID_ARG, "dx is NULL");
    if (!dweight) return fail(EFLA_ERR_INVALID_ARG, "dweight is NULL");
    const Span el[] = {in[0], in[1], in[2], in[3], out[0], out[1], out[2]};
    const size_t es[] = {e, we, e, 8, e, we, we};
    if ((st = check_elems(el, es, 7)) != EFLA_OK) return st;
    if ((st = check_ptrs(nullptr, 0, out + 3, 1)) != EFLA_OK) return st;
    if ((st = check_alias(out, 4, in, 4)) != EFLA_OK) return st;
    const size_t need = efla::norm_bwd_ws_bytes(d);
    if (!workspace || workspace_bytes < need)
        return fail(EFLA_ERR_WORKSPACE, "workspace %zu bytes < required %zu", workspace_bytes, need);
    g_used_norm = true;
    efla::prof_mark(nullptr, stream);
    const cudaError_t r = efla::launch_norm_bwd(d, x, weight, dy, stats, dx, dweight, dbias, workspace, stream);
    return r == cudaSuccess ? EFLA_OK : cuda_fail(r, "efla_norm_bwd");
}

}  // extern "C"

// ------------------------------------------------------------------ profiling
#include <string.h>
#include <vector>

namespace {
struct ProfRec {
    const char* name;   // nullptr: an entry point's start mark
    cudaEvent_t ev;
};
thread_local bool g_prof_on = false;
thread_local std::vector<ProfRec>* g_prof = nullptr;
}  // namespace

void efla::prof_mark(const char* name, cudaStream_t st) {
    if (!g_prof_on) return;
    cudaEvent_t ev;
    if (cudaEventCreate(&ev) != cudaSuccess) return;
    cudaEventRecord(ev, st);
    g_prof->push_back(ProfRec{name, ev});
}

extern "C" efla_status efla_profile_begin(void) {
    if (!g_prof) g_prof = new std::vector<ProfRec>();
    for (auto& r : *g_prof) cudaEventDestroy(r.ev);
    g_prof->clear();
    g_prof_on = true;
    return EFLA_OK;
}

extern "C" int efla_profile_end(int cap, const char** names, float* total_ms, int* launches) {
    g_prof_on = false;
    if (!g_prof) return 0;
    int n = 0;
    bool err = false;
    for (size_t i = 1; i < g_prof->size(); ++i) {
        const ProfRec& r = (*g_prof)[i];
        if (!r.name) continue;
        float ms = 0.f;
        if (cudaEventSynchronize(r.ev) != cudaSuccess ||
            cudaEventElapsedTime(&ms, (*g_prof)[i - 1].ev, r.ev) != cudaSuccess) {
            err = true;
            break;
        }
        int j = 0;
        while (j < n && strcmp(names[j], r.name) != 0) ++j;
        if (j == n) {
            if (n == cap) continue;
            names[n] = r.name;
            total_ms[n] = 0.f;
            launches[n] = 0;
            ++n;
        }
        total_ms[j] += ms;
        launches[j] += 1;
    }
    for (auto& r : *g_prof) cudaEventDestroy(r.ev);
    g_prof->clear();
    return err ? -1 : n;
}
