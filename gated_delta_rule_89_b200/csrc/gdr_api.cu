// C entry points of libgdr.so: argument validation, dispatch, status codes.
// The declarations and the contract of every call are in include/gdr.h.
#include <stdint.h>

#include "gdr.h"
#include "gdr_internal.cuh"
#include "ssm_internal.cuh"

#define GDR_API extern "C" __attribute__((visibility("default")))

namespace {

thread_local int tl_last_cuda_error = 0;
thread_local int tl_last_launches = 0;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int finish(cudaError_t e, int launches)
{
    if (e != cudaSuccess) {
        tl_last_cuda_error = (int)e;
        return GDR_ERR_CUDA;
    }
    tl_last_launches = launches;
    return GDR_OK;
}

bool size_ok(int d) { return d == 64 || d == 128; }

// Debug mode only: GDR_ERR_GATE_RANGE when an element of g is positive or not
// finite (n elements), GDR_ERR_CUDA when the check itself failed, else GDR_OK.
int gate_guard(const float *g, size_t n, cudaStream_t st)
{
    if (!gdr::debug_checks_enabled()) return GDR_OK;
    bool bad = false;
    const cudaError_t e = gdr::check_gate_range(g, n, st, &bad);
    if (e != cudaSuccess) {
        tl_last_cuda_error = (int)e;
        return GDR_ERR_CUDA;
    }
    return bad ? GDR_ERR_GATE_RANGE : GDR_OK;
}

size_t gate_elems(long long heads, int T, int dk, int gate_mode)
{
    return (size_t)heads * (size_t)T * (gate_mode == GDR_GATE_PER_CHANNEL ? (size_t)dk : 1u);
}

}  // namespace

GDR_API const char *gdr_status_string(int status)
{
    switch (status) {
        case GDR_OK: return "GDR_OK";
        case GDR_ERR_INVALID_ARG: return "GDR_ERR_INVALID_ARG";
        case GDR_ERR_UNSUPPORTED: return "GDR_ERR_UNSUPPORTED";
        case GDR_ERR_ALIGNMENT: return "GDR_ERR_ALIGNMENT";
        case GDR_ERR_CUDA: return "GDR_ERR_CUDA";
        case GDR_ERR_GATE_RANGE: return "GDR_ERR_GATE_RANGE";
        case GDR_ERR_TIMEOUT: return "GDR_ERR_TIMEOUT";
        default: return "GDR_ERR_UNKNOWN";
    }
}

GDR_API int gdr_last_cuda_error(void) { return tl_last_cuda_error; }

GDR_API int gdr_last_launch_count(void) { return tl_last_launches; }

GDR_API void gdr_debug_set_wait_budget(long long cycles) { gdr::set_wait_budget(cycles); }

GDR_API size_t gdr_chunk_fwd_workspace_size(int B, int H, int T, int dk, int dv, int C, int gate_mode, int dtype)
{
    if (B <= 0 || H <= 0 || T <= 0) return 0;
    if (gate_mode != GDR_GATE_PER_CHANNEL && gate_mode != GDR_GATE_SCALAR) return 0;
    gdr::ChunkArgs a = {};
    a.B = B; a.H = H; a.T = T; a.dk = dk; a.dv = dv; a.C = C;
    a.scalar_gate = (gate_mode == GDR_GATE_SCALAR);
    a.bf16 = (dtype == GDR_BF16);
    return gdr::chunk_tc_supports(a) ? gdr::chunk_tc_workspace_bytes(B, H, T) : 0;
}

GDR_API int gdr_device_status(void *stream)
{
    int v = 0;
    cudaError_t e = gdr::read_device_status(static_cast<cudaStream_t>(stream), &v);
    if (e != cudaSuccess) {
        tl_last_cuda_error = (int)e;
        return GDR_ERR_CUDA;
    }
    return v;
}

GDR_API int gdr_chunk_fwd(const void *q, const void *k, const void *v, const float *g, const float *beta,
                          const float *S0, void *O, float *S_T,
                          int B, int H, int T, int dk, int dv, int C, int gate_mode, int dtype,
                          void *workspace, size_t ws_bytes, void *stream)
{
    if (B < 0 || H < 0 || T < 0) return GDR_ERR_INVALID_ARG;
    if (gate_mode != GDR_GATE_PER_CHANNEL && gate_mode != GDR_GATE_SCALAR) return GDR_ERR_INVALID_ARG;
    if (dtype != GDR_F32 && dtype != GDR_BF16) return GDR_ERR_INVALID_ARG;
    if (dk <= 0 || dv <= 0 || C <= 0) return GDR_ERR_INVALID_ARG;
    if (!size_ok(dk) || !size_ok(dv) || !(C == 16 || C == 32 || C == 64)) return GDR_ERR_UNSUPPORTED;
    if ((long long)B * H * T * (dk > dv ? dk : dv) >= (1LL << 40)) return GDR_ERR_UNSUPPORTED;
    const size_t ws_need = gdr_chunk_fwd_workspace_size(B, H, T, dk, dv, C, gate_mode, dtype);
    if (ws_bytes < ws_need || (ws_need && !workspace)) return GDR_ERR_INVALID_ARG;
    const long long heads = (long long)B * H;
    if (heads == 0) {
        tl_last_launches = 0;
        return GDR_OK;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        // nothing to read or write per token; the final state is the initial one
        if (S_T && !aligned16(S_T)) return GDR_ERR_ALIGNMENT;
        if (S0 && !aligned16(S0)) return GDR_ERR_ALIGNMENT;
        cudaError_t e = cudaSuccess;
        const size_t bytes = sizeof(float) * (size_t)heads * dv * dk;
        if (S_T && S0 && S_T != S0) e = cudaMemcpyAsync(S_T, S0, bytes, cudaMemcpyDeviceToDevice, st);
        else if (S_T && !S0) e = cudaMemsetAsync(S_T, 0, bytes, st);
        return finish(e, 0);
    }
    if (!q || !k || !v || !g || !beta || !O) return GDR_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, g, beta, S0, O, S_T, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDR_ERR_ALIGNMENT;

    gdr::ChunkArgs a;
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.S0 = S0; a.O = O; a.S_T = S_T;
    a.B = B; a.H = H; a.T = T; a.dk = dk; a.dv = dv; a.C = C;
    a.scalar_gate = (gate_mode == GDR_GATE_SCALAR);
    a.bf16 = (dtype == GDR_BF16);
    a.workspace = workspace;
    if (const int gs = gate_guard(g, gate_elems(heads, T, dk, gate_mode), st)) return gs;
    int launches = 0;
    cudaError_t e = gdr::chunk_tc_supports(a) ? gdr::launch_chunk_tc(a, st, &launches)
                                              : gdr::launch_chunk_simt(a, st, &launches);
    return finish(e, launches);
}

GDR_API int gdr_chunk_fwd_prologue(const void *q_raw, const void *k_raw, const void *v, const void *a,
                                   const float *A_log, const float *dt_bias, const float *b_logit,
                                   const float *S0, void *O, float *S_T,
                                   int B, int H, int T, int dk, int dv, int C, int gate_mode, int dtype,
                                   void *workspace, size_t ws_bytes, void *stream)
{
    if (B < 0 || H < 0 || T < 0) return GDR_ERR_INVALID_ARG;
    if (gate_mode != GDR_GATE_PER_CHANNEL && gate_mode != GDR_GATE_SCALAR) return GDR_ERR_INVALID_ARG;
    if (dtype != GDR_F32 && dtype != GDR_BF16) return GDR_ERR_INVALID_ARG;
    if (dk <= 0 || dv <= 0 || C <= 0) return GDR_ERR_INVALID_ARG;
    gdr::ChunkArgs a_;
    a_.dk = dk; a_.dv = dv; a_.C = C; a_.bf16 = (dtype == GDR_BF16);
    if (!gdr::chunk_tc_supports(a_)) return GDR_ERR_UNSUPPORTED;   // bf16, d_k = d_v = 128, C = 64 only
    if ((long long)B * H * T * 128 >= (1LL << 40)) return GDR_ERR_UNSUPPORTED;
    const size_t ws_need = gdr_chunk_fwd_workspace_size(B, H, T, dk, dv, C, gate_mode, dtype);
    if (ws_bytes < ws_need || (ws_need && !workspace)) return GDR_ERR_INVALID_ARG;
    const long long heads = (long long)B * H;
    if (heads == 0) {
        tl_last_launches = 0;
        return GDR_OK;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        if (S_T && !aligned16(S_T)) return GDR_ERR_ALIGNMENT;
        if (S0 && !aligned16(S0)) return GDR_ERR_ALIGNMENT;
        cudaError_t e = cudaSuccess;
        const size_t bytes = sizeof(float) * (size_t)heads * dv * dk;
        if (S_T && S0 && S_T != S0) e = cudaMemcpyAsync(S_T, S0, bytes, cudaMemcpyDeviceToDevice, st);
        else if (S_T && !S0) e = cudaMemsetAsync(S_T, 0, bytes, st);
        return finish(e, 0);
    }
    if (!q_raw || !k_raw || !v || !a || !A_log || !dt_bias || !b_logit || !O) return GDR_ERR_INVALID_ARG;
    const void *ptrs[] = {q_raw, k_raw, v, a, dt_bias, S0, O, S_T, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDR_ERR_ALIGNMENT;
    if (reinterpret_cast<uintptr_t>(A_log) % 4 || reinterpret_cast<uintptr_t>(b_logit) % 4) return GDR_ERR_ALIGNMENT;

    gdr::ChunkArgs c;
    c.q = q_raw; c.k = k_raw; c.v = v;
    c.g = static_cast<const float *>(a);   // the bf16 pre-activation, reinterpreted by the prologue kernel
    c.beta = b_logit; c.S0 = S0; c.O = O; c.S_T = S_T;
    c.B = B; c.H = H; c.T = T; c.dk = dk; c.dv = dv; c.C = C;
    c.scalar_gate = (gate_mode == GDR_GATE_SCALAR);
    c.bf16 = true;
    c.workspace = workspace;
    c.prologue = true;
    c.A_log = A_log;
    c.dt_bias = dt_bias;
    int launches = 0;
    cudaError_t e = gdr::launch_chunk_tc(c, st, &launches);
    return finish(e, launches);
}

GDR_API int gdr_chunk_fwd_gated(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                const void *gate, const float *norm_w, float eps,
                                const float *S0, void *Y, float *S_T,
                                int B, int H, int T, int dk, int dv, int C, int gate_mode, int dtype,
                                void *workspace, size_t ws_bytes, void *stream)
{
    if (B < 0 || H < 0 || T < 0) return GDR_ERR_INVALID_ARG;
    if (gate_mode != GDR_GATE_PER_CHANNEL && gate_mode != GDR_GATE_SCALAR) return GDR_ERR_INVALID_ARG;
    if (dtype != GDR_F32 && dtype != GDR_BF16) return GDR_ERR_INVALID_ARG;
    if (dk <= 0 || dv <= 0 || C <= 0) return GDR_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || eps > 1e30f) return GDR_ERR_INVALID_ARG;   // also rejects NaN
    gdr::ChunkArgs a_;
    a_.dk = dk; a_.dv = dv; a_.C = C; a_.bf16 = (dtype == GDR_BF16);
    if (!gdr::chunk_tc_supports(a_)) return GDR_ERR_UNSUPPORTED;   // bf16, d_k = d_v = 128, C = 64 only
    if ((long long)B * H * T * 128 >= (1LL << 40)) return GDR_ERR_UNSUPPORTED;
    const size_t ws_need = gdr_chunk_fwd_workspace_size(B, H, T, dk, dv, C, gate_mode, dtype);
    if (ws_bytes < ws_need || (ws_need && !workspace)) return GDR_ERR_INVALID_ARG;
    const long long heads = (long long)B * H;
    if (heads == 0) {
        tl_last_launches = 0;
        return GDR_OK;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        if (S_T && !aligned16(S_T)) return GDR_ERR_ALIGNMENT;
        if (S0 && !aligned16(S0)) return GDR_ERR_ALIGNMENT;
        cudaError_t e = cudaSuccess;
        const size_t bytes = sizeof(float) * (size_t)heads * dv * dk;
        if (S_T && S0 && S_T != S0) e = cudaMemcpyAsync(S_T, S0, bytes, cudaMemcpyDeviceToDevice, st);
        else if (S_T && !S0) e = cudaMemsetAsync(S_T, 0, bytes, st);
        return finish(e, 0);
    }
    if (!q || !k || !v || !g || !beta || !gate || !norm_w || !Y) return GDR_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, g, beta, gate, S0, Y, S_T, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDR_ERR_ALIGNMENT;
    if (reinterpret_cast<uintptr_t>(norm_w) % 4) return GDR_ERR_ALIGNMENT;

    gdr::ChunkArgs c;
    c.q = q; c.k = k; c.v = v; c.g = g; c.beta = beta; c.S0 = S0; c.O = Y; c.S_T = S_T;
    c.B = B; c.H = H; c.T = T; c.dk = dk; c.dv = dv; c.C = C;
    c.scalar_gate = (gate_mode == GDR_GATE_SCALAR);
    c.bf16 = true;
    c.workspace = workspace;
    c.gated_out = true;
    c.ogate = gate;
    c.norm_w = norm_w;
    c.eps = eps;
    if (const int gs = gate_guard(g, gate_elems(heads, T, dk, gate_mode), st)) return gs;
    int launches = 0;
    cudaError_t e = gdr::launch_chunk_tc(c, st, &launches);
    return finish(e, launches);
}

GDR_API size_t gdr_chunk_bwd_workspace_size(int B, int H, int T, int dk, int dv, int C, int gate_mode, int dtype)
{
    if (B <= 0 || H <= 0 || T <= 0) return 0;
    if (gate_mode != GDR_GATE_PER_CHANNEL && gate_mode != GDR_GATE_SCALAR) return 0;
    if (dtype != GDR_F32 && dtype != GDR_BF16) return 0;
    if (dk != dv || !size_ok(dk) || C != 64) return 0;
    return gdr::chunk_bwd_workspace_bytes(B, H, T, dk);
}

GDR_API int gdr_chunk_bwd(const void *q, const void *k, const void *v, const float *g, const float *beta,
                          const float *S0, const void *dO, const float *dS_T,
                          void *dq, void *dk, void *dv, float *dg, float *dbeta, float *dS0,
                          int B, int H, int T, int dk_, int dv_, int C, int gate_mode, int dtype,
                          void *workspace, size_t ws_bytes, void *stream)
{
    if (B < 0 || H < 0 || T < 0) return GDR_ERR_INVALID_ARG;
    if (gate_mode != GDR_GATE_PER_CHANNEL && gate_mode != GDR_GATE_SCALAR) return GDR_ERR_INVALID_ARG;
    if (dtype != GDR_F32 && dtype != GDR_BF16) return GDR_ERR_INVALID_ARG;
    if (dk_ <= 0 || dv_ <= 0 || C <= 0) return GDR_ERR_INVALID_ARG;
    if (dk_ != dv_ || !size_ok(dk_) || C != 64) return GDR_ERR_UNSUPPORTED;
    if ((long long)B * H * T * dk_ >= (1LL << 40)) return GDR_ERR_UNSUPPORTED;
    const long long heads = (long long)B * H;
    if (heads == 0) {
        tl_last_launches = 0;
        return GDR_OK;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        // no tokens: S_T = S0, so dS0 = dS_T
        if (dS0 && !aligned16(dS0)) return GDR_ERR_ALIGNMENT;
        if (dS_T && !aligned16(dS_T)) return GDR_ERR_ALIGNMENT;
        cudaError_t e = cudaSuccess;
        const size_t bytes = sizeof(float) * (size_t)heads * dv_ * dk_;
        if (dS0 && dS_T && dS0 != dS_T) e = cudaMemcpyAsync(dS0, dS_T, bytes, cudaMemcpyDeviceToDevice, st);
        else if (dS0 && !dS_T) e = cudaMemsetAsync(dS0, 0, bytes, st);
        return finish(e, 0);
    }
    const size_t ws_need = gdr_chunk_bwd_workspace_size(B, H, T, dk_, dv_, C, gate_mode, dtype);
    if (ws_bytes < ws_need || !workspace) return GDR_ERR_INVALID_ARG;
    if (!q || !k || !v || !g || !beta || !dO || !dq || !dk || !dv || !dg || !dbeta) return GDR_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, g, beta, S0, dO, dS_T, dq, dk, dv, dg, dbeta, dS0, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDR_ERR_ALIGNMENT;
    gdr::BwdArgs a;
    a.q = q; a.k = k; a.v = v; a.dO = dO; a.g = g; a.beta = beta; a.S0 = S0; a.dS_T = dS_T;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.dS0 = dS0;
    a.B = B; a.H = H; a.T = T; a.D = dk_;
    a.scalar_gate = (gate_mode == GDR_GATE_SCALAR);
    a.bf16 = (dtype == GDR_BF16);
    a.workspace = workspace;
    if (const int gs = gate_guard(g, gate_elems(heads, T, dk_, gate_mode), st)) return gs;
    int launches = 0;
    cudaError_t e = gdr::launch_chunk_bwd(a, st, &launches);
    return finish(e, launches);
}

GDR_API size_t gdr2_chunk_fwd_workspace_size(int B, int H, int T, int dk, int dv, int C, int gate_mode, int dtype)
{
    if (B <= 0 || H <= 0 || T <= 0) return 0;
    if (gate_mode != GDR_GATE_PER_CHANNEL && gate_mode != GDR_GATE_SCALAR) return 0;
    gdr::ChunkArgs a = {};
    a.dk = dk; a.dv = dv; a.C = C;
    a.bf16 = (dtype == GDR_BF16);
    return gdr::chunk_tc_supports(a) ? gdr::chunk_tc_workspace_bytes(B, H, T, true) : 0;
}

GDR_API int gdr2_chunk_fwd(const void *q, const void *k, const void *v, const float *g, const void *b,
                           const void *w, const float *S0, void *O, float *S_T,
                           int B, int H, int T, int dk, int dv, int C, int gate_mode, int dtype,
                           void *workspace, size_t ws_bytes, void *stream)
{
    if (B < 0 || H < 0 || T < 0) return GDR_ERR_INVALID_ARG;
    if (gate_mode != GDR_GATE_PER_CHANNEL && gate_mode != GDR_GATE_SCALAR) return GDR_ERR_INVALID_ARG;
    if (dtype != GDR_F32 && dtype != GDR_BF16) return GDR_ERR_INVALID_ARG;
    if (dk <= 0 || dv <= 0 || C <= 0) return GDR_ERR_INVALID_ARG;
    gdr::ChunkArgs a_;
    a_.dk = dk; a_.dv = dv; a_.C = C; a_.bf16 = (dtype == GDR_BF16);
    if (!gdr::chunk_tc_supports(a_)) return GDR_ERR_UNSUPPORTED;   // bf16, d_k = d_v = 128, C = 64 only
    if ((long long)B * H * T * 128 >= (1LL << 40)) return GDR_ERR_UNSUPPORTED;
    const size_t ws_need = gdr2_chunk_fwd_workspace_size(B, H, T, dk, dv, C, gate_mode, dtype);
    if (ws_bytes < ws_need || (ws_need && !workspace)) return GDR_ERR_INVALID_ARG;
    const long long heads = (long long)B * H;
    if (heads == 0) {
        tl_last_launches = 0;
        return GDR_OK;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        if (S_T && !aligned16(S_T)) return GDR_ERR_ALIGNMENT;
        if (S0 && !aligned16(S0)) return GDR_ERR_ALIGNMENT;
        cudaError_t e = cudaSuccess;
        const size_t bytes = sizeof(float) * (size_t)heads * dv * dk;
        if (S_T && S0 && S_T != S0) e = cudaMemcpyAsync(S_T, S0, bytes, cudaMemcpyDeviceToDevice, st);
        else if (S_T && !S0) e = cudaMemsetAsync(S_T, 0, bytes, st);
        return finish(e, 0);
    }
    if (!q || !k || !v || !g || !b || !w || !O) return GDR_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, g, b, w, S0, O, S_T, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDR_ERR_ALIGNMENT;

    gdr::ChunkArgs c;
    c.q = q; c.k = k; c.v = v; c.g = g; c.beta = nullptr; c.S0 = S0; c.O = O; c.S_T = S_T;
    c.B = B; c.H = H; c.T = T; c.dk = dk; c.dv = dv; c.C = C;
    c.scalar_gate = (gate_mode == GDR_GATE_SCALAR);
    c.bf16 = true;
    c.workspace = workspace;
    c.gdr2 = true;
    c.erase = b;
    c.write = w;
    if (const int gs = gate_guard(g, gate_elems(heads, T, dk, gate_mode), st)) return gs;
    int launches = 0;
    cudaError_t e = gdr::launch_chunk_tc(c, st, &launches);
    return finish(e, launches);
}

GDR_API int gdr2_recurrent_step(const void *q, const void *k, const void *v, const float *g, const void *b,
                                const void *w, float *S, void *o, int B, int H, int dk, int dv, int gate_mode,
                                int dtype, void *stream)
{
    if (B < 0 || H < 0) return GDR_ERR_INVALID_ARG;
    if (gate_mode != GDR_GATE_PER_CHANNEL && gate_mode != GDR_GATE_SCALAR) return GDR_ERR_INVALID_ARG;
    if (dtype != GDR_F32 && dtype != GDR_BF16) return GDR_ERR_INVALID_ARG;
    if (dk <= 0 || dv <= 0) return GDR_ERR_INVALID_ARG;
    if (!size_ok(dk) || !size_ok(dv)) return GDR_ERR_UNSUPPORTED;
    if ((long long)B * H * dv * dk >= (1LL << 40)) return GDR_ERR_UNSUPPORTED;
    if ((long long)B * H == 0) {
        tl_last_launches = 0;
        return GDR_OK;
    }
    if (!q || !k || !v || !g || !b || !w || !S || !o) return GDR_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, g, b, w, S, o};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDR_ERR_ALIGNMENT;
    gdr::StepArgs a;
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = nullptr; a.S = S; a.o = o;
    a.B = B; a.H = H; a.dk = dk; a.dv = dv;
    a.scalar_gate = (gate_mode == GDR_GATE_SCALAR);
    a.bf16 = (dtype == GDR_BF16);
    a.gdr2 = true;
    a.erase = b;
    a.write = w;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (const int gs = gate_guard(g, gate_elems((long long)B * H, 1, dk, gate_mode), st)) return gs;
    int launches = 0;
    cudaError_t e = gdr::launch_recurrent_step(a, st, &launches);
    return finish(e, launches);
}

GDR_API int gdr_recurrent_step(const void *q, const void *k, const void *v, const float *g, const float *beta,
                               float *S, void *o, int B, int H, int dk, int dv, int gate_mode, int dtype,
                               void *stream)
{
    if (B < 0 || H < 0) return GDR_ERR_INVALID_ARG;
    if (gate_mode != GDR_GATE_PER_CHANNEL && gate_mode != GDR_GATE_SCALAR) return GDR_ERR_INVALID_ARG;
    if (dtype != GDR_F32 && dtype != GDR_BF16) return GDR_ERR_INVALID_ARG;
    if (dk <= 0 || dv <= 0) return GDR_ERR_INVALID_ARG;
    if (!size_ok(dk) || !size_ok(dv)) return GDR_ERR_UNSUPPORTED;
    if ((long long)B * H * dv * dk >= (1LL << 40)) return GDR_ERR_UNSUPPORTED;
    if ((long long)B * H == 0) {
        tl_last_launches = 0;
        return GDR_OK;
    }
    if (!q || !k || !v || !g || !beta || !S || !o) return GDR_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, g, beta, S, o};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDR_ERR_ALIGNMENT;
    gdr::StepArgs a;
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.S = S; a.o = o;
    a.B = B; a.H = H; a.dk = dk; a.dv = dv;
    a.scalar_gate = (gate_mode == GDR_GATE_SCALAR);
    a.bf16 = (dtype == GDR_BF16);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (const int gs = gate_guard(g, gate_elems((long long)B * H, 1, dk, gate_mode), st)) return gs;
    int launches = 0;
    cudaError_t e = gdr::launch_recurrent_step(a, st, &launches);
    return finish(e, launches);
}

// ---------------------------------------------- short convolution and state space scan

namespace {

// Bytes of one element, 0 for a bad dtype.
size_t elem_bytes(int dtype) { return dtype == GDR_F32 ? 4 : dtype == GDR_BF16 ? 2 : 0; }

bool any_misaligned(const void *const *p, int n, size_t bytes)
{
    for (int i = 0; i < n; ++i)
        if (p[i] && !gdr::aligned_to(p[i], bytes)) return true;
    return false;
}

bool any_null(const void *const *p, int n)
{
    for (int i = 0; i < n; ++i)
        if (!p[i]) return true;
    return false;
}

bool any_negative(const long long *s, int n)
{
    for (int i = 0; s && i < n; ++i)
        if (s[i] < 0) return true;
    return false;
}

// Sizes both operators share; the limits keep every token index, block count
// and channel index inside 32 bits (offsets are 64-bit throughout).
int sequence_sizes(int B, int T, long long D)
{
    if (B < 0 || T < 0 || D < 0) return GDR_ERR_INVALID_ARG;
    if (B > (1 << 20) || T >= (1 << 30) || D > (1 << 20)) return GDR_ERR_UNSUPPORTED;
    if ((long long)B * (T ? T : 1) * (D ? D : 1) >= (1LL << 40)) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

int conv_sizes(int B, int H, int T, int d, int W, int act, int dtype)
{
    if (H < 0 || d < 0 || W <= 0 || !elem_bytes(dtype)) return GDR_ERR_INVALID_ARG;
    if (act != GDR_ACT_NONE && act != GDR_ACT_SILU) return GDR_ERR_INVALID_ARG;
    if (W < 2 || W > 4) return GDR_ERR_UNSUPPORTED;
    return sequence_sizes(B, T, (long long)H * d);
}

gdr::RowStrides rows_or_dense(const long long *s, int H, int T, int d)
{
    if (s) return {s[0], s[1], s[2]};
    return {(long long)H * T * d, (long long)T * d, d};
}

int scan_sizes(int B, int T, int D, int G, int N, int dtype)
{
    if (!elem_bytes(dtype) || G <= 0 || N <= 0) return GDR_ERR_INVALID_ARG;
    if (const int e = sequence_sizes(B, T, D)) return e;
    if (D % G) return GDR_ERR_INVALID_ARG;
    if (N != 8 && N != 16 && N != 32 && N != 64) return GDR_ERR_UNSUPPORTED;
    if ((long long)B * G * ((D / G + 7) / 8) >= (1LL << 31)) return GDR_ERR_UNSUPPORTED;
    if ((long long)B * D * N >= (1LL << 40)) return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

// Whether the dense block of `count` elements at `out` shares memory with one
// of the B x H x T rows of `row` elements at `in` (elements of `bytes`).
bool overlap(const void *out, long long count, const void *in, const gdr::RowStrides &s, int B, int H, int T,
             long long row, size_t bytes)
{
    if (!out || !in || count <= 0 || row <= 0 || B <= 0 || H <= 0 || T <= 0) return false;
    const long long e = (long long)bytes, first = (long long)(reinterpret_cast<uintptr_t>(in));
    const long long lo = (long long)(reinterpret_cast<uintptr_t>(out)), hi = lo + count * e;
    if (hi <= first || first + ((B - 1) * s.b + (H - 1) * s.h + (T - 1) * s.t + row) * e <= lo) return false;
    for (int b = 0; b < B; ++b)
        for (int h = 0; h < H; ++h) {
            const long long base = first + (b * s.b + h * s.h) * e, step = s.t * e, before = lo - base - row * e;
            // the first row that ends behind lo
            const long long t = before < 0 || step == 0 ? 0 : before / step + 1, at = base + t * step;
            if (t < T && at < hi && at + row * e > lo) return true;
        }
    return false;
}

// As overlap(), for outputs whose kernel reads every element of `in` in the
// thread that later writes its place: those may be the same dense tensor.
bool overlap_elsewhere(const void *out, long long count, const void *in, const gdr::BatchToken &s, int B, int T,
                       long long row, size_t bytes)
{
    if (out == in && (T == 1 || s.t == row) && (B == 1 || s.b == T * row)) return false;
    return overlap(out, count, in, {s.b, 0, s.t}, B, 1, T, row, bytes);
}

// Whether y lies in an input that the kernels may still read.
bool scan_overlap(const gdr::ScanArgs &a)
{
    const size_t e = a.bf16 ? 2 : 4;
    const long long outs = (long long)a.B * a.T * a.D, GN = (long long)a.G * a.N;
    return overlap_elsewhere(a.y, outs, a.x, a.xs, a.B, a.T, a.D, e) ||
           overlap_elsewhere(a.y, outs, a.dt, a.dts, a.B, a.T, a.D, e) ||
           overlap_elsewhere(a.y, outs, a.z, a.zs, a.B, a.T, a.D, e) ||
           overlap(a.y, outs, a.Bm, {a.bs.b, 0, a.bs.t}, a.B, 1, a.T, GN, e) ||
           overlap(a.y, outs, a.Cm, {a.cs.b, 0, a.cs.t}, a.B, 1, a.T, GN, e);
}

gdr::BatchToken tokens_or_dense(const long long *s, int T, long long row)
{
    if (s) return {s[0], s[1]};
    return {(long long)T * row, row};
}

int nothing_to_do()
{
    tl_last_launches = 0;
    return GDR_OK;
}

}  // namespace

GDR_API int gdr_short_conv_fwd(const void *x, const float *weight, const float *bias, const void *state,
                               const int *lengths, void *y, void *state_out, const long long *x_strides, int zero_tail,
                               int B, int H, int T, int d, int W, int act, int dtype, void *stream)
{
    if (const int e = conv_sizes(B, H, T, d, W, act, dtype)) return e;
    if (any_negative(x_strides, 3)) return GDR_ERR_INVALID_ARG;
    if (B == 0 || H == 0 || d == 0 || (T == 0 && !state_out)) return nothing_to_do();
    if (!weight || (T > 0 && (!x || !y))) return GDR_ERR_INVALID_ARG;
    const void *rows[] = {x, state, y, state_out}, *words[] = {weight, bias, lengths};
    if (any_misaligned(rows, 4, elem_bytes(dtype)) || any_misaligned(words, 3, 4)) return GDR_ERR_ALIGNMENT;
    gdr::ConvArgs a = {x, rows_or_dense(x_strides, H, T, d), weight, bias, state, lengths, y, state_out,
                       B, H, T, d, W, act == GDR_ACT_SILU, dtype == GDR_BF16, lengths && zero_tail};
    // y's rows are written while other threads still read x's rows around them
    const long long outs = (long long)B * H * T * d, D = (long long)H * d;
    if (overlap(y, outs, x, a.xs, B, H, T, d, elem_bytes(dtype)) ||
        overlap(y, outs, state, {(W - 1) * D, 0, D}, B, 1, W - 1, D, elem_bytes(dtype)))
        return GDR_ERR_INVALID_ARG;
    int launches = 0;
    const cudaError_t e = gdr::launch_short_conv_fwd(a, static_cast<cudaStream_t>(stream), &launches);
    return finish(e, launches);
}

GDR_API int gdr_short_conv_step(const void *x, const float *weight, const float *bias, void *state, void *y,
                                long long x_stride, int B, int D, int W, int act, int dtype, void *stream)
{
    if (const int e = conv_sizes(B, 1, 1, D, W, act, dtype)) return e;
    if (x_stride < 0) return GDR_ERR_INVALID_ARG;
    if (B == 0 || D == 0) return nothing_to_do();
    if (!x || !weight || !state || !y) return GDR_ERR_INVALID_ARG;
    const void *rows[] = {x, state, y}, *words[] = {weight, bias};
    if (any_misaligned(rows, 3, elem_bytes(dtype)) || any_misaligned(words, 2, 4)) return GDR_ERR_ALIGNMENT;
    gdr::ConvArgs a = {x, {x_stride, 0, 0}, weight, bias, state, nullptr, y, state,
                       B, 1, 1, D, W, act == GDR_ACT_SILU, dtype == GDR_BF16, false};
    const size_t bytes = elem_bytes(dtype);
    if (overlap_elsewhere(y, (long long)B * D, x, {x_stride, 0}, B, 1, D, bytes) ||
        overlap(y, (long long)B * D, state, {(W - 1LL) * D, 0, D}, B, 1, W - 1, D, bytes))
        return GDR_ERR_INVALID_ARG;
    int launches = 0;
    const cudaError_t e = gdr::launch_short_conv_step(a, static_cast<cudaStream_t>(stream), &launches);
    return finish(e, launches);
}

GDR_API size_t gdr_short_conv_bwd_workspace_size(int B, int H, int T, int d, int W, int dtype)
{
    if (conv_sizes(B, H, T, d, W, GDR_ACT_NONE, dtype) || B == 0 || H == 0 || d == 0) return 0;
    return gdr::short_conv_bwd_workspace_bytes(B, H, T, d, W);
}

GDR_API int gdr_short_conv_bwd(const void *x, const float *weight, const float *bias, const void *state,
                               const int *lengths, const void *dy, const void *dstate_out,
                               void *dx, float *dweight, float *dbias, void *dstate,
                               const long long *x_strides, const long long *dy_strides, const long long *dx_strides,
                               int B, int H, int T, int d, int W, int act, int dtype,
                               void *workspace, size_t ws_bytes, void *stream)
{
    if (const int e = conv_sizes(B, H, T, d, W, act, dtype)) return e;
    if (any_negative(x_strides, 3) || any_negative(dy_strides, 3) || any_negative(dx_strides, 3))
        return GDR_ERR_INVALID_ARG;
    if (H == 0 || d == 0) return nothing_to_do();
    if (!weight || !dweight || (B > 0 && T > 0 && (!x || !dy || !dx))) return GDR_ERR_INVALID_ARG;
    const void *rows[] = {x, dy, dx, state, dstate_out, dstate};
    const void *words[] = {weight, bias, lengths, dweight, dbias};
    if (any_misaligned(rows, 6, elem_bytes(dtype)) || any_misaligned(words, 5, 4) || !aligned16(workspace))
        return GDR_ERR_ALIGNMENT;
    const size_t need = gdr_short_conv_bwd_workspace_size(B, H, T, d, W, dtype);
    if (ws_bytes < need || (need && !workspace)) return GDR_ERR_INVALID_ARG;
    if (B > 0 && T > 0 && (dx == x || dx == dy)) return GDR_ERR_INVALID_ARG;   // read around the rows that are written
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (B == 0) {   // the sums over no rows
        cudaError_t e = cudaMemsetAsync(dweight, 0, sizeof(float) * (size_t)H * d * W, st);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, sizeof(float) * (size_t)H * d, st);
        return finish(e, 0);
    }
    gdr::ConvBwdArgs a = {x, dy, rows_or_dense(x_strides, H, T, d), rows_or_dense(dy_strides, H, T, d),
                          rows_or_dense(dx_strides, H, T, d), weight, bias, state, dstate_out, lengths, dx, dstate,
                          dweight, dbias, B, H, T, d, W, act == GDR_ACT_SILU, dtype == GDR_BF16, workspace};
    int launches = 0;
    const cudaError_t e = gdr::launch_short_conv_bwd(a, st, &launches);
    return finish(e, launches);
}

GDR_API size_t gdr_ssm_scan_fwd_workspace_size(int B, int T, int D, int G, int N, int dtype)
{
    if (scan_sizes(B, T, D, G, N, dtype) || B == 0 || T == 0 || D == 0) return 0;
    return gdr::ssm_scan_fwd_workspace_bytes(B, T, D, G, N);
}

GDR_API int gdr_ssm_scan_fwd(const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                             const float *D_skip, const void *z, const float *dt_bias, const float *h0,
                             const int *lengths, void *y, float *h_T, const long long *strides, int zero_tail,
                             int B, int T, int D, int G, int N, int dt_softplus, int dtype,
                             void *workspace, size_t ws_bytes, void *stream)
{
    if (const int e = scan_sizes(B, T, D, G, N, dtype)) return e;
    if (any_negative(strides, 10)) return GDR_ERR_INVALID_ARG;
    if (B == 0 || D == 0 || (T == 0 && !h_T)) return nothing_to_do();
    const void *need[] = {x, dt, Bm, Cm, y};
    if (!A || (T > 0 && any_null(need, 5))) return GDR_ERR_INVALID_ARG;
    const void *rows[] = {x, dt, Bm, Cm, z, y}, *words[] = {D_skip, dt_bias, lengths};
    const void *lines[] = {A, h0, h_T, workspace};
    if (any_misaligned(rows, 6, elem_bytes(dtype)) || any_misaligned(words, 3, 4) || any_misaligned(lines, 4, 16))
        return GDR_ERR_ALIGNMENT;
    const size_t ws_need = gdr_ssm_scan_fwd_workspace_size(B, T, D, G, N, dtype);
    if (ws_bytes < ws_need || (ws_need && !workspace)) return GDR_ERR_INVALID_ARG;
    const long long *s = strides;
    gdr::ScanArgs a = {x, dt, Bm, Cm, z, tokens_or_dense(s, T, D), tokens_or_dense(s ? s + 2 : s, T, D),
                       tokens_or_dense(s ? s + 4 : s, T, (long long)G * N),
                       tokens_or_dense(s ? s + 6 : s, T, (long long)G * N), tokens_or_dense(s ? s + 8 : s, T, D),
                       A, D_skip, dt_bias, h0, lengths, y, h_T, B, T, D, G, N, dt_softplus != 0, dtype == GDR_BF16,
                       workspace, lengths && zero_tail};
    if (scan_overlap(a)) return GDR_ERR_INVALID_ARG;
    int launches = 0;
    const cudaError_t e = gdr::launch_ssm_scan_fwd(a, static_cast<cudaStream_t>(stream), &launches);
    return finish(e, launches);
}

GDR_API int gdr_ssm_scan_step(const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                              const float *D_skip, const void *z, const float *dt_bias, float *h, void *y,
                              const long long *strides, int B, int D, int G, int N, int dt_softplus, int dtype,
                              void *stream)
{
    if (const int e = scan_sizes(B, 1, D, G, N, dtype)) return e;
    if (any_negative(strides, 5)) return GDR_ERR_INVALID_ARG;
    if (B == 0 || D == 0) return nothing_to_do();
    const void *need[] = {x, dt, A, Bm, Cm, h, y};
    if (any_null(need, 7)) return GDR_ERR_INVALID_ARG;
    const void *rows[] = {x, dt, Bm, Cm, z, y}, *words[] = {D_skip, dt_bias}, *lines[] = {A, h};
    if (any_misaligned(rows, 6, elem_bytes(dtype)) || any_misaligned(words, 2, 4) || any_misaligned(lines, 2, 16))
        return GDR_ERR_ALIGNMENT;
    const long long dense[] = {D, D, (long long)G * N, (long long)G * N, D};
    const long long *s = strides ? strides : dense;
    gdr::ScanArgs a = {x, dt, Bm, Cm, z, {s[0], 0}, {s[1], 0}, {s[2], 0}, {s[3], 0}, {s[4], 0},
                       A, D_skip, dt_bias, nullptr, nullptr, y, h, B, 1, D, G, N, dt_softplus != 0,
                       dtype == GDR_BF16, nullptr, false};
    if (scan_overlap(a)) return GDR_ERR_INVALID_ARG;
    int launches = 0;
    const cudaError_t e = gdr::launch_ssm_scan_step(a, static_cast<cudaStream_t>(stream), &launches);
    return finish(e, launches);
}

GDR_API size_t gdr_ssm_scan_bwd_workspace_size(int B, int T, int D, int G, int N, int dtype)
{
    if (scan_sizes(B, T, D, G, N, dtype) || B == 0 || D == 0) return 0;
    if ((long long)B * (T ? T : 1) * G * N >= (1LL << 38)) return 0;
    return gdr::ssm_scan_bwd_workspace_bytes(B, T, D, G, N);
}

GDR_API int gdr_ssm_scan_bwd(const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                             const float *D_skip, const void *z, const float *dt_bias, const float *h0,
                             const int *lengths, const void *dy, const float *dh_T,
                             void *dx, void *ddt, float *dA, void *dB, void *dC, float *dD, void *dz, float *ddt_bias,
                             float *dh0, const long long *strides, int B, int T, int D, int G, int N, int dt_softplus,
                             int dtype, void *workspace, size_t ws_bytes, void *stream)
{
    if (const int e = scan_sizes(B, T, D, G, N, dtype)) return e;
    if ((long long)B * (T ? T : 1) * G * N >= (1LL << 38)) return GDR_ERR_UNSUPPORTED;
    if (any_negative(strides, 12)) return GDR_ERR_INVALID_ARG;
    if (D == 0) return nothing_to_do();
    const void *need[] = {x, dt, Bm, Cm, dy, dx, ddt, dB, dC};
    if (!A || !dA || (z && B > 0 && T > 0 && !dz) || (B > 0 && T > 0 && any_null(need, 9))) return GDR_ERR_INVALID_ARG;
    const void *rows[] = {x, dt, Bm, Cm, z, dy, dx, ddt, dB, dC, dz};
    const void *words[] = {D_skip, dt_bias, lengths, dD, ddt_bias}, *lines[] = {A, h0, dh_T, dA, dh0, workspace};
    if (any_misaligned(rows, 11, elem_bytes(dtype)) || any_misaligned(words, 5, 4) || any_misaligned(lines, 6, 16))
        return GDR_ERR_ALIGNMENT;
    const size_t ws_need = gdr_ssm_scan_bwd_workspace_size(B, T, D, G, N, dtype);
    if (ws_bytes < ws_need || (ws_need && !workspace)) return GDR_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (B == 0) {   // the sums over no rows
        cudaError_t e = cudaMemsetAsync(dA, 0, sizeof(float) * (size_t)D * N, st);
        if (e == cudaSuccess && dD) e = cudaMemsetAsync(dD, 0, sizeof(float) * (size_t)D, st);
        if (e == cudaSuccess && ddt_bias) e = cudaMemsetAsync(ddt_bias, 0, sizeof(float) * (size_t)D, st);
        return finish(e, 0);
    }
    const long long *s = strides;
    gdr::ScanBwdArgs a = {
        {x, dt, Bm, Cm, z, tokens_or_dense(s, T, D), tokens_or_dense(s ? s + 2 : s, T, D),
         tokens_or_dense(s ? s + 4 : s, T, (long long)G * N), tokens_or_dense(s ? s + 6 : s, T, (long long)G * N),
         tokens_or_dense(s ? s + 8 : s, T, D), A, D_skip, dt_bias, h0, lengths, nullptr, nullptr, B, T, D, G, N,
         dt_softplus != 0, dtype == GDR_BF16, nullptr, false},
        dy, tokens_or_dense(s ? s + 10 : s, T, D), dh_T, dx, ddt, dB, dC, z ? dz : nullptr, dA, dD, ddt_bias, dh0,
        workspace};
    int launches = 0;
    const cudaError_t e = gdr::launch_ssm_scan_bwd(a, st, &launches);
    return finish(e, launches);
}
