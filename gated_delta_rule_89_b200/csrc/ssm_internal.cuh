// Declarations shared by the short causal convolution and the selective state
// space scan: argument structures (already validated by the C entry points),
// launchers, and the scalar functions both use.
#pragma once

#include <atomic>

#include "gdr_internal.cuh"

namespace gdr {

// Element strides of a [B, H, T, d] tensor whose last dimension is dense.
struct RowStrides {
    long long b, h, t;
};

// Short causal depthwise convolution; D = H * d channels, channel c = h * d + j.
struct ConvArgs {
    const void *x;
    RowStrides xs;
    const float *weight, *bias;   // [D, W]; [D] or NULL
    const void *state;            // [B, W-1, D] or NULL (zeros)
    const int *lengths;           // [B] or NULL (every row has T tokens)
    void *y, *state_out;          // [B, H, T, d]; [B, W-1, D] or NULL
    int B, H, T, d, W;
    bool silu, bf16;
    bool zero_tail;               // y is set to zero behind a row's end (otherwise left as it is)
};

struct ConvBwdArgs {
    const void *x, *dy;
    RowStrides xs, dys, dxs;
    const float *weight, *bias;
    const void *state, *dstate_out;
    const int *lengths;
    void *dx, *dstate;            // dstate [B, W-1, D] or NULL
    float *dweight, *dbias;       // [D, W]; [D] or NULL
    int B, H, T, d, W;
    bool silu, bf16;
    void *workspace;              // short_conv_bwd_workspace_bytes()
};

cudaError_t launch_short_conv_fwd(const ConvArgs &a, cudaStream_t stream, int *launches);
cudaError_t launch_short_conv_step(const ConvArgs &a, cudaStream_t stream, int *launches);
cudaError_t launch_short_conv_bwd(const ConvBwdArgs &a, cudaStream_t stream, int *launches);
size_t short_conv_bwd_workspace_bytes(int B, int H, int T, int d, int W);

// Selective state space scan.  x, dt, z, y [B, T, D]; Bm, Cm [B, T, G, N];
// strides in elements, the last dimension (the last two of Bm and Cm) dense.
struct BatchToken {
    long long b, t;
};
struct ScanArgs {
    const void *x, *dt, *Bm, *Cm, *z;             // z NULL: no output gate
    BatchToken xs, dts, bs, cs, zs;
    const float *A, *D_skip, *dt_bias, *h0;       // [D, N]; [D] or NULL; [D] or NULL; [B, D, N] or NULL
    const int *lengths;
    void *y;                                      // [B, T, D] dense
    float *h_T;                                   // [B, D, N] or NULL
    int B, T, D, G, N;
    bool softplus, bf16;
    void *workspace;                              // ssm_scan_fwd_workspace_bytes()
    bool zero_tail;                               // as ConvArgs
};

cudaError_t launch_ssm_scan_fwd(const ScanArgs &a, cudaStream_t stream, int *launches);
// one token: x, dt, z, y [B, D], Bm, Cm [B, G, N] (the .t strides unused); h_T is updated in place
cudaError_t launch_ssm_scan_step(const ScanArgs &a, cudaStream_t stream, int *launches);
size_t ssm_scan_fwd_workspace_bytes(int B, int T, int D, int G, int N);

// The states ahead of every kCheckpoint-th token: [B][ceil(T / kCheckpoint)][D][N]
// (those of tokens that a row does not have are not written).  Only the inputs
// of the recurrence are read (x, dt, Bm, A, dt_bias, h0); a.workspace as for
// launch_ssm_scan_fwd.
constexpr int kCheckpoint = 8;
cudaError_t launch_ssm_scan_checkpoints(const ScanArgs &a, float *states, cudaStream_t stream, int *launches);

// For rows cut into `pieces` of `tokens` (a multiple of 32): what pieces 1 ..
// pieces - 1 hand to the one ahead of them as the gradient of the state when
// nothing comes from behind (slots[piece][B][D][N]) and their sums of delta
// (sums[piece][B][D]).  `a` holds dy as x, Cm as Bm, and dt, A, z, dt_bias,
// lengths of the forward.  Pieces behind a row's end are not written.
cudaError_t launch_ssm_scan_adjoint(const ScanArgs &a, int pieces, int tokens, float *slots, float *sums,
                                    cudaStream_t stream, int *launches);

struct ScanBwdArgs {
    ScanArgs f;                                   // the forward's inputs (y, h_T unused)
    const void *dy;
    BatchToken dys;
    const float *dh_T;                            // [B, D, N] or NULL
    void *dx, *ddt, *dB, *dC, *dz;                // dense; dz NULL without a gate
    float *dA, *dD, *ddt_bias, *dh0;              // dD, ddt_bias, dh0 may be NULL
    void *workspace;                              // ssm_scan_bwd_workspace_bytes()
};
cudaError_t launch_ssm_scan_bwd(const ScanBwdArgs &a, cudaStream_t stream, int *launches);
size_t ssm_scan_bwd_workspace_bytes(int B, int T, int D, int G, int N);

constexpr float kLog2e = 1.4426950408889634f;

// 2^x, from the hardware's approximation: measured over [-16, 0] it is off by
// at most 1.5e-7 of the value and 5e-8 at the mean, about the rounding of its
// fp32 result.
__device__ __forceinline__ float exp2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float sigmoid_f32(float x) { return rcp_approx(1.f + exp2_approx(-kLog2e * x)); }

// Two fp32 in a 64-bit register pair: one issue slot for two products.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 make_f32x2(float lo, float hi)
{
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float lo_f32(f32x2 v) { return __uint_as_float((unsigned)v); }
__device__ __forceinline__ float hi_f32(f32x2 v) { return __uint_as_float((unsigned)(v >> 32)); }
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 both(float v) { return make_f32x2(v, v); }
__device__ __forceinline__ f32x2 exp2_approx2(f32x2 x)
{
    return make_f32x2(exp2_approx(lo_f32(x)), exp2_approx(hi_f32(x)));
}
// The same operations on one value, for code written for either.
__device__ __forceinline__ float mul2(float a, float b) { return a * b; }
__device__ __forceinline__ float add2(float a, float b) { return a + b; }
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float sigmoid2(float x) { return sigmoid_f32(x); }
__device__ __forceinline__ f32x2 sigmoid2(f32x2 x)
{
    const f32x2 d = add2(exp2_approx2(mul2(x, both(-kLog2e))), both(1.f));
    return make_f32x2(rcp_approx(lo_f32(d)), rcp_approx(hi_f32(d)));
}
// VEC values as register pairs, or one value.
template <int VEC> struct Lanes {
    using P = f32x2;
    static constexpr int N = VEC / 2;
    static __device__ __forceinline__ P all(float v) { return both(v); }
    static __device__ __forceinline__ void join(const float *f, P *p)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = make_f32x2(f[2 * i], f[2 * i + 1]);
    }
    static __device__ __forceinline__ void split(const P *p, float *f)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) f[2 * i] = lo_f32(p[i]), f[2 * i + 1] = hi_f32(p[i]);
    }
};
template <> struct Lanes<1> {
    using P = float;
    static constexpr int N = 1;
    static __device__ __forceinline__ P all(float v) { return v; }
    static __device__ __forceinline__ void join(const float *f, P *p) { p[0] = f[0]; }
    static __device__ __forceinline__ void split(const P *p, float *f) { f[0] = p[0]; }
};

// The decay 2^(delta A2) of a state, and of two.  The hardware's 2^x lies below the
// exact value by 2e-8 at the mean where it is close to 1, and a slowly
// decaying state multiplies a thousand of them; raising the exponent by 2e-8
// leaves a mean error under 1e-8 between 2^-16 and 2^-1 (measured), at no
// cost, and 2^(2e-8) is still exactly 1, so a time step of 0 keeps the state.
__device__ __forceinline__ float decay(float delta, float A2) { return exp2_approx(fmaf(delta, A2, 2e-8f)); }
__device__ __forceinline__ f32x2 decay2(f32x2 delta, f32x2 A2)
{
    return exp2_approx2(fma2(delta, A2, both(2e-8f)));
}

// decay2(delta, A2) h + v for the decay over a whole piece of a row.  Where a
// state grows, that decay can pass fp32's range while the state is 0 or tiny
// (0 has to stay 0), so what is above 2^126 goes to h first; elsewhere h is
// multiplied by exactly 1.
__device__ __forceinline__ f32x2 fold2(f32x2 delta, f32x2 A2, f32x2 h, f32x2 v)
{
    const f32x2 e = fma2(delta, A2, both(2e-8f));
    const float lo = lo_f32(e), hi = hi_f32(e);
    const f32x2 above = make_f32x2(fminf(fmaxf(lo - 126.f, 0.f), 127.f), fminf(fmaxf(hi - 126.f, 0.f), 127.f));
    return fma2(exp2_approx2(make_f32x2(fminf(lo, 126.f), fminf(hi, 126.f))), mul2(exp2_approx2(above), h), v);
}

// log(1 + e) for e in [0, 1], as e times a polynomial of degree 9 in e (a
// weighted least-squares fit to log(1 + e) / e; with the coefficients rounded
// to fp32 its relative error is 4e-8, and evaluated in fp32 1.6e-7).  A logarithm of
// 1 + e would lose the digits of a small e in the sum; and time steps of 1e-3
// have an e of 1e-3.  It also spares the special-function pipe one operation.
// (One value at a time: the coefficients are then immediate operands, while
// the packed form wants each of them in a register pair.)
__device__ __forceinline__ float log1p_unit(float e)
{
    float p = -0.0032440515f;
    p = fmaf(p, e, 0.01985158f);
    p = fmaf(p, e, -0.056959756f);
    p = fmaf(p, e, 0.106036775f);
    p = fmaf(p, e, -0.15305606f);
    p = fmaf(p, e, 0.19675943f);
    p = fmaf(p, e, -0.24954134f);
    p = fmaf(p, e, 0.33329964f);
    p = fmaf(p, e, -0.49999902f);
    p = fmaf(p, e, 1.f);
    return p * e;
}
// log(1 + exp(x)) = max(x, 0) + log(1 + exp(-|x|)); a NaN stays one.  `e`
// receives exp(-|x|).
__device__ __forceinline__ float softplus_f32(float x, float &e)
{
    e = exp2_approx(-kLog2e * fabsf(x));
    return fmaxf(x, 0.f) + log1p_unit(e);
}

// Sums v[0..COUNT) over the lanes that differ in the bits from MASK up to
// END / 2.  Each step a lane hands half of its values to its partner and keeps
// the other half, so COUNT / (lanes) values stay with every lane (one,
// replicated, when the lanes outnumber the values); `which` is the first index
// it kept.
template <int COUNT, int MASK, int END>
__device__ __forceinline__ void lane_sums(float *v, int lane, int &which)
{
    if constexpr (MASK < END) {
        if constexpr (COUNT > 1) {
            constexpr int H = COUNT / 2;
            const bool up = lane & MASK;
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float send = up ? v[i] : v[i + H], keep = up ? v[i + H] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, MASK);
            }
            if (up) which += H;
            lane_sums<H, MASK * 2, END>(v, lane, which);
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], MASK);
            lane_sums<1, MASK * 2, END>(v, lane, which);
        }
    }
}

// N consecutive elements from / to memory as fp32.  VECTOR: one access of
// N * sizeof(T) bytes (aligned to that); otherwise one access per element.
template <typename T, int N> struct Pack;
template <> struct Pack<float, 4> { using V = float4; };
template <> struct Pack<__nv_bfloat16, 4> { using V = uint2; };
template <> struct Pack<__nv_bfloat16, 8> { using V = uint4; };
template <> struct Pack<float, 1> { using V = float; };
template <> struct Pack<__nv_bfloat16, 1> { using V = unsigned short; };

// The two bf16 of a 32-bit word are widened by a shift and a mask.
__device__ __forceinline__ float bf16_lo(unsigned w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(unsigned w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ unsigned bf16_pair(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const unsigned *>(&p);
}

__device__ __forceinline__ void unpack(float4 v, float *f) { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }
__device__ __forceinline__ void unpack(uint2 v, float *f)
{
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
}
__device__ __forceinline__ void unpack(uint4 v, float *f)
{
    unpack(make_uint2(v.x, v.y), f);
    unpack(make_uint2(v.z, v.w), f + 4);
}
__device__ __forceinline__ void unpack(float v, float *f) { f[0] = v; }
__device__ __forceinline__ void unpack(unsigned short v, float *f) { f[0] = bf16_lo(v); }
__device__ __forceinline__ void pack(float4 &v, const float *f) { v = make_float4(f[0], f[1], f[2], f[3]); }
__device__ __forceinline__ void pack(uint2 &v, const float *f)
{
    v = make_uint2(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]));
}
__device__ __forceinline__ void pack(uint4 &v, const float *f)
{
    v = make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
}
__device__ __forceinline__ void pack(float &v, const float *f) { v = f[0]; }
__device__ __forceinline__ void pack(unsigned short &v, const float *f) { v = (unsigned short)bf16_pair(f[0], 0.f); }

template <typename V> __device__ __forceinline__ V zero_pack();
template <> __device__ __forceinline__ float4 zero_pack<float4>() { return make_float4(0.f, 0.f, 0.f, 0.f); }
template <> __device__ __forceinline__ uint2 zero_pack<uint2>() { return make_uint2(0u, 0u); }
template <> __device__ __forceinline__ float zero_pack<float>() { return 0.f; }
template <> __device__ __forceinline__ unsigned short zero_pack<unsigned short>() { return 0; }

// The number of tokens of row b: T, or lengths[b] brought into [0, T].
__device__ __forceinline__ int row_length(const int *lengths, int b, int T)
{
    return lengths ? min(max(lengths[b], 0), T) : T;
}

// A read-only load that a predicate can leave out (then 0), without a branch:
// a thread's loads stay together instead of waiting for one another.
__device__ __forceinline__ float4 load_if(const float4 *p, bool on)
{
    float4 v;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\t"
        "mov.b32 %3, 0;\n\t@p ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&f"(v.x), "=&f"(v.y), "=&f"(v.z), "=&f"(v.w) : "l"(p), "r"((int)on));
    return v;
}
__device__ __forceinline__ uint2 load_if(const uint2 *p, bool on)
{
    uint2 v;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
        "@p ld.global.nc.v2.u32 {%0, %1}, [%2];\n\t}"
        : "=&r"(v.x), "=&r"(v.y) : "l"(p), "r"((int)on));
    return v;
}
__device__ __forceinline__ float load_if(const float *p, bool on)
{
    float v;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.nc.f32 %0, [%1];\n\t}"
        : "=&f"(v) : "l"(p), "r"((int)on));
    return v;
}
__device__ __forceinline__ unsigned short load_if(const unsigned short *p, bool on)
{
    unsigned short v;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %2, 0;\n\tmov.b16 %0, 0;\n\t@p ld.global.nc.u16 %0, [%1];\n\t}"
        : "=&h"(v) : "l"(p), "r"((int)on));
    return v;
}

// A read-only load that stays where it is written, ahead of the work that hides it.
__device__ __forceinline__ float4 load_always(const float4 *p)
{
    float4 v;
    asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 load_always(const uint2 *p)
{
    uint2 v;
    asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// 4 consecutive elements, of which the first `valid` exist (the rest are 0).
// VECTOR: groups are whole and aligned, so valid is <= 0 or >= 4.  ALL: they
// all exist.
template <typename T, bool VECTOR, bool ALL = false>
__device__ __forceinline__ typename Pack<T, 4>::V load4(const T *p, int valid)
{
    using V = typename Pack<T, 4>::V;
    if constexpr (VECTOR && ALL) {
        return load_always((const V *)p);
    } else if constexpr (VECTOR) {
        return load_if((const V *)p, valid > 0);
    } else {
        using E = typename Pack<T, 1>::V;
        float f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) unpack(load_if((const E *)p + k, k < valid), f + k);
        V v;
        pack(v, f);
        return v;
    }
}
template <typename T, bool VECTOR>
__device__ __forceinline__ void store4(T *p, const float *f, int valid)
{
    using V = typename Pack<T, 4>::V;
    if (VECTOR) {
        if (valid > 0) {
            V v;
            pack(v, f);
            *(V *)p = v;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < valid) p[k] = from_f32<T>(f[k]);
    }
}

// 4 states' B or C as they lie in shared memory, in the inputs' type, and in
// two register pairs.  bf16 is widened by the lanes: 8 integer operations, but
// half the shared-memory traffic, which otherwise bounds the scan.
template <typename T> struct Quad;
template <> struct Quad<float> {
    ulonglong2 v;
    __device__ __forceinline__ f32x2 lo() const { return v.x; }
    __device__ __forceinline__ f32x2 hi() const { return v.y; }
};
template <> struct Quad<__nv_bfloat16> {
    uint2 v;
    __device__ __forceinline__ f32x2 lo() const { return make_f32x2(bf16_lo(v.x), bf16_hi(v.x)); }
    __device__ __forceinline__ f32x2 hi() const { return make_f32x2(bf16_lo(v.y), bf16_hi(v.y)); }
};

// Lets `kernel` have `bytes` of shared memory; `done` (one for each kernel)
// holds the devices where that has been said.
template <typename K>
cudaError_t allow_shared(K kernel, size_t bytes, std::atomic<unsigned long long> &done)
{
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = device < 64 ? 1ull << device : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

inline bool aligned_to(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

}  // namespace gdr
