// Selective state space scan: prompt and single token.
//
// For every batch row, channel d (in group g = d / (D/G)) and state n < N:
//
//   delta_t = softplus(dt_t[d] + dt_bias[d])              (or without the softplus)
//   h_t[n]  = exp(delta_t A[d,n]) h_{t-1}[n] + delta_t x_t[d] B_t[g,n]
//   y_t[d]  = (sum_n C_t[g,n] h_t[n] + D_skip[d] x_t[d]) * silu(z_t[d])
//
// It is the diagonal relative of the gated delta rule's recurrence ("Token
// Mixer I", section "Mamba2: Linear Attention with Decay", with a decay of
// its own for every channel and state and no delta term).
//
// Every (token, channel, state) costs one exponential, and the special
// function pipe gives 16 of them per clock and SM: with N = 16 that is 12
// times what the same pipe would need for the tensors' bytes at HBM speed, so
// the prompt form is bound by exponentials, not by HBM.  The rest of the work
// is arranged to fit into the issue slots beside them.
#include "ssm_internal.cuh"

namespace gdr {
namespace {

constexpr int kSms = 148;
constexpr int kScanLanes = 128;            // scan threads of a block: 4 states each
constexpr int kScanThreads = 2 * kScanLanes;
constexpr int kTile = 32;                  // tokens between two block barriers

// A block's share and its shared memory for state size N.
template <int N> struct Shape {
    static constexpr int LPC = N / 4;                    // scan lanes of a channel
    static constexpr int CB = kScanLanes / LPC;          // channels of a block
    static constexpr int GR = CB / 4;                    // groups of 4 channels
    static constexpr int TPP = kScanLanes / GR;          // tokens the helpers cover at a time
    static constexpr int R = TPP >= kTile ? 1 : kTile / TPP;
    static constexpr int GRB = N / 4;                    // groups of 4 states
    static constexpr int TPB = kScanLanes / GRB;
    static constexpr int RB = TPB >= kTile ? 1 : kTile / TPB;
    static constexpr int P = kTile * CB * 4;             // floats: {delta, delta, u, u} per (token, channel)
    static constexpr int S = kTile * N;                  // floats: B, and as many for C
    static constexpr int Y = kTile * kScanLanes;         // floats: partial sums of C h
    static constexpr int BUF = P + 2 * S + Y;
    static constexpr size_t smem = 2 * BUF * sizeof(float);
};

// Shared-memory position of a 16-byte chunk: the helpers touch every 4th
// (N = 16) chunk at a time, the scan lanes consecutive ones; with two bits of
// the row of 8 folded in, both meet 8 different banks.
__device__ __forceinline__ int swz(int chunk) { return chunk ^ ((chunk >> 3) & 3); }

enum Mode {
    FULL,    // the outputs and the final state
    LOCAL,   // the state that a piece of a row ends with when it starts from zero
    POINTS   // the states ahead of every kCheckpoint-th token, for the backward
};

// pieces of a row (time is split when there are few channels), tokens of a
// piece, and the piece states: slot [s][B][D][N] is what piece s starts from
// (slot 0: h0) before the pieces ahead of it are folded in, and
// sums [s][B][D] the sum of delta over piece s - 1.
struct Pieces {
    int count, tokens;
    float *slots, *sums;
    float *points;   // POINTS: [B][ceil(T / kCheckpoint)][D][N]
};

template <typename T, int N, bool VECTOR, Mode MODE>
__global__ void __launch_bounds__(kScanThreads)
ssm_scan_kernel(const ScanArgs a, const Pieces pc, int blocks_per_group)
{
    using S = Shape<N>;
    using V = typename Pack<T, 4>::V;
    extern __shared__ __align__(16) float sm[];

    const int per_row = blocks_per_group * a.G;
    const int b = blockIdx.x / per_row;
    const int gi = (blockIdx.x - b * per_row) / blocks_per_group;
    const int cpg = a.D / a.G;
    const int cfirst = gi * cpg + (blockIdx.x - b * per_row - gi * blocks_per_group) * S::CB;
    const int cend = min(cfirst + S::CB, (gi + 1) * cpg);     // channels [cfirst, cend)
    const int piece = blockIdx.y;
    const int len = row_length(a.lengths, b, a.T);
    const int t0 = piece * pc.tokens, t1 = min(t0 + pc.tokens, len);
    if (piece > 0 && t0 >= t1) return;                        // the whole block
    const int tiles = t1 > t0 ? (t1 - t0 + kTile - 1) / kTile : 0;
    const int tid = threadIdx.x;

    if (tid < kScanLanes) {
        // -------------------------------------------------- the recurrence
        const int ch = tid / S::LPC, n0 = (tid % S::LPC) * 4;
        const int c = cfirst + ch;
        const bool on = c < cend;
        const size_t slot = (size_t)a.B * a.D * N, at = ((size_t)b * a.D + c) * N + n0;
        float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
        f32x2 A0 = 0, A1 = 0;
        if (on) {
            const float4 A = *(const float4 *)(a.A + (size_t)c * N + n0);
            A0 = make_f32x2(A.x * kLog2e, A.y * kLog2e);
            A1 = make_f32x2(A.z * kLog2e, A.w * kLog2e);
            if (MODE == LOCAL) {
                if (piece == 0) {
                    // the second pass reads h0 from the slot, so that h_T may be the same buffer
                    if (a.h0) h = *(const float4 *)(a.h0 + at);
                    *(float4 *)(pc.slots + at) = h;
                    h = make_float4(0.f, 0.f, 0.f, 0.f);
                }
            } else if (pc.count > 1) {
                h = *(const float4 *)(pc.slots + at);
            } else if (a.h0) {
                h = *(const float4 *)(a.h0 + at);
            }
        }
        f32x2 h0 = make_f32x2(h.x, h.y), h1 = make_f32x2(h.z, h.w);
        if (MODE != LOCAL && on)
            for (int s = 1; s <= piece; ++s) {   // fold in the pieces ahead
                const float sum = pc.sums[((size_t)s * a.B + b) * a.D + c];
                const float4 q = *(const float4 *)(pc.slots + s * slot + at);
                const f32x2 ss = make_f32x2(sum, sum);
                h0 = fma2(decay2(ss, A0), h0, make_f32x2(q.x, q.y));
                h1 = fma2(decay2(ss, A1), h1, make_f32x2(q.z, q.w));
            }
        float sum = 0.f;
        float *points = nullptr;
        if (MODE == POINTS)
            points = pc.points + (((size_t)b * ((a.T + kCheckpoint - 1) / kCheckpoint) + t0 / kCheckpoint) * a.D + c) * N + n0;
        __syncthreads();
        // Four tokens' operands are loaded ahead of the four in work, and ahead of the stores of
        // their outputs: shared-memory loads are not moved across stores, and a warp that waited
        // for each token's loads would spend most of its time there.
        constexpr int G = 4;
        struct Token {
            ulonglong2 du, b, c;
        };
        for (int i = 0; i < tiles; ++i) {
            const float *buf = sm + (i & 1) * S::BUF;
            const float *p = buf + swz(ch) * 4, *sb = buf + S::P + n0, *sc = sb + S::S;
            float *py = sm + (i & 1) * S::BUF + S::P + 2 * S::S + swz(tid >> 2) * 4 + (tid & 3);
            Token now[G], next[G];
            auto fetch = [&](Token *k, int t) {
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    k[j].du = *(const ulonglong2 *)(p + (t + j) * S::CB * 4);
                    k[j].b = *(const ulonglong2 *)(sb + (t + j) * N);
                    if (MODE == FULL) k[j].c = *(const ulonglong2 *)(sc + (t + j) * N);
                }
            };
            fetch(now, 0);
#pragma unroll
            for (int t = 0; t < kTile; t += G) {
                if (MODE == POINTS && t % kCheckpoint == 0 && on && t0 + i * kTile + t < t1)
                    *(ulonglong2 *)(points + (size_t)(i * kTile + t) / kCheckpoint * a.D * N) = make_ulonglong2(h0, h1);
                if (t + G < kTile) fetch(next, t + G);
                float y[G];
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    const Token &k = now[j];
                    h0 = fma2(decay2(k.du.x, A0), h0, mul2(k.du.y, k.b.x));
                    h1 = fma2(decay2(k.du.x, A1), h1, mul2(k.du.y, k.b.y));
                    if (MODE == FULL) {
                        const f32x2 s = fma2(h1, k.c.y, mul2(h0, k.c.x));
                        y[j] = lo_f32(s) + hi_f32(s);
                    } else if (MODE == LOCAL) {
                        sum += lo_f32(k.du.x);
                    }
                }
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    if (MODE == FULL) py[(t + j) * kScanLanes] = y[j];
                    now[j] = next[j];
                }
            }
            __syncthreads();
        }
        h = make_float4(lo_f32(h0), hi_f32(h0), lo_f32(h1), hi_f32(h1));
        if (on && MODE == LOCAL) {
            *(float4 *)(pc.slots + (piece + 1) * slot + at) = h;
            if (n0 == 0) pc.sums[((size_t)(piece + 1) * a.B + b) * a.D + c] = sum;
        }
        if (on && MODE == FULL && a.h_T && (t1 == len || pc.count == 1)) *(float4 *)(a.h_T + at) = h;
    } else {
        // ------------- loads, time steps and outputs, one tile ahead and behind
        const int ht = tid - kScanLanes;
        const int gr = ht % S::GR, tok = ht / S::GR;           // 4 channels, token of a pass
        const int grb = ht % S::GRB, tokb = ht / S::GRB;       // 4 states
        const int c = cfirst + gr * 4;
        const int have = cend - c;                             // channels of the group that exist
        // every group of 4 whole: the tiles that lie inside the piece take no bounds checks
        const bool whole = cfirst + S::CB <= cend;
        // running pointers to this thread's first element of the tile that is fetched next
        const long long first = (long long)t0 + tok, firstb = (long long)t0 + tokb;
        const T *px = (const T *)a.x + b * a.xs.b + c + first * a.xs.t;
        const T *pdt = (const T *)a.dt + b * a.dts.b + c + first * a.dts.t;
        const T *pB = (const T *)a.Bm + b * a.bs.b + (size_t)gi * N + grb * 4 + firstb * a.bs.t;
        const T *pC = (const T *)a.Cm + b * a.cs.b + (size_t)gi * N + grb * 4 + firstb * a.cs.t;
        const T *pxo = px;                                     // and of the tile that is finished next
        const T *pzo = a.z ? (const T *)a.z + b * a.zs.b + c + first * a.zs.t : nullptr;
        T *py = (T *)a.y + ((size_t)b * a.T + first) * a.D + c;
        f32x2 bias[2], skip[2];
        {
            float f[4], g[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                f[v] = a.dt_bias && v < have ? a.dt_bias[c + v] : 0.f;
                g[v] = MODE == FULL && a.D_skip && v < have ? a.D_skip[c + v] : 0.f;
            }
            bias[0] = make_f32x2(f[0], f[1]), bias[1] = make_f32x2(f[2], f[3]);
            skip[0] = make_f32x2(g[0], g[1]), skip[1] = make_f32x2(g[2], g[3]);
        }

        V rx[S::R], rdt[S::R], rB[S::RB], rC[S::RB], ex[S::R], ez[S::R];
        auto fetch = [&](int tile) {
            const int tb = t0 + tile * kTile;
            const bool full = whole && tb + kTile <= t1;
#pragma unroll
            for (int r = 0; r < S::R; ++r) {
                const int k = tok + r * S::TPP;
                const int valid = full && S::TPP <= kTile ? 4 : k < kTile && tb + k < t1 ? have : 0;
                rx[r] = load4<T, VECTOR>(px + r * S::TPP * a.xs.t, valid);
                rdt[r] = load4<T, VECTOR>(pdt + r * S::TPP * a.dts.t, valid);
            }
#pragma unroll
            for (int r = 0; r < S::RB; ++r) {
                const int k = tokb + r * S::TPB;
                const int valid = full && S::TPB <= kTile ? 4 : k < kTile && tb + k < t1 ? 4 : 0;
                rB[r] = load4<T, VECTOR>(pB + r * S::TPB * a.bs.t, valid);
                if (MODE == FULL) rC[r] = load4<T, VECTOR>(pC + r * S::TPB * a.cs.t, valid);
            }
            px += kTile * a.xs.t;
            pdt += kTile * a.dts.t;
            pB += kTile * a.bs.t;
            pC += kTile * a.cs.t;
        };
        auto fetch_out = [&](int tile) {
            const int tb = t0 + tile * kTile;
            const bool full = whole && tb + kTile <= t1;
#pragma unroll
            for (int r = 0; r < S::R; ++r) {
                const int k = tok + r * S::TPP;
                const int valid = full && S::TPP <= kTile ? 4 : k < kTile && tb + k < t1 ? have : 0;
                if (a.D_skip) ex[r] = load4<T, VECTOR>(pxo + r * S::TPP * a.xs.t, valid);
                if (pzo) ez[r] = load4<T, VECTOR>(pzo + r * S::TPP * a.zs.t, valid);
            }
            pxo += kTile * a.xs.t;
            if (pzo) pzo += kTile * a.zs.t;
        };
        auto prepare = [&](int tile) {
            float *buf = sm + (tile & 1) * S::BUF;
            const int tb = t0 + tile * kTile;
            const bool full = whole && tb + kTile <= t1;
#pragma unroll
            for (int r = 0; r < S::R; ++r) {
                const int k = tok + r * S::TPP;
                if (S::TPP > kTile && k >= kTile) continue;
                float fx[4], fd[4];
                unpack(rx[r], fx);
                unpack(rdt[r], fd);
                float *q = buf + k * S::CB * 4;
#pragma unroll
                for (int v = 0; v < 4; v += 2) {
                    f32x2 e, d = add2(make_f32x2(fd[v], fd[v + 1]), bias[v / 2]);
                    if (a.softplus) d = softplus2(d, e);
                    if (!full) {                               // the state stands still
                        const bool live = tb + k < t1;
                        d = make_f32x2(live && v < have ? lo_f32(d) : 0.f, live && v + 1 < have ? hi_f32(d) : 0.f);
                    }
                    const f32x2 u = mul2(d, make_f32x2(fx[v], fx[v + 1]));
                    *(float4 *)(q + swz(gr * 4 + v) * 4) = make_float4(lo_f32(d), lo_f32(d), lo_f32(u), lo_f32(u));
                    *(float4 *)(q + swz(gr * 4 + v + 1) * 4) = make_float4(hi_f32(d), hi_f32(d), hi_f32(u), hi_f32(u));
                }
            }
#pragma unroll
            for (int r = 0; r < S::RB; ++r) {
                const int k = tokb + r * S::TPB;
                if (S::TPB > kTile && k >= kTile) continue;
                float f[4];
                unpack(rB[r], f);
                *(float4 *)(buf + S::P + k * N + grb * 4) = make_float4(f[0], f[1], f[2], f[3]);
                if (MODE == FULL) {
                    unpack(rC[r], f);
                    *(float4 *)(buf + S::P + S::S + k * N + grb * 4) = make_float4(f[0], f[1], f[2], f[3]);
                }
            }
        };
        auto finish = [&](int tile) {
            const float *y = sm + (tile & 1) * S::BUF + S::P + 2 * S::S;
            const int tb = t0 + tile * kTile;
            const bool full = whole && tb + kTile <= t1;
#pragma unroll
            for (int r = 0; r < S::R; ++r) {
                const int k = tok + r * S::TPP;
                if (!full && tb + k >= t1) continue;
                if (S::TPP > kTile && k >= kTile) continue;
                float part[N];                                  // the LPC partial sums of 4 channels
#pragma unroll
                for (int q = 0; q < N / 4; ++q)
                    *(float4 *)(part + 4 * q) = *(const float4 *)(y + k * kScanLanes + swz(gr * (N / 4) + q) * 4);
                float out[4], fx[4], fz[4];
                unpack(ex[r], fx);
                unpack(ez[r], fz);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    float s = part[v * S::LPC];
#pragma unroll
                    for (int l = 1; l < S::LPC; ++l) s += part[v * S::LPC + l];
                    out[v] = s;
                }
#pragma unroll
                for (int v = 0; v < 4; v += 2) {
                    f32x2 s = make_f32x2(out[v], out[v + 1]);
                    if (a.D_skip) s = fma2(skip[v / 2], make_f32x2(fx[v], fx[v + 1]), s);
                    if (pzo)
                        s = mul2(s, mul2(make_f32x2(fz[v], fz[v + 1]),
                                         make_f32x2(sigmoid_f32(fz[v]), sigmoid_f32(fz[v + 1]))));
                    out[v] = lo_f32(s);
                    out[v + 1] = hi_f32(s);
                }
                store4<T, VECTOR>(py + (size_t)(r * S::TPP) * a.D, out, full ? 4 : have);
            }
            py += (size_t)kTile * a.D;
        };

        if (tiles) {
            fetch(0);
            prepare(0);
            if (tiles > 1) fetch(1);
        }
        __syncthreads();
        for (int i = 0; i < tiles; ++i) {
            if (i + 1 < tiles) prepare(i + 1);
            if (i + 2 < tiles) fetch(i + 2);
            if (MODE == FULL) {
                if (i > 0) finish(i - 1);
                fetch_out(i);
            }
            __syncthreads();
        }
        if (MODE == FULL && tiles) finish(tiles - 1);
    }
}

// ------------------------------------------------------------ single token
//
// The state is read once and written once (8 N bytes a channel) and bounds
// the step; a thread owns 4 states, so a warp's accesses are whole lines.
template <typename T, int N>
__global__ void __launch_bounds__(256) ssm_step_kernel(const ScanArgs a, int blocks_per_row)
{
    constexpr int LPC = N / 4, CB = 256 / LPC;
    const int b = blockIdx.x / blocks_per_row;
    const int c = (blockIdx.x - b * blocks_per_row) * CB + threadIdx.x / LPC;
    const int n0 = (threadIdx.x % LPC) * 4;
    const bool on = c < a.D;
    float y = 0.f;
    if (on) {
        float4 *ph = (float4 *)(a.h_T + ((size_t)b * a.D + c) * N + n0);
        const float4 h = __ldcs(ph);
        const float4 A = *(const float4 *)(a.A + (size_t)c * N + n0);
        const float x = to_f32<T>(((const T *)a.x)[b * a.xs.b + c]);
        float d = to_f32<T>(((const T *)a.dt)[b * a.dts.b + c]);
        const int g = c / (a.D / a.G);
        const T *pB = (const T *)a.Bm + b * a.bs.b + (size_t)g * N + n0;
        const T *pC = (const T *)a.Cm + b * a.cs.b + (size_t)g * N + n0;
        if (a.dt_bias) d += a.dt_bias[c];
        if (a.softplus) {
            f32x2 e;
            d = lo_f32(softplus2(both(d), e));
        }
        const float u = d * x, d2 = d * kLog2e;
        float4 r;
        r.x = fmaf(exp2_approx(d2 * A.x), h.x, u * to_f32<T>(pB[0]));
        r.y = fmaf(exp2_approx(d2 * A.y), h.y, u * to_f32<T>(pB[1]));
        r.z = fmaf(exp2_approx(d2 * A.z), h.z, u * to_f32<T>(pB[2]));
        r.w = fmaf(exp2_approx(d2 * A.w), h.w, u * to_f32<T>(pB[3]));
        __stcs(ph, r);
        y = to_f32<T>(pC[0]) * r.x;
        y = fmaf(to_f32<T>(pC[1]), r.y, y);
        y = fmaf(to_f32<T>(pC[2]), r.z, y);
        y = fmaf(to_f32<T>(pC[3]), r.w, y);
        if (n0 == 0 && a.D_skip) y = fmaf(a.D_skip[c], x, y);
    }
#pragma unroll
    for (int o = LPC / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (on && n0 == 0) {
        if (a.z) {
            const float z = to_f32<T>(((const T *)a.z)[b * a.zs.b + c]);
            y *= z * sigmoid_f32(z);
        }
        ((T *)a.y)[(size_t)b * a.D + c] = from_f32<T>(y);
    }
}

// --------------------------------------------------------------- launches

int blocks_per_group(int D, int G, int N)
{
    const int cb = 512 / N;
    return (D / G + cb - 1) / cb;
}

// Few channels leave most of the machine idle; then a row is cut into pieces
// that run side by side: a first pass finds the state each piece would end
// with from a zero start, and the second starts every piece from the states
// ahead of it.  That doubles the exponentials, so it pays from half the
// machine down.
Pieces plan(int B, int T, int D, int G, int N, void *workspace)
{
    Pieces p = {1, T, nullptr, nullptr, nullptr};
    const long long blocks = (long long)B * G * blocks_per_group(D, G, N);
    if (blocks > 0 && blocks * 2 <= kSms && T >= 8 * kTile) {
        long long count = 2 * kSms / blocks;
        if (count > T / (4 * kTile)) count = T / (4 * kTile);
        p.tokens = (int)((T + count - 1) / count + kTile - 1) / kTile * kTile;
        p.count = (T + p.tokens - 1) / p.tokens;
    }
    if (p.count > 1) {
        p.slots = (float *)workspace;
        p.sums = p.slots + (size_t)p.count * B * D * N;
    }
    return p;
}

// 4 elements at a time: every group of 4 channels or states starts on a
// boundary of 4 elements, and belongs to one group of channels.
template <typename T> bool scan_vectors(const ScanArgs &a)
{
    const void *ptrs[] = {a.x, a.dt, a.Bm, a.Cm, a.z, a.y};
    const BatchToken *s[] = {&a.xs, &a.dts, &a.bs, &a.cs, &a.zs};
    if ((a.D / a.G) % 4) return false;
    for (const void *p : ptrs)
        if (p && !aligned_to(p, 4 * sizeof(T))) return false;
    for (const BatchToken *q : s)
        if (q->b % 4 || q->t % 4) return false;
    return true;
}

template <typename T, int N, bool VECTOR, Mode MODE>
cudaError_t run_scan(const ScanArgs &a, const Pieces &p, int pieces, cudaStream_t st)
{
    auto k = ssm_scan_kernel<T, N, VECTOR, MODE>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape<N>::smem);
    if (e != cudaSuccess) return e;
    const int bpg = blocks_per_group(a.D, a.G, N);
    k<<<dim3((unsigned)((long long)a.B * a.G * bpg), pieces), kScanThreads, Shape<N>::smem, st>>>(a, p, bpg);
    return cudaGetLastError();
}

template <typename T, int N, bool VECTOR>
cudaError_t scan_typed(const ScanArgs &a, float *points, cudaStream_t st, int *launches)
{
    Pieces p = plan(a.B, a.T, a.D, a.G, N, a.workspace);
    cudaError_t e = cudaSuccess;
    if (p.count > 1) {
        e = run_scan<T, N, VECTOR, LOCAL>(a, p, p.count - 1, st);
        if (e != cudaSuccess) return e;
        *launches += 1;
    }
    p.points = points;
    e = points ? run_scan<T, N, VECTOR, POINTS>(a, p, p.count, st) : run_scan<T, N, VECTOR, FULL>(a, p, p.count, st);
    if (e == cudaSuccess) *launches += 1;
    return e;
}

template <typename T, int N>
cudaError_t step_typed(const ScanArgs &a, cudaStream_t st)
{
    const int cb = 1024 / N, bpr = (a.D + cb - 1) / cb;
    ssm_step_kernel<T, N><<<(unsigned)((long long)a.B * bpr), 256, 0, st>>>(a, bpr);
    return cudaGetLastError();
}

template <int N>
cudaError_t scan_n(const ScanArgs &a, float *points, cudaStream_t st, int *launches)
{
    if (a.bf16)
        return scan_vectors<__nv_bfloat16>(a) ? scan_typed<__nv_bfloat16, N, true>(a, points, st, launches)
                                              : scan_typed<__nv_bfloat16, N, false>(a, points, st, launches);
    return scan_vectors<float>(a) ? scan_typed<float, N, true>(a, points, st, launches)
                                  : scan_typed<float, N, false>(a, points, st, launches);
}

cudaError_t any_n(const ScanArgs &a, float *points, cudaStream_t st, int *launches)
{
    switch (a.N) {
        case 8: return scan_n<8>(a, points, st, launches);
        case 16: return scan_n<16>(a, points, st, launches);
        case 32: return scan_n<32>(a, points, st, launches);
        default: return scan_n<64>(a, points, st, launches);
    }
}

}  // namespace

size_t ssm_scan_fwd_workspace_bytes(int B, int T, int D, int G, int N)
{
    const Pieces p = plan(B, T, D, G, N, nullptr);
    return p.count > 1 ? (size_t)p.count * B * D * (N + 1) * sizeof(float) : 0;
}

cudaError_t launch_ssm_scan_fwd(const ScanArgs &a, cudaStream_t stream, int *launches)
{
    return any_n(a, nullptr, stream, launches);
}

cudaError_t launch_ssm_scan_checkpoints(const ScanArgs &a, float *states, cudaStream_t stream, int *launches)
{
    return any_n(a, states, stream, launches);
}

cudaError_t launch_ssm_scan_step(const ScanArgs &a, cudaStream_t stream, int *launches)
{
    cudaError_t e;
    switch (a.N) {
        case 8: e = a.bf16 ? step_typed<__nv_bfloat16, 8>(a, stream) : step_typed<float, 8>(a, stream); break;
        case 16: e = a.bf16 ? step_typed<__nv_bfloat16, 16>(a, stream) : step_typed<float, 16>(a, stream); break;
        case 32: e = a.bf16 ? step_typed<__nv_bfloat16, 32>(a, stream) : step_typed<float, 32>(a, stream); break;
        default: e = a.bf16 ? step_typed<__nv_bfloat16, 64>(a, stream) : step_typed<float, 64>(a, stream); break;
    }
    if (e == cudaSuccess) *launches += 1;
    return e;
}

}  // namespace gdr
