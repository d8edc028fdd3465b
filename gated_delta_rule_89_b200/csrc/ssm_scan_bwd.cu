// Backward of the selective state space scan.
//
// With a_t[n] = exp(delta_t A[n]), u_t = delta_t x_t, dc_t = dy_t silu(z_t) and the states h_t,
//
//   g_t[n]   = dc_t C_t[n] + a_{t+1}[n] g_{t+1}[n]         (the gradient of h_t; g_T takes dh_T)
//   dC_t[n]  = sum_d dc_t h_t[n]         dB_t[n] = sum_d g_t[n] u_t       (over a group's channels)
//   w_t[n]   = a_t[n] g_t[n] h_{t-1}[n]  dA[n]   = sum_t w_t[n] delta_t
//   du_t     = sum_n g_t[n] B_t[n]       ddelta_t = du_t x_t + sum_n w_t[n] A[n]
//   dx_t     = du_t delta_t + dc_t D     dD = sum dc_t x_t     dz_t = dy_t (C_t h_t + D x_t) silu'(z_t)
//   ddt_t    = ddelta_t softplus'        dh0 = a_1 g_1
//
// The states are needed from the last to the first.  A forward pass without
// outputs stores them ahead of every 8th token (N/2 bytes per token and
// channel); the walk back recomputes 8 tokens at a time and keeps their
// decays and states in registers, so every exponential is taken once in each
// pass.
//
// Issue slots bound the walk: per (token, channel, state) it takes the sums
// over n (three), over the channels (two) and over tokens (one).  A thread
// owns 4 states of 2 channels: sums over n start in the thread and end with
// the helper warps (through shared memory), sums over channels start in the
// thread and go through the warp by an exchange that halves the number of
// values at each step.  Blocks' parts of dB and dC, and batch rows' parts of
// dA, dD and ddt_bias, are added by a last kernel in a fixed order: no atomics,
// equal calls give equal bits.
#include "ssm_internal.cuh"

namespace gdr {
namespace {

constexpr int kLanes = 128;              // threads that walk: 4 states x 2 channels each
constexpr int kThreads = 2 * kLanes;     // and as many helpers
constexpr int kTile = 16;                // tokens between two block barriers
constexpr int kSub = kCheckpoint;        // tokens recomputed at a time

template <int N> struct Shape {
    static constexpr int LN = N / 4;                   // lanes of a channel
    static constexpr int CL = 32 / LN;                 // channels side by side in a warp
    static constexpr int CW = 2 * CL;                  // channels of a warp
    static constexpr int CB = 4 * CW;                  // channels of a block
    static constexpr int GR = CB / 4;
    static constexpr int TPP = kLanes / GR;
    static constexpr int R = TPP >= kTile ? 1 : kTile / TPP;
    static constexpr int GRB = N / 4;
    static constexpr int TPB = kLanes / GRB;
    static constexpr int RB = TPB >= kTile ? 1 : kTile / TPB;
    // floats of one buffer
    static constexpr int P = kTile * CB * 4;           // {delta, delta, u, u}
    static constexpr int DC = kTile * CB * 2;          // {dc, dc}
    static constexpr int S = kTile * N;                // B, then C
    static constexpr int Y2 = kTile * 2 * kLanes * 2;  // {du, sum w A2} of each lane and channel
    static constexpr int Y1 = kTile * 2 * kLanes;      // C h of each lane and channel
    static constexpr int Q = kTile * 4 * 2 * N;        // the warps' sums of dB and dC
    static constexpr int BUF = P + DC + 2 * S + Y2 + Y1 + Q;
    static constexpr size_t smem = 2 * BUF * sizeof(float);
};

// Shared-memory position of a 16-byte chunk.  The helpers touch chunks 2, 4 or
// 8 apart, the walking lanes consecutive ones; folding the bits above a row of
// 8 into the position gives both different banks.
__device__ __forceinline__ int swz(int chunk) { return chunk ^ ((chunk >> 3) & 7); }

struct BwdParts {
    float *points;     // states ahead of every kSub-th token
    float *bc;         // [blocks of a group][B][T][G][2][N]: parts of dB and dC
    float *dA;         // [B][D][N]
    float *dD, *dbias; // [B][D]
};

// Sums v[0..COUNT) over the lanes that differ in the bits from MASK up to 16.
// Each step a lane hands half of its values to its partner and keeps the other
// half, so COUNT / CL values stay with every lane (one, replicated, when the
// lanes outnumber the values); `which` is the first index it kept.
template <int COUNT, int MASK>
__device__ __forceinline__ void lane_sums(float *v, int lane, int &which)
{
    if constexpr (MASK < 32) {
        if constexpr (COUNT > 1) {
            constexpr int H = COUNT / 2;
            const bool up = lane & MASK;
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float send = up ? v[i] : v[i + H], keep = up ? v[i + H] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, MASK);
            }
            if (up) which += H;
            lane_sums<H, MASK * 2>(v, lane, which);
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], MASK);
            lane_sums<1, MASK * 2>(v, lane, which);
        }
    }
}

template <typename T, int N, bool VECTOR>
__global__ void __launch_bounds__(kThreads, 1)
ssm_bwd_kernel(const ScanBwdArgs a, const BwdParts parts, int blocks_per_group)
{
    using S = Shape<N>;
    using V = typename Pack<T, 4>::V;
    extern __shared__ __align__(16) float sm[];
    const ScanArgs &f = a.f;

    const int per_row = blocks_per_group * f.G;
    const int b = blockIdx.x / per_row;
    const int gi = (blockIdx.x - b * per_row) / blocks_per_group;
    const int blk = blockIdx.x - b * per_row - gi * blocks_per_group;
    const int cpg = f.D / f.G;
    const int cfirst = gi * cpg + blk * S::CB;
    const int cend = min(cfirst + S::CB, (gi + 1) * cpg);
    const int len = row_length(f.lengths, b, f.T);
    const int tiles = (len + kTile - 1) / kTile;
    const int tid = threadIdx.x;

    if (tid < kLanes) {
        const int warp = tid >> 5, lane = tid & 31;
        const int ln = lane % S::LN, n0 = ln * 4;
        int ch[2];
        bool on[2];
        size_t at[2];
        f32x2 A[2][2], carry[2][2], dA[2][2];
        const float *point[2];
        const size_t pstride = (size_t)f.D * N;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            ch[k] = warp * S::CW + k * S::CL + lane / S::LN;
            const int c = cfirst + ch[k];
            on[k] = c < cend;
            at[k] = ((size_t)b * f.D + c) * N + n0;
            float4 q = make_float4(0.f, 0.f, 0.f, 0.f), r = q;
            if (on[k]) {
                q = *(const float4 *)(f.A + (size_t)c * N + n0);
                if (a.dh_T) r = *(const float4 *)(a.dh_T + at[k]);
            }
            A[k][0] = make_f32x2(q.x * kLog2e, q.y * kLog2e);
            A[k][1] = make_f32x2(q.z * kLog2e, q.w * kLog2e);
            carry[k][0] = make_f32x2(r.x, r.y);
            carry[k][1] = make_f32x2(r.z, r.w);
            dA[k][0] = dA[k][1] = 0;
            point[k] = parts.points + ((size_t)b * ((f.T + kSub - 1) / kSub) * f.D + c) * N + n0;
        }
        // the stored state ahead of the sub-tile that comes next
        ulonglong2 next[2] = {make_ulonglong2(0, 0), make_ulonglong2(0, 0)};
        auto fetch_state = [&](int sub) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (on[k] && sub >= 0 && sub * kSub < len)
                    next[k] = *(const ulonglong2 *)(point[k] + (size_t)sub * pstride);
        };
        fetch_state((tiles - 1) * (kTile / kSub) + kTile / kSub - 1);
        __syncthreads();
        for (int i = 0; i < tiles; ++i) {
            const int tile = tiles - 1 - i;
            float *buf = sm + (i & 1) * S::BUF;
            const float *sB = buf + S::P + S::DC + n0, *sC = sB + S::S;
            float *y2 = buf + S::P + S::DC + 2 * S::S, *y1 = y2 + S::Y2, *sq = y1 + S::Y1;
            const float *p[2], *pd[2];
            float *o2[2], *o1[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                p[k] = buf + swz(ch[k]) * 4;
                pd[k] = buf + S::P + swz(ch[k] >> 1) * 4 + (ch[k] & 1) * 2;
                const int s = ch[k] * S::LN + ln;
                o2[k] = y2 + swz(s >> 1) * 4 + (s & 1) * 2;
                o1[k] = y1 + swz(s >> 2) * 4 + (s & 3);
            }
            for (int sub = kTile / kSub - 1; sub >= 0; --sub) {
                const int tb = sub * kSub;
                f32x2 av[kSub][2][2], hv[kSub + 1][2][2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    hv[0][k][0] = next[k].x;
                    hv[0][k][1] = next[k].y;
                }
                // a sub-tile behind the row's end has no stored state; its tokens change nothing and
                // what is computed for them is not written, but the state must be finite
                fetch_state(tile * (kTile / kSub) + sub - 1);
#pragma unroll
                for (int t = 0; t < kSub; ++t) {
                    const ulonglong2 bb = *(const ulonglong2 *)(sB + (tb + t) * N);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const ulonglong2 du = *(const ulonglong2 *)(p[k] + (tb + t) * S::CB * 4);
                        av[t][k][0] = decay2(du.x, A[k][0]);
                        av[t][k][1] = decay2(du.x, A[k][1]);
                        hv[t + 1][k][0] = fma2(av[t][k][0], hv[t][k][0], mul2(du.y, bb.x));
                        hv[t + 1][k][1] = fma2(av[t][k][1], hv[t][k][1], mul2(du.y, bb.y));
                    }
                }
#pragma unroll
                for (int t = kSub - 1; t >= 0; --t) {
                    const ulonglong2 bb = *(const ulonglong2 *)(sB + (tb + t) * N);
                    const ulonglong2 cc = *(const ulonglong2 *)(sC + (tb + t) * N);
                    f32x2 dB[2], dC[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const ulonglong2 du = *(const ulonglong2 *)(p[k] + (tb + t) * S::CB * 4);
                        const f32x2 dc = *(const f32x2 *)(pd[k] + (tb + t) * S::CB * 2);
                        const f32x2 g0 = fma2(dc, cc.x, carry[k][0]), g1 = fma2(dc, cc.y, carry[k][1]);
                        dB[0] = k ? fma2(g0, du.y, dB[0]) : mul2(g0, du.y);
                        dB[1] = k ? fma2(g1, du.y, dB[1]) : mul2(g1, du.y);
                        dC[0] = k ? fma2(dc, hv[t + 1][k][0], dC[0]) : mul2(dc, hv[t + 1][k][0]);
                        dC[1] = k ? fma2(dc, hv[t + 1][k][1], dC[1]) : mul2(dc, hv[t + 1][k][1]);
                        const f32x2 su = fma2(g1, bb.y, mul2(g0, bb.x));
                        carry[k][0] = mul2(av[t][k][0], g0);
                        carry[k][1] = mul2(av[t][k][1], g1);
                        const f32x2 w0 = mul2(carry[k][0], hv[t][k][0]), w1 = mul2(carry[k][1], hv[t][k][1]);
                        const f32x2 sw = fma2(w1, A[k][1], mul2(w0, A[k][0]));
                        dA[k][0] = fma2(w0, du.x, dA[k][0]);
                        dA[k][1] = fma2(w1, du.x, dA[k][1]);
                        *(float2 *)(o2[k] + (tb + t) * kLanes * 4) =
                            make_float2(lo_f32(su) + hi_f32(su), lo_f32(sw) + hi_f32(sw));
                        if (f.z) {
                            const f32x2 y = fma2(hv[t + 1][k][1], cc.y, mul2(hv[t + 1][k][0], cc.x));
                            o1[k][(tb + t) * kLanes * 2] = lo_f32(y) + hi_f32(y);
                        }
                    }
                    float v[8] = {lo_f32(dB[0]), hi_f32(dB[0]), lo_f32(dB[1]), hi_f32(dB[1]),
                                  lo_f32(dC[0]), hi_f32(dC[0]), lo_f32(dC[1]), hi_f32(dC[1])};
                    int which = 0;
                    lane_sums<8, S::LN>(v, lane, which);
                    constexpr int left = 8 / S::CL > 1 ? 8 / S::CL : 1;
                    if (S::CL <= 8 || lane < 16) {
                        float *o = sq + ((tb + t) * 4 + warp) * 2 * N + (which >> 2) * N + n0 + (which & 3);
#pragma unroll
                        for (int j = 0; j < left; ++j) o[j] = v[j];
                    }
                }
            }
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (on[k]) {
                *(float4 *)(parts.dA + at[k]) =
                    make_float4(lo_f32(dA[k][0]), hi_f32(dA[k][0]), lo_f32(dA[k][1]), hi_f32(dA[k][1]));
                if (a.dh0)
                    *(float4 *)(a.dh0 + at[k]) = make_float4(lo_f32(carry[k][0]), hi_f32(carry[k][0]),
                                                             lo_f32(carry[k][1]), hi_f32(carry[k][1]));
            }
    } else {
        const int ht = tid - kLanes;
        const int gr = ht % S::GR, tok = ht / S::GR;
        const int grb = ht % S::GRB, tokb = ht / S::GRB;
        const int c = cfirst + gr * 4, have = cend - c;
        const T *px = (const T *)f.x + b * f.xs.b + c, *pdt = (const T *)f.dt + b * f.dts.b + c;
        const T *pdy = (const T *)a.dy + b * a.dys.b + c;
        const T *pz = f.z ? (const T *)f.z + b * f.zs.b + c : nullptr;
        const T *pB = (const T *)f.Bm + b * f.bs.b + (size_t)gi * N + grb * 4;
        const T *pC = (const T *)f.Cm + b * f.cs.b + (size_t)gi * N + grb * 4;
        const size_t row = (size_t)b * f.T * f.D + c;
        float bias[4], skip[4], sumD[4] = {}, sumb[4] = {};
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            bias[v] = f.dt_bias && v < have ? f.dt_bias[c + v] : 0.f;
            skip[v] = f.D_skip && v < have ? f.D_skip[c + v] : 0.f;
        }
        struct Set {
            V x[S::R], dt[S::R], dy[S::R], z[S::R];
        };
        Set in, out;
        V rB[S::RB], rC[S::RB];
        auto fetch = [&](Set &s, int tile) {
#pragma unroll
            for (int r = 0; r < S::R; ++r) {
                const int k = tok + r * S::TPP;
                const long long t = (long long)tile * kTile + k;
                const int valid = k < kTile && t < len ? have : 0;
                s.x[r] = load4<T, VECTOR>(px + t * f.xs.t, valid);
                s.dt[r] = load4<T, VECTOR>(pdt + t * f.dts.t, valid);
                s.dy[r] = load4<T, VECTOR>(pdy + t * a.dys.t, valid);
                if (pz) s.z[r] = load4<T, VECTOR>(pz + t * f.zs.t, valid);
            }
        };
        auto fetch_bc = [&](int tile) {
#pragma unroll
            for (int r = 0; r < S::RB; ++r) {
                const int k = tokb + r * S::TPB;
                const long long t = (long long)tile * kTile + k;
                const int valid = k < kTile && t < len ? 4 : 0;
                rB[r] = load4<T, VECTOR>(pB + t * f.bs.t, valid);
                rC[r] = load4<T, VECTOR>(pC + t * f.cs.t, valid);
            }
        };
        auto prepare = [&](int i) {
            float *buf = sm + (i & 1) * S::BUF;
            const int tile = tiles - 1 - i;
#pragma unroll
            for (int r = 0; r < S::R; ++r) {
                const int k = tok + r * S::TPP;
                if (k >= kTile) continue;
                const bool live = tile * kTile + k < len;
                float fx[4], fd[4], fy[4], fz[4], dc[4];
                unpack(in.x[r], fx);
                unpack(in.dt[r], fd);
                unpack(in.dy[r], fy);
                if (pz) unpack(in.z[r], fz);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    float d = fd[v] + bias[v];
                    if (f.softplus) { float e; d = softplus_f32(d, e); }
                    if (!live || v >= have) d = 0.f;
                    const float u = d * fx[v];
                    dc[v] = pz ? fy[v] * (fz[v] * sigmoid_f32(fz[v])) : fy[v];
                    *(float4 *)(buf + ((size_t)k * S::CB + swz(gr * 4 + v)) * 4) = make_float4(d, d, u, u);
                }
                float *q = buf + S::P + (size_t)k * S::CB * 2;
                *(float4 *)(q + swz(gr * 2) * 4) = make_float4(dc[0], dc[0], dc[1], dc[1]);
                *(float4 *)(q + swz(gr * 2 + 1) * 4) = make_float4(dc[2], dc[2], dc[3], dc[3]);
            }
#pragma unroll
            for (int r = 0; r < S::RB; ++r) {
                const int k = tokb + r * S::TPB;
                if (k >= kTile) continue;
                float g[4];
                float *q = buf + S::P + S::DC + k * N + grb * 4;
                unpack(rB[r], g);
                *(float4 *)q = make_float4(g[0], g[1], g[2], g[3]);
                unpack(rC[r], g);
                *(float4 *)(q + S::S) = make_float4(g[0], g[1], g[2], g[3]);
            }
        };
        auto finish = [&](int i) {
            const float *buf = sm + (i & 1) * S::BUF;
            const float *y2 = buf + S::P + S::DC + 2 * S::S, *y1 = y2 + S::Y2, *sq = y1 + S::Y1;
            const int tile = tiles - 1 - i;
#pragma unroll
            for (int r = 0; r < S::R; ++r) {
                const int k = tok + r * S::TPP;
                const long long t = (long long)tile * kTile + k;
                if (k >= kTile || t >= f.T) continue;
                float gx[4] = {}, gd[4] = {}, gz[4] = {};
                if (t < len) {
                    float fx[4], fd[4], fy[4], fz[4];
                    unpack(out.x[r], fx);
                    unpack(out.dt[r], fd);
                    unpack(out.dy[r], fy);
                    if (pz) unpack(out.z[r], fz);
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int s0 = (gr * 4 + v) * S::LN;      // LN partial sums of the channel
                        float du = 0.f, sw = 0.f, sy = 0.f;
#pragma unroll
                        for (int q = 0; q < S::LN / 2; ++q) {
                            const float4 w =
                                *(const float4 *)(y2 + (size_t)k * kLanes * 4 + swz((s0 >> 1) + q) * 4);
                            du += w.x + w.z;
                            sw += w.y + w.w;
                        }
                        if (pz) {
                            if (S::LN >= 4) {
#pragma unroll
                                for (int q = 0; q < S::LN / 4; ++q) {
                                    const float4 w =
                                        *(const float4 *)(y1 + (size_t)k * kLanes * 2 + swz((s0 >> 2) + q) * 4);
                                    sy += (w.x + w.y) + (w.z + w.w);
                                }
                            } else {
                                const float2 w = *(const float2 *)(y1 + (size_t)k * kLanes * 2 +
                                                                   swz(s0 >> 2) * 4 + (s0 & 3));
                                sy = w.x + w.y;
                            }
                        }
                        const float pre = fd[v] + bias[v];
                        float e2; const float delta = f.softplus ? softplus_f32(pre, e2) : pre;
                        float dc = fy[v];
                        if (pz) {
                            const float s = sigmoid_f32(fz[v]);
                            dc = fy[v] * (fz[v] * s);
                            gz[v] = fy[v] * fmaf(skip[v], fx[v], sy) * fmaf(fz[v] * s, 1.f - s, s);
                        }
                        gx[v] = fmaf(du, delta, dc * skip[v]);
                        float dd = fmaf(du, fx[v], sw * 0.6931471805599453f);
                        if (f.softplus) dd *= sigmoid_f32(pre);
                        gd[v] = dd;
                        if (v < have) {
                            sumD[v] = fmaf(dc, fx[v], sumD[v]);
                            sumb[v] += dd;
                        }
                    }
                }
                store4<T, VECTOR>((T *)a.dx + row + t * f.D, gx, have);
                store4<T, VECTOR>((T *)a.ddt + row + t * f.D, gd, have);
                if (pz) store4<T, VECTOR>((T *)a.dz + row + t * f.D, gz, have);
            }
            // the four warps' sums of dB and dC
            for (int q = ht; q < kTile * N / 2; q += kLanes) {
                const int k = q / (N / 2), e = (q - k * (N / 2)) * 4;
                const long long t = (long long)tile * kTile + k;
                if (t >= len) continue;
                float4 s = *(const float4 *)(sq + (size_t)k * 8 * N + e);
#pragma unroll
                for (int w = 1; w < 4; ++w) {
                    const float4 m = *(const float4 *)(sq + ((size_t)k * 4 + w) * 2 * N + e);
                    s.x += m.x;
                    s.y += m.y;
                    s.z += m.z;
                    s.w += m.w;
                }
                *(float4 *)(parts.bc + ((((size_t)blk * f.B + b) * f.T + t) * f.G + gi) * 2 * N + e) = s;
            }
        };

        // behind the row's end the gradients are zero
        const float zero[4] = {};
        for (long long t = (long long)tiles * kTile + tok; t < f.T; t += S::TPP) {
            store4<T, VECTOR>((T *)a.dx + row + t * f.D, zero, have);
            store4<T, VECTOR>((T *)a.ddt + row + t * f.D, zero, have);
            if (pz) store4<T, VECTOR>((T *)a.dz + row + t * f.D, zero, have);
        }
        if (tiles) {
            fetch(in, tiles - 1);
            fetch_bc(tiles - 1);
            prepare(0);
            if (tiles > 1) {
                fetch(in, tiles - 2);
                fetch_bc(tiles - 2);
            }
        }
        __syncthreads();
        for (int i = 0; i < tiles; ++i) {
            if (i + 1 < tiles) prepare(i + 1);
            if (i + 2 < tiles) {
                fetch(in, tiles - 3 - i);
                fetch_bc(tiles - 3 - i);
            }
            if (i > 0) finish(i - 1);
            fetch(out, tiles - 1 - i);
            __syncthreads();
        }
        if (tiles) finish(tiles - 1);
        // the walk is over: its shared memory takes the helpers' sums over tokens, and only they meet
        asm volatile("bar.sync 1, 128;" ::: "memory");
        float *red = sm;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            red[(tok * S::CB + gr * 4 + v) * 2] = sumD[v];
            red[(tok * S::CB + gr * 4 + v) * 2 + 1] = sumb[v];
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        for (int k = ht; k < S::CB; k += kLanes)
            if (cfirst + k < cend) {
                float d = 0.f, m = 0.f;
                for (int q = 0; q < S::TPP; ++q) {
                    d += red[(q * S::CB + k) * 2];
                    m += red[(q * S::CB + k) * 2 + 1];
                }
                parts.dD[(size_t)b * f.D + cfirst + k] = d;
                parts.dbias[(size_t)b * f.D + cfirst + k] = m;
            }
    }
}

// The sums of the parts.  The first `bc_blocks` blocks add the blocks' parts of dB and dC, 4
// values a thread; the rest add the batch rows' parts of dA, dD and ddt_bias.
template <typename T>
__global__ void __launch_bounds__(256)
ssm_bwd_sum_kernel(const ScanBwdArgs a, const BwdParts parts, int blocks_per_group, unsigned bc_blocks)
{
    const ScanArgs &f = a.f;
    const int N = f.N;
    if (blockIdx.x < bc_blocks) {
        const long long rows = (long long)f.B * f.T * f.G, q = (long long)blockIdx.x * 256 + threadIdx.x;
        const long long r = q / (N / 2);                 // (b, t, g)
        if (r >= rows) return;
        const int e = (int)(q - r * (N / 2)) * 4;
        const int b = (int)(r / ((long long)f.T * f.G));
        const int t = (int)((r - (long long)b * f.T * f.G) / f.G);
        float s[4] = {};
        if (t < row_length(f.lengths, b, f.T)) {
            const float *p = parts.bc + r * 2 * N + e;
            for (int k = 0; k < blocks_per_group; ++k) {
                const float4 m = *(const float4 *)(p + (size_t)k * rows * 2 * N);
                s[0] += m.x;
                s[1] += m.y;
                s[2] += m.z;
                s[3] += m.w;
            }
        }
        T *o = e < N ? (T *)a.dB + r * N + e : (T *)a.dC + r * N + e - N;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = from_f32<T>(s[k]);
        return;
    }
    const long long i = (long long)(blockIdx.x - bc_blocks) * 256 + threadIdx.x;
    const long long DN = (long long)f.D * N;
    const float *p;
    float *o;
    long long stride;
    if (i < DN) {
        p = parts.dA + i;
        o = a.dA + i;
        stride = DN;
    } else if (i < DN + 2 * f.D) {
        const long long c = i - DN;
        p = c < f.D ? parts.dD + c : parts.dbias + c - f.D;
        o = c < f.D ? (a.dD ? a.dD + c : nullptr) : (a.ddt_bias ? a.ddt_bias + c - f.D : nullptr);
        stride = f.D;
    } else {
        return;
    }
    if (!o) return;
    float s = 0.f;
    for (int b = 0; b < f.B; ++b) s += p[(size_t)b * stride];
    *o = s;
}

int blocks_per_group(int D, int G, int N)
{
    const int cb = 1024 / N;
    return (D / G + cb - 1) / cb;
}

struct Layout {
    size_t points, bc, dA, dD, scan, total;   // offsets in bytes, 256-byte steps
};
Layout layout(int B, int T, int D, int G, int N)
{
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    Layout l;
    size_t at = 0;
    l.points = at;
    at += up((size_t)B * ((T + kSub - 1) / kSub) * D * N * 4);
    l.bc = at;
    at += up((size_t)blocks_per_group(D, G, N) * B * T * G * 2 * N * 4);
    l.dA = at;
    at += up((size_t)B * D * N * 4);
    l.dD = at;
    at += up((size_t)B * D * 2 * 4);
    l.scan = at;
    l.total = at + ssm_scan_fwd_workspace_bytes(B, T, D, G, N);
    return l;
}

template <typename T> bool bwd_vectors(const ScanBwdArgs &a)
{
    const ScanArgs &f = a.f;
    const void *ptrs[] = {f.x, f.dt, f.Bm, f.Cm, f.z, a.dy, a.dx, a.ddt, a.dz};
    const BatchToken *s[] = {&f.xs, &f.dts, &f.bs, &f.cs, &f.zs, &a.dys};
    if ((f.D / f.G) % 4) return false;
    for (const void *p : ptrs)
        if (p && !aligned_to(p, 4 * sizeof(T))) return false;
    for (const BatchToken *q : s)
        if (q->b % 4 || q->t % 4) return false;
    return true;
}

template <typename T, int N, bool VECTOR>
cudaError_t run_bwd(const ScanBwdArgs &a, const BwdParts &p, cudaStream_t st)
{
    auto k = ssm_bwd_kernel<T, N, VECTOR>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape<N>::smem);
    if (e != cudaSuccess) return e;
    const int bpg = blocks_per_group(a.f.D, a.f.G, N);
    k<<<(unsigned)((long long)a.f.B * a.f.G * bpg), kThreads, Shape<N>::smem, st>>>(a, p, bpg);
    return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_typed(const ScanBwdArgs &a, const BwdParts &p, cudaStream_t st)
{
    const bool v = bwd_vectors<T>(a);
    switch (a.f.N) {
        case 8: return v ? run_bwd<T, 8, true>(a, p, st) : run_bwd<T, 8, false>(a, p, st);
        case 16: return v ? run_bwd<T, 16, true>(a, p, st) : run_bwd<T, 16, false>(a, p, st);
        case 32: return v ? run_bwd<T, 32, true>(a, p, st) : run_bwd<T, 32, false>(a, p, st);
        default: return v ? run_bwd<T, 64, true>(a, p, st) : run_bwd<T, 64, false>(a, p, st);
    }
}

}  // namespace

size_t ssm_scan_bwd_workspace_bytes(int B, int T, int D, int G, int N) { return layout(B, T, D, G, N).total; }

cudaError_t launch_ssm_scan_bwd(const ScanBwdArgs &a, cudaStream_t stream, int *launches)
{
    const ScanArgs &f = a.f;
    const Layout l = layout(f.B, f.T, f.D, f.G, f.N);
    unsigned char *ws = (unsigned char *)a.workspace;
    BwdParts p;
    p.points = (float *)(ws + l.points);
    p.bc = (float *)(ws + l.bc);
    p.dA = (float *)(ws + l.dA);
    p.dD = (float *)(ws + l.dD);
    p.dbias = p.dD + (size_t)f.B * f.D;
    cudaError_t e;
    if (f.T > 0) {
        ScanArgs s = f;
        s.y = nullptr;
        s.z = nullptr;
        s.workspace = ws + l.scan;
        e = launch_ssm_scan_checkpoints(s, p.points, stream, launches);
        if (e != cudaSuccess) return e;
    }
    e = f.bf16 ? bwd_typed<__nv_bfloat16>(a, p, stream) : bwd_typed<float>(a, p, stream);
    if (e != cudaSuccess) return e;
    const int bpg = blocks_per_group(f.D, f.G, f.N);
    const unsigned bcb = (unsigned)(((long long)f.B * f.T * f.G * (f.N / 2) + 255) / 256);
    const unsigned rest = (unsigned)(((long long)f.D * (f.N + 2) + 255) / 256);
    if (f.bf16) ssm_bwd_sum_kernel<__nv_bfloat16><<<bcb + rest, 256, 0, stream>>>(a, p, bpg, bcb);
    else ssm_bwd_sum_kernel<float><<<bcb + rest, 256, 0, stream>>>(a, p, bpg, bcb);
    e = cudaGetLastError();
    if (e == cudaSuccess) *launches += 2;
    return e;
}

}  // namespace gdr
