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
// owns 4 states of a channel: sums over n start in the thread and end with
// the helper warps (through shared memory), sums over channels go through the
// warp by an exchange that halves the number of values at each step and end
// with the helpers too.  Blocks' parts of dB and dC, and batch rows' parts of
// dA, dD and ddt_bias, are added by a last kernel in a fixed order: no atomics,
// equal calls give equal bits.  4 x 4096 x 2048, N = 16, bf16: 911 us, of which
// the storing pass takes about 180, the walk 720 (72% of the issue slots of the
// SMs that have a block: 128 of 148; 250 instructions per 16 channels and token)
// and the last kernel 14.
#include <type_traits>

#include "ssm_internal.cuh"

namespace gdr {
namespace {

constexpr int kSms = 148;
constexpr int kLanes = 256;              // threads that walk: 4 states of a channel each
constexpr int kHelpers = 256;            // threads that load, form the time steps and write the results
constexpr int kThreads = kLanes + kHelpers;
constexpr int kWarps = kLanes / 32;
constexpr int kSub = kCheckpoint;        // tokens recomputed at a time
// Registers a thread: the launch gives every thread 128; the walk keeps 8
// tokens' decays and states and takes 144, which the helpers make room for
// (256 * 144 + 256 * 112 = 512 * 128).
constexpr int kWalkRegs = 144, kHelperRegs = 112;

template <typename T, int N> struct Shape {
    static constexpr int LN = N / 4;                   // lanes of a channel
    static constexpr int CL = 32 / LN;                 // channels of a warp
    static constexpr int CB = kWarps * CL;             // channels of a block
    static constexpr int kTile = N == 16 || N == 32 ? 16 : 8;   // tokens between two block barriers
    static constexpr int GR = CB / 4;
    static constexpr int TPP = kHelpers / GR;
    static constexpr int R = TPP >= kTile ? 1 : kTile / TPP;
    static constexpr int GRB = N / 4;
    static constexpr int TPB = kHelpers / GRB;
    static constexpr int RB = TPB >= kTile ? 1 : kTile / TPB;
    // floats of one buffer
    static constexpr int P = kTile * CB * 2;           // {delta, u}
    static constexpr int DC = kTile * CB;              // dc
    static constexpr int S = kTile * N * sizeof(T) / 4;   // B, then C, in the inputs' type
    static constexpr int Y2 = kTile * kLanes * 2;      // {du, sum w A2} of each lane
    static constexpr int Y1 = kTile * kLanes;          // C h of each lane
    static constexpr int Q = kTile * kWarps * 2 * N;   // the warps' sums of dB and dC
    static constexpr int BUF = P + DC + 2 * S + Y2 + Y1 + Q;
    static constexpr size_t smem = 2 * BUF * sizeof(float);
};

// Pieces that a row is walked in (side by side, when there are few channels),
// tokens of a piece, and what the pieces behind hand on: launch_ssm_scan_adjoint.
struct BackPieces {
    int count, tokens;
    float *slots, *sums;
};

// Shared-memory position of a 16-byte chunk.  The helpers touch chunks 2, 4 or
// 8 apart, the walking lanes consecutive ones; folding the bits above a row of
// 8 into the position gives both different banks.
__device__ __forceinline__ int swz(int chunk) { return chunk ^ ((chunk >> 3) & 7); }

struct BwdParts {
    float *points;     // states ahead of every kSub-th token
    float *bc;         // [blocks of a group][B][T][G][2][N]: parts of dB and dC
    float *dA;         // [pieces * B][D][N]
    float *dD, *dbias; // [pieces * B][D]
    BackPieces pc;
};

// A lane's 4 states in the order in which the exchange between the lanes gives
// them away: position j holds state j ^ order, the bits of `order` being the
// lane's bits of the first two steps.  Then "keep half, send half" is the same
// registers in every lane, and no value has to be selected.
struct Order {
    int first;                 // 2 * bit 1 of the order: where the pair of positions 0, 1 lies
    bool swap;                 // bit 0: the two of a pair change places
    unsigned low, high;        // byte selectors that widen the bf16 of positions 0 and 1 of a pair
    __device__ Order(int order)
        : first(order & 2), swap(order & 1), low(swap ? 0x3244u : 0x1044u), high(swap ? 0x1044u : 0x3244u) {}
    __device__ __forceinline__ int state(int j) const { return j ^ (first | (int)swap); }
    __device__ __forceinline__ f32x2 pair(float2 v) const { return swap ? make_f32x2(v.y, v.x) : make_f32x2(v.x, v.y); }
    // both pairs of 4 values in memory, and back
    __device__ __forceinline__ void load(const float *p, f32x2 &a, f32x2 &b) const
    {
        a = pair(*(const float2 *)(p + first));
        b = pair(*(const float2 *)(p + (first ^ 2)));
    }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, f32x2 &a, f32x2 &b) const
    {
        const unsigned u = *(const unsigned *)(p + first), v = *(const unsigned *)(p + (first ^ 2));
        a = make_f32x2(__uint_as_float(__byte_perm(u, 0, low)), __uint_as_float(__byte_perm(u, 0, high)));
        b = make_f32x2(__uint_as_float(__byte_perm(v, 0, low)), __uint_as_float(__byte_perm(v, 0, high)));
    }
    __device__ __forceinline__ void store(float *p, f32x2 a, f32x2 b) const
    {
        *(f32x2 *)(p + first) = pair(make_float2(lo_f32(a), hi_f32(a)));
        *(f32x2 *)(p + (first ^ 2)) = pair(make_float2(lo_f32(b), hi_f32(b)));
    }
};

// The sums of 4 values of dB and 4 of dC, in a lane's order, over the channels
// of a warp (lanes LN, 2 LN, ... apart), stored by the lane that has them.
template <int N, int LN, int CL>
__device__ __forceinline__ void store_sums(f32x2 dB0, f32x2 dB1, f32x2 dC0, f32x2 dC1, int lane, const Order &order,
                                           float *out)
{
    constexpr unsigned all = 0xffffffffu;
    float b0 = lo_f32(dB0) + __shfl_xor_sync(all, lo_f32(dB1), LN), b1 = hi_f32(dB0) + __shfl_xor_sync(all, hi_f32(dB1), LN);
    float c0 = lo_f32(dC0) + __shfl_xor_sync(all, lo_f32(dC1), LN), c1 = hi_f32(dC0) + __shfl_xor_sync(all, hi_f32(dC1), LN);
    if constexpr (CL == 2) {
        *(float2 *)(out + order.state(0)) = make_float2(b0, b1);
        *(float2 *)(out + N + order.state(0)) = make_float2(c0, c1);
    } else {
        b0 += __shfl_xor_sync(all, b1, 2 * LN);
        c0 += __shfl_xor_sync(all, c1, 2 * LN);
        if constexpr (CL == 4) {
            out[order.state(0)] = b0;
            out[N + order.state(0)] = c0;
        } else {
            const bool up = lane & (4 * LN);
            float v = (up ? c0 : b0) + __shfl_xor_sync(all, up ? b0 : c0, 4 * LN);
            if constexpr (CL == 16) v += __shfl_xor_sync(all, v, 8 * LN);
            if (CL == 8 || lane < 16) out[(up ? N : 0) + order.state(0)] = v;
        }
    }
}

template <typename T, int N, bool VECTOR>
__global__ void __launch_bounds__(kThreads, 1)
ssm_bwd_kernel(const ScanBwdArgs a, const BwdParts parts, int blocks_per_group)
{
    using S = Shape<T, N>;
    using V = typename Pack<T, 4>::V;
    constexpr int kTile = S::kTile;
    extern __shared__ __align__(16) float sm[];
    const ScanArgs &f = a.f;
    const BackPieces &pc = parts.pc;

    const int per_row = blocks_per_group * f.G;
    const int b = blockIdx.x / per_row;
    const int gi = (blockIdx.x - b * per_row) / blocks_per_group;
    const int blk = blockIdx.x - b * per_row - gi * blocks_per_group;
    const int cpg = f.D / f.G;
    const int cfirst = gi * cpg + blk * S::CB;
    const int cend = min(cfirst + S::CB, (gi + 1) * cpg);
    const int len = row_length(f.lengths, b, f.T);
    const int piece = blockIdx.y, t0 = piece * pc.tokens;     // a multiple of kTile
    const int stop = min(t0 + pc.tokens, f.T);                // rows [t0, stop) are this piece's
    const int t1 = min(stop, len);
    const int tiles = t1 > t0 ? (t1 - t0 + kTile - 1) / kTile : 0;
    const int tid = threadIdx.x;
    const size_t row_of_parts = (size_t)piece * f.B + b;

    if (tid < kLanes) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWalkRegs));
        const int warp = tid >> 5, lane = tid & 31;
        const int ln = lane % S::LN, n0 = ln * 4;
        const int ch = warp * S::CL + lane / S::LN, c = cfirst + ch;
        const bool on = c < cend;
        const size_t at = ((size_t)b * f.D + c) * N + n0;
        const Order order(((lane / S::LN) & 1) * 2 + (S::CL >= 4 ? (lane / (2 * S::LN)) & 1 : 0));
        f32x2 A0 = 0, A1 = 0, carry0 = 0, carry1 = 0, dA0 = 0, dA1 = 0;
        if (on) {
            order.load(f.A + (size_t)c * N + n0, A0, A1);
            if (a.dh_T) order.load(a.dh_T + at, carry0, carry1);
        }
        A0 = mul2(A0, both(kLog2e));
        A1 = mul2(A1, both(kLog2e));
        // fold in the pieces behind, the last that the row has first
        if (pc.count > 1 && on)
#pragma unroll 4
            for (int s = (len - 1) / pc.tokens; s > piece; --s) {
                const f32x2 sum = both(pc.sums[((size_t)s * f.B + b) * f.D + c]);
                f32x2 v0, v1;
                order.load(pc.slots + (size_t)s * f.B * f.D * N + at, v0, v1);
                carry0 = fold2(sum, A0, carry0, v0);
                carry1 = fold2(sum, A1, carry1, v1);
            }
        // the stored state ahead of the sub-tile that comes next
        const size_t pstride = (size_t)f.D * N;
        const float *point = parts.points + ((size_t)b * ((f.T + kSub - 1) / kSub) * f.D + c) * N + n0;
        float2 state0 = make_float2(0.f, 0.f), state1 = state0;
        auto fetch_state = [&](int t) {
            if (t >= t0 && t < t1 && on) {
                state0 = *(const float2 *)(point + (size_t)(t / kSub) * pstride + order.first);
                state1 = *(const float2 *)(point + (size_t)(t / kSub) * pstride + (order.first ^ 2));
            }
        };
        fetch_state(t0 + tiles * kTile - kSub);
        __syncthreads();
        for (int i = 0; i < tiles; ++i) {
            const int tb0 = t0 + (tiles - 1 - i) * kTile;
            float *buf = sm + (i & 1) * S::BUF;
            const float *p = buf + swz(ch >> 1) * 4 + (ch & 1) * 2, *pd = buf + S::P + swz(ch >> 2) * 4 + (ch & 3);
            const T *sB = (const T *)(buf + S::P + S::DC) + n0, *sC = (const T *)(buf + S::P + S::DC + S::S) + n0;
            float *y2 = buf + S::P + S::DC + 2 * S::S, *y1 = y2 + S::Y2;
            float *sq = y1 + S::Y1 + warp * 2 * N + n0;
            float *o2 = y2 + swz(tid >> 1) * 4 + (tid & 1) * 2, *o1 = y1 + swz(tid >> 2) * 4 + (tid & 3);
#pragma unroll 1
            for (int sub = kTile / kSub - 1; sub >= 0; --sub) {
                const int tb = sub * kSub;
                f32x2 a0[kSub], a1[kSub], h0[kSub + 1], h1[kSub + 1];
                h0[0] = order.pair(state0);
                h1[0] = order.pair(state1);
                // A sub-tile behind the row's end has no stored state (it is 0 then); its tokens
                // have delta = dc = 0 and change nothing.
                fetch_state(tb0 + tb - kSub);
#pragma unroll
                for (int t = 0; t < kSub; ++t) {
                    const float2 du = *(const float2 *)(p + (tb + t) * S::CB * 2);
                    f32x2 b0, b1;
                    order.load(sB + (tb + t) * N, b0, b1);
                    const f32x2 d = both(du.x), u = both(du.y);
                    a0[t] = decay2(d, A0);
                    a1[t] = decay2(d, A1);
                    h0[t + 1] = fma2(a0[t], h0[t], mul2(u, b0));
                    h1[t + 1] = fma2(a1[t], h1[t], mul2(u, b1));
                }
                // A token's operands are loaded while the one before is in work, and its sums and
                // stores wait until the next one's work is under way: loads stay behind stores, and
                // stores behind the exchange between the lanes, which takes about 100 cycles.
                struct Token {
                    float2 du;
                    float dc;
                    f32x2 b0, b1, c0, c1;
                } now, next;
                struct Sums {
                    f32x2 dB0, dB1, dC0, dC1;
                    float su, sw, sy;
                } done;
                auto fetch = [&](Token &k, int t) {
                    k.du = *(const float2 *)(p + t * S::CB * 2);
                    k.dc = pd[t * S::CB];
                    order.load(sB + t * N, k.b0, k.b1);
                    order.load(sC + t * N, k.c0, k.c1);
                };
                auto store = [&](const Sums &k, int t) {
                    store_sums<N, S::LN, S::CL>(k.dB0, k.dB1, k.dC0, k.dC1, lane, order, sq + t * kWarps * 2 * N);
                    *(float2 *)(o2 + t * kLanes * 2) = make_float2(k.su, k.sw);
                    if (f.z) o1[t * kLanes] = k.sy;
                };
                fetch(now, tb + kSub - 1);
#pragma unroll
                for (int t = kSub - 1; t >= 0; --t) {
                    if (t > 0) fetch(next, tb + t - 1);
                    const f32x2 d = both(now.du.x), u = both(now.du.y), dc = both(now.dc);
                    const f32x2 c0 = now.c0, c1 = now.c1;
                    const f32x2 g0 = fma2(dc, c0, carry0), g1 = fma2(dc, c1, carry1);
                    const f32x2 dB0 = mul2(g0, u), dB1 = mul2(g1, u), dC0 = mul2(dc, h0[t + 1]), dC1 = mul2(dc, h1[t + 1]);
                    const f32x2 pu = fma2(g1, now.b1, mul2(g0, now.b0));
                    carry0 = mul2(a0[t], g0);
                    carry1 = mul2(a1[t], g1);
                    const f32x2 w0 = mul2(carry0, h0[t]), w1 = mul2(carry1, h1[t]);
                    const f32x2 pw = fma2(w1, A1, mul2(w0, A0));
                    dA0 = fma2(w0, d, dA0);
                    dA1 = fma2(w1, d, dA1);
                    const f32x2 y = fma2(h1[t + 1], c1, mul2(h0[t + 1], c0));
                    if (t < kSub - 1) store(done, tb + t + 1);
                    done = {dB0, dB1, dC0, dC1, lo_f32(pu) + hi_f32(pu), lo_f32(pw) + hi_f32(pw), lo_f32(y) + hi_f32(y)};
                    now = next;
                }
                store(done, tb);
            }
            __syncthreads();
        }
        if (on) {
            order.store(parts.dA + (row_of_parts * f.D + c) * N + n0, dA0, dA1);
            if (a.dh0 && piece == 0) order.store(a.dh0 + at, carry0, carry1);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kHelperRegs));
        const int ht = tid - kLanes;
        const int gr = ht % S::GR, tok = ht / S::GR;
        const int grb = ht % S::GRB, tokb = ht / S::GRB;
        const int c = cfirst + gr * 4, have = cend - c;
        const bool whole = cfirst + S::CB <= cend;
        auto token_of = [&](int i) { return t0 + (tiles - 1 - i) * kTile; };   // of the i-th tile, from the end
        // running pointers to this thread's first element of the tile that is fetched next
        const long long first = (long long)t0 + (tiles ? (long long)(tiles - 1) * kTile : 0);
        const T *px = (const T *)f.x + b * f.xs.b + c + (first + tok) * f.xs.t;
        const T *pdt = (const T *)f.dt + b * f.dts.b + c + (first + tok) * f.dts.t;
        const T *pdy = (const T *)a.dy + b * a.dys.b + c + (first + tok) * a.dys.t;
        const T *pz = f.z ? (const T *)f.z + b * f.zs.b + c + (first + tok) * f.zs.t : nullptr;
        const T *pB = (const T *)f.Bm + b * f.bs.b + (size_t)gi * N + grb * 4 + (first + tokb) * f.bs.t;
        const T *pC = (const T *)f.Cm + b * f.cs.b + (size_t)gi * N + grb * 4 + (first + tokb) * f.cs.t;
        const size_t row = (size_t)b * f.T * f.D + c;
        size_t out = row + (first + tok) * f.D;               // and of the tile that is finished next
        float *pbc = parts.bc + ((((size_t)blk * f.B + b) * f.T + first) * f.G + gi) * 2 * N;
        float bias[4], skip[4], sumD[4] = {}, sumb[4] = {};
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            bias[v] = f.dt_bias && v < have ? f.dt_bias[c + v] : 0.f;
            skip[v] = f.D_skip && v < have ? f.D_skip[c + v] : 0.f;
        }
        V rx[S::R], rdt[S::R], rdy[S::R], rz[S::R], rB[S::RB], rC[S::RB];
        // what a tile's last step needs of its first, one and two tiles old: x, the slope of the
        // softplus, and dy silu'(z)
        struct Kept {
            V x[S::R];
            float slope[S::R][4], dz[S::R][4];
        } old, mid;
        // tiles inside the piece load without predicates
        auto fetch_as = [&](int tb, auto inside) {
            constexpr bool FULL_TILE = decltype(inside)::value;
#pragma unroll
            for (int r = 0; r < S::R; ++r) {
                const int k = tok + r * S::TPP;
                const int valid = FULL_TILE ? 4 : k < kTile && tb + k < t1 ? have : 0;
                rx[r] = load4<T, VECTOR, FULL_TILE>(px + r * S::TPP * f.xs.t, valid);
                rdt[r] = load4<T, VECTOR, FULL_TILE>(pdt + r * S::TPP * f.dts.t, valid);
                rdy[r] = load4<T, VECTOR, FULL_TILE>(pdy + r * S::TPP * a.dys.t, valid);
                if (pz) rz[r] = load4<T, VECTOR, FULL_TILE>(pz + r * S::TPP * f.zs.t, valid);
            }
#pragma unroll
            for (int r = 0; r < S::RB; ++r) {
                const int k = tokb + r * S::TPB;
                const int valid = FULL_TILE ? 4 : k < kTile && tb + k < t1 ? 4 : 0;
                if (S::TPB > kTile && k >= kTile) continue;
                rB[r] = load4<T, VECTOR, FULL_TILE>(pB + r * S::TPB * f.bs.t, valid);
                rC[r] = load4<T, VECTOR, FULL_TILE>(pC + r * S::TPB * f.cs.t, valid);
            }
        };
        auto fetch = [&](int i) {
            const int tb = token_of(i);
            if (whole && tb + kTile <= t1 && S::TPP <= kTile) fetch_as(tb, std::true_type{});
            else fetch_as(tb, std::false_type{});
            px -= kTile * f.xs.t;
            pdt -= kTile * f.dts.t;
            pdy -= kTile * a.dys.t;
            if (pz) pz -= kTile * f.zs.t;
            pB -= kTile * f.bs.t;
            pC -= kTile * f.cs.t;
        };
        auto prepare = [&](int i, Kept &keep) {
            float *buf = sm + (i & 1) * S::BUF;
            const int tb = token_of(i);
            const bool full = whole && tb + kTile <= t1;
#pragma unroll
            for (int r = 0; r < S::R; ++r) {
                const int k = tok + r * S::TPP;
                if (S::TPP > kTile && k >= kTile) continue;
                float fx[4], fd[4], fy[4], fz[4];
                unpack(rx[r], fx);
                unpack(rdt[r], fd);
                unpack(rdy[r], fy);
                if (pz) unpack(rz[r], fz);
                keep.x[r] = rx[r];
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    float e, d = fd[v] + bias[v], slope = 1.f;
                    if (f.softplus) {
                        const float pre = d;
                        d = softplus_f32(pre, e);
                        const float q = rcp_approx(1.f + e);      // sigmoid(|pre|)
                        slope = pre < 0.f ? e * q : q;
                    }
                    if (!full && (tb + k >= t1 || v >= have)) d = 0.f;
                    fd[v] = d;
                    fx[v] *= d;
                    keep.slope[r][v] = slope;
                    if (pz) {
                        const float q = sigmoid_f32(fz[v]), zq = fz[v] * q;
                        keep.dz[r][v] = fy[v] * fmaf(zq, 1.f - q, q);
                        fy[v] *= zq;
                    }
                }
                float *q = buf + k * S::CB * 2;
                *(float4 *)(q + swz(gr * 2) * 4) = make_float4(fd[0], fx[0], fd[1], fx[1]);
                *(float4 *)(q + swz(gr * 2 + 1) * 4) = make_float4(fd[2], fx[2], fd[3], fx[3]);
                *(float4 *)(buf + S::P + k * S::CB + swz(gr) * 4) = make_float4(fy[0], fy[1], fy[2], fy[3]);
            }
#pragma unroll
            for (int r = 0; r < S::RB; ++r) {
                const int k = tokb + r * S::TPB;
                if (S::TPB > kTile && k >= kTile) continue;
                T *q = (T *)(buf + S::P + S::DC) + k * N + grb * 4;
                *(V *)q = rB[r];
                *(V *)(q + kTile * N) = rC[r];
            }
        };
        auto finish = [&](int i, const Kept &keep) {
            const float *buf = sm + (i & 1) * S::BUF;
            const float *y2 = buf + S::P + S::DC + 2 * S::S, *y1 = y2 + S::Y2, *sq = y1 + S::Y1;
            const int tb = token_of(i);
            const bool full = whole && tb + kTile <= t1;
#pragma unroll
            for (int r = 0; r < S::R; ++r) {
                const int k = tok + r * S::TPP;
                if (S::TPP > kTile && k >= kTile) continue;
                if (!full && tb + k >= stop) continue;
                const bool live = full || tb + k < t1;
                // this thread's own entries of the buffer
                const float *q = buf + k * S::CB * 2;
                const float4 d01 = *(const float4 *)(q + swz(gr * 2) * 4), d23 = *(const float4 *)(q + swz(gr * 2 + 1) * 4);
                const float4 dc4 = *(const float4 *)(buf + S::P + k * S::CB + swz(gr) * 4);
                const float delta[4] = {d01.x, d01.z, d23.x, d23.z}, dc[4] = {dc4.x, dc4.y, dc4.z, dc4.w};
                float fx[4], gx[4], gd[4], gz[4];
                unpack(keep.x[r], fx);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int s0 = (gr * 4 + v) * S::LN;          // LN partial sums of the channel
                    float du = 0.f, sw = 0.f, sy = 0.f;
#pragma unroll
                    for (int l = 0; l < S::LN / 2; ++l) {
                        const float4 w = *(const float4 *)(y2 + k * kLanes * 2 + swz((s0 >> 1) + l) * 4);
                        du += w.x + w.z;
                        sw += w.y + w.w;
                    }
                    gx[v] = fmaf(du, delta[v], dc[v] * skip[v]);
                    gd[v] = fmaf(du, fx[v], sw * 0.6931471805599453f) * keep.slope[r][v];
                    if (pz) {
                        if (S::LN >= 4) {
#pragma unroll
                            for (int l = 0; l < S::LN / 4; ++l) {
                                const float4 w = *(const float4 *)(y1 + k * kLanes + swz((s0 >> 2) + l) * 4);
                                sy += (w.x + w.y) + (w.z + w.w);
                            }
                        } else {
                            const float2 w = *(const float2 *)(y1 + k * kLanes + swz(s0 >> 2) * 4 + (s0 & 3));
                            sy = w.x + w.y;
                        }
                        gz[v] = keep.dz[r][v] * fmaf(skip[v], fx[v], sy);
                    }
                    if (!live) gx[v] = gd[v] = gz[v] = 0.f;
                    if (full || (live && v < have)) {
                        sumD[v] = fmaf(dc[v], fx[v], sumD[v]);
                        sumb[v] += gd[v];
                    }
                }
                const size_t o = out + (size_t)(r * S::TPP) * f.D;
                const int n = full ? 4 : have;
                store4<T, VECTOR>((T *)a.dx + o, gx, n);
                store4<T, VECTOR>((T *)a.ddt + o, gd, n);
                if (pz) store4<T, VECTOR>((T *)a.dz + o, gz, n);
            }
            out -= (size_t)kTile * f.D;
            // the warps' sums of dB and dC
#pragma unroll
            for (int q = 0; q < kTile * N / 2; q += kHelpers) {
                const int j = q + ht, k = j / (N / 2), e = (j - k * (N / 2)) * 4;
                if ((kTile * N / 2 < kHelpers && j >= kTile * N / 2) || tb + k >= t1) continue;
                float4 s = *(const float4 *)(sq + k * kWarps * 2 * N + e);
#pragma unroll
                for (int w = 1; w < kWarps; ++w) {
                    const float4 m = *(const float4 *)(sq + (k * kWarps + w) * 2 * N + e);
                    s.x += m.x;
                    s.y += m.y;
                    s.z += m.z;
                    s.w += m.w;
                }
                *(float4 *)(pbc + (size_t)k * f.G * 2 * N + e) = s;
            }
            pbc -= (size_t)kTile * f.G * 2 * N;
        };

        // behind the row's end the gradients are zero
        const float zero[4] = {};
        for (long long t = (long long)t0 + tiles * kTile + tok; t < stop; t += S::TPP) {
            store4<T, VECTOR>((T *)a.dx + row + t * f.D, zero, have);
            store4<T, VECTOR>((T *)a.ddt + row + t * f.D, zero, have);
            if (pz) store4<T, VECTOR>((T *)a.dz + row + t * f.D, zero, have);
        }
        if (tiles) {
            fetch(0);
            prepare(0, mid);
            if (tiles > 1) fetch(1);
        }
        __syncthreads();
        for (int i = 0; i < tiles; ++i) {
            if (i > 0) finish(i - 1, old);     // ahead of the entries' next use
            old = mid;
            if (i + 1 < tiles) prepare(i + 1, mid);
            if (i + 2 < tiles) fetch(i + 2);
            __syncthreads();
        }
        if (tiles) finish(tiles - 1, old);
        // the walk is over: its shared memory takes the helpers' sums over tokens, and only they meet
        asm volatile("bar.sync 1, %0;" ::"n"(kHelpers) : "memory");
        float *red = sm;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            red[(tok * S::CB + gr * 4 + v) * 2] = sumD[v];
            red[(tok * S::CB + gr * 4 + v) * 2 + 1] = sumb[v];
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kHelpers) : "memory");
        for (int k = ht; k < S::CB; k += kHelpers)
            if (cfirst + k < cend) {
                float d = 0.f, m = 0.f;
                for (int q = 0; q < S::TPP; ++q) {
                    d += red[(q * S::CB + k) * 2];
                    m += red[(q * S::CB + k) * 2 + 1];
                }
                parts.dD[row_of_parts * f.D + cfirst + k] = d;
                parts.dbias[row_of_parts * f.D + cfirst + k] = m;
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
    for (int b = 0; b < f.B * parts.pc.count; ++b) s += p[(size_t)b * stride];
    *o = s;
}

int blocks_per_group(int D, int G, int N)
{
    const int cb = 1024 / N;
    return (D / G + cb - 1) / cb;
}

// As in the forward: few channels, then pieces side by side.  A piece's
// gradient from behind costs another pass of exponentials (about a third of
// the walk), so it pays from half the machine down.
BackPieces plan(int B, int T, int D, int G, int N)
{
    BackPieces p = {1, T > 0 ? T : 1, nullptr, nullptr};
    const long long blocks = (long long)B * G * blocks_per_group(D, G, N);
    if (blocks > 0 && blocks * 2 <= kSms && T >= 96) {
        long long count = kSms / blocks;
        if (count > T / 32) count = T / 32;
        p.tokens = (int)((T + count - 1) / count + 31) / 32 * 32;
        p.count = (T + p.tokens - 1) / p.tokens;
    }
    return p;
}

struct Layout {
    size_t points, bc, dA, dD, slots, sums, scan, total;   // offsets in bytes, 256-byte steps
};
Layout layout(int B, int T, int D, int G, int N)
{
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    const size_t pieces = plan(B, T, D, G, N).count;
    Layout l;
    size_t at = 0;
    l.points = at;
    at += up((size_t)B * ((T + kSub - 1) / kSub) * D * N * 4);
    l.bc = at;
    at += up((size_t)blocks_per_group(D, G, N) * B * T * G * 2 * N * 4);
    l.dA = at;
    at += up(pieces * B * D * N * 4);
    l.dD = at;
    at += up(pieces * B * D * 2 * 4);
    l.slots = at;
    at += pieces > 1 ? up(pieces * B * D * N * 4) : 0;
    l.sums = at;
    at += pieces > 1 ? up(pieces * B * D * 4) : 0;
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
    using S = Shape<T, N>;
    auto k = ssm_bwd_kernel<T, N, VECTOR>;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = allow_shared(k, S::smem, done);
    if (e != cudaSuccess) return e;
    const int bpg = blocks_per_group(a.f.D, a.f.G, N);
    k<<<dim3((unsigned)((long long)a.f.B * a.f.G * bpg), p.pc.count), kThreads, S::smem, st>>>(a, p, bpg);
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
    p.pc = plan(f.B, f.T, f.D, f.G, f.N);
    p.pc.slots = (float *)(ws + l.slots);
    p.pc.sums = (float *)(ws + l.sums);
    p.dbias = p.dD + (size_t)p.pc.count * f.B * f.D;
    cudaError_t e;
    if (f.T > 0) {
        ScanArgs s = f;
        s.y = nullptr;
        s.z = nullptr;
        s.workspace = ws + l.scan;
        e = launch_ssm_scan_checkpoints(s, p.points, stream, launches);
        if (e != cudaSuccess) return e;
    }
    if (p.pc.count > 1) {
        ScanArgs s = f;
        s.x = a.dy;
        s.xs = a.dys;
        s.Bm = f.Cm;
        s.bs = f.cs;
        s.D_skip = s.h0 = nullptr;
        s.y = nullptr;
        e = launch_ssm_scan_adjoint(s, p.pc.count, p.pc.tokens, p.pc.slots, p.pc.sums, stream, launches);
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
