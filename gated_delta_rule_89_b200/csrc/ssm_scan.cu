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
// Every (token, channel, state) costs one exponential, and every (token,
// channel) three more special functions for the time step and the gate.  The
// pipe gives 16 of them per clock and SM: at N = 16 that is 3.3 times as long
// as the tensors' bytes take at HBM speed, so the prompt form is bound by
// exponentials, and after them by issue slots.  2 x 8192 x 4096 channels, bf16:
// 520 us, where the exponentials alone need 274 (and the 256 blocks keep 86%
// of the SMs busy).
//
// A block's first four warps run the recurrence, one channel (or two) and 4
// states a thread; the others, one tile ahead and behind, load, form delta and
// delta x, add the partial sums of C h, and write the outputs.  The two meet at
// one barrier a tile, in double-buffered shared memory.
#include <type_traits>

#include "ssm_internal.cuh"

namespace gdr {
namespace {

constexpr int kSms = 148;
constexpr int kScanLanes = 128;            // threads of a block that run the recurrence
constexpr int kUnit = 32;                  // pieces of a row are multiples of it

enum Mode {
    FULL,    // the outputs and the final state
    LOCAL,   // the state that a piece of a row ends with when it starts from zero
    POINTS,  // the states ahead of every kCheckpoint-th token, for the backward
    ADJOINT  // the gradient of the state ahead of a piece when that behind it is zero: a walk back
             // with dy silu(z) in the place of u and C in the place of B
};

// A block's share and its shared memory, for state size N and CPT channels a
// scan thread (4 states of each).  With two channels the B and C that a thread
// loads serve twice: shared memory returns 128 bytes a clock, and one channel's
// loads of a token take 24 (bf16) or 40 (fp32) clocks of an SM against 32 for
// its exponentials.  With one channel there are twice as many blocks.
template <typename T, int N, int CPT, Mode MODE> struct Shape {
    static constexpr int H = CPT == 1 && N > 16 ? kScanLanes : 2 * kScanLanes;   // helper threads
    static constexpr int THREADS = kScanLanes + H;
    static constexpr int LPC = N / 4;                    // scan lanes of a channel
    static constexpr int CB = kScanLanes / LPC * CPT;    // channels of a block
    // Tokens between two block barriers: 64 where two blocks still fit on an SM (at one block
    // an SM, 1 x 4096 channels, 309 us against 408 with 32; at two 520 and 527); the passes
    // without outputs have less to do between the barriers and are 2% to 4% faster with 32.
    static constexpr int kTile = MODE == FULL && CPT == 1 && N >= 16 && sizeof(T) == 2 ? 64 : 32;
    static constexpr int GR = CB / 4;                    // groups of 4 channels
    static constexpr int TPP = H / GR;                   // tokens the helpers cover at a time
    static constexpr int R = TPP >= kTile ? 1 : kTile / TPP;
    static constexpr int GRB = N / 4;                    // groups of 4 states
    static constexpr int TPB = H / GRB;
    static constexpr int RB = TPB >= kTile ? 1 : kTile / TPB;
    static constexpr int P = kTile * CB * 2;             // floats: {delta, u} per (token, channel)
    static constexpr int S = kTile * N * sizeof(T) / 4;  // floats: B, and as many for C, in the inputs' type
    static constexpr int Y = kTile * CB * LPC;           // floats: partial sums of C h
    static constexpr int BUF = P + 2 * S + Y;
    static constexpr size_t smem = 2 * BUF * sizeof(float);
};

// Shared-memory position of a 16-byte chunk: the helpers touch every 2nd or
// 4th chunk, the scan lanes consecutive ones; with the bits above a row of 8
// folded in, both meet 8 different banks.
__device__ __forceinline__ int swz(int chunk) { return chunk ^ ((chunk >> 3) & 7); }

// pieces of a row (time is split when there are few channels), tokens of a
// piece, and the piece states: slot [s][B][D][N] is what piece s starts from
// (slot 0: h0) before the pieces ahead of it are folded in, and
// sums [s][B][D] the sum of delta over piece s - 1.
struct Pieces {
    int count, tokens;
    float *slots, *sums;
    float *points;   // POINTS: [B][ceil(T / kCheckpoint)][D][N]
};
// ADJOINT takes dy as x and Cm as Bm, and writes piece s's result to slots[s]
// and its sum of delta to sums[s].

template <typename T, int N, int CPT, bool VECTOR, Mode MODE>
__global__ void __launch_bounds__(Shape<T, N, CPT, MODE>::THREADS, 2)
ssm_scan_kernel(const ScanArgs a, const Pieces pc, int blocks_per_group)
{
    using S = Shape<T, N, CPT, MODE>;
    using V = typename Pack<T, 4>::V;
    constexpr int kTile = S::kTile;
    extern __shared__ __align__(16) float sm[];

    const int per_row = blocks_per_group * a.G;
    const int b = blockIdx.x / per_row;
    const int gi = (blockIdx.x - b * per_row) / blocks_per_group;
    const int cpg = a.D / a.G;
    const int cfirst = gi * cpg + (blockIdx.x - b * per_row - gi * blocks_per_group) * S::CB;
    const int cend = min(cfirst + S::CB, (gi + 1) * cpg);     // channels [cfirst, cend)
    const int piece = blockIdx.y + (MODE == ADJOINT);         // nothing lies ahead of piece 0
    constexpr bool kBack = MODE == ADJOINT;
    const int len = row_length(a.lengths, b, a.T);
    const int t0 = piece * pc.tokens, t1 = min(t0 + pc.tokens, len);
    if (MODE == FULL && a.zero_tail) {                        // the piece's tokens behind the row's end
        const int stop = min(t0 + pc.tokens, a.T), from = max(t0, len), wide = cend - cfirst;
        T *y = (T *)a.y + ((size_t)b * a.T + from) * a.D + cfirst;
        for (long long k = threadIdx.x; k < (long long)(stop - from) * wide; k += S::THREADS)
            y[k / wide * a.D + k % wide] = from_f32<T>(0.f);
    }
    if (piece > 0 && t0 >= t1) return;                        // the whole block
    const int tiles = t1 > t0 ? (t1 - t0 + kTile - 1) / kTile : 0;
    const int tid = threadIdx.x;

    if (tid < kScanLanes) {
        // -------------------------------------------------- the recurrence
        const int ch = tid / S::LPC * CPT, ln = tid % S::LPC, n0 = ln * 4;
        const size_t slot = (size_t)a.B * a.D * N, at = ((size_t)b * a.D + cfirst + ch) * N + n0;
        bool on[CPT];
        f32x2 A[CPT][2], h[CPT][2];
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            on[k] = cfirst + ch + k < cend;
            const size_t ak = at + k * N;
            float4 q = make_float4(0.f, 0.f, 0.f, 0.f), r = q;
            if (on[k]) {
                q = *(const float4 *)(a.A + (size_t)(cfirst + ch + k) * N + n0);
                if (MODE == LOCAL) {
                    if (piece == 0) {
                        // the second pass reads h0 from the slot, so that h_T may be the same buffer
                        if (a.h0) r = *(const float4 *)(a.h0 + ak);
                        *(float4 *)(pc.slots + ak) = r;
                        r = make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                } else if (MODE == ADJOINT) {
                } else if (pc.count > 1) {
                    r = *(const float4 *)(pc.slots + ak);
                } else if (a.h0) {
                    r = *(const float4 *)(a.h0 + ak);
                }
            }
            A[k][0] = make_f32x2(q.x * kLog2e, q.y * kLog2e);
            A[k][1] = make_f32x2(q.z * kLog2e, q.w * kLog2e);
            h[k][0] = make_f32x2(r.x, r.y);
            h[k][1] = make_f32x2(r.z, r.w);
            if ((MODE == FULL || MODE == POINTS) && on[k])
#pragma unroll 4
                for (int s = 1; s <= piece; ++s) {   // fold in the pieces ahead
                    const f32x2 sum = both(pc.sums[((size_t)s * a.B + b) * a.D + cfirst + ch + k]);
                    const ulonglong2 v = *(const ulonglong2 *)(pc.slots + s * slot + ak);
                    h[k][0] = fold2(sum, A[k][0], h[k][0], v.x);
                    h[k][1] = fold2(sum, A[k][1], h[k][1], v.y);
                }
        }
        float sum[CPT] = {};
        float *points = nullptr;
        if (MODE == POINTS)
            points = pc.points +
                     (((size_t)b * ((a.T + kCheckpoint - 1) / kCheckpoint) + t0 / kCheckpoint) * a.D + cfirst + ch) * N + n0;
        __syncthreads();
        // Four tokens' operands are loaded ahead of the four in work, and ahead of the stores of
        // their outputs: shared-memory loads are not moved across stores, and a warp that waited
        // for each token's loads would spend most of its time there.
        constexpr int G = 4;
        struct Token {
            float du[2 * CPT];
            Quad<T> b, c;
        };
        for (int i = 0; i < tiles; ++i) {
            const float *buf = sm + (i & 1) * S::BUF;
            const float *p = buf + swz(ch >> 1) * 4 + (ch & 1) * 2;
            const T *sb = (const T *)(buf + S::P) + n0, *sc = (const T *)(buf + S::P + S::S) + n0;
            float *py[CPT];
#pragma unroll
            for (int k = 0; k < CPT; ++k) {
                const int s = (ch + k) * S::LPC + ln;
                py[k] = sm + (i & 1) * S::BUF + S::P + 2 * S::S + swz(s >> 2) * 4 + (s & 3);
            }
            Token now[G], next[G];
            auto fetch = [&](Token *k, int t) {
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    const int at = kBack ? kTile - 1 - (t + j) : t + j;
                    const float *q = p + at * S::CB * 2;
                    if (CPT == 2) *(float4 *)k[j].du = *(const float4 *)q;
                    else *(float2 *)k[j].du = *(const float2 *)q;
                    k[j].b = *(const Quad<T> *)(sb + at * N);
                    if (MODE == FULL) k[j].c = *(const Quad<T> *)(sc + at * N);
                }
            };
            // four tokens from t on; `more`: four others follow
            auto work = [&](int t, bool more) {
                if (MODE == POINTS && t % kCheckpoint == 0 && t0 + i * kTile + t < t1) {
                    float *q = points + (size_t)(i * kTile + t) / kCheckpoint * a.D * N;
#pragma unroll
                    for (int k = 0; k < CPT; ++k)
                        if (on[k]) *(ulonglong2 *)(q + k * N) = make_ulonglong2(h[k][0], h[k][1]);
                }
                if (more) fetch(next, t + G);
                float y[G][CPT];
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    const Token &o = now[j];
                    const f32x2 b0 = o.b.lo(), b1 = o.b.hi();
#pragma unroll
                    for (int k = 0; k < CPT; ++k) {
                        const f32x2 d = both(o.du[2 * k]), u = both(o.du[2 * k + 1]);
                        if (kBack) {   // u is dy silu(z), b is C
                            h[k][0] = mul2(decay2(d, A[k][0]), fma2(u, b0, h[k][0]));
                            h[k][1] = mul2(decay2(d, A[k][1]), fma2(u, b1, h[k][1]));
                        } else {
                            h[k][0] = fma2(decay2(d, A[k][0]), h[k][0], mul2(u, b0));
                            h[k][1] = fma2(decay2(d, A[k][1]), h[k][1], mul2(u, b1));
                        }
                        if (MODE == FULL) {
                            const f32x2 s = fma2(h[k][1], o.c.hi(), mul2(h[k][0], o.c.lo()));
                            y[j][k] = lo_f32(s) + hi_f32(s);
                        } else if (MODE != POINTS) {
                            sum[k] += o.du[2 * k];
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    if (MODE == FULL)
#pragma unroll
                        for (int k = 0; k < CPT; ++k) py[k][(t + j) * S::CB * S::LPC] = y[j][k];
                    now[j] = next[j];
                }
            };
            fetch(now, 0);
            const int count = t1 - t0 - i * kTile;
            if (kBack || count >= kTile) {
#pragma unroll
                for (int t = 0; t < kTile; t += G) work(t, t + G < kTile);
            } else {   // a row's last tile, as far as it has tokens (in fours: the rest change nothing)
#pragma unroll 1
                for (int t = 0; t < count; t += G) work(t, t + G < kTile);
            }
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            if (!on[k]) continue;
            const ulonglong2 v = make_ulonglong2(h[k][0], h[k][1]);
            if (MODE == LOCAL || MODE == ADJOINT) {
                const int s = kBack ? piece : piece + 1;
                *(ulonglong2 *)(pc.slots + s * slot + at + k * N) = v;
                if (ln == 0) pc.sums[((size_t)s * a.B + b) * a.D + cfirst + ch + k] = sum[k];
            }
            if (MODE == FULL && a.h_T && (t1 == len || pc.count == 1)) *(ulonglong2 *)(a.h_T + at + k * N) = v;
        }
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
        constexpr int kStep = kBack ? -kTile : kTile;
        const long long begin = (long long)t0 + (kBack && tiles ? (long long)(tiles - 1) * kTile : 0);
        const long long first = begin + tok, firstb = begin + tokb;
        auto token_of = [&](int i) { return t0 + (kBack ? tiles - 1 - i : i) * kTile; };   // of the i-th tile
        const T *px = (const T *)a.x + b * a.xs.b + c + first * a.xs.t;
        const T *pdt = (const T *)a.dt + b * a.dts.b + c + first * a.dts.t;
        const T *pB = (const T *)a.Bm + b * a.bs.b + (size_t)gi * N + grb * 4 + firstb * a.bs.t;
        const T *pC = (const T *)a.Cm + b * a.cs.b + (size_t)gi * N + grb * 4 + firstb * a.cs.t;
        const T *pxo = px;                                     // and of the tile that is finished next
        const T *pzo = a.z ? (const T *)a.z + b * a.zs.b + c + first * a.zs.t : nullptr;
        T *py = (T *)a.y + ((size_t)b * a.T + first) * a.D + c;
        float bias[4], skip[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            bias[v] = a.dt_bias && v < have ? a.dt_bias[c + v] : 0.f;
            skip[v] = MODE == FULL && a.D_skip && v < have ? a.D_skip[c + v] : 0.f;
        }

        V rx[S::R], rdt[S::R], rB[S::RB], rC[S::RB], ex[S::R], ez[S::R], rz[S::R];
        const T *pz = kBack ? pzo : nullptr;
        // Tiles inside the piece load without predicates (which cost three instructions a load).
        auto fetch_as = [&](int tb, auto inside) {
            constexpr bool FULL_TILE = decltype(inside)::value;
#pragma unroll
            for (int r = 0; r < S::R; ++r) {
                const int k = tok + r * S::TPP;
                const int valid = FULL_TILE ? 4 : k < kTile && tb + k < t1 ? have : 0;
                rx[r] = load4<T, VECTOR, FULL_TILE>(px + r * S::TPP * a.xs.t, valid);
                rdt[r] = load4<T, VECTOR, FULL_TILE>(pdt + r * S::TPP * a.dts.t, valid);
                if (kBack && pz) rz[r] = load4<T, VECTOR, FULL_TILE>(pz + r * S::TPP * a.zs.t, valid);
            }
#pragma unroll
            for (int r = 0; r < S::RB; ++r) {
                const int k = tokb + r * S::TPB;
                const int valid = FULL_TILE ? 4 : k < kTile && tb + k < t1 ? 4 : 0;
                if (S::TPB > kTile && k >= kTile) continue;
                rB[r] = load4<T, VECTOR, FULL_TILE>(pB + r * S::TPB * a.bs.t, valid);
                if (MODE == FULL) rC[r] = load4<T, VECTOR, FULL_TILE>(pC + r * S::TPB * a.cs.t, valid);
            }
        };
        auto inside = [&](int tb) { return whole && tb + kTile <= t1 && S::TPP <= kTile; };
        auto fetch = [&](int i) {
            const int tb = token_of(i);
            if (inside(tb)) fetch_as(tb, std::true_type{});
            else fetch_as(tb, std::false_type{});
            px += kStep * a.xs.t;
            pdt += kStep * a.dts.t;
            pB += kStep * a.bs.t;
            if (MODE == FULL) pC += kStep * a.cs.t;
            if (kBack && pz) pz += kStep * a.zs.t;
        };
        auto fetch_out_as = [&](int tb, auto inside) {
            constexpr bool FULL_TILE = decltype(inside)::value;
#pragma unroll
            for (int r = 0; r < S::R; ++r) {
                const int k = tok + r * S::TPP;
                const int valid = FULL_TILE ? 4 : k < kTile && tb + k < t1 ? have : 0;
                if (a.D_skip) ex[r] = load4<T, VECTOR, FULL_TILE>(pxo + r * S::TPP * a.xs.t, valid);
                if (pzo) ez[r] = load4<T, VECTOR, FULL_TILE>(pzo + r * S::TPP * a.zs.t, valid);
            }
        };
        auto fetch_out = [&](int tile) {
            const int tb = t0 + tile * kTile;
            if (inside(tb)) fetch_out_as(tb, std::true_type{});
            else fetch_out_as(tb, std::false_type{});
            pxo += kTile * a.xs.t;
            if (pzo) pzo += kTile * a.zs.t;
        };
        auto prepare = [&](int i) {
            float *buf = sm + (i & 1) * S::BUF;
            const int tb = token_of(i);
            const bool full = whole && tb + kTile <= t1;
#pragma unroll
            for (int r = 0; r < S::R; ++r) {
                const int k = tok + r * S::TPP;
                if (S::TPP > kTile && k >= kTile) continue;
                float fx[4], fd[4], fz[4];
                unpack(rx[r], fx);
                unpack(rdt[r], fd);
                if (kBack && pz) unpack(rz[r], fz);
                float *q = buf + k * S::CB * 2;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    float e, d = fd[v] + bias[v];
                    if (a.softplus) d = softplus_f32(d, e);
                    if (!full && (tb + k >= t1 || v >= have)) d = 0.f;   // the state stands still
                    fd[v] = d;
                    if (!kBack) fx[v] *= d;
                    else if (pz) fx[v] *= fz[v] * sigmoid_f32(fz[v]);
                }
                *(float4 *)(q + swz(gr * 2) * 4) = make_float4(fd[0], fx[0], fd[1], fx[1]);
                *(float4 *)(q + swz(gr * 2 + 1) * 4) = make_float4(fd[2], fx[2], fd[3], fx[3]);
            }
#pragma unroll
            for (int r = 0; r < S::RB; ++r) {
                const int k = tokb + r * S::TPB;
                if (S::TPB > kTile && k >= kTile) continue;
                *(V *)((T *)(buf + S::P) + k * N + grb * 4) = rB[r];
                if (MODE == FULL) *(V *)((T *)(buf + S::P + S::S) + k * N + grb * 4) = rC[r];
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
                    *(float4 *)(part + 4 * q) = *(const float4 *)(y + k * S::CB * S::LPC + swz(gr * (N / 4) + q) * 4);
                float out[4], fx[4], fz[4];
                unpack(ex[r], fx);
                unpack(ez[r], fz);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    float s = part[v * S::LPC];
#pragma unroll
                    for (int l = 1; l < S::LPC; ++l) s += part[v * S::LPC + l];
                    if (a.D_skip) s = fmaf(skip[v], fx[v], s);
                    if (pzo) s *= fz[v] * sigmoid_f32(fz[v]);
                    out[v] = s;
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
// the step.  A thread owns 4 states of a channel in ROWS batch rows, so a
// warp's accesses are whole lines, several loads are in flight, and A is read
// once for the rows; each of a channel's lanes forms the time step and the
// output of one row.  256 x 4096 channels, N = 16, bf16: 28.8 us, 143 MB at
// 5.0 TB/s, with 4 rows and 5 blocks an SM; one row a thread took 39.
template <typename T, int N, bool VECTOR>
__global__ void __launch_bounds__(256, 5) ssm_step_kernel(const ScanArgs a, int blocks_per_row)
{
    constexpr int LPC = N / 4, CB = 256 / LPC, ROWS = LPC < 4 ? LPC : 4;
    const int group = blockIdx.x / blocks_per_row, b0 = group * ROWS;
    const int c = (blockIdx.x - group * blocks_per_row) * CB + threadIdx.x / LPC;
    const int ln = threadIdx.x % LPC, n0 = ln * 4;
    const bool on = c < a.D;
    float4 *ph = (float4 *)(a.h_T + ((size_t)b0 * a.D + c) * N + n0);
    const size_t hrow = (size_t)a.D * N / 4;
    float4 h[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
        h[r] = on && b0 + r < a.B ? __ldcs(ph + r * hrow) : make_float4(0.f, 0.f, 0.f, 0.f);
    // the row whose sum lane_sums leaves with this lane
    const int mine = ROWS == 4 ? (ln & 1) * 2 + (ln >> 1 & 1) : ln & 1;
    const int bm = b0 + mine;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    float x = 0.f, d = 0.f, z = 0.f;
    if (on) {
        A = *(const float4 *)(a.A + (size_t)c * N + n0);
        if (bm < a.B) {
            x = to_f32<T>(((const T *)a.x)[bm * a.xs.b + c]);
            d = to_f32<T>(((const T *)a.dt)[bm * a.dts.b + c]);
            if (a.z) z = to_f32<T>(((const T *)a.z)[bm * a.zs.b + c]);
            if (a.dt_bias) d += a.dt_bias[c];
            if (a.softplus) {
                float e;
                d = softplus_f32(d, e);
            }
        }
    }
    const int g = on ? c / (a.D / a.G) : 0;
    const T *pB = (const T *)a.Bm + (size_t)g * N + n0, *pC = (const T *)a.Cm + (size_t)g * N + n0;
    const float u = d * x, d2 = d * kLog2e;
    float y[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int from = ROWS == 4 ? (r >> 1) + (r & 1) * 2 : r;      // the lane whose row r is
        const float dr = __shfl_sync(0xffffffffu, d2, from, LPC), ur = __shfl_sync(0xffffffffu, u, from, LPC);
        y[r] = 0.f;
        if (on && b0 + r < a.B) {
            float fb[4], fc[4];
            unpack(load4<T, VECTOR>(pB + (b0 + r) * a.bs.b, 4), fb);
            unpack(load4<T, VECTOR>(pC + (b0 + r) * a.cs.b, 4), fc);
            float4 &s = h[r];
            s.x = fmaf(decay(dr, A.x), s.x, ur * fb[0]);
            s.y = fmaf(decay(dr, A.y), s.y, ur * fb[1]);
            s.z = fmaf(decay(dr, A.z), s.z, ur * fb[2]);
            s.w = fmaf(decay(dr, A.w), s.w, ur * fb[3]);
            __stcs(ph + r * hrow, s);
            y[r] = fmaf(fc[3], s.w, fmaf(fc[2], s.z, fmaf(fc[1], s.y, fc[0] * s.x)));
        }
    }
    int which = 0;
    lane_sums<ROWS, 1, LPC>(y, ln, which);
    if (on && ln < ROWS && bm < a.B) {
        float out = y[0];
        if (a.D_skip) out = fmaf(a.D_skip[c], x, out);
        if (a.z) out *= z * sigmoid_f32(z);
        ((T *)a.y)[(size_t)bm * a.D + c] = from_f32<T>(out);
    }
}

// --------------------------------------------------------------- launches

int blocks_per_group(int D, int G, int N, int cpt)
{
    const int cb = 512 * cpt / N;
    return (D / G + cb - 1) / cb;
}

// Where two channels a thread can pay: with outputs only (the pass that stores
// states for the backward is never faster with two: a whole backward of 2048 x
// 9472, bf16, N = 16, 544 and 606 us; N = 32, 1024 and 1022).  At N = 8 their
// shared memory leaves an SM one block, and in fp32 at N = 16 they spill 536
// bytes a thread: 2048 tokens of 37888 channels, one and two channels a thread,
// N = 8: bf16 349 and 419 us, fp32 362 and 807; 18944 channels, N = 16, fp32:
// 276 and 300.  (Kernels that are chosen spill too: in fp32 one channel a thread
// 192 bytes at N = 8 and 16, two 532 at N = 32 and 876 at N = 64; in bf16 two
// channels 140 bytes at N = 16 and 32, 420 at N = 64.)
template <typename T, int N> constexpr bool kTwoChannels = sizeof(T) == 2 ? N >= 16 : N >= 32;

// And whether they do, by how the blocks fill the SMs (two on each either way).
// In us per 4096 tokens (N = 16, bf16): one channel 260 for a full set of 296
// blocks and 154 for half of one, two channels 467 and 287; in fp32 at N = 64
// half a set takes as long as a full one (but not one element at a time, where
// the helpers bound it).  2048 tokens, with as many blocks of one channel a
// thread as named, one and two channels a thread in us:
//                     296          444          592          888
//   N = 16, bf16   140  146     211  239     265  241     388  359
//   N = 32, bf16   127  129     198  215     244  217     360  327
//   N = 64, bf16   142  149     216  242     276  244     411  386
//   N = 32, fp32   140  164     236  254     272  254     403  392
//   N = 64, fp32   173  217     278  319     341  321     508  624
// and one element at a time at 592: 341 279, 312 239, 369 242, 366 285, 438 320.
template <typename T, int N, bool VECTOR> bool two_channels(int B, int D, int G)
{
    const long long set = 2 * kSms, groups = (long long)B * G;
    auto cost = [&](int cpt, int full, int half) {
        const long long blocks = groups * blocks_per_group(D, G, N, cpt), rest = blocks % set;
        return blocks / set * full + (rest == 0 ? 0 : rest <= kSms ? half : full);
    };
    return cost(2, 467, sizeof(T) == 4 && N == 64 && VECTOR ? 467 : 287) < cost(1, 260, 154);
}

// Few channels leave most of the machine idle; then a row is cut into pieces
// that run side by side: a first pass finds the state each piece would end
// with from a zero start, and the second starts every piece from the states
// ahead of it.  That doubles the exponentials, so it pays from half the
// machine down.  Two sets of blocks rather than one let the short rows of a
// ragged batch make room for the long ones (2 x 20011 x 520, N = 8, fp32, eight
// draws of the short row's length: 201 us with one set at the mean, 184 with
// two, 168 to 202; whole rows 201 and 201), up to 64 pieces: every piece folds
// in all those ahead (128 channels x 65536 tokens, N = 16, bf16: 116 us with 74
// pieces, 134 with 148).
Pieces plan(int B, int T, int D, int G, int N, void *workspace)
{
    Pieces p = {1, T, nullptr, nullptr, nullptr};
    const long long blocks = (long long)B * G * blocks_per_group(D, G, N, 1);   // two channels a thread need more
    if (blocks > 0 && blocks * 2 <= kSms && T >= 8 * kUnit) {
        long long count = 4 * kSms / blocks;
        if (count > 64) count = 2 * kSms / blocks > 64 ? 2 * kSms / blocks : 64;
        if (count > T / (2 * kUnit)) count = T / (2 * kUnit);
        p.tokens = (int)((T + count - 1) / count + kUnit - 1) / kUnit * kUnit;
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

template <typename T, int N, int CPT, bool VECTOR, Mode MODE>
cudaError_t run_scan(const ScanArgs &a, const Pieces &p, int pieces, cudaStream_t st)
{
    using S = Shape<T, N, CPT, MODE>;
    auto k = ssm_scan_kernel<T, N, CPT, VECTOR, MODE>;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = allow_shared(k, S::smem, done);
    if (e != cudaSuccess) return e;
    const int bpg = blocks_per_group(a.D, a.G, N, CPT);
    k<<<dim3((unsigned)((long long)a.B * a.G * bpg), pieces), S::THREADS, S::smem, st>>>(a, p, bpg);
    return cudaGetLastError();
}

// What a call wants besides the outputs: the states for the backward, or only
// the backward's walk over its pieces.
struct Extra {
    float *points = nullptr;
    bool adjoint = false;
    Pieces back = {};
};

template <typename T, int N, bool VECTOR>
cudaError_t scan_typed(const ScanArgs &a, const Extra &x, cudaStream_t st, int *launches)
{
    cudaError_t e = cudaSuccess;
    if (x.adjoint) {
        e = run_scan<T, N, 1, VECTOR, ADJOINT>(a, x.back, x.back.count - 1, st);
        if (e == cudaSuccess) *launches += 1;
        return e;
    }
    Pieces p = plan(a.B, a.T, a.D, a.G, N, a.workspace);
    if (p.count > 1) {
        e = run_scan<T, N, 1, VECTOR, LOCAL>(a, p, p.count - 1, st);
        if (e != cudaSuccess) return e;
        *launches += 1;
    }
    p.points = x.points;
    *launches += 1;
    if (x.points) return run_scan<T, N, 1, VECTOR, POINTS>(a, p, p.count, st);
    if constexpr (kTwoChannels<T, N>)
        if (two_channels<T, N, VECTOR>(a.B, a.D, a.G)) return run_scan<T, N, 2, VECTOR, FULL>(a, p, p.count, st);
    return run_scan<T, N, 1, VECTOR, FULL>(a, p, p.count, st);
}

template <typename T, int N>
cudaError_t scan_by_layout(const ScanArgs &a, const Extra &x, cudaStream_t st, int *launches)
{
    return scan_vectors<T>(a) ? scan_typed<T, N, true>(a, x, st, launches) : scan_typed<T, N, false>(a, x, st, launches);
}

template <typename T, int N>
cudaError_t step_typed(const ScanArgs &a, cudaStream_t st)
{
    const int cb = 1024 / N, bpr = (a.D + cb - 1) / cb, rows = N / 4 < 4 ? N / 4 : 4;
    const unsigned blocks = (unsigned)((long long)((a.B + rows - 1) / rows) * bpr);
    const size_t quad = 4 * sizeof(T);
    if (aligned_to(a.Bm, quad) && aligned_to(a.Cm, quad) && a.bs.b % 4 == 0 && a.cs.b % 4 == 0)
        ssm_step_kernel<T, N, true><<<blocks, 256, 0, st>>>(a, bpr);
    else
        ssm_step_kernel<T, N, false><<<blocks, 256, 0, st>>>(a, bpr);
    return cudaGetLastError();
}

template <int N>
cudaError_t scan_n(const ScanArgs &a, const Extra &x, cudaStream_t st, int *launches)
{
    return a.bf16 ? scan_by_layout<__nv_bfloat16, N>(a, x, st, launches)
                  : scan_by_layout<float, N>(a, x, st, launches);
}

cudaError_t any_n(const ScanArgs &a, const Extra &x, cudaStream_t st, int *launches)
{
    switch (a.N) {
        case 8: return scan_n<8>(a, x, st, launches);
        case 16: return scan_n<16>(a, x, st, launches);
        case 32: return scan_n<32>(a, x, st, launches);
        default: return scan_n<64>(a, x, st, launches);
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
    return any_n(a, Extra{}, stream, launches);
}

cudaError_t launch_ssm_scan_checkpoints(const ScanArgs &a, float *states, cudaStream_t stream, int *launches)
{
    Extra x;
    x.points = states;
    return any_n(a, x, stream, launches);
}

cudaError_t launch_ssm_scan_adjoint(const ScanArgs &a, int pieces, int tokens, float *slots, float *sums,
                                    cudaStream_t stream, int *launches)
{
    Extra x;
    x.adjoint = true;
    x.back = {pieces, tokens, slots, sums, nullptr};
    return any_n(a, x, stream, launches);
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
