// Short causal depthwise convolution with an optional SiLU, in front of a
// token mixer: prompt, backward and single token.
//
//   pre[t, c] = bias[c] + sum_{j<W} weight[c, j] x[t - (W-1) + j, c],   y = pre or pre * sigmoid(pre)
//
// where the W-1 rows before a sequence are its carried state.  ("Token Mixer
// I", section "The Kimi Linear Model Architecture": q, k and v are
// Swish(ShortConv(W x)).)  Channels are independent and tokens touch only
// their W-1 predecessors, so the work is bound by HBM: each input row is read
// once and each output row written once.
//
// Every thread owns a few neighbouring channels (4, and 8 in a step, where the
// layout allows) and walks a run of tokens with the last W-1 rows in
// registers; neighbouring threads own neighbouring channels, so every access
// of a warp is one contiguous run of a token row.
#include <type_traits>

#include "ssm_internal.cuh"

namespace gdr {
namespace {

constexpr int kConvThreads = 128;
constexpr int kSms = 148;

// A vector in memory as register pairs, and back.
template <int VEC, typename V> __device__ __forceinline__ void widen(V v, typename Lanes<VEC>::P *p)
{
    float f[VEC];
    unpack(v, f);
    Lanes<VEC>::join(f, p);
}
template <int VEC, typename V> __device__ __forceinline__ V narrow(const typename Lanes<VEC>::P *p)
{
    float f[VEC];
    Lanes<VEC>::split(p, f);
    V v;
    pack(v, f);
    return v;
}

// The W taps of VEC neighbouring channels, and their biases.
template <int VEC, int W>
__device__ __forceinline__ void load_taps(const float *weight, const float *bias, int c0,
                                          typename Lanes<VEC>::P (*w)[Lanes<VEC>::N], typename Lanes<VEC>::P *b)
{
    const float *p = weight + (size_t)c0 * W;
    float f[W][VEC], g[VEC];
    if (W == 4 && (reinterpret_cast<uintptr_t>(weight) & 15) == 0) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float4 q = *(const float4 *)(p + v * W);
            f[0][v] = q.x;
            f[1][v] = q.y;
            f[2 < W ? 2 : 0][v] = q.z;
            f[3 < W ? 3 : 0][v] = q.w;
        }
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v)
#pragma unroll
            for (int j = 0; j < W; ++j) f[j][v] = p[v * W + j];
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) g[v] = bias ? bias[c0 + v] : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) Lanes<VEC>::join(f[j], w[j]);
    Lanes<VEC>::join(g, b);
}

// blockDim.x channel vectors by blockDim.y token runs.  Blocks are numbered
// along the channels first, so that those at work together read whole token
// rows (memory pages), not strips of far apart rows.
struct ConvGrid {
    dim3 block;
    int run, runs;        // tokens of a run, runs of a row
    int across;           // blocks along the channels
    long long down;       // blocks along the (batch, run) pairs
    unsigned blocks() const { return (unsigned)(across * down); }
};
// This thread's channel vector and (batch, run) pair.
struct ConvPlace {
    int vector;
    long long piece;
    long long row;        // of the block
};
__device__ __forceinline__ ConvPlace conv_place(int across)
{
    const unsigned down = blockIdx.x / across;
    return {(int)((blockIdx.x - down * across) * blockDim.x + threadIdx.x),
            (long long)down * blockDim.y + threadIdx.y, down};
}

// The run length: long enough that the W-1 rows read again at its start (and,
// backward, at its end) cost little, short enough that small problems still
// spread over the machine.
ConvGrid conv_grid(int B, int T, long long vectors, int widest, int threads_per_sm, int longest)
{
    ConvGrid g;
    int bx = 1;
    while (bx < widest && bx < vectors) bx *= 2;
    // whole warps along the channels; drop to 32 where a wider block would idle on the last vectors
    while (bx > 32 && (vectors + bx - 1) / bx * bx - vectors >= 32) bx /= 2;
    g.block = dim3(bx, kConvThreads / bx);
    const long long want = (long long)kSms * threads_per_sm;
    long long run = ((long long)B * T * vectors + want - 1) / want;
    run = (run + 7) / 8 * 8;
    g.run = (int)(run < 8 ? 8 : run > longest ? longest : run);
    g.runs = T > 0 ? (T + g.run - 1) / g.run : 1;
    const long long rows = (long long)B * g.runs;
    g.across = (int)((vectors + bx - 1) / bx);
    g.down = (rows + g.block.y - 1) / g.block.y;
    return g;
}

// Four rows a step and 64 registers keep 8 blocks on an SM: 2 x 8192 x 4096
// bf16 53 us (5.1 TB/s), against 71 with 16-byte vectors, eight rows and 4
// blocks.  The two special-function operations of a sigmoid take 30 of them.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kConvThreads, 8) conv_fwd_kernel(ConvArgs a, int run, int runs, int across)
{
    using V = typename Pack<T, VEC>::V;
    // rows in work; as many more are on their way from memory meanwhile
    constexpr int U = VEC * sizeof(T) > 8 ? 2 : 4;
    const int D = a.H * a.d;
    const ConvPlace at = conv_place(across);
    const int c0 = at.vector * VEC;
    const long long piece = at.piece;
    const int b = (int)(piece / runs);
    if (c0 >= D || b >= a.B) return;
    const int t0 = (int)(piece - (long long)b * runs) * run;
    const int head = c0 / a.d, j0 = c0 - head * a.d;
    const int len = row_length(a.lengths, b, a.T);

    const T *x = (const T *)a.x + b * a.xs.b + head * a.xs.h + j0;
    const T *st = a.state ? (const T *)a.state + (size_t)b * (W - 1) * D + c0 : nullptr;

    // the W-1 rows before the run, oldest first
    V before[W - 1];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        const int r = t0 - (W - 1) + i;
        before[i] = r >= 0 ? (r < len ? *(const V *)(x + r * a.xs.t) : zero_pack<V>())
                           : (st ? *(const V *)(st + (size_t)(W - 1 + r) * D) : zero_pack<V>());
    }
    // The thread of a row's first run also writes its final state.  `before` is
    // the whole carried state there, in registers, so state_out may be the same
    // buffer, and a row shorter than W-1 keeps what it has to keep.
    if (t0 == 0 && a.state_out) {
        T *so = (T *)a.state_out + (size_t)b * (W - 1) * D + c0;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const int r = len - (W - 1) + i;
            V v = zero_pack<V>();
            if (r >= 0) v = *(const V *)(x + r * a.xs.t);
#pragma unroll
            for (int k = 0; k < W - 1; ++k)
                if (r == k - (W - 1)) v = before[k];
            *(V *)(so + (size_t)i * D) = v;
        }
    }
    if (a.zero_tail) {
        T *tail = (T *)a.y + ((size_t)b * a.H + head) * a.T * a.d + j0;
        for (int t = max(t0, len); t < min(t0 + run, a.T); ++t) *(V *)(tail + (size_t)t * a.d) = zero_pack<V>();
    }
    int left = min(t0 + run, len) - t0;
    if (left <= 0) return;

    x += t0 * a.xs.t;
    T *y = (T *)a.y + (((size_t)b * a.H + head) * a.T + t0) * a.d + j0;
    V now[U], next[U];
    auto fetch = [&](V *rows, int n) {   // the next U rows, of which n exist
#pragma unroll
        for (int u = 0; u < U; ++u) {
            rows[u] = load_if((const V *)x, u < n);
            x += a.xs.t;
        }
    };
    fetch(now, left);
    using L = Lanes<VEC>;
    using P = typename L::P;
    P w[W][L::N], bias[L::N], win[W - 1][L::N];
    load_taps<VEC, W>(a.weight, a.bias, c0, w, bias);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) widen<VEC>(before[i], win[i]);
    for (; left > 0; left -= U) {
        fetch(next, left - U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            P cur[L::N], acc[L::N];
            widen<VEC>(now[u], cur);
#pragma unroll
            for (int v = 0; v < L::N; ++v) {
                P s = bias[v];
#pragma unroll
                for (int i = 0; i < W - 1; ++i) s = fma2(w[i][v], win[i][v], s);
                s = fma2(w[W - 1][v], cur[v], s);
                acc[v] = a.silu ? mul2(s, sigmoid2(s)) : s;
#pragma unroll
                for (int i = 0; i + 1 < W - 1; ++i) win[i][v] = win[i + 1][v];
                win[W - 2][v] = cur[v];
            }
            if (u < left) *(V *)y = narrow<VEC, V>(acc);
            y += a.d;
            now[u] = next[u];
        }
    }
}

// One token per row: x [B, D] (row stride xs.b), state [B, W-1, D] shifted in
// place.  A thread takes ROWS batch rows, so the taps are read once for them
// and all of its rows' loads are in flight together.
constexpr int kStepRows = 4;
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(ConvArgs a, int across)
{
    using V = typename Pack<T, VEC>::V;
    const int D = a.d;
    const ConvPlace at = conv_place(across);
    const int c0 = at.vector * VEC, b0 = (int)at.piece * kStepRows;
    if (c0 >= D) return;
    V rows[kStepRows][W];
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
        if (b0 + r >= a.B) break;
        const T *st = (const T *)a.state_out + (size_t)(b0 + r) * (W - 1) * D + c0;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) rows[r][i] = *(const V *)(st + (size_t)i * D);
        rows[r][W - 1] = *(const V *)((const T *)a.x + (b0 + r) * a.xs.b + c0);
    }
    using L = Lanes<VEC>;
    using P = typename L::P;
    P w[W][L::N], bias[L::N];
    load_taps<VEC, W>(a.weight, a.bias, c0, w, bias);
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
        if (b0 + r >= a.B) break;
        P acc[L::N];
#pragma unroll
        for (int v = 0; v < L::N; ++v) acc[v] = bias[v];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            P f[L::N];
            widen<VEC>(rows[r][i], f);
#pragma unroll
            for (int v = 0; v < L::N; ++v) acc[v] = fma2(w[i][v], f[v], acc[v]);
        }
        if (a.silu) {
#pragma unroll
            for (int v = 0; v < L::N; ++v) acc[v] = mul2(acc[v], sigmoid2(acc[v]));
        }
        *(V *)((T *)a.y + (size_t)(b0 + r) * D + c0) = narrow<VEC, V>(acc);
        T *st = (T *)a.state_out + (size_t)(b0 + r) * (W - 1) * D + c0;
#pragma unroll
        for (int i = 0; i < W - 1; ++i) *(V *)(st + (size_t)i * D) = rows[r][i + 1];
    }
}

// ------------------------------------------------------------- backward
//
//   dpre[t] = dy[t] act'(pre[t])   (0 behind the row's end),
//   dx[r]   = sum_j weight[j] dpre[r + W-1-j],   dweight[j] = sum_t dpre[t] x[t - (W-1) + j],
//   dbias   = sum_t dpre[t];   rows r < 0 are the gradient of the carried state, and the final
//   state's gradient adds to the rows it was copied from.
//
// One walk forward over a run and W-1 tokens beyond it: at token t the
// pre-activation is recomputed from the window of x, and row t-(W-1), whose
// last term that was, is written.  A thread sums dweight and dbias of its run
// in registers, a block over its runs in shared memory, and the blocks'
// partial sums are added by a second kernel in a fixed order, so the result
// does not depend on scheduling.  4 x 4096 x 2048 bf16: 58 us, 201 MB at 3.5
// TB/s (51 and, for the second kernel, 7); 128 registers a thread (and 28 bytes
// spilled at W = 4) leave 16 warps on an SM, and half of the issue slots are used (two channels a thread and more warps: 110 us and more).
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kConvThreads, 4) conv_bwd_kernel(ConvBwdArgs a, int run, int runs, int across, float *part)
{
    using V = typename Pack<T, VEC>::V;
    constexpr int U = VEC == 1 ? 8 : sizeof(T) == 4 ? 2 : 4;   // as in the forward
    const int D = a.H * a.d;
    const ConvPlace at = conv_place(across);
    const int c0 = at.vector * VEC;
    const long long piece = at.piece;
    const int b = (int)(piece / runs);
    using L = Lanes<VEC>;
    using P = typename L::P;
    P dw[W][L::N] = {}, db[L::N] = {};   // all bits 0 is 0

    if (c0 < D && b < a.B) {
        const int t0 = (int)(piece - (long long)b * runs) * run;
        const int head = c0 / a.d, j0 = c0 - head * a.d;
        const int len = row_length(a.lengths, b, a.T);
        const int t1 = min(t0 + run, a.T);            // rows [t0, t1) are this run's
        const bool first = t0 == 0;
        const T *x = (const T *)a.x + b * a.xs.b + head * a.xs.h + j0;
        const T *dy = (const T *)a.dy + b * a.dys.b + head * a.dys.h + j0;
        T *dx = (T *)a.dx + b * a.dxs.b + head * a.dxs.h + j0;
        const T *st = a.state ? (const T *)a.state + (size_t)b * (W - 1) * D + c0 : nullptr;
        const T *dso = a.dstate_out ? (const T *)a.dstate_out + (size_t)b * (W - 1) * D + c0 : nullptr;
        T *dst = a.dstate ? (T *)a.dstate + (size_t)b * (W - 1) * D + c0 : nullptr;

        P w[W][L::N], bias[L::N], win[W - 1][L::N], dp[W][L::N] = {};
        load_taps<VEC, W>(a.weight, a.bias, c0, w, bias);
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const int r = t0 - (W - 1) + i;
            V v = r >= 0 ? (r < len ? *(const V *)(x + r * a.xs.t) : zero_pack<V>())
                         : (st ? *(const V *)(st + (size_t)(W - 1 + r) * D) : zero_pack<V>());
            widen<VEC>(v, win[i]);
        }
        // rows the walk completes: [-(W-1), t1) from a row's first run, [t0, t1) from the others
        const int tend = t1 + (W - 1), live_end = min(len, tend), rmin = first ? -(W - 1) : t0;
        const T *xr = x + t0 * a.xs.t, *gr = dy + t0 * a.dys.t;
        V xin[U], gin[U], xnext[U], gnext[U];
        auto fetch = [&](V *xs, V *gs, int t) {   // U rows from t on
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool live = t + u < live_end;
                xs[u] = load_if((const V *)xr, live);
                gs[u] = load_if((const V *)gr, live);
                xr += a.xs.t;
                gr += a.dys.t;
            }
        };
        // U tokens; `inside`: all of them are the run's and live, and so are the rows they complete
        auto walk = [&](int t, auto inside) {
            constexpr bool FULL = decltype(inside)::value;
            T *dxr = dx + (t - (W - 1)) * a.dxs.t;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int tt = t + u;
                P cur[L::N], g[L::N], out[L::N];
                widen<VEC>(xin[u], cur);
                widen<VEC>(gin[u], g);
#pragma unroll
                for (int v = 0; v < L::N; ++v) {
                    P s = bias[v];
#pragma unroll
                    for (int i = 0; i < W - 1; ++i) s = fma2(w[i][v], win[i][v], s);
                    s = fma2(w[W - 1][v], cur[v], s);
                    P p = g[v];
                    if (a.silu) {   // q + s q (1 - q)
                        const P q = sigmoid2(s);
                        p = mul2(p, fma2(mul2(s, q), fma2(q, L::all(-1.f), L::all(1.f)), q));
                    }
                    if (!FULL && tt >= live_end) p = L::all(0.f);
#pragma unroll
                    for (int i = 0; i < W - 1; ++i) dp[i][v] = dp[i + 1][v];
                    dp[W - 1][v] = p;
                    if (FULL || tt < t1) {
#pragma unroll
                        for (int i = 0; i < W - 1; ++i) dw[i][v] = fma2(p, win[i][v], dw[i][v]);
                        dw[W - 1][v] = fma2(p, cur[v], dw[W - 1][v]);
                        db[v] = add2(db[v], p);
                    }
                    P acc = mul2(w[0][v], dp[W - 1][v]);
#pragma unroll
                    for (int j = 1; j < W; ++j) acc = fma2(w[j][v], dp[W - 1 - j][v], acc);
                    out[v] = acc;
#pragma unroll
                    for (int i = 0; i + 1 < W - 1; ++i) win[i][v] = win[i + 1][v];
                    win[W - 2][v] = cur[v];
                }
                const int r = tt - (W - 1);
                if (FULL || (r >= rmin && r < t1)) {
                    if (!FULL && dso && r >= len - (W - 1) && r < len) {
                        P f[L::N];
                        widen<VEC>(*(const V *)(dso + (size_t)(r - len + W - 1) * D), f);
#pragma unroll
                        for (int v = 0; v < L::N; ++v) out[v] = add2(out[v], f[v]);
                    }
                    const V o = narrow<VEC, V>(out);
                    if (FULL || r >= 0) *(V *)dxr = o;
                    else if (dst) *(V *)(dst + (size_t)(r + W - 1) * D) = o;
                }
                dxr += a.dxs.t;
            }
        };
        fetch(xin, gin, t0);
        for (int t = t0; t < tend; t += U) {
            fetch(xnext, gnext, t + U);
            if (t >= t0 + W - 1 && t + U <= t1 && t + U <= len) walk(t, std::true_type{});
            else walk(t, std::false_type{});
#pragma unroll
            for (int u = 0; u < U; ++u) {
                xin[u] = xnext[u];
                gin[u] = gnext[u];
            }
        }
    }

    // the block's runs, added in the order of threadIdx.y
    __shared__ float sum[kConvThreads][VEC];
    const int tid = threadIdx.y * blockDim.x + threadIdx.x;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        L::split(j < W ? dw[j < W ? j : 0] : db, sum[tid]);
        __syncthreads();
        if (threadIdx.y == 0 && c0 < D) {
            for (int k = 1; k < (int)blockDim.y; ++k)
#pragma unroll
                for (int v = 0; v < VEC; ++v) sum[tid][v] += sum[tid + k * blockDim.x][v];
#pragma unroll
            for (int v = 0; v < VEC; ++v) part[((size_t)at.row * (W + 1) + j) * D + c0 + v] = sum[tid][v];
        }
        __syncthreads();
    }
}

// Adds the blocks' partial sums [parts][W+1][D]: 32 columns a block, each by
// 32 threads that take every 32nd partial sum and join in a fixed tree.
__global__ void __launch_bounds__(1024)
conv_bwd_sum_kernel(const float *part, int parts, int D, int W, float *dweight, float *dbias)
{
    __shared__ float s[32][33];
    const int n = (W + 1) * D, col = blockIdx.x * 32 + threadIdx.x;
    float acc = 0.f;
    if (col < n)
        for (int p = threadIdx.y; p < parts; p += 32) acc += part[(size_t)p * n + col];
    s[threadIdx.y][threadIdx.x] = acc;
    for (int k = 16; k > 0; k >>= 1) {
        __syncthreads();
        if ((int)threadIdx.y < k) s[threadIdx.y][threadIdx.x] += s[threadIdx.y + k][threadIdx.x];
    }
    if (threadIdx.y == 0 && col < n) {
        const int j = col / D, c = col - j * D;
        if (j < W) dweight[(size_t)c * W + j] = s[0][threadIdx.x];
        else if (dbias) dbias[c] = s[0][threadIdx.x];
    }
}

// 16-byte accesses need every pointer and every stride to keep 16-byte
// alignment and the channels of a head to be a whole number of vectors.
template <typename T> bool conv_vectors(int d, int vec, const void *const *ptrs, int np, const RowStrides *s, int ns)
{
    if (d % vec) return false;
    for (int i = 0; i < np; ++i)
        if (ptrs[i] && !aligned_to(ptrs[i], vec * sizeof(T))) return false;
    for (int i = 0; i < ns; ++i)
        if (s[i].b % vec || s[i].h % vec || s[i].t % vec) return false;
    return true;
}

template <typename T, int VEC, int W>
cudaError_t conv_fwd(const ConvArgs &a, cudaStream_t st)
{
    const ConvGrid g = conv_grid(a.B, a.T, (long long)a.H * a.d / VEC, kConvThreads, 1024, 256);
    conv_fwd_kernel<T, VEC, W><<<g.blocks(), g.block, 0, st>>>(a, g.run, g.runs, g.across);
    return cudaGetLastError();
}

template <typename T, int VEC, int W>
cudaError_t conv_step(const ConvArgs &a, cudaStream_t st)
{
    const ConvGrid g = conv_grid((a.B + kStepRows - 1) / kStepRows, 1, a.d / VEC, kConvThreads, 512, 8);
    conv_step_kernel<T, VEC, W><<<g.blocks(), g.block, 0, st>>>(a, g.across);
    return cudaGetLastError();
}

// Four runs a block, so that a block's partial sums of dweight are few.
ConvGrid conv_bwd_grid(int B, int T, long long vectors) { return conv_grid(B, T, vectors, 32, 512, 256); }

template <typename T, int VEC, int W>
cudaError_t conv_bwd(const ConvBwdArgs &a, cudaStream_t st)
{
    const int D = a.H * a.d;
    const ConvGrid g = conv_bwd_grid(a.B, a.T, D / VEC);
    conv_bwd_kernel<T, VEC, W><<<g.blocks(), g.block, 0, st>>>(a, g.run, g.runs, g.across, (float *)a.workspace);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    conv_bwd_sum_kernel<<<((W + 1) * D + 31) / 32, dim3(32, 32), 0, st>>>((const float *)a.workspace, (int)g.down,
                                                                            D, W, a.dweight, a.dbias);
    return cudaGetLastError();
}

enum Form { FWD, STEP };

template <typename T, int VEC, int W, Form F>
cudaError_t conv_form(const ConvArgs &a, cudaStream_t st)
{
    if constexpr (F == FWD) return conv_fwd<T, VEC, W>(a, st);
    else return conv_step<T, VEC, W>(a, st);
}

template <typename T, int VEC, Form F>
cudaError_t by_width(const ConvArgs &a, cudaStream_t st)
{
    switch (a.W) {
        case 2: return conv_form<T, VEC, 2, F>(a, st);
        case 3: return conv_form<T, VEC, 3, F>(a, st);
        default: return conv_form<T, VEC, 4, F>(a, st);
    }
}

template <Form F>
cudaError_t by_type(const ConvArgs &a, cudaStream_t st)
{
    const void *p[] = {a.x, a.state, a.y, a.state_out};
    if (a.bf16)
        return conv_vectors<__nv_bfloat16>(a.d, F == FWD ? 4 : 8, p, 4, &a.xs, 1)
                   ? by_width<__nv_bfloat16, F == FWD ? 4 : 8, F>(a, st) : by_width<__nv_bfloat16, 1, F>(a, st);
    return conv_vectors<float>(a.d, 4, p, 4, &a.xs, 1) ? by_width<float, 4, F>(a, st) : by_width<float, 1, F>(a, st);
}

template <typename T, int VEC>
cudaError_t bwd_by_width(const ConvBwdArgs &a, cudaStream_t st)
{
    switch (a.W) {
        case 2: return conv_bwd<T, VEC, 2>(a, st);
        case 3: return conv_bwd<T, VEC, 3>(a, st);
        default: return conv_bwd<T, VEC, 4>(a, st);
    }
}

}  // namespace

cudaError_t launch_short_conv_fwd(const ConvArgs &a, cudaStream_t stream, int *launches)
{
    cudaError_t e = by_type<FWD>(a, stream);
    if (e == cudaSuccess) *launches += 1;
    return e;
}

cudaError_t launch_short_conv_step(const ConvArgs &a, cudaStream_t stream, int *launches)
{
    cudaError_t e = by_type<STEP>(a, stream);
    if (e == cudaSuccess) *launches += 1;
    return e;
}

size_t short_conv_bwd_workspace_bytes(int B, int H, int T, int d, int W)
{
    // the partial sums of whichever access width the call will take
    const long long D = (long long)H * d;
    const long long wide = d % 4 == 0 ? conv_bwd_grid(B, T, D / 4).down : 0, narrow = conv_bwd_grid(B, T, D).down;
    return (size_t)(wide > narrow ? wide : narrow) * (size_t)(W + 1) * (size_t)D * sizeof(float);
}

cudaError_t launch_short_conv_bwd(const ConvBwdArgs &a, cudaStream_t stream, int *launches)
{
    const void *p[] = {a.x, a.dy, a.dx, a.state, a.dstate_out, a.dstate};
    const RowStrides s[] = {a.xs, a.dys, a.dxs};
    cudaError_t e;
    if (a.bf16)
        e = conv_vectors<__nv_bfloat16>(a.d, 4, p, 6, s, 3) ? bwd_by_width<__nv_bfloat16, 4>(a, stream)
                                                            : bwd_by_width<__nv_bfloat16, 1>(a, stream);
    else
        e = conv_vectors<float>(a.d, 4, p, 6, s, 3) ? bwd_by_width<float, 4>(a, stream)
                                                    : bwd_by_width<float, 1>(a, stream);
    if (e == cudaSuccess) *launches += 2;
    return e;
}

}  // namespace gdr
