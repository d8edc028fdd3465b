"""fp64 CPU oracle of the short causal convolution and the selective state
space scan -- TEST INFRASTRUCTURE, as the rest of this package.

Plain walks over the tokens in numpy, written from the formulas:

    conv   pre[t,c] = bias[c] + sum_j w[c,j] x[t-(W-1)+j, c],  y = pre or pre sigmoid(pre)
    scan   h_t[n] = exp(delta_t A[n]) h_{t-1}[n] + delta_t x_t B_t[n],
           y_t = (sum_n C_t[n] h_t[n] + D x_t) z_t sigmoid(z_t)

Token rows are [B,T,D], states [B,W-1,D] and [B,D,N].

``*_bound`` give, for every element of a result, how far fp32 arithmetic in
any order may take it from the exact value (before the result is rounded to
its own type).  Each result is a sum of products of inputs, decays and gates.
With every factor replaced by its absolute value, and every factor that is
computed with a relative error e multiplied by 1 + e, the sum grows by at
least what the errors can change; the difference of the two sums is the bound.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24            # half a unit in the last place of fp32, relative
EX2 = 4 * U               # the hardware's 2^x (measured 2.4 U)
LOG1P = 3 * U             # the polynomial of log(1 + e)


def _f64(x):
    if x is None:
        return None
    if hasattr(x, "detach"):
        x = x.detach().double().cpu().numpy()
    return np.asarray(x, np.float64)


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-x))


def _sigmoid_err(x):
    """Relative error of the fp32 sigmoid: the exponent's two roundings times its size, 2^x, 1 + ., 1 / ."""
    return 2 * np.abs(x) * U + EX2 + 4 * U


def _ends(lengths, B, T):
    return np.full(B, T) if lengths is None else np.clip(np.asarray(_f64(lengths), np.int64), 0, T)


# ------------------------------------------------------------- convolution

def _conv_src(x, W, state, ends):
    B, T, D = x.shape
    src = np.zeros((B, W - 1 + T, D))
    if state is not None:
        src[:, :W - 1] = state
    for b in range(B):
        src[b, W - 1:W - 1 + ends[b]] = x[b, :ends[b]]
    return src


def conv_fwd(x, weight, bias=None, state=None, act=True, lengths=None):
    """(y, state_out, bound of y); y is 0 behind a row's end."""
    x, w, bias, state = _f64(x), _f64(weight), _f64(bias), _f64(state)
    B, T, D = x.shape
    W = w.shape[1]
    ends = _ends(lengths, B, T)
    src = _conv_src(x, W, state, ends)
    y, bound = np.zeros((B, T, D)), np.zeros((B, T, D))
    for b in range(B):
        for t in range(ends[b]):
            taps = w.T * src[b, t:t + W]
            pre = taps.sum(0) + (0 if bias is None else bias)
            mag = np.abs(taps).sum(0) + (0 if bias is None else np.abs(bias))
            err = (W + 1) * U * mag
            if act:
                y[b, t] = pre * sigmoid(pre)
                # |d silu| < 1.1, and the sigmoid's own error and the product's
                bound[b, t] = 1.1 * err + np.abs(y[b, t]) * (_sigmoid_err(pre) + U)
            else:
                y[b, t], bound[b, t] = pre, err
    out = np.stack([src[b, ends[b]:ends[b] + W - 1] for b in range(B)]) if B else np.zeros((0, W - 1, D))
    return y, out, bound * 1.01


def conv_bwd(x, weight, dy, bias=None, state=None, dstate_out=None, act=True, lengths=None):
    """dict name -> (gradient, bound) for dx, dweight, dbias, dstate."""
    x, w, dy = _f64(x), _f64(weight), _f64(dy)
    bias, state, dso = _f64(bias), _f64(state), _f64(dstate_out)
    B, T, D = x.shape
    W = w.shape[1]
    ends = _ends(lengths, B, T)
    src = _conv_src(x, W, state, ends)
    dsrc, msrc = np.zeros_like(src), np.zeros_like(src)
    dw, mw = np.zeros((D, W)), np.zeros((D, W))
    db, mb = np.zeros(D), np.zeros(D)
    n = 0
    for b in range(B):
        for t in range(ends[b]):
            n += 1
            taps = w.T * src[b, t:t + W]
            pre = taps.sum(0) + (0 if bias is None else bias)
            mag = np.abs(taps).sum(0) + (0 if bias is None else np.abs(bias))
            p, e = dy[b, t].copy(), np.zeros(D)
            if act:
                q = sigmoid(pre)
                slope = q + pre * q * (1 - q)
                # |silu''| <= 1/2; terms of the slope are at most 1 and 0.3
                e = np.abs(p) * (0.5 * (W + 1) * U * mag + (1 + 0.3) * (2 * _sigmoid_err(pre) + 4 * U))
                p = p * slope
            dsrc[b, t:t + W] += w.T * p
            msrc[b, t:t + W] += np.abs(w.T) * (np.abs(p) * (W + 2) * U + e)
            dw += (p * src[b, t:t + W]).T
            mw += (np.abs(src[b, t:t + W]) * e).T
            mb += e
            db += p
    # sums over n terms in fp32, in any order of at most n + 1 roundings each
    aw, ab = np.zeros((D, W)), np.zeros(D)
    for b in range(B):
        for t in range(ends[b]):
            taps = w.T * src[b, t:t + W]
            pre = taps.sum(0) + (0 if bias is None else bias)
            p = np.abs(dy[b, t])
            if act:
                q = sigmoid(pre)
                p = p * np.abs(q + pre * q * (1 - q))
            aw += (p * np.abs(src[b, t:t + W])).T
            ab += p
    mw += (n + 2) * U * aw
    mb += (n + 2) * U * ab
    if dso is not None:
        for b in range(B):
            dsrc[b, ends[b]:ends[b] + W - 1] += dso[b]
            msrc[b, ends[b]:ends[b] + W - 1] += 2 * U * np.abs(dsrc[b, ends[b]:ends[b] + W - 1])
    return {"dx": (dsrc[:, W - 1:], msrc[:, W - 1:] * 1.01), "dweight": (dw, mw * 1.01), "dbias": (db, mb * 1.01),
            "dstate": (dsrc[:, :W - 1], msrc[:, :W - 1] * 1.01)}


# --------------------------------------------------------------------- scan

class _Scan:
    """The scan's factors in fp64; with `worst`, their absolute values grown by their fp32 errors."""

    def __init__(self, x, dt, A, Bm, Cm, D_skip, z, dt_bias, softplus, lengths, worst):
        x, dt, A, Bm, Cm = (_f64(t) for t in (x, dt, A, Bm, Cm))
        D_skip, z, dt_bias = _f64(D_skip), _f64(z), _f64(dt_bias)
        B, T, D = x.shape
        G, N = Bm.shape[2:]
        self.shape = B, T, D, G, N
        ends = _ends(lengths, B, T)
        live = (np.arange(T)[None] < ends[:, None])[..., None]
        self.live = live
        p = np.where(live, dt, 0) + (0 if dt_bias is None else dt_bias)
        if softplus:
            delta = np.maximum(p, 0) + np.log1p(np.exp(-np.abs(p)))
            slope = sigmoid(p)
        else:
            delta, slope = p, np.ones_like(p)
        x = np.where(live, x, 0)
        delta, slope = np.where(live, delta, 0), np.where(live, slope, 0)
        Bc = np.where(live[..., None], np.repeat(Bm, D // G, axis=2), 0)
        Cc = np.where(live[..., None], np.repeat(Cm, D // G, axis=2), 0)
        gate = np.ones_like(x) if z is None else np.where(live, z * sigmoid(z), 0)
        dgate = np.zeros_like(x) if z is None else np.where(live, sigmoid(z) * (1 + z * (1 - sigmoid(z))), 0)
        skip = np.zeros(D) if D_skip is None else D_skip
        a = np.exp(delta[..., None] * A)
        grow = 1.0
        if worst:
            # the bias's rounding moves the softplus by U |p| at most; its exponential has two
            # roundings of the exponent, 2^x and the polynomial; and the sum
            ed = (3 * np.abs(p) * U + EX2 + LOG1P + 3 * U) if softplus else U * np.ones_like(p)
            # the exponent delta A log2(e): three roundings and delta's error, times its size; 2^x
            a = a * (1 + (np.abs(delta[..., None] * A) * (3 * U + ed[..., None]) + EX2) + 2 * U)
            delta = np.abs(delta) * (1 + ed)
            es = 0 if z is None else _sigmoid_err(z)
            gate = np.abs(gate) * (1 + es + 2 * U)
            dgate = (np.zeros_like(x) if z is None else
                     np.where(live, sigmoid(z) * (1 + np.abs(z) * (1 - sigmoid(z))), 0) * (1 + 3 * es + 6 * U))
            slope = slope * (1 + (_sigmoid_err(p) + np.abs(p) * U if softplus else 0))
            x, Bc, Cc, A, skip = np.abs(x), np.abs(Bc), np.abs(Cc), np.abs(A), np.abs(skip)
            grow = 1 + 4 * U          # the roundings of one term of a sum over tokens
        self.x, self.delta, self.slope, self.B, self.C, self.A = x, delta, slope, Bc, Cc, A
        self.gate, self.dgate, self.skip, self.a, self.grow = gate, dgate, skip, a, grow
        self.worst = worst

    def states(self, h0):
        B, T, D, G, N = self.shape
        h = np.zeros((B, D, N)) if h0 is None else (np.abs(_f64(h0)) if self.worst else _f64(h0).copy())
        hs = [h]
        for t in range(T):
            h = self.a[:, t] * h + (self.delta[:, t] * self.x[:, t])[..., None] * self.B[:, t] * self.grow
            hs.append(h)
        return hs

    def fwd(self, h0):
        B, T, D, G, N = self.shape
        hs = self.states(h0)
        sums = 1 + (N + 2) * U if self.worst else 1.0
        core = np.stack([(self.C[:, t] * hs[t + 1]).sum(-1) for t in range(T)], 1) if T else np.zeros((B, 0, D))
        core = (core + self.skip * self.x) * sums
        return hs, np.where(self.live, core, 0)

    def bwd(self, dy, h0, dh_T):
        B, T, D, G, N = self.shape
        dy = np.where(self.live, _f64(dy), 0)
        g = np.zeros((B, D, N)) if dh_T is None else _f64(dh_T).copy()
        if self.worst:
            dy, g = np.abs(dy), np.abs(g)
        hs, core = self.fwd(h0)
        dz, dcore = dy * core * self.dgate, dy * self.gate
        over_n = 1 + (N + 4) * U if self.worst else 1.0
        over_d = 1 + (D // G + 4) * U if self.worst else 1.0
        over_t = 1 + (B * T + 4) * U if self.worst else 1.0
        dx, dp = np.zeros((B, T, D)), np.zeros((B, T, D))
        dB, dC, dA = np.zeros((B, T, G, N)), np.zeros((B, T, G, N)), np.zeros((D, N))
        for t in range(T - 1, -1, -1):
            g = g + dcore[:, t, :, None] * self.C[:, t] * self.grow
            dC[:, t] = (dcore[:, t, :, None] * hs[t + 1]).reshape(B, G, D // G, N).sum(2)
            dB[:, t] = (g * (self.delta[:, t] * self.x[:, t])[..., None]).reshape(B, G, D // G, N).sum(2)
            w = self.a[:, t] * g * hs[t]
            du = (g * self.B[:, t]).sum(-1)
            dp[:, t] = (du * self.x[:, t] + (w * self.A).sum(-1)) * self.slope[:, t]
            dx[:, t] = du * self.delta[:, t] + dcore[:, t] * self.skip
            dA += (w * self.delta[:, t, :, None]).sum(0)
            g = self.a[:, t] * g
        dp = np.where(self.live, dp, 0)
        return {"dx": dx * over_n, "ddt": dp * over_n, "dA": dA * over_t, "dB": dB * over_d, "dC": dC * over_d,
                "dD": (dcore * self.x).sum((0, 1)) * over_t, "dz": dz, "ddt_bias": dp.sum((0, 1)) * over_t * over_n,
                "dh0": g}


def scan_fwd(x, dt, A, Bm, Cm, D_skip=None, z=None, dt_bias=None, softplus=True, h0=None, lengths=None):
    """(y, h_T, bound of y, bound of h_T); y is 0 behind a row's end."""
    out = []
    for worst in (False, True):
        s = _Scan(x, dt, A, Bm, Cm, D_skip, z, dt_bias, softplus, lengths, worst)
        hs, core = s.fwd(h0)
        out.append((core * s.gate, hs[-1]))
    s = _Scan(x, dt, A, Bm, Cm, D_skip, z, dt_bias, softplus, lengths, False)
    # the growth of the absolute sums: |sum| with errors minus |sum| without
    hs, core = _plain_abs(s).fwd(None if h0 is None else np.abs(_f64(h0)))
    base = (core * np.abs(s.gate), hs[-1])
    return out[0][0], out[0][1], (out[1][0] - base[0]) * 1.01, (out[1][1] - base[1]) * 1.01


def _plain_abs(s):
    for k in ("x", "delta", "B", "C", "A", "skip", "gate"):
        setattr(s, k, np.abs(getattr(s, k)))
    return s


def scan_bwd(x, dt, A, Bm, Cm, dy, D_skip=None, z=None, dt_bias=None, softplus=True, h0=None, dh_T=None,
             lengths=None):
    """dict name -> (gradient, bound); dz is 0 without a gate, dD without a skip."""
    args = (x, dt, A, Bm, Cm, D_skip, z, dt_bias, softplus, lengths)
    exact = _Scan(*args, False).bwd(dy, h0, dh_T)
    worst = _Scan(*args, True).bwd(dy, h0, dh_T)
    s = _plain_abs(_Scan(*args, False))
    zz = None if z is None else _f64(z)
    if zz is not None:
        s.dgate = np.where(s.live, sigmoid(zz) * (1 + np.abs(zz) * (1 - sigmoid(zz))), 0)
    base = s.bwd(np.abs(_f64(dy)), None if h0 is None else np.abs(_f64(h0)),
                 None if dh_T is None else np.abs(_f64(dh_T)))
    return {k: (exact[k], (worst[k] - base[k]) * 1.01) for k in exact}
