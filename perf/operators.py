"""The short causal convolution and the selective state space scan, as measured operators.

A case names one operator (``op``) and its sizes.  ``run`` makes one pass: with ``own`` through
the library's entry points, otherwise in plain torch operations in 32 bits.  ``exact`` restates
every operator in 64 bits as a walk over the tokens.

Shapes (channels D, or heads x head width for the convolution that feeds the gated delta rule;
taps W; state size N; groups G that share B and C):

    short convolution   x [B,T,D] or [B,H,T,d], weight [D,W], bias [D], state [B,W-1,D]
    selective scan      x, dt, z [B,T,D], A [D,N], Bm, Cm [B,T,G,N], D_skip, dt_bias [D], h0 [B,D,N]

A row with ``lengths`` ends before T: what lies behind is no input, the output is zero there and
the state is the one at the row's length.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def _conv(op, name=None, B=1, T=1, heads=1, d=128, W=4, dtype="bf16", act=True, bias=True, state=True, ragged=False):
    c = dict(op=op, B=B, T=T, heads=heads, d=d, W=W, dtype=dtype, act=act, bias=bias, state=state, ragged=ragged)
    return dict(c, name=name) if name else c


def _scan(op, name=None, B=1, T=1, D=128, N=16, G=1, dtype="bf16", z=True, skip=True, softplus=True, state=True,
          ragged=False):
    c = dict(op=op, B=B, T=T, D=D, N=N, G=G, dtype=dtype, z=z, skip=skip, softplus=softplus, state=state,
             ragged=ragged)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the convolution in front of a gated delta rule layer's prompt: a projection's token rows in,
        # the layer's [B,H,T,d] out
        _conv("conv_fwd", "conv_prompt", B=2, T=8192, heads=32, d=128),
        # a batch of prompts of different lengths, an odd width, three taps, no activation
        _conv("conv_fwd", "conv_prompt_ragged", B=5, T=1037, d=1001, W=3, dtype="fp32", act=False, bias=False,
              ragged=True),
        # one training step's gradients
        _conv("conv_bwd", "conv_train", B=4, T=4096, d=2048, state=False),
        # gradients of a small odd problem with a carried state and ragged rows
        _conv("conv_bwd", "conv_train_odd", B=3, T=333, d=130, dtype="fp32", ragged=True),
        # one token for every row of a full serving batch
        _conv("conv_step", "conv_step_b256", B=256, d=4096),
        # one token of one request: latency
        _conv("conv_step", "conv_step_b1", B=1, d=2048, dtype="fp32"),
        # a prompt through the scan, gated, x and z being the halves of one projection
        _scan("scan_fwd", "scan_prompt", B=2, T=8192, D=4096),
        # few channels and long prompts of different lengths, two groups
        _scan("scan_fwd", "scan_long_ragged", B=2, T=20011, D=520, N=8, G=2, dtype="fp32", z=False, ragged=True),
        # one training step's gradients
        _scan("scan_bwd", "scan_train", B=4, T=4096, D=2048),
        # gradients of a small odd problem with a carried state and ragged rows
        _scan("scan_bwd", "scan_train_odd", B=3, T=333, D=130, N=8, dtype="fp32", ragged=True),
        # one token for every row of a full serving batch: the state is read and written
        _scan("scan_step", "scan_step_b256", B=256, D=4096),
        # one token of one request: latency
        _scan("scan_step", "scan_step_b1", B=1, D=2048, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_bwd", "scan_step"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    step = op.endswith("step")
    B = _log(rng, 1, 256) if step else _log(rng, 1, 8)
    D = _log(rng, 32, 4096)
    if rng.random() < 0.6:
        D = max(32, D // 32 * 32)      # whole vectors, as projections have; else any width
    # a pass costs no more than the largest listed one of its kind
    most = (1 << 20) if step else (1 << 26) if op.startswith("conv") and op.endswith("fwd") else (1 << 25)
    T = 1 if step else max(1, min(_log(rng, 1, 32768), most // (2 * B * D)))
    if op.startswith("conv"):
        heads = rng.choice([1, 1, 4]) if D % 32 == 0 and not step else 1
        return _conv(op, B=B, T=T, heads=heads, d=D // heads, W=rng.choice([2, 3, 4, 4]), dtype=dtype,
                     act=rng.random() < 0.8, bias=rng.random() < 0.5, state=step or rng.random() < 0.5,
                     ragged=not step and rng.random() < 0.4)
    G = rng.choice([1, 1, 2, 4]) if D % 4 == 0 else 1
    return _scan(op, B=B, T=T, D=D, N=rng.choice([8, 16, 16]), G=G, dtype=dtype, z=rng.random() < 0.6,
                 skip=rng.random() < 0.8, softplus=rng.random() < 0.8, state=step or rng.random() < 0.5,
                 ragged=not step and rng.random() < 0.4)


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev) * scale).to(dtype)

    B, T, op = case["B"], case["T"], case["op"]
    s = {"op": op}
    if case["ragged"]:
        n = torch.randint(0, T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        n[-1] = T                  # one whole row
        if B > 2:
            n[0] = 0               # one empty row
        s["lengths"] = n
    else:
        s["lengths"] = None
    if op.startswith("conv"):
        H, d, W = case["heads"], case["d"], case["W"]
        D = H * d
        # a depthwise weight as it is initialised: uniform in 1/sqrt(taps)
        s["weight"] = (torch.rand(D, W, generator=g, device=dev) * 2 - 1) * W ** -0.5
        s["bias"] = normal(D, scale=0.2, dtype=torch.float32) if case["bias"] else None
        s["act"] = "silu" if case["act"] else None
        if op == "conv_step":
            s["x"], s["state"] = normal(B, D), normal(B, W - 1, D)
            return s
        s["x"] = normal(B, T, H, d).transpose(1, 2) if H > 1 else normal(B, T, D)
        s["state"] = normal(B, W - 1, D) if case["state"] else None
        if op == "conv_bwd":
            s["dy"] = normal(B, H, T, d) if H > 1 else normal(B, T, D)
            s["dstate_out"] = normal(B, W - 1, D) if case["state"] else None
        return s
    D, N, G = case["D"], case["N"], case["G"]
    # A and the time step as the layer is initialised: A around -(1..N), softplus(dt_bias)
    # log-uniform in [0.001, 0.1]
    s["A"] = -torch.arange(1, N + 1, device=dev, dtype=torch.float32) * torch.exp(
        normal(D, N, scale=0.1, dtype=torch.float32))
    step = torch.exp(torch.rand(D, generator=g, device=dev) * math.log(100.0) + math.log(0.001))
    s["softplus"] = case["softplus"]
    s["D_skip"] = 1 + normal(D, scale=0.1, dtype=torch.float32) if case["skip"] else None
    lead = (B,) if op == "scan_step" else (B, T)
    if case["softplus"]:
        s["dt"] = normal(*lead, D, scale=0.5)
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    else:
        s["dt"] = (step * (0.5 + torch.rand(*lead, D, generator=g, device=dev))).to(dt)
        s["dt_bias"] = None
    # x and z are the halves of one projection's rows; dt's low-rank part, B and C share another's
    if case["z"]:
        xz = normal(*lead, 2 * D)
        s["x"], s["z"] = xz[..., :D], xz[..., D:]
    else:
        s["x"], s["z"] = normal(*lead, D), None
    R, GN = max(16, D // 16 // 16 * 16), G * N
    rbc = normal(*lead, R + 2 * GN)
    s["Bm"] = rbc[..., R:R + GN].unflatten(-1, (G, N))
    s["Cm"] = rbc[..., R + GN:].unflatten(-1, (G, N))
    if op == "scan_step":
        s["h"] = normal(B, D, N, scale=0.3, dtype=torch.float32)
        return s
    s["h0"] = normal(B, D, N, scale=0.3, dtype=torch.float32) if case["state"] else None
    if op == "scan_bwd":
        s["dy"] = normal(B, T, D)
        s["dh_T"] = normal(B, D, N, dtype=torch.float32) if case["state"] else None
    return s


# ------------------------------------------------------ one pass, each way

def run(s):
    op = s["op"]
    if own:
        import gated_delta_rule_89_b200 as gdr
        if op == "conv_fwd":
            y, st = gdr.short_conv_fwd(s["x"], s["weight"], s["bias"], s["state"], activation=s["act"],
                                       lengths=s["lengths"])
            return {"y": y, "state": st}
        if op == "conv_step":
            y = gdr.short_conv_step(s["x"], s["state"], s["weight"], s["bias"], activation=s["act"])
            return {"y": y, "state": s["state"]}
        if op == "conv_bwd":
            dx, dw, db, ds = gdr.short_conv_bwd(s["x"], s["weight"], s["dy"], s["bias"], s["state"], s["dstate_out"],
                                                activation=s["act"], lengths=s["lengths"])
            return {"dx": dx, "dweight": dw, "dbias": db, "dstate": ds}
        if op == "scan_fwd":
            y, h = gdr.ssm_scan_fwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], D_skip=s["D_skip"], z=s["z"],
                                    dt_bias=s["dt_bias"], dt_softplus=s["softplus"], h0=s["h0"], lengths=s["lengths"])
            return {"y": y, "h": h}
        if op == "scan_step":
            y = gdr.ssm_scan_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["h"], D_skip=s["D_skip"], z=s["z"],
                                  dt_bias=s["dt_bias"], dt_softplus=s["softplus"])
            return {"y": y, "h": s["h"]}
        names = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")
        return dict(zip(names, gdr.ssm_scan_bwd(
            s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dy"], D_skip=s["D_skip"], z=s["z"], dt_bias=s["dt_bias"],
            dt_softplus=s["softplus"], h0=s["h0"], dh_T=s["dh_T"], lengths=s["lengths"])))
    return {"conv_fwd": _conv_fwd, "conv_step": _conv_step, "conv_bwd": _conv_bwd,
            "scan_fwd": _scan_fwd, "scan_step": _scan_step, "scan_bwd": _scan_bwd}[op](s)


def _rows(x):
    """[B,H,T,d] or [B,T,D] as fp32 token rows [B,T,D]."""
    return (x.transpose(1, 2).flatten(2) if x.dim() == 4 else x).float()


def _heads(y, like):
    """Token rows back to the layout and type of `like`."""
    if like.dim() == 4:
        y = y.unflatten(2, (like.shape[1], like.shape[3])).transpose(1, 2)
    return y.to(like.dtype).contiguous()


def _live(s, B, T, device):
    """[B,T,1]: whether a token lies before its row's end."""
    t = torch.arange(T, device=device)
    if s["lengths"] is None:
        return torch.ones(B, T, 1, dtype=torch.bool, device=device)
    return (t < s["lengths"][:, None])[..., None]


def _padded(s, x):
    """The token rows with the W-1 rows before them."""
    B, T, D = x.shape
    before = x.new_zeros(B, s["weight"].shape[1] - 1, D) if s["state"] is None else s["state"].float()
    return torch.cat([before, x], 1)


def _preact(s, xp, T):
    w = s["weight"]
    pre = sum(xp[:, j:j + T] * w[:, j] for j in range(w.shape[1]))
    return pre if s["bias"] is None else pre + s["bias"]


def _tail_rows(s, B, T, device):
    """Indices in the padded rows of the W-1 rows before each row's end, [B,W-1]."""
    n = torch.full((B,), T, device=device) if s["lengths"] is None else s["lengths"].long()
    return n[:, None] + torch.arange(s["weight"].shape[1] - 1, device=device)


def _conv_fwd(s):
    x = _rows(s["x"])
    B, T, D = x.shape
    xp = _padded(s, x)
    y = _preact(s, xp, T)
    if s["act"]:
        y = y * torch.sigmoid(y)
    y = torch.where(_live(s, B, T, x.device), y, 0.0)
    at = _tail_rows(s, B, T, x.device)[..., None].expand(-1, -1, D)
    return {"y": _heads(y, s["x"]), "state": xp.gather(1, at).to(s["x"].dtype)}


def _conv_step(s):
    xp = _padded(s, s["x"].float()[:, None])
    y = _preact(s, xp, 1)[:, 0]
    if s["act"]:
        y = y * torch.sigmoid(y)
    s["state"].copy_(xp[:, 1:])
    return {"y": y.to(s["x"].dtype), "state": s["state"]}


def _conv_bwd(s):
    x, dy, w = _rows(s["x"]), _rows(s["dy"]), s["weight"]
    B, T, D = x.shape
    W = w.shape[1]
    live = _live(s, B, T, x.device)
    xp = _padded(s, torch.where(live, x, 0.0))
    pre = _preact(s, xp, T)
    if s["act"]:
        sg = torch.sigmoid(pre)
        dy = dy * (sg * (1 + pre * (1 - sg)))
    dy = torch.where(live, dy, 0.0)
    dxp = sum(torch.nn.functional.pad(dy * w[:, j], (0, 0, j, W - 1 - j)) for j in range(W))
    if s["dstate_out"] is not None:
        at = _tail_rows(s, B, T, x.device)[..., None].expand(-1, -1, D)
        dxp.scatter_add_(1, at, s["dstate_out"].float())
    dw = torch.stack([(dy * xp[:, j:j + T]).sum((0, 1)) for j in range(W)], 1)
    return {"dx": _heads(dxp[:, W - 1:], s["x"]), "dweight": dw,
            "dbias": None if s["bias"] is None else dy.sum((0, 1)),
            "dstate": None if s["state"] is None else dxp[:, :W - 1].to(s["x"].dtype)}


def _recurrence(a, b):
    """r_t = a_t r_{t-1} + b_t over dim 1, by doubling: after the pass with distance k every entry
    covers the 2k tokens up to it."""
    k = 1
    while k < b.shape[1]:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _delta(s, live):
    """The time steps (0 behind a row's end: the state stands still) and their derivative."""
    p = s["dt"].float()
    if s["dt_bias"] is not None:
        p = p + s["dt_bias"]
    if not s["softplus"]:
        return torch.where(live, p, 0.0), live.to(p.dtype)
    # log(1 + e^p) without loss at either end
    return (torch.where(live, p.clamp(min=0) + torch.log1p(torch.exp(-p.abs())), 0.0),
            torch.where(live, torch.sigmoid(p), 0.0))


def _per_channel(m, D):
    """[...,G,N] as fp32 [...,D,N]: every channel of a group reads the group's row."""
    return m.float().repeat_interleave(D // m.shape[-2], dim=-2)


def _states(s, live):
    x = torch.where(live, s["x"].float(), 0.0)
    delta, slope = _delta(s, live)
    Bd = _per_channel(torch.where(live[..., None], s["Bm"], 0), x.shape[-1])
    a = torch.exp(delta[..., None] * s["A"])
    b = (delta * x)[..., None] * Bd
    if s["h0"] is not None:
        b[:, 0] += a[:, 0] * s["h0"]
    return x, delta, slope, Bd, a, _recurrence(a, b)


def _scan_fwd(s):
    B, T, D = s["x"].shape
    live = _live(s, B, T, s["x"].device)
    x, _, _, _, _, h = _states(s, live)
    y = (h * _per_channel(torch.where(live[..., None], s["Cm"], 0), D)).sum(-1)
    if s["D_skip"] is not None:
        y = y + x * s["D_skip"]
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    return {"y": torch.where(live, y, 0.0).to(s["x"].dtype), "h": h[:, -1].clone()}


def _scan_step(s):
    x, D = s["x"].float(), s["x"].shape[-1]
    delta, _ = _delta(s, torch.ones_like(x, dtype=torch.bool))
    h = torch.exp(delta[..., None] * s["A"]) * s["h"] + (delta * x)[..., None] * _per_channel(s["Bm"], D)
    y = (h * _per_channel(s["Cm"], D)).sum(-1)
    if s["D_skip"] is not None:
        y = y + x * s["D_skip"]
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    s["h"].copy_(h)
    return {"y": y.to(s["x"].dtype), "h": s["h"]}


def _scan_bwd(s):
    B, T, D = s["x"].shape
    G, N = s["Bm"].shape[-2:]
    dt = s["x"].dtype
    live = _live(s, B, T, s["x"].device)
    x, delta, slope, Bd, a, h = _states(s, live)
    Cd = _per_channel(torch.where(live[..., None], s["Cm"], 0), D)
    ds = torch.where(live, s["dy"].float(), 0.0)
    dz = None
    if s["z"] is not None:
        z = torch.where(live, s["z"].float(), 0.0)
        sg = torch.sigmoid(z)
        y = (h * Cd).sum(-1)
        if s["D_skip"] is not None:
            y = y + x * s["D_skip"]
        dz = (ds * y * (sg * (1 + z * (1 - sg)))).to(dt)
        ds = ds * (z * sg)
    dC = (ds[..., None] * h).unflatten(2, (G, D // G)).sum(3).to(dt)
    # the adjoint of the state: g_t = ds_t C_t + a_{t+1} g_{t+1}, a walk from the end
    g = ds[..., None] * Cd
    del Cd
    if s["dh_T"] is not None:
        g[:, -1] += s["dh_T"]
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    g = _recurrence(after.flip(1), g.flip(1)).flip(1)
    del after
    before = h.new_zeros(B, 1, D, N) if s["h0"] is None else s["h0"][:, None]
    w = g * a * torch.cat([before, h[:, :-1]], 1)
    dh0 = None if s["h0"] is None else a[:, 0] * g[:, 0]
    del a, h
    dB = (g * (delta * x)[..., None]).unflatten(2, (G, D // G)).sum(3).to(dt)
    du = (g * Bd).sum(-1)
    dp = (du * x + (w * s["A"]).sum(-1)) * slope
    dx = du * delta
    if s["D_skip"] is not None:
        dx = dx + ds * s["D_skip"]
    return {"dx": dx.to(dt), "ddt": dp.to(dt), "dA": (w * delta[..., None]).sum((0, 1)), "dB": dB, "dC": dC,
            "dD": None if s["D_skip"] is None else (ds * x).sum((0, 1)), "dz": dz,
            "ddt_bias": None if s["dt_bias"] is None else dp.sum((0, 1)), "dh0": dh0}


# ---------------------------------------------------------------- the work

def work(case):
    """Each input read once, each output written once; multiplications, additions and exponentials
    of the formulas."""
    e = 2 if case["dtype"] == "bf16" else 4
    B, T, op = case["B"], case["T"], case["op"]
    if op.startswith("conv"):
        D, W = case["heads"] * case["d"], case["W"]
        params, state = 4 * D * (W + case["bias"]), e * B * (W - 1) * D
        if op == "conv_bwd":
            return {"bytes": 3 * e * B * T * D + 2 * params + (3 * state if case["state"] else 0),
                    "flops": B * T * D * (6 * W + 12 * case["act"])}
        return {"bytes": 2 * e * B * T * D + params + state * (1 + case["state"]),
                "flops": B * T * D * (2 * W + 4 * case["act"])}
    D, N, G = case["D"], case["N"], case["G"]
    params, state = 4 * D * (N + case["skip"] + case["softplus"]), 4 * B * D * N
    rows, shared = e * B * T * D, e * B * T * G * N
    if op == "scan_bwd":
        # x, dt, dy (and z) in, dx, ddt (and dz) out
        return {"bytes": rows * (5 + 2 * case["z"]) + 4 * shared + 2 * params + (3 * state if case["state"] else 0),
                "flops": B * T * D * (22 * N + 20)}
    return {"bytes": rows * (3 + case["z"]) + 2 * shared + params + state * (1 + case["state"]),
            "flops": B * T * D * (7 * N + 12)}


# --------------------------------------------------- the definition, 64 bits

def exact(case, seed):
    s = {k: (v.double() if torch.is_tensor(v) and v.is_floating_point() else v)
         for k, v in prepare(case, seed).items()}
    if case["op"].startswith("conv"):
        return _exact_conv(case, s)
    return _exact_scan(case, s)


def _ends(case, s, device):
    if s.get("lengths") is None:
        return torch.full((case["B"],), case["T"], device=device)
    return s["lengths"].long()


def _exact_conv(case, s):
    W, op, B, T = case["W"], case["op"], case["B"], case["T"]
    H, d = case["heads"], case["d"]
    x = s["x"][:, None] if op == "conv_step" else s["x"].transpose(1, 2).reshape(B, T, H * d) if H > 1 else s["x"]
    D = x.shape[-1]
    end = _ends(case, s, x.device)
    # one tap at a time, through an explicit index of the rows before, inside and behind
    src = torch.zeros(B, W - 1 + T, D, dtype=torch.float64, device=x.device)
    if s["state"] is not None:
        src[:, :W - 1] = s["state"]
    src[:, W - 1:] = x
    row = torch.arange(T, device=x.device)
    inside = (row[None] < end[:, None])[:, :, None]
    pre = torch.zeros(B, T, D, dtype=torch.float64, device=x.device)
    if s["bias"] is not None:
        pre += s["bias"]
    for lag in range(W):
        pre += s["weight"][:, W - 1 - lag] * src[:, row + (W - 1 - lag)]
    tail = torch.stack([src[b, int(end[b]):int(end[b]) + W - 1] for b in range(B)]) if W > 1 else None

    def shaped(y):
        return y.reshape(B, T, H, d).transpose(1, 2).contiguous() if H > 1 else y

    if op != "conv_bwd":
        y = pre / (1 + torch.exp(-pre)) if case["act"] else pre
        y = y * inside
        return {"y": y[:, 0] if op == "conv_step" else shaped(y), "state": tail}
    dy = s["dy"].transpose(1, 2).reshape(B, T, D) if H > 1 else s["dy"]
    if case["act"]:
        q = 1 / (1 + torch.exp(-pre))
        dpre = dy * q + dy * pre * q * (1 - q)
    else:
        dpre = dy
    dpre = torch.where(inside, dpre, 0.0)
    dsrc = torch.zeros_like(src)
    dw = torch.zeros(D, W, dtype=torch.float64, device=x.device)
    for lag in range(W):
        at = row + (W - 1 - lag)
        dsrc[:, at] += s["weight"][:, W - 1 - lag] * dpre
        dw[:, W - 1 - lag] = torch.einsum("btd,btd->d", dpre, src[:, at])
    if s["dstate_out"] is not None:
        for b in range(B):
            dsrc[b, int(end[b]):int(end[b]) + W - 1] += s["dstate_out"][b]
    return {"dx": shaped(dsrc[:, W - 1:]), "dweight": dw, "dbias": dpre.sum((0, 1)) if case["bias"] else None,
            "dstate": dsrc[:, :W - 1] if case["state"] else None}


def _exact_scan(case, s):
    op, B, T, D, N, G = case["op"], case["B"], case["T"], case["D"], case["N"], case["G"]
    if op == "scan_step":
        s = dict(s, h0=s["h"], **{k: s[k][:, None] for k in ("x", "dt", "Bm", "Cm")},
                 z=None if s["z"] is None else s["z"][:, None])
    dev, A = s["x"].device, s["A"]
    end = _ends(case, s, dev)
    group = torch.arange(D, device=dev) // (D // G)
    p = s["dt"] if s["dt_bias"] is None else s["dt"] + s["dt_bias"]
    delta = torch.logaddexp(p, torch.zeros_like(p)) if case["softplus"] else p
    h = torch.zeros(B, D, N, dtype=torch.float64, device=dev) if s["h0"] is None else s["h0"].clone()
    back = op == "scan_bwd"
    kept = [h.clone()] if back else None
    y = torch.zeros(B, T, D, dtype=torch.float64, device=dev)
    for t in range(T):
        on = (t < end)[:, None]
        dl = torch.where(on, delta[:, t], 0.0)[..., None]
        h = torch.exp(dl * A) * h + dl * s["x"][:, t, :, None] * s["Bm"][:, t, group]
        y[:, t] = torch.where(on, (h * s["Cm"][:, t, group]).sum(-1), 0.0)
        if back:
            kept.append(h.clone())
    skip = s["D_skip"] if s["D_skip"] is not None else torch.zeros(D, dtype=torch.float64, device=dev)
    on = (torch.arange(T, device=dev)[None] < end[:, None])[..., None]
    core = y + torch.where(on, s["x"] * skip, 0.0)
    q = None if s["z"] is None else 1 / (1 + torch.exp(-s["z"]))
    if not back:
        out = core if q is None else core * s["z"] * q
        return {"y": out[:, 0] if op == "scan_step" else out, "h": h}
    dy = torch.where(on, s["dy"], 0.0)
    dz = None if q is None else dy * core * (q + s["z"] * q * (1 - q))
    dcore = dy if q is None else dy * s["z"] * q
    dx, dp = torch.zeros_like(dy), torch.zeros_like(dy)
    dB = torch.zeros(B, T, G, N, dtype=torch.float64, device=dev)
    dC = torch.zeros_like(dB)
    dA = torch.zeros_like(A)
    g = torch.zeros_like(h) if s["dh_T"] is None else s["dh_T"].clone()
    for t in range(T - 1, -1, -1):
        live = (t < end)[:, None]
        dl = torch.where(live, delta[:, t], 0.0)
        xt, Bt = s["x"][:, t], s["Bm"][:, t, group]
        dc = dcore[:, t, :, None]
        g = g + dc * s["Cm"][:, t, group]
        dC[:, t] = (dc * kept[t + 1]).reshape(B, G, D // G, N).sum(2)
        dB[:, t] = (g * (dl * xt)[..., None]).reshape(B, G, D // G, N).sum(2)
        a = torch.exp(dl[..., None] * A)
        through = g * a * kept[t]
        gb = (g * Bt).sum(-1)
        dp[:, t] = torch.where(live, gb * xt + (through * A).sum(-1), 0.0)
        dx[:, t] = gb * dl + dcore[:, t] * skip
        dA += (through * dl[..., None]).sum(0)
        g = a * g
    if case["softplus"]:
        dp = dp / (1 + torch.exp(-p))
    return {"dx": dx, "ddt": dp, "dA": dA, "dB": dB, "dC": dC,
            "dD": torch.where(on, dcore * s["x"], 0.0).sum((0, 1)) if case["skip"] else None, "dz": dz,
            "ddt_bias": dp.sum((0, 1)) if case["softplus"] else None, "dh0": g if case["state"] else None}
