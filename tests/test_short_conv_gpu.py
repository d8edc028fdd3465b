"""GPU parity of the short causal convolution (gdr_short_conv_fwd / _step / _bwd) with its fp64 oracle.

Every element is held to the oracle's own error bound for fp32 arithmetic plus half a step of
its type (relative to the value, and to the bound's reach beyond it)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_89_b200 as gdr
from oracle import ssm

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32
TINY = 2.0 ** -126


def rnd(*shape, dtype=FP, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def cuda(t):
    return None if t is None else t.cuda()


def near(got, ref, bound, dtype, name=""):
    """|got - ref| <= bound + half a step of `dtype` of the rounded value."""
    half = torch.finfo(dtype).eps / 2
    got = got.detach().double().cpu().numpy()
    assert got.shape == ref.shape, name
    off = np.abs(got - ref) - (bound + half * (np.abs(ref) + bound) + TINY)
    assert np.isfinite(got).all() and (off <= 0).all(), (name, float(off.max()))


def rows(t):
    """[B,H,T,d] or [B,T,D] as [B,T,D]."""
    return t.transpose(1, 2).flatten(2) if t.dim() == 4 else t


CASES = [
    # B, T, D, W, dtype, act, bias, state, lengths
    (1, 1, 8, 4, BF, True, True, True, None),
    (2, 7, 8, 4, BF, True, False, False, None),
    (1, 2, 64, 3, FP, False, True, True, None),
    (3, 65, 40, 2, BF, True, True, True, [0, 1, 65]),
    (4, 130, 33, 4, FP, True, True, True, [0, 2, 130, 77]),       # an odd width: one element at a time
    (2, 50, 1001, 3, BF, False, False, True, [50, 1]),
    (1, 300, 256, 4, FP, True, True, False, None),
    (5, 17, 12, 4, BF, True, True, True, [3, -4, 99, 16, 17]),    # lengths are brought into [0, T]
    (2, 0, 16, 4, BF, True, True, True, None),
]


def make(case, seed=1):
    B, T, D, W, dt, act, bias, state, lengths = case
    return dict(x=rnd(B, T, D, dtype=dt, seed=seed), weight=rnd(D, W, seed=seed + 1, scale=0.5),
                bias=rnd(D, seed=seed + 2) if bias else None,
                state=rnd(B, W - 1, D, dtype=dt, seed=seed + 3) if state else None,
                lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32))


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    act, dt = case[5], case[4]
    c = make(case)
    y_ref, st_ref, bound = ssm.conv_fwd(**c, act=act)
    d = {k: cuda(v) for k, v in c.items()}
    y, st = gdr.short_conv_fwd(d["x"], d["weight"], d["bias"], d["state"], "silu" if act else None, d["lengths"])
    near(y, y_ref, bound, dt, "y")
    np.testing.assert_array_equal(st.double().cpu().numpy(), st_ref)       # copies
    if c["lengths"] is not None:      # a y made by the call is zero behind a row's end
        for b, n in enumerate(c["lengths"].clamp(0, case[1]).tolist()):
            assert not y[b, n:].any()
    # behind a row's end a given y stays as it is, and the state may be updated in place
    mine = torch.full_like(d["x"], 7.0).contiguous()
    if d["state"] is not None:
        gdr.short_conv_fwd(d["x"], d["weight"], d["bias"], d["state"], "silu" if act else None, d["lengths"], y=mine,
                           state_out=d["state"])
        np.testing.assert_array_equal(d["state"].double().cpu().numpy(), st_ref)
        if c["lengths"] is not None:
            for b, n in enumerate(c["lengths"].clamp(0, case[1]).tolist()):
                assert (mine[b, n:] == 7).all() and torch.equal(mine[b, :n], y[b, :n])


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("shape", [(2, 3, 20, 16), (1, 2, 100, 128), (2, 5, 9, 6)])
def test_head_layout(shape, dt):
    """Token rows [B,T,H*d] in, the gated delta rule's [B,H,T,d] out; and the other way round."""
    B, H, T, d = shape
    x = rnd(B, T, H, d, dtype=dt)
    w, b = rnd(H * d, 4, seed=2), rnd(H * d, seed=3)
    y_ref, st_ref, bound = ssm.conv_fwd(x.flatten(2), w, b)
    y, st = gdr.short_conv_fwd(x.cuda().transpose(1, 2), w.cuda(), b.cuda())
    assert y.shape == (B, H, T, d) and y.is_contiguous()
    near(rows(y), y_ref, bound, dt)
    np.testing.assert_array_equal(st.double().cpu().numpy(), st_ref)
    y2, _ = gdr.short_conv_fwd(x.cuda().transpose(1, 2).contiguous(), w.cuda(), b.cuda())
    assert torch.equal(y, y2)


def test_strided_slices_and_odd_offsets():
    """Slices of a wider projection, aligned or not, give what their copies give."""
    for off in (0, 8, 3):
        wide = rnd(2, 40, 200, dtype=BF).cuda()
        x = wide[..., off:off + 96]
        w = rnd(96, 4, seed=2).cuda()
        a = gdr.short_conv_fwd(x, w)
        b = gdr.short_conv_fwd(x.contiguous(), w)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_steps_continue_a_prompt():
    for dt, D in ((BF, 64), (FP, 64), (BF, 37)):
        x, w, b = rnd(3, 20, D, dtype=dt).cuda(), rnd(D, 4, seed=2).cuda(), rnd(D, seed=3).cuda()
        whole, end = gdr.short_conv_fwd(x, w, b)
        y, st = gdr.short_conv_fwd(x[:, :15], w, b)
        outs = [y] + [gdr.short_conv_step(x[:, t], st, w, b)[:, None] for t in range(15, 20)]
        assert torch.equal(st, end)
        # the same sums in the same order
        np.testing.assert_allclose(torch.cat(outs, 1).float().cpu(), whole.float().cpu(), rtol=2.0 ** -7, atol=1e-6)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("B,D", [(1, 8), (3, 33), (17, 2048), (256, 64)])
def test_step(B, D, dt, W):
    x, w, b = rnd(B, 1, D, dtype=dt), rnd(D, W, seed=2), rnd(D, seed=3)
    st = rnd(B, W - 1, D, dtype=dt, seed=4)
    y_ref, st_ref, bound = ssm.conv_fwd(x, w, b, st)
    s = st.cuda()
    y = gdr.short_conv_step(x[:, 0].cuda(), s, w.cuda(), b.cuda())
    near(y[:, None], y_ref, bound, dt)
    np.testing.assert_array_equal(s.double().cpu().numpy(), st_ref)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    B, T, D, W, dt, act, bias, state, lengths = case
    c = make(case)
    dy = rnd(B, T, D, dtype=dt, seed=9)
    dso = rnd(B, W - 1, D, dtype=dt, seed=10) if state else None
    ref = ssm.conv_bwd(c["x"], c["weight"], dy, c["bias"], c["state"], dso, act, c["lengths"])
    d = {k: cuda(v) for k, v in c.items()}
    args = (d["x"], d["weight"], dy.cuda(), d["bias"], d["state"], cuda(dso), "silu" if act else None, d["lengths"])
    got = dict(zip(("dx", "dweight", "dbias", "dstate"), gdr.short_conv_bwd(*args)))
    assert (got["dbias"] is None) == (not bias) and (got["dstate"] is None) == (not state)
    for k, v in got.items():
        if v is not None:
            near(v, *ref[k], v.dtype, k)
    again = gdr.short_conv_bwd(*args)
    assert all(a is None or torch.equal(a, b) for a, b in zip(again, got.values()))


def test_backward_does_not_read_behind_a_row():
    """NaN behind a row's end, in x and dy, touches nothing."""
    c = make((3, 40, 24, 4, BF, True, True, True, [0, 13, 40]))
    dy = rnd(3, 40, 24, dtype=BF, seed=9)
    d = {k: cuda(v) for k, v in c.items()}
    clean = gdr.short_conv_bwd(d["x"], d["weight"], dy.cuda(), d["bias"], d["state"], None, "silu", d["lengths"])
    y0, s0 = gdr.short_conv_fwd(d["x"], d["weight"], d["bias"], d["state"], "silu", d["lengths"])
    x, dyn = c["x"].clone(), dy.clone()
    for b, n in enumerate([0, 13, 40]):
        x[b, n:], dyn[b, n:] = float("nan"), float("inf")
    dirty = gdr.short_conv_bwd(x.cuda(), d["weight"], dyn.cuda(), d["bias"], d["state"], None, "silu", d["lengths"])
    y1, s1 = gdr.short_conv_fwd(x.cuda(), d["weight"], d["bias"], d["state"], "silu", d["lengths"])
    assert all(torch.equal(a, b) for a, b in zip(clean, dirty))
    assert torch.equal(y0, y1) and torch.equal(s0, s1)


def test_backward_keeps_token_rows():
    """The gradient of a projection's rows seen as heads is made in those rows."""
    x = rnd(2, 30, 4, 16, dtype=BF).cuda().transpose(1, 2)
    dy = rnd(2, 4, 30, 16, dtype=BF, seed=1).cuda()
    w = rnd(64, 4, seed=2).cuda()
    dx, dw, _, _ = gdr.short_conv_bwd(x, w, dy)
    assert dx.shape == x.shape and dx.transpose(1, 2).is_contiguous()
    dx2, dw2, _, _ = gdr.short_conv_bwd(x.contiguous(), w, dy)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_other_stream_and_host_tensors():
    c = make((2, 90, 64, 4, BF, True, True, True, None))
    d = {k: cuda(v) for k, v in c.items()}
    y, st = gdr.short_conv_fwd(d["x"], d["weight"], d["bias"], d["state"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y2, st2 = gdr.short_conv_fwd(d["x"], d["weight"], d["bias"], d["state"], stream=s)
    s.synchronize()
    assert torch.equal(y, y2) and torch.equal(st, st2)
    y3, st3 = gdr.short_conv_fwd(c["x"], c["weight"], c["bias"], c["state"])
    assert not y3.is_cuda and torch.equal(y.cpu(), y3) and torch.equal(st.cpu(), st3)


def test_refusals():
    c = make((2, 9, 16, 4, BF, True, True, True, None))
    d = {k: cuda(v) for k, v in c.items()}
    call = lambda **kw: gdr.short_conv_fwd(**{**d, **kw})   # noqa: E731
    for bad, err in ((dict(weight=d["weight"].bfloat16()), TypeError), (dict(weight=d["weight"][:8]), ValueError),
                     (dict(bias=d["bias"][:8]), ValueError), (dict(state=d["state"].float()), TypeError),
                     (dict(state=d["state"][:, :2]), ValueError), (dict(activation="relu"), ValueError),
                     (dict(lengths=torch.ones(2, dtype=torch.int64, device="cuda")), TypeError),
                     (dict(lengths=torch.ones(3, dtype=torch.int32, device="cuda")), ValueError),
                     (dict(weight=d["weight"].cpu()), ValueError), (dict(y=d["x"].transpose(0, 1)), ValueError),
                     (dict(x=d["x"].half()), TypeError), (dict(x=d["x"][0]), ValueError),
                     (dict(weight=None), ValueError),
                     (dict(weight=torch.zeros(16, 5, device="cuda"), state=None), gdr.GDRError)):
        with pytest.raises(err):
            call(**bad)


def test_graph_capture():
    c = make((2, 90, 64, 4, BF, True, True, True, None))
    d = {k: cuda(v) for k, v in c.items()}
    dy = rnd(2, 90, 64, dtype=BF, seed=5).cuda()

    def both():
        return (*gdr.short_conv_fwd(d["x"], d["weight"], d["bias"], d["state"]),
                *gdr.short_conv_bwd(d["x"], d["weight"], dy, d["bias"], d["state"]))
    ref = both()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = both()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, out))
    d["x"].add_(1)
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(both(), out))


def test_feeds_the_gated_delta_rule():
    """A layer's path: three convolutions over one projection's rows, then the chunk forward with
    the fused prologue; a prompt in one call and in two with the carried states agree."""
    B, H, T, d = 1, 2, 192, 128
    D = H * d
    qkv = rnd(B, T, 3 * D, dtype=BF, scale=0.7).cuda()
    w = [rnd(D, 4, seed=s, scale=0.5).cuda() for s in (1, 2, 3)]
    a, bl = rnd(B, H, T, d, dtype=BF, seed=4).cuda(), rnd(B, H, T, seed=5).cuda()
    A_log, dtb = rnd(H, seed=6).cuda(), rnd(H, d, seed=7, scale=0.5).cuda()

    def layer(lo, hi, states, S):
        xs = [qkv[:, lo:hi, i * D:(i + 1) * D].unflatten(2, (H, d)).transpose(1, 2) for i in range(3)]
        out = [gdr.short_conv_fwd(x, wi, state=st) for x, wi, st in zip(xs, w, states)]
        O, S = gdr.chunk_fwd_prologue(*(y for y, _ in out), a[:, :, lo:hi].contiguous(), A_log, dtb,
                                      bl[:, :, lo:hi].contiguous(), S)
        return O, [st for _, st in out], S
    O, st, S = layer(0, T, [None] * 3, None)
    O1, st1, S1 = layer(0, 128, [None] * 3, None)
    O2, st2, S2 = layer(128, T, st1, S1)
    assert all(torch.equal(p, q) for p, q in zip(st, st2))
    assert torch.equal(O[:, :, :128], O1)
    # the carried state is fp32 and chunks start at the same tokens: the same arithmetic
    err = (O[:, :, 128:].float() - O2.float()).abs().max() / O.float().abs().max()
    assert err <= 2e-2 and (S - S2).abs().max() <= 2e-2 * S.abs().max()


def test_outputs_beside_and_in_the_inputs():
    """y right behind x, or between far apart rows of x, is taken; y in x is not, but a step's may be x."""
    D, T = 24, 40
    buf = rnd(4, T, D, dtype=BF).cuda()
    w = rnd(D, 4, seed=2).cuda()
    ref, _ = gdr.short_conv_fwd(buf[:1].clone(), w)
    y, _ = gdr.short_conv_fwd(buf[:1], w, y=buf[1:2])
    assert torch.equal(y, ref) and torch.equal(buf[1:2], ref)
    buf = rnd(4, T, D, dtype=BF).cuda()
    far = buf[::3]                                 # rows 0 and 3; y is rows 1 and 2
    ref, _ = gdr.short_conv_fwd(far.contiguous(), w)
    gdr.short_conv_fwd(far, w, y=buf[1:3])
    assert torch.equal(buf[1:3], ref)
    for y in (buf[:2], buf[1:3]):
        with pytest.raises(gdr.GDRError):
            gdr.short_conv_fwd(buf[:2], w, y=y)
    x, st = rnd(5, D, dtype=BF).cuda(), rnd(5, 3, D, dtype=BF, seed=3).cuda()
    st2 = st.clone()
    ref = gdr.short_conv_step(x, st, w)
    assert torch.equal(gdr.short_conv_step(x, st2, w, y=x), ref) and torch.equal(x, ref) and torch.equal(st, st2)
