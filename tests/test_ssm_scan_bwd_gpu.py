"""GPU parity of the scan's backward (gdr_ssm_scan_bwd) with the fp64 oracle's reverse walk.

Every element of every gradient is held to the oracle's error bound for fp32 arithmetic plus
half a step of its type."""
import numpy as np
import pytest
import torch

import gated_delta_rule_89_b200 as gdr
from oracle import ssm
from test_ssm_scan_gpu import BF, FP, cuda, make, near, rnd

pytestmark = pytest.mark.gpu

NAMES = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")


def gradients(c, dy, dh, softplus=True, **kw):
    d = {k: cuda(v) for k, v in c.items()}
    return dict(zip(NAMES, gdr.ssm_scan_bwd(**d, dy=cuda(dy), dh_T=cuda(dh), dt_softplus=softplus, **kw)))


def check(c, dy, dh, softplus=True):
    ref = ssm.scan_bwd(c["x"], c["dt"], c["A"], c["Bm"], c["Cm"], dy, c["D_skip"], c["z"], c["dt_bias"], softplus,
                       c["h0"], dh, c["lengths"])
    got = gradients(c, dy, dh, softplus)
    for k, key in (("dD", "D_skip"), ("dz", "z"), ("ddt_bias", "dt_bias"), ("dh0", "h0")):
        assert (got[k] is None) == (c[key] is None), k
    for k, v in got.items():
        if v is not None:
            near(v, *ref[k], v.dtype, k)
    return got


CASES = [
    dict(B=1, T=1, D=4, N=16),
    dict(B=2, T=16, D=64, N=16, z=False),
    dict(B=1, T=33, D=36, N=8, dt=FP, skip=False),
    dict(B=2, T=40, D=132, N=8),                                     # two blocks of channels
    dict(B=2, T=50, D=68, N=32, bias=False),
    dict(B=1, T=41, D=24, N=64, dt=FP),
    dict(B=1, T=23, D=36, N=64),
    dict(B=3, T=50, D=66, N=16, G=2, lengths=[0, 1, 50]),            # odd groups: one element at a time
    dict(B=2, T=97, D=33, N=8, dt=FP, lengths=[97, 40]),
    dict(B=2, T=90, D=288, N=16, G=4, dt=FP, state=False),           # blocks end inside a group
    dict(B=4, T=40, D=8, N=32, G=2, lengths=[-3, 99, 8, 39]),
    dict(B=1, T=400, D=40, N=16),                                    # pieces of a row
    dict(B=3, T=520, D=20, N=8, G=2, dt=FP, lengths=[520, 130, 0]),
    dict(B=2, T=300, D=18, N=32, lengths=[160, 161]),                # a row that ends with a piece
    dict(B=1, T=270, D=12, N=64, z=False),
    dict(B=2, T=0, D=16, N=16),
]


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case, softplus):
    c = make(**case)
    if not softplus:
        c["dt"] = (c["dt"].float().abs() * 0.2).to(c["dt"].dtype)
        c["dt_bias"] = None if c["dt_bias"] is None else c["dt_bias"].abs() * 0.02
    B, T, D, N = case["B"], case["T"], case["D"], case["N"]
    dy = rnd(B, T, D, dtype=c["x"].dtype, seed=30)
    dh = rnd(B, D, N, seed=31) if c["h0"] is not None else None
    got = check(c, dy, dh, softplus)
    again = gradients(c, dy, dh, softplus)
    assert all(v is None or torch.equal(v, again[k]) for k, v in got.items())


def test_strided_and_unaligned_inputs():
    B, T, D, N = 2, 45, 64, 16
    c = make(B, T, D, N)
    dy = rnd(B, T, D, dtype=BF, seed=30).cuda()
    d = {k: cuda(v) for k, v in c.items()}
    for off in (0, 3):
        xz, rbc = rnd(B, T, 2 * D + 8, dtype=BF).cuda(), rnd(B, T, 16 + 2 * N + 8, dtype=BF, seed=1).cuda()
        wide = torch.zeros(B, T, D + 8, dtype=BF, device="cuda")
        wide[..., off:off + D] = dy
        d.update(x=xz[..., off:off + D], z=xz[..., D + off:2 * D + off],
                 Bm=rbc[..., 16 + off:16 + off + N][:, :, None],
                 Cm=rbc[..., 16 + N + off:16 + 2 * N + off][:, :, None])
        a = gdr.ssm_scan_bwd(**d, dy=wide[..., off:off + D])
        b = gdr.ssm_scan_bwd(**{k: v.contiguous() if v is not None else None for k, v in d.items()}, dy=dy)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_nothing_behind_a_row_is_read():
    ends = [0, 13, 50]
    c = make(3, 50, 36, 16, lengths=ends)
    dy, dh = rnd(3, 50, 36, dtype=BF, seed=30), rnd(3, 36, 16, seed=31)
    clean = gradients(c, dy, dh)
    for k in ("x", "dt", "Bm", "Cm", "z"):
        c[k] = c[k].clone()
        for b, n in enumerate(ends):
            c[k][b, n:] = float("nan")
    dy = dy.clone()
    for b, n in enumerate(ends):
        dy[b, n:] = float("inf")
    dirty = gradients(c, dy, dh)
    for k in NAMES:
        assert torch.equal(clean[k], dirty[k]), k
    for k in ("dx", "ddt", "dB", "dC", "dz"):
        for b, n in enumerate(ends):
            assert not dirty[k][b, n:].any()
    assert torch.equal(dirty["dh0"][0], dh[0].cuda())     # an empty row hands the gradient through


def test_against_differences_of_the_forward():
    """The library's own forward, differenced along random directions in fp32.

    The loss sums m = sum |y dy| + |h dh| of size 1e3 with relative errors of a few fp32 roundings
    per term (random signs), 1e-6 m together; the step 2^-6 divides that by 2^-5: 0.03 absolute,
    against slopes of the order of 30.  The third derivative adds (2^-6)^2 / 6 = 4e-5 of it."""
    c = make(2, 60, 32, 16, dt=FP)
    dy, dh = rnd(2, 60, 32, seed=30), rnd(2, 32, 16, seed=31)
    got = gradients(c, dy, dh)
    eps = 2.0 ** -6
    for name, key in (("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("Bm", "dB"), ("Cm", "dC"), ("D_skip", "dD"),
                      ("z", "dz"), ("dt_bias", "ddt_bias"), ("h0", "dh0")):
        v = rnd(*c[name].shape, seed=77)
        if name == "A":
            v = v * 0.1
        loss = []
        for sign in (1, -1):
            d = {k: cuda(t) for k, t in c.items()}
            d[name] = (c[name] + sign * eps * v).cuda()
            y, h = gdr.ssm_scan_fwd(**d)
            loss.append(float((y.double() * dy.cuda()).sum() + (h.double() * dh.cuda()).sum()))
        slope = float((got[key].double() * v.cuda()).sum())
        size = float((got[key].double().abs() * v.cuda().abs()).sum())
        assert abs((loss[0] - loss[1]) / (2 * eps) - slope) <= 0.03 + 2e-3 * size, name


def test_stream_host_and_capture():
    c = make(2, 70, 64, 16)
    dy, dh = rnd(2, 70, 64, dtype=BF, seed=30), rnd(2, 64, 16, seed=31)
    ref = gradients(c, dy, dh)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other = gradients(c, dy, dh, stream=s)
    s.synchronize()
    host = dict(zip(NAMES, gdr.ssm_scan_bwd(**c, dy=dy, dh_T=dh)))
    d = {k: cuda(v) for k, v in c.items()}
    dyc, dhc = dy.cuda(), dh.cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = gdr.ssm_scan_bwd(**d, dy=dyc, dh_T=dhc)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for k, o in zip(NAMES, out):
        assert torch.equal(ref[k], other[k]) and torch.equal(ref[k].cpu(), host[k]) and torch.equal(ref[k], o), k


def test_a_training_step_through_both():
    """Gradients of a mixer (convolution, then scan) chained by hand, against autograd in fp64."""
    B, T, D, N = 2, 37, 32, 16
    c = make(B, T, D, N, dt=FP, state=False)
    x, w, b = rnd(B, T, D, seed=40), rnd(D, 4, seed=41, scale=0.5), rnd(D, seed=42)
    dy = rnd(B, T, D, seed=43)
    u, _ = gdr.short_conv_fwd(x.cuda(), w.cuda(), b.cuda())
    d = {k: cuda(v) for k, v in c.items()}
    d["x"] = u
    g = dict(zip(NAMES, gdr.ssm_scan_bwd(**d, dy=dy.cuda())))
    dx, dw, db, _ = gdr.short_conv_bwd(x.cuda(), w.cuda(), g["dx"], b.cuda())

    leaf = [t.double().requires_grad_() for t in (x, w, b)]
    xp = torch.nn.functional.pad(leaf[0], (0, 0, 3, 0))
    pre = sum(xp[:, j:j + T] * leaf[1][:, j] for j in range(4)) + leaf[2]
    uu = torch.nn.functional.silu(pre)
    f = {k: (v.double() if v is not None else None) for k, v in c.items()}
    delta = torch.nn.functional.softplus(f["dt"] + f["dt_bias"])
    h, ys = torch.zeros(B, D, N, dtype=torch.float64), []
    for t in range(T):
        h = torch.exp(delta[:, t, :, None] * f["A"]) * h + (delta[:, t] * uu[:, t])[..., None] * f["Bm"][:, t]
        ys.append((h * f["Cm"][:, t]).sum(-1) + f["D_skip"] * uu[:, t])
    y = torch.stack(ys, 1) * torch.nn.functional.silu(f["z"])
    (y * dy).sum().backward()
    for got, want in ((dx, leaf[0].grad), (dw, leaf[1].grad), (db, leaf[2].grad)):
        # fp32 along chains of about 50 roundings each, whose terms partly cancel
        assert (got.double().cpu() - want).abs().max() <= 2e-5 * want.abs().max()


def test_no_channels():
    """Sums over no channels: dB and dC are zero, whatever their memory held."""
    for dt in (BF, FP):
        c = make(2, 5, 0, 16, dt=dt)
        junk = [torch.full((2, 5, 1, 16), 7.0, dtype=dt, device="cuda") for _ in range(4)]
        del junk
        got = gradients(c, rnd(2, 5, 0, dtype=dt), rnd(2, 0, 16))
        assert got["dB"].shape == got["dC"].shape == (2, 5, 1, 16)
        assert not got["dB"].any() and not got["dC"].any()
        assert got["dx"].shape == (2, 5, 0) and got["dA"].shape == (0, 16)


@pytest.mark.parametrize("T,D,N", [(700, 40, 16), (400, 24, 8), (270, 12, 64)])
def test_growing_states_across_pieces(T, D, N):
    """States that grow (A > 0) by more than fp32 holds over a piece, where nothing has come in:
    0 stays 0.  x is there for the last 8 tokens only and dy for the first 8, so the states and
    their gradients are 0 or small wherever they are used."""
    c = make(1, T, D, N, dt=FP, bias=False, state=False)
    c["A"] = 4 + rnd(D, N, seed=50) * 0.1
    c["dt"] = torch.ones(1, T, D)
    c["x"][:, :-8] = 0
    dy = rnd(1, T, D, seed=30)
    y_ref, h_ref, by, bh = ssm.scan_fwd(**c, softplus=False)
    y, h = gdr.ssm_scan_fwd(**{k: cuda(v) for k, v in c.items()}, dt_softplus=False)
    near(y, y_ref, by, FP, "y")
    near(h, h_ref, bh, FP, "h")
    dy[:, 8:] = 0
    got = check(c, dy, None, softplus=False)
    assert got["dx"][:, :8].any() and not got["dx"][:, 8:].any()


@pytest.mark.parametrize("case", [
    dict(B=230, T=35, D=36, N=16, lengths=[35, 0, 1, 33, 32] * 46),
    dict(B=230, T=33, D=69, N=8, dt=FP),
    dict(B=115, T=40, D=36, N=32, G=2, z=False),
    dict(B=230, T=20, D=10, N=64, skip=False),
    dict(B=230, T=20, D=12, N=64, dt=FP),
], ids=str)
def test_many_rows(case):
    """More blocks than the machine holds at a time, in the storing pass and in the walk."""
    c = make(**case)
    check(c, rnd(case["B"], case["T"], case["D"], dtype=c["x"].dtype, seed=30),
          rnd(case["B"], case["D"], case["N"], seed=31))


def test_pieces_are_taken():
    """The cases above that are meant to be walked in pieces are: their workspace holds more than the
    stored states, one block's share of dB and dC, and one part of dA, dD and ddt_bias a row."""
    def pieces(B, T, D, N, G=1):
        up = lambda n: (n + 255) // 256 * 256   # noqa: E731
        groups = -(-(D // G) // (1024 // N))
        rest = (gdr.ssm_scan_bwd_workspace_size(B, T, D, G, N) - gdr.ssm_scan_fwd_workspace_size(B, T, D, G, N) -
                up(B * -(-T // 8) * D * N * 4) - up(groups * B * T * G * 2 * N * 4))
        one = up(B * D * N * 4) + up(B * D * 8)
        if rest == one:
            return 1
        for n in range(2, 200):      # as many parts, the gradients between the pieces, and their sums of delta
            if rest == up(n * B * D * N * 4) * 2 + up(n * B * D * 8) + up(n * B * D * 4):
                return n
        raise AssertionError("the workspace is laid out otherwise")
    assert pieces(2, 50, 68, 32) == 1 and pieces(230, 35, 36, 16) == 1
    for size in ((1, 400, 40, 16), (3, 520, 20, 8, 2), (2, 300, 18, 32), (1, 270, 12, 64), (1, 700, 40, 16)):
        assert pieces(*size) > 2, size
