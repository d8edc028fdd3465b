"""CPU pins of the convolution's and the scan's fp64 oracle (oracle/ssm.py): closed forms,
torch's convolution, and gradients against central differences."""
import numpy as np
import pytest
import torch

from oracle import ssm

RNG = np.random.default_rng


def conv_case(B=2, T=7, D=3, W=4, seed=0):
    r = RNG(seed)
    return dict(x=r.normal(size=(B, T, D)), weight=r.normal(size=(D, W)), bias=r.normal(size=D),
                state=r.normal(size=(B, W - 1, D)))


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 2, 9])
def test_conv_is_torch_conv1d(W, T):
    c = conv_case(T=T, W=W)
    y, st, _ = ssm.conv_fwd(**c, act=False)
    xp = torch.tensor(np.concatenate([c["state"], c["x"]], 1)).transpose(1, 2)
    ref = torch.nn.functional.conv1d(xp, torch.tensor(c["weight"])[:, None], torch.tensor(c["bias"]), groups=3)
    np.testing.assert_allclose(y, ref.transpose(1, 2).numpy(), atol=1e-13)
    np.testing.assert_array_equal(st, np.concatenate([c["state"], c["x"]], 1)[:, -(W - 1):])


def test_conv_splits_and_ends():
    c = conv_case(T=9)
    whole, end, _ = ssm.conv_fwd(**c)
    a, mid, _ = ssm.conv_fwd(c["x"][:, :4], c["weight"], c["bias"], c["state"])
    b, end2, _ = ssm.conv_fwd(c["x"][:, 4:], c["weight"], c["bias"], mid)
    np.testing.assert_allclose(np.concatenate([a, b], 1), whole, atol=1e-14)
    np.testing.assert_array_equal(end, end2)
    y, st, _ = ssm.conv_fwd(**c, lengths=[0, 2])
    assert not y[0].any() and not y[1, 2:].any()
    np.testing.assert_array_equal(st[0], c["state"][0])
    np.testing.assert_array_equal(st[1], np.concatenate([c["state"][1, 2:], c["x"][1, :2]]))


def differences(loss, value, grad, eps=1e-6):
    """Every entry of `grad` against the central difference of `loss` in that entry.

    The step's own error is of the order eps^2 = 1e-12 of the third derivative; what counts is the
    rounding of the two losses: each is a sum whose terms amount to m and carry a few times 2^-53,
    so the quotient is off by about 4 * 2^-53 * m / eps (2e-6 at m = 5e3).
    """
    m = loss()[1]
    flat = value.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + eps
        up = loss()[0]
        flat[i] = keep - eps
        down = loss()[0]
        flat[i] = keep
        assert abs((up - down) / (2 * eps) - grad.reshape(-1)[i]) < \
            2e-7 * max(1, abs(grad.reshape(-1)[i])) + 4 * 2.0 ** -53 * m / eps, i


@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("lengths", [None, [5, 1]])
def test_conv_gradients(act, lengths):
    c = conv_case(T=5, D=2)
    r = RNG(1)
    dy, dso = r.normal(size=c["x"].shape), r.normal(size=c["state"].shape)
    g = ssm.conv_bwd(c["x"], c["weight"], dy, c["bias"], c["state"], dso, act, lengths)

    def loss():
        y, st, _ = ssm.conv_fwd(**c, act=act, lengths=lengths)
        return (y * dy).sum() + (st * dso).sum(), np.abs(y * dy).sum() + np.abs(st * dso).sum()
    for name, key in (("x", "dx"), ("weight", "dweight"), ("bias", "dbias"), ("state", "dstate")):
        differences(loss, c[name], g[key][0])


def scan_case(B=2, T=5, D=4, N=8, G=2, seed=0):
    r = RNG(seed)
    return dict(x=r.normal(size=(B, T, D)), dt=r.normal(size=(B, T, D)) - 1, A=-np.exp(r.normal(size=(D, N))),
                Bm=r.normal(size=(B, T, G, N)), Cm=r.normal(size=(B, T, G, N)), D_skip=r.normal(size=D),
                z=r.normal(size=(B, T, D)), dt_bias=r.normal(size=D), h0=r.normal(size=(B, D, N)))


def test_scan_without_decay_is_a_cumulative_sum():
    c = scan_case(G=1)
    c["A"][:] = 0
    c.update(D_skip=None, z=None, h0=None, dt_bias=None, dt=np.ones_like(c["dt"]))
    y, h, _, _ = ssm.scan_fwd(**c, softplus=False)
    run = np.cumsum(c["x"][..., None] * c["Bm"], 1)
    np.testing.assert_allclose(y, (run * c["Cm"]).sum(-1), atol=1e-13)
    np.testing.assert_allclose(h, run[:, -1], atol=1e-13)


def test_scan_is_the_sum_over_the_past():
    """y_t = sum_{s<=t} C_t . (exp(A (S_t - S_s)) * B_s) delta_s x_s with S the running sum of delta."""
    c = scan_case(T=6, G=1)
    delta = np.log1p(np.exp(c["dt"] + c["dt_bias"]))
    S = np.cumsum(delta, 1)
    B, T, D = c["x"].shape
    ref = np.zeros((B, T, D))
    for t in range(T):
        for s in range(t + 1):
            k = np.exp((S[:, t] - S[:, s])[..., None] * c["A"])
            ref[:, t] += (c["Cm"][:, t] * k * c["Bm"][:, s]).sum(-1) * delta[:, s] * c["x"][:, s]
        ref[:, t] += (c["Cm"][:, t] * np.exp(S[:, t][..., None] * c["A"]) * c["h0"]).sum(-1)
    ref = (ref + c["D_skip"] * c["x"]) * c["z"] / (1 + np.exp(-c["z"]))
    np.testing.assert_allclose(ssm.scan_fwd(**c)[0], ref, atol=1e-12)


def test_scan_splits_and_ends():
    c = scan_case(T=7)
    y, h, _, _ = ssm.scan_fwd(**c)
    seq = ("x", "dt", "Bm", "Cm", "z")
    cut = lambda lo, hi: {k: (v[:, lo:hi] if k in seq else v) for k, v in c.items()}   # noqa: E731
    a, mid, _, _ = ssm.scan_fwd(**cut(0, 3))
    b, end, _, _ = ssm.scan_fwd(**{**cut(3, 7), "h0": mid})
    np.testing.assert_allclose(np.concatenate([a, b], 1), y, atol=1e-14)
    np.testing.assert_allclose(end, h, atol=1e-14)
    y, h, _, _ = ssm.scan_fwd(**c, lengths=[3, 0])
    np.testing.assert_allclose(h[0], mid[0], atol=1e-14)
    np.testing.assert_array_equal(h[1], c["h0"][1])
    assert not y[1].any() and not y[0, 3:].any()


@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("lengths", [None, [4, 0]])
def test_scan_gradients(G, softplus, lengths):
    c = scan_case(T=4, N=8, G=G)
    if not softplus:
        c["dt"] = np.abs(c["dt"]) * 0.3
    r = RNG(1)
    dy, dh = r.normal(size=c["x"].shape), r.normal(size=c["h0"].shape)
    g = ssm.scan_bwd(c["x"], c["dt"], c["A"], c["Bm"], c["Cm"], dy, c["D_skip"], c["z"], c["dt_bias"], softplus,
                     c["h0"], dh, lengths)

    def loss():
        y, h, _, _ = ssm.scan_fwd(**c, softplus=softplus, lengths=lengths)
        return (y * dy).sum() + (h * dh).sum(), np.abs(y * dy).sum() + np.abs(h * dh).sum()
    for name, key in (("x", "dx"), ("dt", "ddt"), ("A", "dA"), ("Bm", "dB"), ("Cm", "dC"), ("D_skip", "dD"),
                      ("z", "dz"), ("dt_bias", "ddt_bias"), ("h0", "dh0")):
        differences(loss, c[name], g[key][0])


def test_bounds_cover_fp32_and_not_much_more():
    """The same walks in fp32 stay inside the bounds, and the bounds are a few hundred roundings."""
    c = scan_case(T=40, N=16)
    f = {k: v.astype(np.float32) for k, v in c.items()}
    y, h, by, bh = ssm.scan_fwd(**f)
    p = f["dt"] + f["dt_bias"]
    delta = np.log1p(np.exp(p)).astype(np.float32)
    st = f["h0"].copy()
    for t in range(40):
        rep = lambda m: np.repeat(m[:, t], 2, axis=1)   # noqa: E731
        st = np.exp(delta[:, t, :, None] * f["A"]) * st + (delta[:, t] * f["x"][:, t])[..., None] * rep(f["Bm"])
        core = (rep(f["Cm"]) * st).sum(-1) + f["D_skip"] * f["x"][:, t]
        out = core * f["z"][:, t] / (1 + np.exp(-f["z"][:, t]))
        assert out.dtype == np.float32
        assert (np.abs(out - y[:, t]) <= by[:, t] + ssm.U * np.abs(y[:, t])).all()
    assert (np.abs(st - h) <= bh).all()
    assert by.max() < 1e-3 * np.abs(y).max() and bh.max() < 1e-3 * np.abs(h).max()
