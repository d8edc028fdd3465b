"""GPU parity of the selective state space scan (gdr_ssm_scan_fwd / _step) with its fp64 oracle.

Every element is held to the oracle's own error bound for fp32 arithmetic plus half a step of
its type."""
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
    return t.cuda() if isinstance(t, torch.Tensor) else t


def near(got, ref, bound, dtype, name=""):
    half = torch.finfo(dtype).eps / 2
    got = got.detach().double().cpu().numpy()
    assert got.shape == ref.shape, name
    off = np.abs(got - ref) - (bound + half * (np.abs(ref) + bound) + TINY)
    assert np.isfinite(got).all() and (off <= 0).all(), (name, float(off.max()))


def make(B, T, D, N=16, G=1, dt=BF, z=True, skip=True, bias=True, state=True, lengths=None, seed=1):
    return dict(x=rnd(B, T, D, dtype=dt, seed=seed), dt=rnd(B, T, D, dtype=dt, seed=seed + 1, scale=0.5),
                A=-torch.exp(rnd(D, N, seed=seed + 2)), Bm=rnd(B, T, G, N, dtype=dt, seed=seed + 3),
                Cm=rnd(B, T, G, N, dtype=dt, seed=seed + 4), D_skip=rnd(D, seed=seed + 5) if skip else None,
                z=rnd(B, T, D, dtype=dt, seed=seed + 6) if z else None,
                dt_bias=rnd(D, seed=seed + 7) - 2 if bias else None,
                h0=rnd(B, D, N, seed=seed + 8) if state else None,
                lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32))


CASES = [
    dict(B=1, T=1, D=4, N=16),
    dict(B=2, T=31, D=32, N=16, z=False),
    dict(B=1, T=33, D=36, N=8, dt=FP, skip=False),
    dict(B=2, T=64, D=20, N=32, bias=False),
    dict(B=1, T=70, D=24, N=64, dt=FP),
    dict(B=1, T=65, D=12, N=64),
    dict(B=3, T=50, D=66, N=16, G=2, lengths=[0, 1, 50]),            # odd groups: one element at a time
    dict(B=2, T=97, D=33, N=8, dt=FP, lengths=[97, 40]),
    dict(B=2, T=90, D=144, N=16, G=4, dt=FP, state=False),           # blocks end inside a group
    dict(B=4, T=40, D=8, N=32, G=2, lengths=[-3, 99, 32, 39]),
    dict(B=1, T=700, D=40, N=16),                                    # pieces of a row
    dict(B=2, T=1100, D=8, N=8, G=2, dt=FP, lengths=[1100, 130]),
    dict(B=2, T=0, D=16, N=16),
    # two channels a thread: as many blocks of twice the channels as fill two on most SMs
    dict(B=230, T=37, D=36, N=16, lengths=[37, 0, 1, 33, 32] * 46),
    dict(B=230, T=33, D=69, N=8, dt=FP),
    dict(B=115, T=40, D=36, N=32, G=2, z=False),
    dict(B=230, T=34, D=10, N=64, skip=False),
]


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case, softplus):
    c = make(**case)
    if not softplus:
        c["dt"] = (c["dt"].float().abs() * 0.2).to(c["dt"].dtype)
        c["dt_bias"] = None if c["dt_bias"] is None else c["dt_bias"].abs() * 0.02
    y_ref, h_ref, by, bh = ssm.scan_fwd(**c, softplus=softplus)
    d = {k: cuda(v) for k, v in c.items()}
    y, h = gdr.ssm_scan_fwd(**d, dt_softplus=softplus)
    near(y, y_ref, by, c["x"].dtype, "y")
    near(h, h_ref, bh, FP, "h")
    # in place of h0, and a y of the caller's
    mine = torch.full_like(d["x"], 7.0)
    d["h_T"] = d["h0"]
    if d["h0"] is not None:
        gdr.ssm_scan_fwd(**d, dt_softplus=softplus, y=mine)
        assert torch.equal(d["h0"], h)
        T = case["T"]
        for b in range(case["B"]):
            n = T if c["lengths"] is None else int(c["lengths"][b].clamp(0, T))
            assert torch.equal(mine[b, :n], y[b, :n]) and (mine[b, n:] == 7).all() and not y[b, n:].any()


def test_pieces_are_taken():
    """The cases above that are meant to be cut into pieces are."""
    assert gdr.ssm_scan_fwd_workspace_size(1, 700, 40, 1, 16) > 0
    assert gdr.ssm_scan_fwd_workspace_size(2, 1100, 8, 2, 8) > 0
    assert gdr.ssm_scan_fwd_workspace_size(2, 8192, 4096, 1, 16) == 0


def test_strided_slices():
    """x | z halves of one projection, dt | B | C slices of another, aligned or not."""
    B, T, D, N = 2, 45, 64, 16
    for off in (0, 3):
        xz, rbc = rnd(B, T, 2 * D + 8, dtype=BF).cuda(), rnd(B, T, 16 + 2 * N + 8, dtype=BF, seed=1).cuda()
        c = make(B, T, D, N)
        d = {k: cuda(v) for k, v in c.items()}
        d.update(x=xz[..., off:off + D], z=xz[..., D + off:2 * D + off],
                 Bm=rbc[..., 16 + off:16 + off + N][:, :, None],
                 Cm=rbc[..., 16 + N + off:16 + 2 * N + off][:, :, None])
        y, h = gdr.ssm_scan_fwd(**d)
        y2, h2 = gdr.ssm_scan_fwd(**{k: v.contiguous() if v is not None else None for k, v in d.items()})
        assert torch.equal(h, h2) and torch.equal(y, y2)
    # B and C shared by the batch and the tokens through strides of 0
    one = rnd(1, 1, 1, N, dtype=BF, seed=5).cuda()
    d.update(Bm=one.expand(B, T, 1, N), Cm=one.expand(B, T, 1, N))
    y, h = gdr.ssm_scan_fwd(**d)
    d.update(Bm=one.expand(B, T, 1, N).contiguous(), Cm=one.expand(B, T, 1, N).contiguous())
    y2, h2 = gdr.ssm_scan_fwd(**d)
    assert torch.equal(y, y2) and torch.equal(h, h2)


def test_nothing_behind_a_row_is_read():
    c = make(3, 300, 36, 16, lengths=[0, 130, 300])
    d = {k: cuda(v) for k, v in c.items()}
    y, h = gdr.ssm_scan_fwd(**d)
    for k in ("x", "dt", "Bm", "Cm", "z"):
        v = c[k].clone()
        for b, n in enumerate([0, 130, 300]):
            v[b, n:] = float("nan")
        d[k] = v.cuda()
    y2, h2 = gdr.ssm_scan_fwd(**d)
    assert torch.equal(y, y2) and torch.equal(h, h2)


def test_non_finite_values_stay_in_their_channel_and_row():
    c = make(2, 80, 40, 16)
    d = {k: cuda(v) for k, v in c.items()}
    y, h = gdr.ssm_scan_fwd(**d)
    x = c["x"].clone()
    x[0, 33, 5] = float("nan")
    y2, h2 = gdr.ssm_scan_fwd(**{**d, "x": x.cuda()})
    assert torch.isnan(y2[0, 33:, 5]).all() and torch.isnan(h2[0, 5]).all()
    y2[0, 33:, 5], h2[0, 5] = y[0, 33:, 5], h[0, 5]
    assert torch.equal(y, y2) and torch.equal(h, h2)


def test_extreme_time_steps():
    """Time steps from 0 to far past the exponential's range: full decay, no decay, no NaN."""
    c = make(1, 64, 32, 16, dt=FP, bias=False)
    c["dt"] = torch.linspace(-120, 200, 64)[None, :, None].expand(1, 64, 32).contiguous()
    y_ref, h_ref, by, bh = ssm.scan_fwd(**c)
    y, h = gdr.ssm_scan_fwd(**{k: cuda(v) for k, v in c.items()})
    near(y, y_ref, by, FP, "y")
    near(h, h_ref, bh, FP, "h")


@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("B,D,G", [(1, 4, 1), (3, 66, 2), (2, 257, 1), (33, 128, 4)])
def test_step(B, D, G, dt, N):
    c = make(B, 1, D, N, G, dt, seed=B)
    y_ref, h_ref, by, bh = ssm.scan_fwd(**c)
    h = c.pop("h0").cuda()
    c.pop("lengths")
    d = {k: cuda(v[:, 0] if k in ("x", "dt", "z", "Bm", "Cm") else v) for k, v in c.items()}
    y = gdr.ssm_scan_step(**d, h=h)
    near(y[:, None], y_ref, by, dt, "y")
    near(h, h_ref, bh, FP, "h")


def test_steps_continue_a_prompt():
    c = make(2, 40, 48, 16, dt=FP)
    d = {k: cuda(v) for k, v in c.items()}
    y_ref, h_ref, by, bh = ssm.scan_fwd(**c)
    seq = ("x", "dt", "z", "Bm", "Cm")
    y, h = gdr.ssm_scan_fwd(**{k: (v[:, :30] if k in seq else v) for k, v in d.items()})
    outs = [y]
    for t in range(30, 40):
        one = {k: (v[:, t] if k in seq else v) for k, v in d.items() if k not in ("h0", "lengths")}
        outs.append(gdr.ssm_scan_step(**one, h=h)[:, None])
    near(torch.cat(outs, 1), y_ref, by, FP, "y")
    near(h, h_ref, bh, FP, "h")


def test_streams_host_and_repeats():
    c = make(2, 600, 64, 16)
    d = {k: cuda(v) for k, v in c.items()}
    y, h = gdr.ssm_scan_fwd(**d)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [gdr.ssm_scan_fwd(**d, stream=s) for s in streams for _ in range(3)]   # two at a time
    torch.cuda.synchronize()
    assert all(torch.equal(y, a) and torch.equal(h, b) for a, b in outs)
    y2, h2 = gdr.ssm_scan_fwd(**c)
    assert not y2.is_cuda and torch.equal(y.cpu(), y2) and torch.equal(h.cpu(), h2)


def test_stream_handles_workspaces_and_options():
    c = make(1, 700, 40, 16)
    d = {k: cuda(v) for k, v in c.items()}
    y, h = gdr.ssm_scan_fwd(**d)
    ws = torch.empty(gdr.ssm_scan_fwd_workspace_size(1, 700, 40, 1, 16) + 256, dtype=torch.uint8, device="cuda")
    for kw in (dict(workspace=ws), dict(stream=torch.cuda.current_stream()), dict(stream=0),
               dict(stream=torch.cuda.current_stream().cuda_stream)):
        y2, h2 = gdr.ssm_scan_fwd(**d, **kw)
        assert torch.equal(y, y2) and torch.equal(h, h2)
    y2, none = gdr.ssm_scan_fwd(**d, final_state=False)
    assert none is None and torch.equal(y, y2)
    with pytest.raises(ValueError):
        gdr.ssm_scan_fwd(**{**d, "dt": d["dt"][:, :-1]})
    with pytest.raises(ValueError):
        gdr.ssm_scan_fwd(**{**d, "x": d["x"].transpose(1, 2)})
    with pytest.raises(ValueError):
        gdr.ssm_scan_fwd(**{**d, "A": d["A"].cpu()})
    with pytest.raises(TypeError):
        gdr.ssm_scan_fwd(**{**d, "z": d["z"].float()})
    with pytest.raises(TypeError):
        gdr.ssm_scan_fwd(**{**d, "A": None})
    with pytest.raises(gdr.GDRError):
        gdr.ssm_scan_fwd(**{**d, "A": d["A"][:, :4].contiguous(), "Bm": d["Bm"][..., :4].contiguous(),
                            "Cm": d["Cm"][..., :4].contiguous(), "h0": None})


def test_rows_far_apart():
    """Rows more than 2^31 elements apart (4.3 GB of address space, little of it touched)."""
    B, T, D, N = 2, 40, 16, 8
    c = make(B, T, D, N)
    d = {k: cuda(v) for k, v in c.items()}
    far = torch.empty(2 ** 31 + 16 + T * D, dtype=BF, device="cuda").as_strided((B, T, D), (2 ** 31 + 16, D, 1))
    far.copy_(d["x"])
    y, h = gdr.ssm_scan_fwd(**d)
    y2, h2 = gdr.ssm_scan_fwd(**{**d, "x": far})
    assert torch.equal(y, y2) and torch.equal(h, h2)
    w = rnd(D, 4, seed=3).cuda()
    assert torch.equal(gdr.short_conv_fwd(far, w)[0], gdr.short_conv_fwd(d["x"], w)[0])
    g, g2 = gdr.short_conv_bwd(far, w, far), gdr.short_conv_bwd(d["x"], w, d["x"])
    assert torch.equal(g[0], g2[0]) and torch.equal(g[1], g2[1])


def test_graph_capture():
    c = make(1, 700, 40, 16)
    d = {k: cuda(v) for k, v in c.items()}
    one = {k: (v[:, 0] if k in ("x", "dt", "z", "Bm", "Cm") else v) for k, v in d.items() if k not in ("h0", "lengths")}
    st = d["h0"].clone()
    ref = gdr.ssm_scan_fwd(**d)
    gdr.ssm_scan_step(**one, h=st)
    st.copy_(d["h0"])
    torch.cuda.synchronize()
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = gdr.ssm_scan_fwd(**d)
    with torch.cuda.graph(g2):
        step = gdr.ssm_scan_step(**one, h=st)
    for _ in range(3):
        g.replay()
        g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(ref[0], out[0]) and torch.equal(ref[1], out[1])
    want = d["h0"].clone()
    for _ in range(3):
        y = gdr.ssm_scan_step(**one, h=want)
    assert torch.equal(want, st) and torch.equal(y, step)


def test_a_whole_mixer():
    """Convolution, scan and single tokens as a layer runs them: one prompt, cut anywhere, and the
    last tokens one by one give the same outputs and states."""
    B, T, D, N = 2, 60, 64, 16
    dt = FP
    proj = rnd(B, T, 2 * D, dtype=dt).cuda()
    c = make(B, T, D, N, dt=dt)
    p = {k: cuda(c[k]) for k in ("A", "D_skip", "dt_bias")}
    w, b = rnd(D, 4, seed=20, scale=0.5).cuda(), rnd(D, seed=21).cuda()
    to_dt, to_bc = rnd(D, D, seed=22, scale=D ** -0.5).cuda(), rnd(D, 2 * N, seed=23, scale=D ** -0.5).cuda()

    def prompt(rows, conv, h):
        u, conv = gdr.short_conv_fwd(rows[..., :D], w, b, conv)
        bc = u @ to_bc
        y, h = gdr.ssm_scan_fwd(u, u @ to_dt, Bm=bc[..., None, :N], Cm=bc[..., None, N:], z=rows[..., D:], h0=h, **p)
        return y, conv, h
    whole, conv, h = prompt(proj, None, None)
    y1, conv1, h1 = prompt(proj[:, :41], None, None)
    outs = [y1]
    for t in range(41, T):
        u = gdr.short_conv_step(proj[:, t, :D], conv1, w, b)
        bc = u @ to_bc
        outs.append(gdr.ssm_scan_step(u, u @ to_dt, Bm=bc[:, None, :N], Cm=bc[:, None, N:], h=h1, z=proj[:, t, D:],
                                      **p)[:, None])
    assert torch.equal(conv, conv1)
    # the projections are library products whose order of sums may differ between the two runs
    y = torch.cat(outs, 1)
    assert (y - whole).abs().max() <= 1e-4 * whole.abs().max() and (h - h1).abs().max() <= 1e-4 * h.abs().max()


@pytest.mark.parametrize("case", [dict(B=2, T=75, D=40), dict(B=1, T=700, D=40, dt=FP), dict(B=3, T=50, D=66, G=2),
                                  dict(B=230, T=37, D=36)], ids=str)
def test_y_in_place(case):
    """y may be x, dt or z itself; one that meets them otherwise is refused."""
    c = make(**case)
    d = {k: cuda(v) for k, v in c.items()}
    ref, h = gdr.ssm_scan_fwd(**d)
    for k in ("x", "dt", "z"):
        e = {**d, k: d[k].clone()}
        y, h2 = gdr.ssm_scan_fwd(**e, y=e[k])
        assert torch.equal(y, ref) and torch.equal(e[k], ref) and torch.equal(h, h2), k
    wide = torch.zeros(2, *d["x"].shape, dtype=d["x"].dtype, device="cuda")
    wide[0] = d["x"]
    with pytest.raises(gdr.GDRError):
        gdr.ssm_scan_fwd(**{**d, "x": wide[0]}, y=wide.view(-1)[8:8 + d["x"].numel()].view_as(d["x"]))
    if case["B"] < 100:
        one = {k: (v[:, 0].contiguous() if k in ("x", "dt", "z", "Bm", "Cm") else v) for k, v in d.items()
               if k not in ("h0", "lengths")}
        a, b = d["h0"].clone(), d["h0"].clone()
        ref = gdr.ssm_scan_step(**one, h=a)
        assert torch.equal(gdr.ssm_scan_step(**one, h=b, y=one["x"]), ref) and torch.equal(a, b)


# Two channels a thread are taken where twice the channels still fill two blocks on most SMs, in bf16 from
# N = 16 and in fp32 from N = 32 on; a last block with one channel of a thread's two, and rows that end.
@pytest.mark.parametrize("case", [
    dict(B=230, T=35, D=36, N=16),
    dict(B=230, T=35, D=41, N=16, lengths=[35, 3, 0, 32, 31] * 46),
    dict(B=230, T=35, D=20, N=32),
    dict(B=230, T=35, D=20, N=32, dt=FP, lengths=[35, 3, 0, 32, 31] * 46),
    dict(B=230, T=35, D=17, N=32, dt=FP),
    dict(B=230, T=35, D=12, N=64),
    dict(B=230, T=35, D=12, N=64, dt=FP),
    dict(B=230, T=35, D=9, N=64, dt=FP, lengths=[35, 3, 0, 32, 31] * 46),
    dict(B=230, T=35, D=40, N=16, dt=FP),      # and sizes that would, of a type and N that do not
    dict(B=230, T=35, D=72, N=8),
], ids=str)
def test_many_rows(case):
    c = make(**case)
    y_ref, h_ref, by, bh = ssm.scan_fwd(**c)
    y, h = gdr.ssm_scan_fwd(**{k: cuda(v) for k, v in c.items()})
    near(y, y_ref, by, c["x"].dtype, "y")
    near(h, h_ref, bh, FP, "h")
