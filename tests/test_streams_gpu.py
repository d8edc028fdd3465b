"""Calls on another stream than the current one: whose memory is whose.

A side stream is kept busy by a spinning kernel, so that what the call on it reads and writes is
in use when the test's own allocations ask for memory."""
import pytest
import torch

import gated_delta_rule_89_b200 as gdr
from test_ssm_scan_gpu import BF, rnd

pytestmark = pytest.mark.gpu

B, H, T, D, N = 2, 2, 192, 128, 16


def rule(**kw):
    return dict(q=torch.nn.functional.normalize(rnd(B, H, T, D), dim=-1).to(BF),
                k=torch.nn.functional.normalize(rnd(B, H, T, D, seed=1), dim=-1).to(BF),
                v=rnd(B, H, T, D, dtype=BF, seed=2), g=-rnd(B, H, T, D, seed=3).abs() * 0.1,
                beta=torch.sigmoid(rnd(B, H, T, seed=4)), **kw)


def token(**kw):
    return {**{k: v[:, :, 0].contiguous() for k, v in rule().items()}, "S": rnd(B, H, D, D, seed=5), **kw}


def conv(**kw):
    return dict(x=rnd(B, T, 264, dtype=BF), weight=rnd(264, 4, seed=1), **kw)


def scan(**kw):
    return dict(x=rnd(B, T, 264), dt=rnd(B, T, 264, seed=1) - 2, A=-torch.exp(rnd(264, N, seed=2)),
                Bm=rnd(B, T, 1, N, seed=3), Cm=rnd(B, T, 1, N, seed=4), **kw)


def one(c):
    return {k: (v[:, 0].contiguous() if k in ("x", "dt", "Bm", "Cm") else v) for k, v in c.items()}


# the call, its inputs, and the input that is dropped right behind it
CALLS = {
    "chunk_fwd": (gdr.chunk_fwd, rule, "v"),
    "chunk_fwd_prologue": (gdr.chunk_fwd_prologue, lambda: dict(
        q_raw=rnd(B, H, T, D, dtype=BF), k_raw=rnd(B, H, T, D, dtype=BF, seed=1), v=rnd(B, H, T, D, dtype=BF, seed=2),
        a=rnd(B, H, T, D, dtype=BF, seed=3), A_log=rnd(H, seed=4), dt_bias=rnd(H, D, seed=5),
        b_logit=rnd(B, H, T, seed=6)), "a"),
    "chunk_fwd_gdr2": (gdr.chunk_fwd_gdr2, lambda: {
        **{k: v for k, v in rule().items() if k != "beta"}, "b": rnd(B, H, T, D, dtype=BF, seed=7, scale=0.1),
        "w": rnd(B, H, T, D, dtype=BF, seed=8, scale=0.1)}, "w"),
    "chunk_fwd_gated": (gdr.chunk_fwd_gated, lambda: rule(gate=rnd(B, H, T, D, dtype=BF, seed=7), norm_w=rnd(D)), "gate"),
    "chunk_bwd": (gdr.chunk_bwd, lambda: rule(dO=rnd(B, H, T, D, dtype=BF, seed=7)), "dO"),
    "recurrent_step": (gdr.recurrent_step, token, "S"),
    "recurrent_step_gdr2": (gdr.recurrent_step_gdr2, lambda: {
        **{k: v for k, v in token().items() if k != "beta"}, "b": rnd(B, H, D, dtype=BF, seed=7, scale=0.1),
        "w": rnd(B, H, D, dtype=BF, seed=8, scale=0.1)}, "S"),
    "short_conv_fwd": (gdr.short_conv_fwd, conv, "x"),
    "short_conv_bwd": (gdr.short_conv_bwd, lambda: conv(dy=rnd(B, T, 264, dtype=BF, seed=2)), "dy"),
    "short_conv_step": (gdr.short_conv_step, lambda: dict(one(conv()), state=rnd(B, 3, 264, dtype=BF)), "state"),
    "ssm_scan_fwd": (gdr.ssm_scan_fwd, scan, "dt"),
    "ssm_scan_bwd": (gdr.ssm_scan_bwd, lambda: scan(dy=rnd(B, T, 264, seed=5)), "dy"),
    "ssm_scan_step": (gdr.ssm_scan_step, lambda: dict(one(scan()), h=rnd(B, 264, N)), "h"),
}


def as_tuple(out):
    return tuple(t for t in (out if isinstance(out, tuple) else (out,)) if t is not None)


def busy(stream):
    """About 50 ms of work on the stream."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100_000_000)


def new_like(t):
    return torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=t.device)


@pytest.mark.parametrize("name", CALLS)
def test_a_dropped_input_is_not_handed_on(name):
    call, make, drop = CALLS[name]
    side = torch.cuda.Stream()
    d = {k: v.cuda() for k, v in make().items()}
    torch.cuda.synchronize()
    call(**d, stream=side)       # loads its kernels and gets its memory, both of which wait for the device
    torch.cuda.synchronize()
    busy(side)
    call(**d, stream=side)
    at, shape, dtype = d[drop].data_ptr(), d[drop].shape, d[drop].dtype
    del d[drop]
    fresh = [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(4)]
    still_busy = not side.query()
    torch.cuda.synchronize()
    assert still_busy, "the side stream was done before the question was asked"
    assert at not in [t.data_ptr() for t in fresh]


@pytest.mark.parametrize("name", CALLS)
def test_outputs_come_from_the_stream_that_writes_them(name):
    """Memory that the current stream has just freed may still be in use there: a call on another
    stream does not write to it.  And the results are the same."""
    call, make, _ = CALLS[name]
    d = {k: v.cuda() for k, v in make().items()}
    ref = as_tuple(call(**{k: v.clone() for k, v in d.items()}))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [new_like(t) for t in ref]
    at = {t.data_ptr() for t in freed}
    del freed
    out = as_tuple(call(**d, stream=side))
    assert at.isdisjoint(t.data_ptr() for t in out)
    side.synchronize()
    assert len(out) == len(ref) and all(torch.equal(a, b) for a, b in zip(ref, out))


@pytest.mark.parametrize("name", [n for n in CALLS if not n.endswith(("step", "step_gdr2"))])
def test_page_locked_inputs_are_copied_on_the_stream(name):
    """Their copies run on the stream of the call, not behind what the current stream has to do."""
    call, make, _ = CALLS[name]
    host = {k: v.pin_memory() for k, v in make().items()}
    ref = as_tuple(call(**{k: v.cuda() for k, v in host.items()}))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy(torch.cuda.current_stream())
    out = as_tuple(call(**host, stream=side))
    assert all(not b.is_cuda and torch.equal(a.cpu(), b) for a, b in zip(ref, out))


def test_stream_by_position_and_by_handle():
    d = {k: v.cuda() for k, v in token().items()}
    ref = gdr.recurrent_step(**{k: v.clone() for k, v in d.items()})
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream, torch.cuda.current_stream().cuda_stream):
        a = [d[k].clone() for k in ("q", "k", "v", "g", "beta", "S")]
        torch.cuda.synchronize()
        o = gdr.recurrent_step(*a, None, None, s)
        torch.cuda.synchronize()
        assert torch.equal(o, ref)


@pytest.mark.parametrize("name", ["chunk_fwd", "chunk_bwd", "short_conv_bwd", "ssm_scan_fwd", "ssm_scan_bwd"])
def test_captured_on_a_forked_stream(name):
    """A call on a stream that a capture has forked to, replayed on new inputs, beside an eager call."""
    call, make, drop = CALLS[name]
    d = {k: v.cuda() for k, v in make().items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(**d, stream=side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        out = as_tuple(call(**d, stream=side))
        torch.cuda.current_stream().wait_stream(side)
    for scale in (1.0, 0.5):
        d[drop].mul_(scale)
        g.replay()
        eager = as_tuple(call(**d))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
