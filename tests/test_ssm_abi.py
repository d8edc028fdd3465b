"""The convolution's and the scan's entry points refuse bad arguments on the host (no GPU needed)."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import gated_delta_rule_89_b200 as gdr
from gated_delta_rule_89_b200 import build as gbuild

OK, INVALID, UNSUPPORTED, ALIGN = 0, 1, 2, 3
P = ctypes.c_void_p
GOOD = P(0x100000)      # never dereferenced: every case below fails validation first


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdr.lib()


def longs(*v):
    return (ctypes.c_longlong * len(v))(*v)


def test_conv_arguments(L):
    def conv(x=GOOD, weight=GOOD, bias=None, state=None, lengths=None, y=GOOD, so=None, strides=None, B=1, H=1, T=4,
             d=8, W=4, act=1, dtype=1):
        return L.gdr_short_conv_fwd(x, weight, bias, state, lengths, y, so, strides, 0, B, H, T, d, W, act, dtype, None)
    for bad in (dict(B=-1), dict(H=-1), dict(T=-1), dict(d=-1), dict(W=0), dict(act=2), dict(dtype=2), dict(x=None),
                dict(weight=None), dict(y=None), dict(strides=longs(1, -1, 1))):
        assert conv(**bad) == INVALID, bad
    for bad in (dict(W=1), dict(W=5), dict(T=1 << 30), dict(d=(1 << 20) + 1), dict(B=1 << 19, T=1 << 20, d=8)):
        assert conv(**bad) == UNSUPPORTED, bad
    for bad in (dict(x=P(0x100001)), dict(weight=P(0x100002)), dict(bias=P(0x100002)), dict(state=P(0x100001)),
                dict(lengths=P(0x100002)), dict(y=P(0x100001)), dict(so=P(0x100001)), dict(x=P(0x100002), dtype=0)):
        assert conv(**bad) == ALIGN, bad
    assert conv(B=0) == OK and conv(d=0) == OK and conv(T=0, x=None, y=None) == OK
    assert L.gdr_last_launch_count() == 0


def test_conv_step_arguments(L):
    def step(x=GOOD, weight=GOOD, bias=None, state=GOOD, y=GOOD, xs=8, B=1, D=8, W=4, act=1, dtype=1):
        return L.gdr_short_conv_step(x, weight, bias, state, y, xs, B, D, W, act, dtype, None)
    for bad in (dict(B=-1), dict(D=-1), dict(act=-1), dict(dtype=7), dict(x=None), dict(state=None), dict(y=None),
                dict(weight=None), dict(xs=-1)):
        assert step(**bad) == INVALID, bad
    assert step(W=8) == UNSUPPORTED
    assert step(state=P(0x100001)) == ALIGN
    assert step(B=0) == OK and step(D=0) == OK


def test_conv_bwd_arguments(L):
    def bwd(x=GOOD, weight=GOOD, dy=GOOD, dx=GOOD, dw=GOOD, db=None, ds=None, xs=None, B=1, H=1, T=4, d=8, W=4, act=1,
            dtype=1, ws=GOOD, size=1 << 40):
        return L.gdr_short_conv_bwd(x, weight, None, None, None, dy, None, dx, dw, db, ds, xs, None, None, B, H, T, d,
                                    W, act, dtype, ws, size, None)
    for bad in (dict(B=-1), dict(x=None), dict(dy=None), dict(dx=None), dict(dw=None), dict(weight=None),
                dict(ws=None), dict(size=0), dict(dtype=3), dict(xs=longs(-1, 0, 0))):
        assert bwd(**bad) == INVALID, bad
    need = L.gdr_short_conv_bwd_workspace_size(1, 1, 4, 8, 4, 1)
    assert need > 0 and bwd(size=need - 1) == INVALID
    assert bwd(W=5) == UNSUPPORTED and L.gdr_short_conv_bwd_workspace_size(1, 1, 4, 8, 5, 1) == 0
    for bad in (dict(ws=P(0x100008)), dict(dy=P(0x100001)), dict(dw=P(0x100002)), dict(db=P(0x100002)),
                dict(ds=P(0x100001))):
        assert bwd(**bad) == ALIGN, bad
    assert bwd(d=0) == OK and bwd(H=0) == OK


def test_scan_arguments(L):
    def scan(x=GOOD, dt=GOOD, A=GOOD, Bm=GOOD, Cm=GOOD, skip=None, z=None, bias=None, h0=None, lengths=None, y=GOOD,
             hT=None, strides=None, B=1, T=4, D=8, G=1, N=16, dtype=1, ws=None, size=0):
        return L.gdr_ssm_scan_fwd(x, dt, A, Bm, Cm, skip, z, bias, h0, lengths, y, hT, strides, 0, B, T, D, G, N, 1,
                                  dtype, ws, size, None)
    for bad in (dict(B=-1), dict(T=-1), dict(D=-1), dict(G=0), dict(N=0), dict(G=3), dict(dtype=2), dict(x=None),
                dict(dt=None), dict(A=None), dict(Bm=None), dict(Cm=None), dict(y=None),
                dict(strides=longs(*[0] * 9, -1)), dict(T=4096)):      # 4096 tokens of 8 channels need a workspace
        assert scan(**bad) == INVALID, bad
    for bad in (dict(N=4), dict(N=24), dict(N=128), dict(T=1 << 30), dict(D=(1 << 20) + 8)):
        assert scan(**bad) == UNSUPPORTED, bad
    for bad in (dict(A=P(0x100008)), dict(h0=P(0x100004)), dict(hT=P(0x100008)), dict(x=P(0x100001)),
                dict(skip=P(0x100002)), dict(lengths=P(0x100001)), dict(z=P(0x100002), dtype=0)):
        assert scan(**bad) == ALIGN, bad
    need = L.gdr_ssm_scan_fwd_workspace_size(1, 4096, 8, 1, 16, 1)
    assert need > 0 and scan(T=4096, ws=GOOD, size=need - 1) == INVALID
    assert L.gdr_ssm_scan_fwd_workspace_size(1, 4096, 8, 1, 24, 1) == 0
    assert scan(B=0) == OK and scan(D=0) == OK and scan(T=0, x=None, y=None) == OK


def test_scan_step_arguments(L):
    def step(x=GOOD, dt=GOOD, A=GOOD, Bm=GOOD, Cm=GOOD, h=GOOD, y=GOOD, strides=None, B=1, D=8, G=1, N=16, dtype=1):
        return L.gdr_ssm_scan_step(x, dt, A, Bm, Cm, None, None, None, h, y, strides, B, D, G, N, 1, dtype, None)
    for bad in (dict(B=-1), dict(G=5), dict(x=None), dict(h=None), dict(y=None), dict(dtype=-1),
                dict(strides=longs(0, 0, 0, 0, -1))):
        assert step(**bad) == INVALID, bad
    assert step(N=12) == UNSUPPORTED and step(h=P(0x100004)) == ALIGN
    assert step(B=0) == OK and step(D=0) == OK


def test_scan_bwd_arguments(L):
    def bwd(x=GOOD, A=GOOD, z=None, dy=GOOD, dx=GOOD, dA=GOOD, dB=GOOD, dD=None, dz=None, dh0=None, strides=None, B=1,
            T=4, D=8, G=1, N=16, dtype=1, ws=GOOD, size=1 << 40):
        return L.gdr_ssm_scan_bwd(x, GOOD, A, GOOD, GOOD, None, z, None, None, None, dy, None, dx, GOOD, dA, dB, GOOD,
                                  dD, dz, None, dh0, strides, B, T, D, G, N, 1, dtype, ws, size, None)
    for bad in (dict(B=-1), dict(G=0), dict(x=None), dict(A=None), dict(dy=None), dict(dx=None), dict(dA=None),
                dict(dB=None), dict(z=GOOD), dict(ws=None), dict(size=0), dict(dtype=4),
                dict(strides=longs(*[0] * 11, -1))):
        assert bwd(**bad) == INVALID, bad
    assert bwd(N=20) == UNSUPPORTED
    assert bwd(B=1 << 19, T=1 << 14, D=32, G=32, N=64) == UNSUPPORTED
    for bad in (dict(A=P(0x100008)), dict(dA=P(0x100008)), dict(dh0=P(0x100004)), dict(dD=P(0x100002)),
                dict(dx=P(0x100001)), dict(ws=P(0x100008))):
        assert bwd(**bad) == ALIGN, bad
    need = L.gdr_ssm_scan_bwd_workspace_size(2, 90, 64, 1, 16, 1)
    # states every 8 tokens, the one block's parts of dB and dC, dA, dD and ddt_bias per row, and
    # what the forward pass wants
    up = lambda n: (n + 255) // 256 * 256   # noqa: E731
    assert need == up(2 * 12 * 64 * 16 * 4) + up(2 * 90 * 32 * 4) + up(2 * 64 * 16 * 4) + up(2 * 64 * 2 * 4) + \
        L.gdr_ssm_scan_fwd_workspace_size(2, 90, 64, 1, 16, 1)
    assert bwd(D=0) == OK


def test_binding_refuses():
    x = torch.zeros(2, 4, 8)
    with pytest.raises(TypeError):
        gdr.short_conv_fwd(x.double(), torch.zeros(8, 4))
    with pytest.raises(TypeError):
        gdr.ssm_scan_fwd("x", x, x, x, x)
    with pytest.raises(ValueError):
        gdr.short_conv_step(x[:, 0], torch.zeros(2, 3, 8), torch.zeros(8, 4))     # host tensors
    with pytest.raises(ValueError):
        gdr.ssm_scan_step(x[:, 0], x[:, 0], torch.zeros(8, 16), torch.zeros(2, 1, 16), torch.zeros(2, 1, 16),
                          torch.zeros(2, 8, 16))


def test_binding_refuses_host_outputs():
    """A host call's results are new tensors: an output that would stay unwritten is refused (before
    any CUDA call is made)."""
    x, w, st = torch.zeros(2, 4, 8), torch.zeros(8, 4), torch.zeros(2, 3, 8)
    for kw in (dict(y=torch.zeros(2, 4, 8)), dict(state_out=st), dict(state_out=torch.zeros(2, 3, 8))):
        with pytest.raises(ValueError, match=next(iter(kw))):
            gdr.short_conv_fwd(x, w, state=st, **kw)
    h, bc = torch.zeros(2, 8, 16), torch.zeros(2, 4, 1, 16)
    for kw in (dict(y=torch.zeros(2, 4, 8)), dict(h_T=h), dict(h_T=torch.zeros(2, 8, 16))):
        with pytest.raises(ValueError, match=next(iter(kw))):
            gdr.ssm_scan_fwd(x, x, torch.zeros(8, 16), bc, bc, h0=h, **kw)


def test_import_without_cuda_in_torch():
    """A torch build without CUDA has no raw device and stream queries; the package and its build
    module still import there."""
    code = ("import torch\n"
            "for n in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "import gated_delta_rule_89_b200, gated_delta_rule_89_b200.build\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(gdr.__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def at(n):
    return P(0x100000 + n)


def test_outputs_in_the_inputs_memory(L):
    """An output that lies in rows which other threads still read is refused.  (Nothing here is launched: what
    is allowed is tried on real memory in the GPU tests.)"""
    def conv(x=GOOD, y=at(1 << 20), state=None, strides=None, B=2, H=2, T=10, d=8, dtype=0):
        return L.gdr_short_conv_fwd(x, at(1 << 24), None, state, None, y, None, strides, 0, B, H, T, d, 4, 1, dtype, None)
    size = 2 * 2 * 10 * 8 * 4
    assert conv(y=GOOD) == INVALID
    assert conv(y=at(size - 4)) == INVALID and conv(x=at(size - 4), y=GOOD) == INVALID
    assert conv(state=at((1 << 20) + size - 16)) == INVALID and conv(state=at((1 << 20) - 16)) == INVALID
    rows = longs(10 * 48, 8, 48)       # a third of a projection's rows; y in its last row
    assert conv(strides=rows, y=at((19 * 48 + 8 + 7) * 4)) == INVALID

    def bwd(dx, dy=at(1 << 20)):
        return L.gdr_short_conv_bwd(GOOD, at(1 << 24), None, None, None, dy, None, dx, at(1 << 25), None, None, None,
                                    None, None, 1, 1, 4, 8, 4, 1, 1, at(1 << 26), 1 << 40, None)
    assert bwd(GOOD) == INVALID and bwd(at(1 << 20)) == INVALID

    def conv_step(y, x=GOOD, xs=8):
        return L.gdr_short_conv_step(x, at(1 << 24), None, at(1 << 22), y, xs, 3, 8, 4, 1, 0, None)
    assert conv_step(at(4)) == INVALID and conv_step(GOOD, xs=16) == INVALID and conv_step(at(1 << 22)) == INVALID

    def scan(y, z=None, strides=None):
        return L.gdr_ssm_scan_fwd(GOOD, at(1 << 16), at(1 << 24), at(1 << 17), at(1 << 18), None, z, None, None, None, y,
                                  None, strides, 0, 2, 10, 8, 1, 16, 1, 0, None, 0, None)
    assert scan(at(4)) == INVALID and scan(at((1 << 16) - 4)) == INVALID and scan(at(1 << 17)) == INVALID
    assert scan(at((1 << 18) + 2 * 10 * 16 * 4 - 4)) == INVALID and scan(at(1 << 19), z=at((1 << 19) + 8)) == INVALID
    assert scan(GOOD, strides=longs(160, 16, 80, 8, 160, 16, 160, 16, 80, 8)) == INVALID     # x strided

    def scan_step(y):
        return L.gdr_ssm_scan_step(GOOD, at(1 << 16), at(1 << 24), at(1 << 17), at(1 << 18), None, None, None, at(1 << 20),
                                   y, None, 2, 8, 1, 16, 1, 0, None)
    assert scan_step(at(8)) == INVALID and scan_step(at(1 << 17)) == INVALID
