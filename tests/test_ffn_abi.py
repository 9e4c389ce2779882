"""Refusals of the feed-forward operators' entry points and their binding that need
no GPU: shapes and arguments are checked on the host before any device call."""
import ctypes

import pytest
import torch

from non_linear_matrix_gb300 import build as nb

A = [ctypes.c_void_p((i + 1) << 40) for i in range(10)]  # addresses far apart
SZ = 1 << 50
NORM_BAD = [
    (None, -1),
    ((-1, 4, 64, 1), -1),             # B < 0
    ((1, -4, 64, 1), -1),             # T < 0
    ((1, 4, 0, 1), -1),               # D < 1
    ((1, 4, 64, 2), -1),              # dtype
    ((1, 4, 60, 1), -2),              # D not a multiple of 8
    ((1 << 16, 1 << 15, 64, 1), -2),  # B * T
    ((1 << 10, 1 << 20, 8192, 1), -2),  # B * T * D
]


@pytest.fixture(scope="module")
def m():
    nb.build()
    from non_linear_matrix_gb300 import m2rnn
    m2rnn.use_library("normal")
    return m2rnn


def norm_fwd(L, s, x=A[0], x_rows=None, res=A[1], res_rows=None, w=A[2], eps=1e-6, r=A[3], y=A[4]):
    return L.m2rnn_add_norm_fwd(s, x, x_rows, res, res_rows, w, eps, r, y, None)


@pytest.mark.parametrize("shape,code", NORM_BAD + [((1, 4, 16392, 1), -2)])
def test_norm_refuses_shapes(m, shape, code):
    L, s = m.lib(), None if shape is None else ctypes.byref(m.NormShape(*shape))
    assert norm_fwd(L, s) == code
    assert L.m2rnn_add_norm_q8(s, A[0], None, A[1], None, A[2], 1e-6, A[3], A[4], A[5], None) == code
    assert L.m2rnn_add_norm_bwd(s, A[0], None, A[1], 1e-6, A[2], A[3], A[4], A[5], A[6], SZ, None) == code
    assert L.m2rnn_add_norm_bwd_workspace_size(s) == 0


@pytest.mark.parametrize("shape,code", NORM_BAD + [((1, 4, (1 << 20) + 8, 1), -2)])
def test_quant_refuses_shapes(m, shape, code):
    s = None if shape is None else ctypes.byref(m.NormShape(*shape))
    assert m.lib().m2rnn_quant_rows(s, A[0], None, A[1], A[2], None) == code


def test_norm_refuses_arguments(m):
    L, s = m.lib(), ctypes.byref(m.NormShape(2, 4, 64, 1))
    rows = lambda b, t: ctypes.byref(m.Rows(b, t))  # noqa: E731
    assert norm_fwd(L, s, eps=-1.0) == -1 and norm_fwd(L, s, eps=float("nan")) == -1
    assert norm_fwd(L, s, x_rows=rows(-64, 64)) == -1 and norm_fwd(L, s, x_rows=rows(256, -64)) == -1
    assert norm_fwd(L, s, x_rows=rows(256, 60)) == -3 and norm_fwd(L, s, res_rows=rows(4, 64)) == -3
    assert norm_fwd(L, s, x_rows=rows(1 << 40, 64)) == -2
    assert norm_fwd(L, s, r=None) == -1 and norm_fwd(L, s, res=None) == -1  # r goes with res
    for at in (A[0], A[1], A[2], A[3]):  # y over an input or r
        assert norm_fwd(L, s, y=at) == -1
    assert norm_fwd(L, s, r=ctypes.c_void_p(A[0].value + 16)) == -1
    assert norm_fwd(L, s, x_rows=rows(288, 72), r=A[0]) == -1  # in place only where rows are contiguous
    bwd = lambda dx, dw: L.m2rnn_add_norm_bwd(s, A[0], None, A[1], 1e-6, A[2], A[3], dx, dw, A[6], SZ, None)  # noqa: E731
    assert bwd(A[0], A[5]) == -1 and bwd(ctypes.c_void_p(A[2].value + 16), A[5]) == -1 and bwd(A[4], A[4]) == -1
    assert L.m2rnn_quant_rows(s, A[0], None, A[0], A[2], None) == -1
    assert L.m2rnn_quant_rows(s, A[0], rows(256, 60), A[1], A[2], None) == -3


GLU_BAD = [
    (None, -1),
    ((-1, 64, 64, 1, 0), -1),
    ((4, 0, 64, 1, 0), -1),
    ((4, 64, 0, 1, 0), -1),
    ((4, 64, 64, 2, 0), -1),             # dtype
    ((4, 64, 64, 1, 2), -1),             # activation
    ((4, 60, 64, 1, 0), -2),
    ((4, 64, 60, 1, 0), -2),
    ((4, (1 << 16) + 16, 64, 1, 0), -2), # D
    ((4, 64, (1 << 20) + 8, 1, 0), -2),  # F
    ((1 << 31, 64, 64, 1, 0), -2),
    ((1 << 30, 64, 2048, 1, 0), -2),     # M * F
]


@pytest.mark.parametrize("shape,code", GLU_BAD)
def test_glu_refuses_shapes(m, shape, code):
    L, s = m.lib(), None if shape is None else ctypes.byref(m.GluShape(*shape))
    assert L.m2rnn_glu_fwd(s, A[0], 1 << 21, A[1], A[2], A[3], A[4], SZ, None) == code
    assert L.m2rnn_glu_bwd(s, A[0], 1 << 21, A[1], A[2], A[3], A[4], A[5], A[6], A[7], SZ, None) == code
    assert L.m2rnn_glu_q8(s, A[0], 1 << 21, A[1], A[2], A[3], A[4], A[5], A[6], None) == code
    assert L.m2rnn_linear_q8(s, A[0], 1 << 21, A[1], A[2], A[3], A[4], 64, A[5], None) == code
    assert L.m2rnn_glu_fwd_workspace_size(s) == 0 and L.m2rnn_glu_bwd_workspace_size(s) == 0


def test_glu_refuses_arguments(m):
    L, s = m.lib(), ctypes.byref(m.GluShape(4, 64, 64, 1, 0))
    fwd = lambda row=64, h=A[3]: L.m2rnn_glu_fwd(s, A[0], row, A[1], A[2], h, None, 0, None)  # noqa: E731
    assert fwd(row=56) == -1 and fwd(row=0) == -1 and fwd(row=68) == -3 and fwd(row=1 << 39) == -2
    assert all(fwd(h=a) == -1 for a in A[:3])
    one = ctypes.byref(m.GluShape(1, 64, 64, 1, 0))  # a row distance beyond a tensor map's
    assert L.m2rnn_glu_fwd(one, A[0], 1 << 39, A[1], A[2], A[3], None, 0, None) == -2
    bwd = lambda dx=A[4], dwg=A[5], dwu=A[6]: L.m2rnn_glu_bwd(  # noqa: E731
        s, A[0], 64, A[1], A[2], A[3], dx, dwg, dwu, A[7], SZ, None)
    assert bwd(dwu=None) == -1 and bwd(dwg=None) == -1  # together
    assert bwd(dx=A[0]) == -1 and bwd(dwg=A[1]) == -1 and bwd(dwu=A[3]) == -1 and bwd(dwg=A[6]) == -1
    f32 = ctypes.byref(m.GluShape(4, 64, 64, 0, 0))
    odd = ctypes.byref(m.GluShape(4, 72, 64, 1, 0))
    for call in (lambda s: L.m2rnn_glu_q8(s, A[0], 80, A[1], A[2], A[3], A[4], A[5], A[6], None),
                 lambda s: L.m2rnn_linear_q8(s, A[0], 80, A[1], A[2], A[3], A[4], 64, A[5], None)):
        assert call(f32) == -1 and call(odd) == -2  # bf16 outputs; D a multiple of 16
    lin = lambda row=64, y=A[5], res_row=64: L.m2rnn_linear_q8(  # noqa: E731
        s, A[0], row, A[1], A[2], A[3], A[4], res_row, y, None)
    assert lin(row=72) == -3 and lin(row=48) == -1 and lin(res_row=60) == -3
    assert all(lin(y=a) == -1 for a in A[:4]) and lin(y=A[4], res_row=72) == -1


def test_sizes(m):
    L = m.lib()
    size = lambda f, *s: f(ctypes.byref(m.GluShape(*s)))  # noqa: E731
    assert size(L.m2rnn_glu_fwd_workspace_size, 1000, 512, 2048, 1, 0) == 0          # bf16: operands as they are
    assert size(L.m2rnn_glu_fwd_workspace_size, 64, 512, 2048, 0, 0) == 0            # few tokens
    assert size(L.m2rnn_glu_fwd_workspace_size, 1000, 512, 2048, 0, 0) >= 6 * 512 * (1000 + 2 * 2048)
    assert size(L.m2rnn_glu_bwd_workspace_size, 1000, 512, 2048, 1, 0) >= 4 * 1000 * 2048
    assert size(L.m2rnn_glu_bwd_workspace_size, 0, 512, 2048, 1, 0) == 0
    s = ctypes.byref(m.NormShape(10, 100, 512, 1))
    assert 0 < L.m2rnn_add_norm_bwd_workspace_size(s) <= 304 * 512 * 4


def test_binding_refuses(m):
    """What the binding finds before it calls the library."""
    x, w = torch.zeros(4, 64).bfloat16(), torch.zeros(8, 64).bfloat16()
    half = x.half()
    for bad, err in ((lambda: m.add_norm_fwd(half), TypeError), (lambda: m.add_norm_fwd(x, x.float()), TypeError),
                     (lambda: m.add_norm_fwd(x, None, torch.zeros(60).bfloat16()), ValueError),
                     (lambda: m.add_norm_fwd(x, out={"r": x}), ValueError),
                     (lambda: m.add_norm_bwd(x, x[:2]), ValueError), (lambda: m.quant_rows(half), TypeError),
                     (lambda: m.glu_fwd(x, w, w, act="relu"), ValueError), (lambda: m.glu_fwd(x, w, w.float()), TypeError),
                     (lambda: m.glu_fwd(x, w[0], w[0]), ValueError),
                     (lambda: m.glu_fwd(x, w, torch.zeros(8, 72).bfloat16()), ValueError),
                     (lambda: m.glu_bwd(x, w, w, x), ValueError), (lambda: m.glu_q8(x, x, w, w, w, w), TypeError),
                     (lambda: m.linear_q8(x.to(torch.float8_e4m3fn), torch.zeros(3), w, w), ValueError)):
        with pytest.raises(err):
            bad()
