"""Refusals of the block operators' entry points that need no GPU: shapes and
arguments are checked on the host before any device call."""
import ctypes

import pytest

from non_linear_matrix_gb300 import build as nb

P = ctypes.c_void_p(16)
SZ = ctypes.c_size_t(1 << 30)


@pytest.fixture(scope="module")
def m():
    nb.build()
    from non_linear_matrix_gb300 import m2rnn
    m2rnn.use_library("normal")
    return m2rnn


@pytest.mark.parametrize("shape,code", [
    (None, -1),
    ((0, 8, 64, 4, 1, 1, 1), -1),   # B < 1
    ((1, -1, 64, 4, 1, 1, 1), -1),  # T < 0
    ((1, 8, 60, 4, 1, 1, 1), -2),   # C not a multiple of 8
    ((1, 8, 64, 5, 1, 1, 1), -2),   # W outside 2..4
    ((1, 8, 64, 1, 1, 1, 1), -2),
    ((1, 8, 64, 4, 7, 1, 1), -1),   # dtype
    ((1, 8, 64, 4, 1, 1, 2), -1),   # activation
    ((1, 8, 1 << 25, 4, 1, 1, 1), -2),          # C > 2^24
    ((1, (1 << 30) + 1, 8, 4, 1, 1, 1), -2),    # T > 2^30
])
def test_conv_refuses(m, shape, code):
    s = None if shape is None else ctypes.byref(m.ConvShape(*shape))
    L = m.lib()
    assert L.m2rnn_conv_fwd(s, P, None, P, P, P, P, None, None) == code
    assert L.m2rnn_conv_bwd(s, P, None, P, P, P, P, None, P, P, P, None, P, SZ, None) == code
    assert L.m2rnn_conv_step(s, P, None, P, P, P, P, P, None) == code


def test_conv_refuses_rows_and_gradient_type(m):
    L, s = m.lib(), ctypes.byref(m.ConvShape(2, 8, 64, 4, 1, 1, 1))
    for rows, code in ((m.Rows(-64, 64), -1), (m.Rows(512, 60), -3), (m.Rows(516, 64), -3)):
        assert L.m2rnn_conv_fwd(s, P, ctypes.byref(rows), P, P, P, P, None, None) == code
    bad = ctypes.byref(m.ConvShape(2, 8, 64, 4, 0, 1, 1))  # bf16 gradient of fp32 inputs
    assert L.m2rnn_conv_bwd(bad, P, None, P, P, P, P, None, P, P, P, None, P, SZ, None) == -1
    assert L.m2rnn_conv_step(s, P, None, P, P, P, P, P, None) == -1  # T != 1


@pytest.mark.parametrize("shape,code", [
    (None, -1),
    ((1, 8, 0, 1, 64, 64, 8, 1, 1, 0), -1),    # Nq < 1
    ((1, 8, 2, 1, 60, 0, 0, 1, 1, 0), -2),     # K not a multiple of 8
    ((1, 8, 2, 1, 264, 0, 0, 1, 1, 0), -2),    # K > 256
    ((1, 8, 2, 1, 64, 72, 8, 1, 1, 0), -2),    # R > K
    ((1, 8, 2, 1, 64, 20, 8, 1, 1, 0), -2),    # R not a multiple of 8
    ((1, 8, 2, 1, 64, 64, 8, 1, 1, 2), -1),    # interleaved
    ((1, 8, 2, 1, 64, 64, 8, 3, 1, 0), -1),    # dtype
])
def test_qk_norm_refuses(m, shape, code):
    s = None if shape is None else ctypes.byref(m.QkShape(*shape))
    L = m.lib()
    assert L.m2rnn_qk_norm_fwd(s, P, None, P, None, P, P, 1e-6, P, P, P, P, P, None) == code
    assert L.m2rnn_qk_norm_bwd(s, P, None, P, None, P, P, 1e-6, P, P, P, P, P, P, P, P, P, P, SZ,
                               None) == code


def test_qk_norm_refuses_eps_tables_positions(m):
    L, s = m.lib(), ctypes.byref(m.QkShape(1, 8, 2, 1, 64, 64, 4, 1, 1, 0))
    fwd = lambda eps, c, n, pos: L.m2rnn_qk_norm_fwd(s, P, None, P, None, P, P, eps, c, n, pos, P, P,  # noqa: E731
                                                     None)
    assert fwd(-1.0, P, P, P) == -1 and fwd(float("nan"), P, P, P) == -1
    assert fwd(1e-6, None, P, P) == -1   # R > 0 without a table
    assert fwd(1e-6, P, P, None) == -1   # 8 tokens, 4 positions


@pytest.mark.parametrize("shape,code", [
    (None, -1),
    ((1, 8, 2, 48, 16, 1, 0, 1), -2),   # K
    ((1, 8, 2, 64, 64, 1, 0, 1), -2),   # V
    ((1, 8, 3, 64, 16, 1, 0, 2), -1),   # Nq does not divide N
    ((1, -2, 2, 64, 16, 1, 0, 1), -1),  # T
    ((1, 8, 2, 64, 16, 5, 0, 1), -1),   # dtype
])
def test_scan_refuses(m, shape, code):
    s = None if shape is None else ctypes.byref(m.Shape(*shape))
    L = m.lib()
    assert L.m2rnn_scan_fwd(s, None, P, P, P, P, P, P, P, None, P, None, None, P, SZ, None) == code
    assert L.m2rnn_scan_bwd(s, None, P, P, P, P, P, P, P, None, None, P, None, P, P, P, P, P, P, P,
                            None, P, SZ, None) == code
    assert L.m2rnn_scan_step(s, None, P, P, P, P, P, P, P, P, P, P, None) == code


def test_scan_sizes(m):
    """The workspace of both passes and what the forward pass keeps: 0 without
    tokens or for a bad shape, less for the backward pass when it is given."""
    L = m.lib()
    s = ctypes.byref(m.Shape(2, 300, 4, 64, 16, 1, 0, 1))
    saved = L.m2rnn_scan_saved_size(s)
    # 5 chunks of one head block (64 x 64 fp32 each) per sequence and their gate values
    assert saved >= 2 * 5 * (64 * 64 * 4 + 4 * 3 * 64 * 4)
    # without a backward pass to come, bf16 inputs' states are kept in bf16
    assert L.m2rnn_scan_fwd_workspace_size(s, 0) == saved - 2 * 5 * 64 * 64 * 2
    assert L.m2rnn_scan_fwd_workspace_size(ctypes.byref(m.Shape(2, 300, 4, 64, 16, 0, 0, 1)), 0) == saved
    assert L.m2rnn_scan_fwd_workspace_size(s, 1) == 0
    assert L.m2rnn_scan_bwd_workspace_size(s, 0) == L.m2rnn_scan_bwd_workspace_size(s, 1) + saved
    for bad in ((2, 0, 4, 64, 16, 1, 0, 1), (2, 300, 4, 60, 16, 1, 0, 1)):
        s = ctypes.byref(m.Shape(*bad))
        assert L.m2rnn_scan_saved_size(s) == 0 and L.m2rnn_scan_bwd_workspace_size(s, 0) == 0


def test_scan_step_needs_one_token(m):
    s = ctypes.byref(m.Shape(2, 2, 4, 64, 16, 1, 0, 1))
    assert m.lib().m2rnn_scan_step(s, None, P, P, P, P, P, P, P, P, P, P, None) == -1
