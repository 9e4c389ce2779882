"""The convolution of whole sequences reads its neighbours' rows while others are
written: outputs over inputs are refused (on the host, before any device call),
outputs between an input's rows or items are not."""
import ctypes

import pytest
import torch

from non_linear_matrix_gb300 import build as nb


@pytest.fixture(scope="module")
def m():
    nb.build()
    from non_linear_matrix_gb300 import m2rnn
    m2rnn.use_library("normal")
    return m2rnn


B, T, C, W = 2, 8, 64, 4
NX, NS = B * T * C * 2, B * (W - 1) * C * 2  # bytes of x and of the state (bf16)
X, S = 1 << 20, 1 << 22                      # addresses that no device call sees


def ptr(x):
    return None if x is None else ctypes.c_void_p(x)


def fwd(m, y, so=None, state=S, rows=None):
    s = ctypes.byref(m.ConvShape(B, T, C, W, 1, 1, 1))
    r = None if rows is None else ctypes.byref(m.Rows(*rows))
    return m.lib().m2rnn_conv_fwd(s, ptr(X), r, ptr(16), None, ptr(state), ptr(y), ptr(so), None)


def bwd(m, dx, ds=None, dy=1 << 24, dso=1 << 25, grad=1):
    s = ctypes.byref(m.ConvShape(B, T, C, W, 1, grad, 1))
    return m.lib().m2rnn_conv_bwd(s, ptr(X), None, ptr(16), None, ptr(S), ptr(dy), ptr(dso), ptr(dx),
                                  ptr(32), None, ptr(ds), ptr(64), ctypes.c_size_t(1 << 30), None)


def test_outputs_over_inputs(m):
    for y in (X, X + 16, X + NX - 16, X - NX + 16, S, S + NS - 16, S - NX + 16):
        assert fwd(m, y) == -1, hex(y)
    far = 1 << 23
    for so in (S, S + 16, X, X + NX - 16, far, far + NX - 16):
        assert fwd(m, far, so) == -1, hex(so)
    for dx in (X, S, 1 << 24, (1 << 24) + NX - 16, 1 << 25):
        assert bwd(m, dx) == -1, hex(dx)
    assert bwd(m, (1 << 24) + 2 * NX - 16, grad=0) == -1  # fp32 dy: twice as long
    for ds in (X, S, 1 << 24, 1 << 25, far):
        assert bwd(m, far, ds) == -1, hex(ds)


def test_rows_with_room_between(m):
    """x of a wide buffer.  (Without a GPU what is not refused goes on to -6.)"""
    batch = 1 << 16
    ok = lambda rc: rc != -1  # noqa: E731
    item = T * C * 2
    assert ok(fwd(m, X + item, rows=(batch, C))) and ok(fwd(m, X + batch * 2 - NX, rows=(batch, C)))
    assert fwd(m, X + item - 16, rows=(batch, C)) == -1
    assert fwd(m, X + batch * 2 - NX + 16, rows=(batch, C)) == -1
    token = 1 << 14  # elements: the whole of y fits between two tokens
    row = C * 2
    for t in (0, 3, T - 2):
        at = X + t * token * 2
        assert ok(fwd(m, at + row, rows=(batch * 16, token)))
        assert ok(fwd(m, at + 2 * token - NX, rows=(batch * 16, token)))
        assert fwd(m, at + row - 16, rows=(batch * 16, token)) == -1
        assert fwd(m, at + 2 * token - NX + 16, rows=(batch * 16, token)) == -1
    assert ok(fwd(m, X + row, rows=(0, 0))) and fwd(m, X + row - 16, rows=(0, 0)) == -1  # one row for all


@pytest.mark.gpu
def test_refused_and_not(m):
    import __graft_entry__
    __graft_entry__.build()
    g = torch.Generator().manual_seed(1)
    buf = torch.randn(2, 3 * 40, 64, generator=g).bfloat16().cuda()
    w = torch.randn(64, 4, generator=g).bfloat16().cuda()
    x = buf[:, :40]
    want = m.conv_fwd(x, w)[0].clone()
    gap = buf[0, 40:].view(2, 40, 64)  # between the items
    y, _ = m.conv_fwd(x, w, out={"y": gap})
    assert y is gap and torch.equal(y, want)
    xc = x.contiguous()
    for call in (lambda: m.conv_fwd(xc, w, out={"y": xc}), lambda: m.conv_bwd(xc, w, want, out={"dx": xc}),
                 lambda: m.conv_bwd(xc, w, want, out={"dx": want})):
        with pytest.raises(m.M2RNNError) as e:
            call()
        assert e.value.code == -1
