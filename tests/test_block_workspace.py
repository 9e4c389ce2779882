"""Scratch and kept buffers of exactly the bytes that the size functions return,
between guard regions, in the normal and the checked build: nothing is written
beside them, nothing is read that the call has not written (the results do
not depend on what they held)."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

GUARD = 4096
TD = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def m2rnn():
    import __graft_entry__
    __graft_entry__.build()
    from non_linear_matrix_gb300 import build as b
    b.build(checked=True)
    from non_linear_matrix_gb300 import m2rnn as m
    m.use_library("normal")
    yield m
    m.use_library("normal")


class Exact:
    """Buffers of n bytes filled with ``fill`` between guards."""

    def __init__(self, fill):
        self.fill, self.bufs = fill, []

    def __call__(self, n):
        n = int(n)
        buf = torch.full((n + 2 * GUARD,), 165, dtype=torch.uint8, device="cuda")
        buf[GUARD:GUARD + n] = self.fill
        self.bufs.append((buf, n))
        return buf[GUARD:GUARD + n]

    def check(self):
        torch.cuda.synchronize()
        for buf, n in self.bufs:
            assert (buf[:GUARD] == 165).all() and (buf[GUARD + n:] == 165).all()


def run_all(m2rnn, call):
    """call(Exact) -> dict of tensors, in both builds and with two fills: one result."""
    first = None
    for which in ("normal", "checked"):
        m2rnn.use_library(which)
        try:
            for fill in (0, 255):
                m2rnn.device_status(clear=True)
                ws = Exact(fill)
                got = call(ws)
                ws.check()
                assert m2rnn.device_status(clear=True) == (0, 0)
                got = {n: t for n, t in got.items() if t is not None}
                first = first or got
                assert got.keys() == first.keys()
                for n, t in got.items():
                    assert torch.equal(t, first[n]), (which, fill, n)
        finally:
            m2rnn.use_library("normal")


def rn_of(seed, td):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g).to(td).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,W", [(1, 1, 8, 4), (3, 37, 136, 4), (2, 5, 40, 2), (1, 3001, 200, 3), (70, 9, 640, 4)])
def test_conv(m2rnn, B, T, C, W, dtype):
    rn = rn_of(T + C, TD[dtype])
    x, w, bias, dy = rn(B, T, C), rn(C, W), rn(C), rn(B, T, C)
    s = m2rnn.ConvShape(B, T, C, W, int(dtype == "bf16"), int(dtype == "bf16"), 1)
    run_all(m2rnn, lambda ws: m2rnn.conv_bwd(
        x, w, dy, bias, workspace=ws(m2rnn.lib().m2rnn_conv_bwd_workspace_size(ctypes.byref(s)))))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,Nq,Nk,K", [(1, 1, 1, 1, 16), (2, 37, 3, 2, 64), (3, 21, 2, 1, 256), (4, 999, 8, 2, 104)])
def test_qk_norm(m2rnn, B, T, Nq, Nk, K, dtype):
    rn = rn_of(T + K, TD[dtype])
    q, k, wq, wk, dq, dk = rn(B, T, Nq, K), rn(B, T, Nk, K), rn(K), rn(K), rn(B, T, Nq, K), rn(B, T, Nk, K)
    s = m2rnn.QkShape(B, T, Nq, Nk, K, 0, 0, int(dtype == "bf16"), int(dtype == "bf16"), 0)
    run_all(m2rnn, lambda ws: m2rnn.qk_norm_bwd(
        q, k, wq, wk, dq, dk, workspace=ws(m2rnn.lib().m2rnn_qk_norm_bwd_workspace_size(ctypes.byref(s)))))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,N,K,V,Nq", [
    (1, 1, 1, 16, 16, 1), (2, 130, 5, 64, 16, 1),   # one segment
    (1, 700, 2, 64, 32, 1), (3, 1500, 6, 128, 32, 2), (2, 900, 7, 32, 16, 7),  # several
    (400, 70, 2, 16, 16, 1)])                        # more pairs than CTAs at a time
def test_scan(m2rnn, B, T, N, K, V, Nq, dtype):
    td = TD[dtype]
    rn = rn_of(T + K, td)
    x = (rn(B, T, Nq, K) * 0.2, rn(B, T, Nq, K) * 0.2, rn(B, T, N, V), rn(B, T, N), rn(N).abs(), rn(N) - 3)
    w_r, dy, H0, dHT = rn(N, V), rn(B, T, N, V), rn(B, N, K, V).float(), rn(B, N, K, V).float()
    s = ctypes.byref(m2rnn.Shape(B, T, N, K, V, int(dtype == "bf16"), 0, Nq))

    def call(ws):
        L = m2rnn.lib()
        size, res = L.m2rnn_scan_saved_size(s), {}
        for n, given in (("least", L.m2rnn_scan_fwd_workspace_size(s, 0)), ("one part", size)):
            res["y " + n], res["H " + n], _ = m2rnn.scan_fwd(*x, w_r, H0, workspace=ws(given))
        res["y kept"], res["H kept"], saved = m2rnn.scan_fwd(*x, w_r, H0, out={"saved": ws(size)})
        for n, kept in (("kept", saved), ("again", None)):
            work = ws(L.m2rnn_scan_bwd_workspace_size(s, int(kept is not None)))
            g = m2rnn.scan_bwd(*x, dy, w_r, H0, dHT, saved=kept, workspace=work, want_dH0=True)
            res.update({f"{a} {n}": t for a, t in g.items()})
        assert torch.equal(res["y least"], res["y one part"]) and torch.equal(res["y kept"], res["y least"])
        assert torch.equal(res["H least"], res["H one part"]) and torch.equal(res["H kept"], res["H least"])
        assert all(torch.equal(t, res[n[:-4] + "again"]) for n, t in res.items()
                   if n.endswith(" kept") and n[:-4] + "again" in res)
        return res
    run_all(m2rnn, call)
