"""The feed-forward operators under the checked build (every computed global index
tested against its array), between guard regions and with scratch of exactly the returned
size, filled with zeros and with NaN: the status word stays clean, the results are the
normal build's bit for bit, no guard and no input changes."""
import ctypes
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

GUARD = 256  # bytes
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


class Guarded:
    """Buffers filled with a byte between guards."""

    def __init__(self, fill):
        self.fill, self.bufs = fill, []

    def __call__(self, shape, dtype=torch.float32):
        n = math.prod(shape) * dtype.itemsize
        buf = torch.full((n + 2 * GUARD + 16,), 165, dtype=torch.uint8, device="cuda")
        buf[GUARD:GUARD + n] = self.fill
        self.bufs.append((buf, n))
        return buf[GUARD:GUARD + n].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for buf, n in self.bufs:
            assert (buf[:GUARD] == 165).all() and (buf[GUARD + n:] == 165).all()


def run_all(m2rnn, inputs, run):
    """run(Guarded) -> tensors, in both builds, with two fills."""
    copies = [t.clone() for t in inputs]
    first = None
    for which in ("normal", "checked"):
        m2rnn.use_library(which)
        try:
            assert m2rnn.lib().m2rnn_checked() == (which == "checked")
            for fill in (0, 255):
                m2rnn.device_status(clear=True)
                gd = Guarded(fill)
                got = run(gd)
                gd.check()
                assert m2rnn.device_status(clear=True) == (0, 0)
                got = [t.contiguous().view(torch.uint8) for t in got if t is not None]
                first = first or [t.clone() for t in got]
                assert len(got) == len(first) and all(torch.equal(a, b) for a, b in zip(got, first))
        finally:
            m2rnn.use_library("normal")
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(copies, inputs))


def rn(seed, *s, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*s, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D", [(1, 8), (37, 136), (330, 520), (65, 2008), (19, 8200), (3, 16384)])
def test_norm(m2rnn, M, D, dtype):
    td = TD[dtype]
    buf, res, w, dy, dr = rn(1, M, D + 16, dtype=td), rn(2, M, D, dtype=td), rn(3, D, dtype=td), rn(4, M, D, dtype=td), rn(5, M, D, dtype=td)
    x = buf[:, 8:8 + D]

    def run(gd):
        y, r = m2rnn.add_norm_fwd(x, res, w, out={"y": gd((M, D), td), "r": gd((M, D), td)})
        q, s, r8 = m2rnn.add_norm_q8(x, res, w, out={"q": gd((M, D), torch.float8_e4m3fn), "scale": gd((M,)), "r": gd((M, D), td)})
        shape = m2rnn.NormShape(1, M, D, m2rnn._dtype_code(x))
        need = m2rnn.lib().m2rnn_add_norm_bwd_workspace_size(ctypes.byref(shape))
        g = m2rnn.add_norm_bwd(x, dy, w, dr, out={"dx": gd((M, D), td), "dw": gd((D,))},
                               workspace=gd((need,), torch.uint8))
        qr, sr = m2rnn.quant_rows(x, out={"q": gd((M, D), torch.float8_e4m3fn), "scale": gd((M,))})
        return y, r, q, s, r8, g["dx"], g["dw"], qr, sr

    run_all(m2rnn, (buf, res, w, dy, dr), run)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D,F", [(1, 8, 8), (7, 136, 72), (16, 40, 264), (40, 264, 24), (65, 72, 200), (130, 520, 264),
                                   (300, 136, 1400), (1554, 520, 392)])
def test_glu(m2rnn, M, D, F, dtype):
    td = TD[dtype]
    buf, wg, wu, dh = rn(1, M, D + 16, dtype=td), rn(2, F, D, dtype=td, scale=0.1), rn(3, F, D, dtype=td, scale=0.1), rn(4, M, F, dtype=td)
    x = buf[:, 8:8 + D]

    def run(gd):
        s = ctypes.byref(m2rnn.GluShape(M, D, F, m2rnn._dtype_code(x), 0))
        L = m2rnn.lib()
        h = m2rnn.glu_fwd(x, wg, wu, out={"h": gd((M, F), td)},
                          workspace=gd((L.m2rnn_glu_fwd_workspace_size(s),), torch.uint8))
        g = m2rnn.glu_bwd(x, wg, wu, dh, workspace=gd((L.m2rnn_glu_bwd_workspace_size(s),), torch.uint8),
                          out={"dx": gd((M, D), td), "dwg": gd((F, D), td), "dwu": gd((F, D), td)})
        return h, g["dx"], g["dwg"], g["dwu"]

    run_all(m2rnn, (buf, wg, wu, dh), run)


def test_glu_pairs_of_ctas(m2rnn):
    M, D, F = 5003, 520, 2824
    x, wg, wu, dh = rn(1, M, D), rn(2, F, D, scale=0.1), rn(3, F, D, scale=0.1), rn(4, M, F)

    def run(gd):
        s = ctypes.byref(m2rnn.GluShape(M, D, F, 1, 0))
        h = m2rnn.glu_fwd(x, wg, wu, out={"h": gd((M, F), torch.bfloat16)})
        g = m2rnn.glu_bwd(x, wg, wu, dh, workspace=gd((m2rnn.lib().m2rnn_glu_bwd_workspace_size(s),), torch.uint8),
                          out={"dx": gd((M, D), torch.bfloat16), "dwg": gd((F, D), torch.bfloat16),
                               "dwu": gd((F, D), torch.bfloat16)})
        return h, g["dx"], g["dwg"], g["dwu"]

    run_all(m2rnn, (x, wg, wu, dh), run)


@pytest.mark.parametrize("M,D,F", [(1, 16, 8), (9, 144, 72), (16, 48, 264), (130, 528, 264), (4100, 272, 2824)])
def test_8_bits(m2rnn, M, D, F):
    (buf, xs), (wg, gs), (wu, us) = (m2rnn.quant_rows(t) for t in (rn(1, M, D + 32), rn(2, F, D), rn(3, F, D)))
    x, res = buf[:, 16:16 + D], rn(4, M, F + 8)

    def run(gd):
        h = m2rnn.glu_q8(x, xs, wg, gs, wu, us, out={"h": gd((M, F), torch.bfloat16)})
        y = m2rnn.linear_q8(x, xs, wg, gs, res[:, 8:], out={"y": gd((M, F), torch.bfloat16)})
        return h, y, m2rnn.linear_q8(x, xs, wu, us, out={"y": gd((M, F), torch.bfloat16)})

    run_all(m2rnn, (buf, xs, wg, gs, wu, us, res), run)


def test_workspace_refusals(m2rnn):
    """A workspace one byte short, or none, is refused before anything is launched."""
    x, w, dh = rn(1, 300, 136, dtype=torch.float32), rn(2, 72, 136, dtype=torch.float32), rn(3, 300, 72, dtype=torch.float32)
    s = ctypes.byref(m2rnn.GluShape(300, 136, 72, 0, 0))
    L = m2rnn.lib()
    for call, need in ((lambda ws: m2rnn.glu_fwd(x, w, w, workspace=ws), L.m2rnn_glu_fwd_workspace_size(s)),
                       (lambda ws: m2rnn.glu_bwd(x, w, w, dh, workspace=ws), L.m2rnn_glu_bwd_workspace_size(s)),
                       (lambda ws: m2rnn.add_norm_bwd(x, x, x[0].contiguous(), workspace=ws), 300 // 8 * 136 * 4)):
        with pytest.raises(m2rnn.M2RNNError) as e:
            call(torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
        assert e.value.code == -5
    assert m2rnn.device_status() == (0, 0)


def test_host_memory_and_alignment_are_refused(m2rnn):
    x, w = rn(1, 64, 136), rn(2, 72, 136)
    with pytest.raises(m2rnn.M2RNNError) as e:
        m2rnn.add_norm_fwd(x, x.cpu(), out={"y": torch.empty_like(x), "r": torch.empty_like(x)})
    assert e.value.code == -4
    with pytest.raises(m2rnn.M2RNNError) as e:
        m2rnn.glu_fwd(x, w, w.cpu())
    assert e.value.code == -4
    odd = torch.empty(64 * 136 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(64, 136)
    for call in (lambda: m2rnn.add_norm_fwd(odd), lambda: m2rnn.glu_fwd(odd, w, w), lambda: m2rnn.quant_rows(odd)):
        with pytest.raises(m2rnn.M2RNNError) as e:
            call()
        assert e.value.code == -3


@pytest.mark.parametrize("M", [3000, 100])  # pairs of CTAs, single ones
def test_a_wait_that_runs_out_is_reported(m2rnn, M):
    """No copies are started and waits end after 20 ms: the call leaves M2RNN_ERR_TIMEOUT in
    the status word and the context usable; the next one is right."""
    x, w = rn(1, M, 264), rn(2, 1032, 264, scale=0.1)
    want = m2rnn.glu_fwd(x, w, w)
    torch.cuda.synchronize()
    m2rnn.set_wait_limit_ns(20_000_000)
    m2rnn.set_fault_injection(1)
    try:
        m2rnn.glu_fwd(x, w, w)
        st, site = m2rnn.device_status(clear=True)
        assert st == -7 and 951 <= site <= 954
    finally:
        m2rnn.set_fault_injection(0)
        m2rnn.set_wait_limit_ns(0)
    assert torch.equal(m2rnn.glu_fwd(x, w, w), want) and m2rnn.device_status() == (0, 0)
