"""Where the selective scan's bf16 outputs leave fp32: at their last rounding
only.  States between kernels are fp32, and the operands that are made on the
way (weights, states) keep more bits than an output does."""
import ctypes
import importlib.util
import os

import pytest
import torch

spec = importlib.util.spec_from_file_location(
    "scan_forms", os.path.join(os.path.dirname(os.path.abspath(__file__)), "test_scan.py"))
forms = importlib.util.module_from_spec(spec)
spec.loader.exec_module(forms)
make, plain, args, rel = forms.make, forms.plain, forms.args, forms.rel


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    from non_linear_matrix_gb300 import m2rnn
    m2rnn.use_library("normal")
    return m2rnn


def rounding(ref):
    """Error of a single rounding to bf16."""
    return rel(ref.float().bfloat16(), ref)


@pytest.mark.parametrize("B", [1, 2, 3, 8])
def test_workspace_holds_fp32_states(B):
    """From the sizes, without a GPU: a call has room for 64 x 64 fp32 states before
    each chunk of at least half of its sequences."""
    from non_linear_matrix_gb300 import build as nb, m2rnn
    nb.build()
    for dtype in (0, 1):
        s = ctypes.byref(m2rnn.Shape(B, 300, 4, 64, 16, dtype, 0, 1))
        least, full = m2rnn.lib().m2rnn_scan_fwd_workspace_size(s, 0), m2rnn.lib().m2rnn_scan_saved_size(s)
        state = 5 * 64 * 64 * 4
        assert full >= B * state and full - least in ((0,) if dtype == 0 else (B // 2 * state,))


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,K,V,Nq", [(1, 1, 16, 16, 1), (2, 6, 64, 16, 2), (3, 2, 128, 32, 1)])
def test_states_are_not_rounded_on_the_way(m, B, N, K, V, Nq):
    """Without decay, and with q a unit vector, y is a row of the state, rounded once,
    wherever the chunk itself adds nothing: every second chunk of 64 has v = 0.  16
    chunks: the state crosses segments.  Tolerance: half an ulp of bf16 and the
    state's own 1e-6."""
    d = make(B, 1024, N, K, V, Nq, "bf16", 5 + K)
    d["alpha"] = torch.zeros_like(d["alpha"])
    d["w_r"] = None
    d["v"].view(B, 8, 2, 64, N, V)[:, :, 1] = 0
    d["q"].zero_()[..., 3] = 1
    ref = plain(d)["y"].view(B, 8, 2, 64, N, V)[:, :, 1]
    scale = ref.abs().max()
    for save in (False, True):
        y = m.scan_fwd(*args(d), None, d["H0"], save=save)[0].view(B, 8, 2, 64, N, V)[:, :, 1].double()
        ulp = torch.exp2(torch.floor(torch.log2(ref.abs().clamp_min(1e-30))) - 7)
        assert ((y - ref).abs() <= 0.5 * ulp + 1e-6 * scale).all(), (save, ((y - ref).abs() / ulp).max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,N,K,V,Nq", [(2, 300, 4, 64, 16, 1), (5, 130, 6, 32, 32, 3), (1, 700, 3, 128, 16, 3)])
def test_least_workspace(m, B, T, N, K, V, Nq, dtype):
    """In two parts: the bits of one part, nothing behind the workspace's end."""
    d = make(B, T, N, K, V, Nq, dtype, T, sliced=True)
    want = m.scan_fwd(*args(d), d["w_r"], d["H0"])
    s = m.Shape(B, T, N, K, V, int(dtype == "bf16"), 0, Nq)
    need = m.lib().m2rnn_scan_fwd_workspace_size(ctypes.byref(s), 0)
    for given in (need, m.lib().m2rnn_scan_saved_size(ctypes.byref(s))):
        buf = torch.full((given + 4096,), 165, dtype=torch.uint8, device="cuda")
        for HT in (True, False):
            y, H, _ = m.scan_fwd(*args(d), d["w_r"], d["H0"], want_HT=HT, workspace=buf[:given])
            assert torch.equal(y, want[0]) and (H is None or torch.equal(H, want[1]))
        assert (buf[given:] == 165).all()
    with pytest.raises(m.M2RNNError):
        m.scan_fwd(*args(d), d["w_r"], d["H0"], workspace=buf[:need - 16])


# B, T, N, K, V, Nq
SHAPES = [(2, 512, 8, 64, 16, 1), (1, 333, 6, 128, 32, 2), (3, 130, 5, 32, 16, 5), (1, 1500, 4, 16, 32, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,N,K,V,Nq", SHAPES)
def test_outputs_are_rounded_once(m, B, T, N, K, V, Nq):
    """Without the skip term, which would hide the scan's own part.  Tolerance: the
    exact values' rounding to bf16, and 2^-14: operands of two bf16 terms (2^-17
    each), their sums' cancellation (a factor of 8)."""
    for sliced, state in [(False, True), (True, False)]:
        d = make(B, T, N, K, V, Nq, "bf16", T + K + 2, sliced, state)
        d["w_r"] = None
        ref = plain(d)["y"]
        for save in (False, True):
            y = m.scan_fwd(*args(d), None, d["H0"], save=save)[0]
            assert rel(y, ref) <= rounding(ref) + 2.0 ** -14, (sliced, save, rel(y, ref), rounding(ref))


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,N,K,V,Nq", SHAPES)
def test_gradients_are_rounded_once(m, B, T, N, K, V, Nq):
    """As the outputs: dq, dk, dv, da."""
    for sliced, state in [(False, True), (True, False)]:
        d = make(B, T, N, K, V, Nq, "bf16", T + K + 3, sliced, state)
        d["w_r"] = None
        ref = plain(d, backward=True)
        g = m.scan_bwd(*args(d), d["dy"], None, d["H0"], d["dHT"])
        bad = {n: (rel(g[n], ref[n]), rounding(ref[n])) for n in ("dq", "dk", "dv", "da")
               if not rel(g[n], ref[n]) <= rounding(ref[n]) + 2.0 ** -14}
        assert not bad, (sliced, bad)
