"""The selective scan where the gate's strength changes within a few tokens
(resets between slow tokens), and the gate's own gradients at extreme gates.

Tolerances, derived (fp32 inputs).  A decay 2^S(j,i) is off by S times a few 2^-24
whatever lies in front of j, a relative error of at most 0.53 ln 2 2^-22 = 9e-8 of the
largest weights (S 2^-S <= 0.53); 2^x and dt 2^-22 each; three-term operands and
sums of 64 products 2^-22 each: below 1e-6 together.  Outputs 2e-6; gradients, which
pass through two such products, 4e-6; the gate's gradients, where parts cancel, 1e-5 of
the parts' size.
bf16 inputs: half an ulp, 4e-3 for outputs; 1e-5 for parameters' gradients."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

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


def with_resets(d, pattern, seed=1):
    """a + 30 at some tokens: "block" the first 10 of every 16, "one" every 16th,
    "random" a quarter of them.  Returns which tokens stay slow."""
    B, T, N = d["a"].shape
    if pattern == "random":
        on = torch.rand(B, T, N, generator=torch.Generator().manual_seed(seed)) < 0.25
    else:
        on = (torch.arange(T) % 16 < (10 if pattern == "block" else 1))[None, :, None].expand(B, T, N)
    on = on.to(d["a"].device)
    d["a"] = torch.where(on, d["a"].float() + 30, d["a"].float()).to(d["a"].dtype)
    return ~on


SHAPES = [(1, 200, 4, 64, 16, 1), (2, 333, 3, 128, 32, 3), (1, 150, 6, 16, 16, 2)]
PATTERNS = ["block", "one", "random"]


@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("B,T,N,K,V,Nq", SHAPES)
def test_slow_tokens_after_resets(m, B, T, N, K, V, Nq, pattern):
    d = make(B, T, N, K, V, Nq, "f32", T, state=False)
    d["w_r"] = None
    slow = with_resets(d, pattern)
    y, HT, _ = m.scan_fwd(*args(d))
    ref = plain(d)
    assert rel(y[slow], ref["y"][slow]) <= 2e-6, rel(y[slow], ref["y"][slow])
    assert rel(y, ref["y"]) <= 2e-6 and rel(HT, ref["HT"]) <= 2e-6


@pytest.mark.parametrize("pattern", PATTERNS)
@pytest.mark.parametrize("B,T,N,K,V,Nq", SHAPES)
def test_gradients_with_resets(m, B, T, N, K, V, Nq, pattern):
    d = make(B, T, N, K, V, Nq, "f32", T + 1)
    slow = with_resets(d, pattern, 2)
    g = m.scan_bwd(*args(d), d["dy"], d["w_r"], d["H0"], d["dHT"], want_dH0=True)
    ref = plain(d, backward=True)
    bad = {n: rel(g[n], ref[n]) for n in ("dq", "dk", "dv", "dw_r", "dH0")
           if not rel(g[n], ref[n]) <= 4e-6}
    bad.update({n: rel(g[n], ref[n]) for n in ("da", "dalpha", "dbeta") if not rel(g[n], ref[n]) <= 1e-5})
    for n, tol in (("dv", 4e-6), ("da", 1e-5)):
        if not rel(g[n][slow], ref[n][slow]) <= tol:
            bad[n + " slow"] = rel(g[n][slow], ref[n][slow])
    assert not bad, bad


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pattern", PATTERNS + [-80.0, 30.0, 200.0])
def test_gate_gradients_at_extremes(m, dtype, pattern):
    """da, dalpha, dbeta.  Where decays vanish dalpha does too: its tolerance is
    1e-5 of its parts' size, dt |f dL/df| + |da|."""
    d = make(1, 150, 4, 64, 16, 1, dtype, 33)
    if isinstance(pattern, str):
        with_resets(d, pattern, 3)
    else:
        d["a"] = (d["a"].float() + pattern).to(d["a"].dtype)
        d["a"][:, 50:60] = -math.inf
    g = m.scan_bwd(*args(d), d["dy"], d["w_r"], d["H0"], d["dHT"])
    ref = plain(d, backward=True)
    parts = ref["da"].abs().sum((0, 1))
    assert rel(g["da"], ref["da"]) <= (4e-3 if dtype == "bf16" else 1e-5), rel(g["da"], ref["da"])
    for n in ("dalpha", "dbeta"):
        err = (g[n].double() - ref[n]).abs()
        assert (err <= 1e-5 * (ref[n].abs() + parts)).all(), (n, err / (ref[n].abs() + parts))
