"""The selective scan's outputs with values that are not finite: y_t depends on
no later token, whatever that holds, and on its own head's and column's values
only."""
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
make, args = forms.make, forms.args


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    from non_linear_matrix_gb300 import m2rnn
    m2rnn.use_library("normal")
    return m2rnn


BAD = [math.inf, -math.inf, math.nan]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t", [0, 21, 31, 70])
@pytest.mark.parametrize("bad", BAD)
def test_outputs_do_not_see_later_tokens(m, dtype, t, bad):
    """A token that is not finite in k, v, a or q changes no bit of the tokens before
    it; v and a of one head none of the other heads, q none of any other token."""
    d = make(2, 100, 5, 64, 16, 1, dtype, 12)
    clean, _, _ = m.scan_fwd(*args(d), d["w_r"], d["H0"])
    assert clean.isfinite().all()
    for name, at in (("k", (1, t, 0, 9)), ("v", (1, t, 2, 5)), ("a", (1, t, 2)), ("q", (1, t, 0, 3))):
        e = dict(d)
        e[name] = d[name].clone()
        e[name][at] = bad
        y = m.scan_fwd(*args(e), d["w_r"], d["H0"])[0]
        same = torch.ones_like(clean, dtype=torch.bool)
        if name == "q":
            same[1, t] = False
        elif name == "k":
            same[1, t:] = False
        else:
            same[1, t:, 2] = False
        assert torch.equal(y[same], clean[same]), name
        if name == "v":  # and the token itself, with the later ones of its column
            assert not y[1, t, 2, 5].isfinite()
            if not math.isnan(bad):
                assert torch.equal(y[1, t, 2, :5], clean[1, t, 2, :5])
        elif name == "k":
            assert not y[1, t].isfinite().any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,Nq", [(16, 4), (32, 2)])
def test_many_tokens_not_finite(m, dtype, V, Nq):
    """Several bad values in one block of 16, in neighbouring columns and heads: each
    column is finite up to its first bad token and has the clean bits there."""
    d = make(1, 80, 4, 32, V, Nq, dtype, 13)
    clean = m.scan_fwd(*args(d), d["w_r"], d["H0"])[0]
    e = dict(d, v=d["v"].clone())
    first = torch.full((4, V), 80)
    for i, (t, n, c) in enumerate([(17, 0, 0), (19, 0, 1), (18, 0, 9), (23, 1, V - 1), (31, 3, 7), (16, 2, 8),
                                   (30, 2, 15), (47, 1, 3), (17, 3, 7)]):
        e["v"][0, t, n, c] = BAD[i % 3]
        first[n, c] = min(first[n, c].item(), t)
    y = m.scan_fwd(*args(e), d["w_r"], d["H0"])[0][0]
    before = torch.arange(80)[:, None, None] < first[None]
    assert torch.equal(y[before.cuda()], clean[0][before.cuda()])
    hit = (first < 80).nonzero()
    for n, c in hit.tolist():
        assert not y[first[n, c], n, c].isfinite()
