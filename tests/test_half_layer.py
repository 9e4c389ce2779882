"""The feed-forward half of examples/layer.py on the same mixer outputs as one prompt and as
single tokens: only the kernels behind the calls differ (few tokens, tiles; rows of a norm by
their number).

Bounds per token, 2-norms.  bf16: y may differ by a rounding step where its sums run in another
order (2^-7 of a value at most), which the products' sums carry on as the same share of g and
u, h = act(g) u as 2.2 times it, and a step of h of its own, 2^-7: together below 2^-5 of the
branch.  8 bits: the codes of y are equal (they do not depend on the order of the row's sum) and
its scale is within 2^-22.  h may differ by a step, 2^-7 of a value, and with it the scale of
its row, so that codes closer to a middle than that change: at most 2^-7 of 2^-3 or more between
two codes, one in 16 of them, by 2^-3 of their value: a 2-norm of 2^-5 and 2^-7 of the scale;
2^-4 of the branch is above their sum.  Both: the sum with the residual rounds on either side, 2^-7 of the
output in all."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def layer():
    import __graft_entry__
    __graft_entry__.build()
    from non_linear_matrix_gb300 import m2rnn
    m2rnn.use_library("normal")
    spec = importlib.util.spec_from_file_location("layer", os.path.join(ROOT, "examples", "layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("B,T", [(3, 200), (16, 5), (1, 33)])
@pytest.mark.parametrize("d,F", [(64, 176), (272, 528)])
def test_single_tokens_and_a_prompt(layer, d, F, B, T, q8):
    net = layer.Layer("scan", d=d, F=F, q8=q8, N=8, K=32, V=16, Nq=2)
    g = torch.Generator().manual_seed(5)
    size = 2.0 ** torch.randint(-3, 4, (B, T, 1), generator=g)  # tokens of sizes of their own
    o, x = ((torch.randn(B, T, d, generator=g) * size).bfloat16().cuda() for _ in range(2))
    whole = net.half(o, x)[0].double()
    branch = whole - (o + x).double()
    assert torch.isfinite(whole).all() and (branch.norm(dim=-1) > 0).all()
    for t in range(min(T, 20)):
        one = net.half(o[:, t], x[:, t])[0].double()
        off = (one - whole[:, t]).norm(dim=-1)
        bound = branch[:, t].norm(dim=-1) * 2.0 ** (-4 if q8 else -5) + whole[:, t].norm(dim=-1) * 2.0 ** -7
        assert (off <= bound).all(), (t, (off / bound).max().item())


@pytest.mark.parametrize("q8", [False, True])
def test_against_64_bits(layer, q8):
    """The branch itself: roundings of y, h and the output in bf16 (2^-8 each), in 8 bits of y, h and
    the weights to codes (2-norm of one such rounding: 2^-4 / 3^(1/2) at most, 2.2 times it
    for y, once for h, once for each weight in the products that it enters: 0.12 in all)."""
    net = layer.Layer("scan", d=272, F=528, q8=q8, N=8, K=32, V=16, Nq=2)
    g = torch.Generator().manual_seed(6)
    o, x = (torch.randn(40, 272, generator=g).bfloat16().cuda() for _ in range(2))
    w = {n: t.double() for n, t in net.w.items()}
    r = (o + x).double()
    y = r * (r.square().mean(-1, keepdim=True) + layer.EPS).rsqrt() * w["norm"]
    a = y @ w["wg"].T
    ref = (a * torch.sigmoid(a) * (y @ w["wu"].T)) @ w["wd"].T
    for rows in (slice(0, 40), slice(0, 3)):
        out = net.half(o[rows], x[rows])[0].double()
        off = (out - r[rows] - ref[rows]).norm(dim=-1)
        assert (off <= ref[rows].norm(dim=-1) * (0.12 if q8 else 2.0 ** -5) + (r + ref)[rows].norm(dim=-1) * 2.0 ** -7).all()
