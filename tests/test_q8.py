"""The 8-bit products (glu_q8, linear_q8) against 64 bits on the same codes and
scales.  Codes' products are exact in fp32; a step of the tensor core (32 k) may cut off one
place of its sum, so a product is off by (D / 32 + 20) 2^-23 of the sum of absolute
products, the scales by three roundings; bf16's half step is 2^-8."""
import pytest
import torch
import torch.nn.functional as nnf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    from non_linear_matrix_gb300 import m2rnn
    m2rnn.use_library("normal")
    return m2rnn


def rn(seed, *s, scale=1.0):
    return (torch.randn(*s, generator=torch.Generator().manual_seed(seed)) * scale).cuda()


def values(q, s):
    return q.double() * s.double()[..., None]


def product(x, w):
    """x w^T and the bound of its error."""
    e = (x.shape[-1] / 32 + 20) * 2.0 ** -23
    return x @ w.T, e * (x.abs() @ w.abs().T)


def within(got, ref, tol, label):
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (label, int(bad.sum()), ((got.double() - ref).abs() / tol.clamp_min(1e-300)).max().item())


SIZES = [(1, 16, 8), (1, 5632, 520), (8, 1024, 264), (9, 144, 72), (16, 528, 136), (17, 112, 56), (33, 272, 264), (64, 2048, 312),
         (65, 128, 64), (128, 128, 256), (129, 144, 8), (200, 16, 264), (257, 1040, 1032), (3000, 528, 1416),
         (5000, 1024, 2816)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,D,F", SIZES)
def test_gated(m, M, D, F, act):
    (x, xs), (wg, gs), (wu, us) = (m.quant_rows(t) for t in (rn(1, M, D), rn(2, F, D, scale=D ** -0.5),
                                                             rn(3, F, D, scale=D ** -0.5)))
    h = m.glu_q8(x, xs, wg, gs, wu, us, act=act)
    assert h.dtype is torch.bfloat16
    X = values(x, xs)
    (g, eg), (u, eu) = product(X, values(wg, gs)), product(X, values(wu, us))
    a = nnf.silu(g) if act == "silu" else nnf.gelu(g, approximate="tanh")
    ref = a * u
    ea = 2.0 ** -20 * (a.abs() + g.abs() * 0.25)
    within(h, ref, (1.13 * eg + ea) * u.abs() + a.abs() * eu + ref.abs() * 2.0 ** -8 * 1.01 + 1e-30, "h")
    assert m.device_status() == (0, 0)


@pytest.mark.parametrize("with_res", [True, False])
@pytest.mark.parametrize("M,D,F", SIZES)
def test_linear(m, M, D, F, with_res):
    (x, xs), (w, ws) = m.quant_rows(rn(1, M, D)), m.quant_rows(rn(2, F, D, scale=D ** -0.5))
    res = rn(3, M, F).bfloat16() if with_res else None
    y = m.linear_q8(x, xs, w, ws, res)
    ref, e = product(values(x, xs), values(w, ws))
    tol = e + 2.0 ** -22 * ref.abs()
    if with_res:
        ref = ref + res.double()
        tol = tol + 2.0 ** -24 * ref.abs()
    within(y, ref, tol + ref.abs() * 2.0 ** -8 * 1.01 + 1e-30, "y")
    if with_res:  # rows of a wider buffer, and in place
        wide = torch.zeros(M, F + 24, dtype=torch.bfloat16, device="cuda")
        wide[:, 8:8 + F] = res
        assert torch.equal(m.linear_q8(x, xs, w, ws, wide[:, 8:8 + F]), y)
        here = res.clone()
        assert m.linear_q8(x, xs, w, ws, here, out={"y": here}) is here and torch.equal(here, y)


@pytest.mark.parametrize("M", [7, 300])
def test_rows_scales_and_codes(m, M):
    """Rows of a wider buffer; all 256 codes (two of them NaN) as the values they stand for;
    rows of scale 0."""
    D, F = 272, 72
    codes = (torch.arange(M * (D + 48), device="cuda") * 37 % 256).to(torch.uint8)
    codes = torch.where((codes & 0x7F) == 0x7F, torch.zeros_like(codes), codes)
    wide = codes.view(M, D + 48).view(torch.float8_e4m3fn)
    x, xs = wide[:, 16:16 + D], rn(1, M).abs()
    w, ws = m.quant_rows(rn(2, F, D))
    y = m.linear_q8(x, xs, w, ws)
    assert torch.equal(y, m.linear_q8(x.contiguous(), xs, w, ws))
    ref, e = product(values(x, xs), values(w, ws))
    within(y, ref, e + ref.abs() * (2.0 ** -8 * 1.01 + 2.0 ** -22) + 1e-30, "y")
    nan = x.contiguous().view(torch.uint8).clone()
    nan[2, 5] = 0x7F
    y2 = m.linear_q8(nan.view(torch.float8_e4m3fn), xs, w, ws)
    keep = [i for i in range(M) if i != 2]
    assert torch.isnan(y2[2]).all() and torch.equal(y2[keep], y[keep])
    xs0 = xs.clone()
    xs0[1] = 0
    assert not m.linear_q8(x, xs0, w, ws)[1].any()


def test_no_tokens(m):
    x, xs = m.quant_rows(rn(1, 0, 64))
    w, ws = m.quant_rows(rn(2, 72, 64))
    assert m.glu_q8(x, xs, w, ws, w, ws).shape == (0, 72) and m.linear_q8(x, xs, w, ws).shape == (0, 72)


@pytest.mark.parametrize("M", [3, 200])
def test_the_half_layer_in_8_bits(m, M):
    """Norm, gated products, quantiser and the way back, one after the other, against 64 bits
    on the codes that each stage handed on."""
    D, F = 272, 528
    x, stream = rn(1, M, D).bfloat16(), rn(2, M, D).bfloat16()
    (wg, gs), (wu, us), (wd, ds) = (m.quant_rows(rn(s, *sh, scale=sh[1] ** -0.5)) for s, sh in
                                    ((3, (F, D)), (4, (F, D)), (5, (D, F))))
    q, qs, r = m.add_norm_q8(x, stream)
    h = m.glu_q8(q, qs, wg, gs, wu, us)
    hq, hs = m.quant_rows(h)
    y = m.linear_q8(hq, hs, wd, ds, r)
    assert torch.equal(r, x + stream)
    X = values(q, qs)
    h64 = nnf.silu(X @ values(wg, gs).T) * (X @ values(wu, us).T)
    assert (h.double() - h64).norm() <= 2.0 ** -8 * h64.norm()
    ref, e = product(values(hq, hs), values(wd, ds))
    ref = ref + r.double()
    within(y, ref, e + ref.abs() * (2.0 ** -8 * 1.01 + 2.0 ** -22) + 1e-6, "y")
