"""The residual's addition with the RMS norm (add_norm_fwd, add_norm_q8,
add_norm_bwd) and the row quantiser (quant_rows) against plain implementations
in 64 bits on the same inputs.

Tolerances, derived.  u = 2^-24 is fp32's half step, b the output type's (bf16
2^-8, fp32 2^-24), relative to the value.
  r: the sum rounded once: equal to torch's.
  y = w r rstd: the sum of D squares in fp32 is off by at most 64 u of itself (at
    most 32 terms in a row per thread, then a tree), the mean, root and
    reciprocal by 4 u; with the two products: |y| (b + 40 u).
  dx = dr + rstd (p - n c), c = mean(p n) over D terms of fp32 products (error 70 u of
    the mean of |p n|): rstd (|p| + |n| mean|p n|) 120 u + b |dx|.
  dw: a group sums M / (2 * 304) rows in order, groups and parts after it: at most
    sqrt-free bound (rows + 320 + 40) u of the sum of |dy n|.
  codes: nearest of an argument that is off by 48 u: half a step, 2^-4 of the value or 2^-10
    of the scale (steps below the smallest normal code), and that much more.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

TD = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    from non_linear_matrix_gb300 import m2rnn
    m2rnn.use_library("normal")
    return m2rnn


def rn(seed, *s, dtype="bf16", scale=1.0):
    return (torch.randn(*s, generator=torch.Generator().manual_seed(seed)) * scale).to(TD[dtype]).cuda()


def within(got, ref, tol, label):
    """|got - ref| <= tol elementwise (tol a tensor)."""
    assert got.shape == ref.shape
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (label, int(bad.sum()), ((got.double() - ref).abs() / tol.clamp_min(1e-300)).max().item())


def norm64(r, w, eps):
    r = r.double()
    inv = (r.square().mean(-1, keepdim=True) + eps).rsqrt()
    n = r * inv
    return n, inv, n if w is None else n * w.double()


SIZES = [(1, 8), (3, 72), (1, 1024), (65, 512), (7, 520), (64, 1024), (301, 1048), (130, 2000), (9, 4096), (700, 264),
         (5, 8192), (33, 8200), (2, 16384), (1300, 1024)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D", SIZES)
def test_forward(m, M, D, dtype):
    x, res, w = rn(1, M, D, dtype=dtype), rn(2, M, D, dtype=dtype, scale=2), rn(3, D, dtype=dtype)
    y, r = m.add_norm_fwd(x, res, w, EPS)
    assert torch.equal(r, x + res)
    ref = norm64(r, w, EPS)[2]
    within(y, ref, ref.abs() * (HALF[dtype] + 40 * U), "y")
    y2, none = m.add_norm_fwd(r, None, w, EPS)  # the norm alone
    assert none is None and torch.equal(y2, y)
    ref = norm64(x, None, 0.0)[2]
    within(m.add_norm_fwd(x, eps=0.0)[0], ref, ref.abs() * (HALF[dtype] + 40 * U), "unweighted")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D", SIZES)
def test_8_bits(m, M, D, dtype):
    x, res, w = rn(4, M, D, dtype=dtype), rn(5, M, D, dtype=dtype), rn(6, D, dtype=dtype)
    q, scale, r = m.add_norm_q8(x, res, w, EPS)
    assert q.dtype is torch.float8_e4m3fn and scale.shape == (M,) and torch.equal(r, x + res)
    ref = norm64(r, w, EPS)[2]
    top = ref.abs().amax(-1)
    within(scale, top / 448, top / 448 * 48 * U, "scale")
    s = scale.double()[:, None]
    within(q.double() * s, ref, ref.abs() * (2.0 ** -4 + 64 * U) + s * 2.0 ** -10 * (1 + 64 * U), "codes")
    q2, s2, none = m.add_norm_q8(r, None, w, EPS)
    assert none is None and torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("with_dr", [True, False])
@pytest.mark.parametrize("M,D", SIZES)
def test_gradient(m, M, D, with_dr, dtype):
    r, w, dy = rn(7, M, D, dtype=dtype, scale=2), rn(8, D, dtype=dtype), rn(9, M, D, dtype=dtype)
    dr = rn(10, M, D, dtype=dtype) if with_dr else None
    g = m.add_norm_bwd(r, dy, w, dr, EPS)
    leaf, wl = r.double().requires_grad_(), w.double().requires_grad_()
    y = leaf / (leaf.square().mean(-1, keepdim=True) + EPS).sqrt() * wl
    dx, dw = torch.autograd.grad(y, (leaf, wl), dy.double())
    n, inv, _ = norm64(r, w, EPS)
    p = dy.double() * w.double()
    size = inv * (p.abs() + n.abs() * (p * n).abs().mean(-1, keepdim=True))
    if with_dr:
        dx = dx + dr.double()
    within(g["dx"], dx, dx.abs() * (HALF[dtype] + U) + size * 120 * U, "dx")
    within(g["dw"], dw, (dy.double() * n).abs().sum(0) * (M / 608 + 400) * U + 1e-30, "dw")
    assert torch.equal(m.add_norm_bwd(r, dy, w, dr, EPS, want_dw=False)["dx"], g["dx"])
    assert m.add_norm_bwd(r, dy, None, dr, EPS)["dw"] is None


@pytest.mark.parametrize("M,D", [(400_000, 64), (60_000, 1032), (20_000, 8200)])
def test_long_sums_of_the_weights_gradient(m, M, D):
    """dw over many rows of one sign, whose sum drifts if it is formed in one run: a run of
    64 rows, then M / (64 groups) runs, then at most 2,432 groups and parts, 8 in a row or in a
    tree: (64 + M / (64 * 152) + 400) u of the sum, and as each rounding is as often up as
    down, a hundredth of what a single run of M rows could lose."""
    r, dy = rn(1, M, D).abs(), rn(2, M, D).abs()
    w = torch.ones(D, device="cuda").bfloat16()
    dw = m.add_norm_bwd(r, dy, w, None, EPS)["dw"]
    ref = torch.zeros(D, dtype=torch.float64, device="cuda")
    for i in range(0, M, 20_000):
        ref += (norm64(r[i:i + 20_000], None, EPS)[0] * dy[i:i + 20_000].double()).sum(0)
    assert (dw.double() - ref).norm() <= 1e-6 * ref.norm()
    within(dw, ref, ref.abs() * (464 + M / 9728) * U, "dw")


def test_gradient_against_differences(m):
    """Central differences of sum(y dy) in fp32 along a direction: the step 2^-6 has a
    curvature term of 2^-12 / 6 of third derivatives of size about one per row, and
    rounding 2^-24 of the sum of |y dy| over 2^-6."""
    M, D = 40, 136
    r, w, dy, d = (rn(s, *sh, dtype="f32") for s, sh in ((1, (M, D)), (2, (D,)), (3, (M, D)), (4, (M, D))))
    h = 2.0 ** -6
    d = d / d.norm() * 4
    up, down = (m.add_norm_fwd(r + k * d, None, w, EPS)[0].double() for k in (h, -h))
    slope = ((up - down) * dy.double()).sum() / (2 * h)
    g = m.add_norm_bwd(r, dy, w, None, EPS)
    want = (g["dx"].double() * d.double()).sum()
    size = (up * dy.double()).abs().sum().item()
    assert abs(slope - want) <= 4 * 2.0 ** -24 * size / h + 2.0 ** -12 * 64


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_wider_buffers_and_in_place(m, dtype):
    B, T, D = 3, 17, 136
    buf, res, w = rn(1, B, T, D + 24, dtype=dtype), rn(2, B, T, 2 * D, dtype=dtype), rn(3, D, dtype=dtype)
    x, rs = buf[..., 8:8 + D], res[..., D:]
    y, r = m.add_norm_fwd(x, rs, w)
    yc, rc = m.add_norm_fwd(x.contiguous(), rs.contiguous(), w)
    assert torch.equal(y, yc) and torch.equal(r, rc) and y.shape == (B, T, D)
    q, s, r8 = m.add_norm_q8(x, rs, w)
    qc, sc, _ = m.add_norm_q8(x.contiguous(), rs.contiguous(), w)
    assert torch.equal(q.view(torch.uint8), qc.view(torch.uint8)) and torch.equal(s, sc) and s.shape == (B, T)
    stream = rs.contiguous()
    y2, r2 = m.add_norm_fwd(x, stream, w, out={"r": stream})  # the stream in place
    assert r2 is stream and torch.equal(stream, rc) and torch.equal(y2, yc)
    xin = x.contiguous()
    assert torch.equal(m.add_norm_fwd(xin, rs, w, out={"r": xin})[0], yc) and torch.equal(xin, rc)
    for part in (x[:, :5], x[1:, 3:9], x[:, :1], x[:1]):  # items and tokens at their own distances
        got, r3 = m.add_norm_fwd(part, part, w)
        c = part.contiguous()
        assert torch.equal(got, m.add_norm_fwd(c, c, w)[0]) and torch.equal(r3, c + c)
        assert torch.equal(m.quant_rows(part)[0].view(torch.uint8), m.quant_rows(c)[0].view(torch.uint8))
        gd = rn(7, *part.shape, dtype=dtype)
        a, b = m.add_norm_bwd(part, gd, w), m.add_norm_bwd(c, gd, w)
        assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dw"], b["dw"])
    one = rn(4, D, dtype=dtype).expand(T, D)  # the same row for every token
    assert torch.equal(m.add_norm_fwd(one, None, w)[0], m.add_norm_fwd(one.contiguous(), None, w)[0])
    dy, dr = rn(5, B, T, D, dtype=dtype), rn(6, B, T, D, dtype=dtype)
    g = m.add_norm_bwd(x, dy, w, dr)
    gc = m.add_norm_bwd(x.contiguous(), dy, w, dr)
    assert torch.equal(g["dx"], gc["dx"]) and torch.equal(g["dw"], gc["dw"])
    for over in (dy, dr):
        d2 = {"dy": dy.clone(), "dr": dr.clone()}
        t = d2["dy" if over is dy else "dr"]
        got = m.add_norm_bwd(x, d2["dy"], w, d2["dr"], out={"dx": t})
        assert got["dx"] is t and torch.equal(t, gc["dx"]) and torch.equal(got["dw"], gc["dw"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_rows(m, dtype):
    x, w = rn(1, 0, 64, dtype=dtype), rn(2, 64, dtype=dtype)
    y, r = m.add_norm_fwd(x, x, w)
    assert y.shape == r.shape == (0, 64)
    assert m.add_norm_q8(x, x, w)[1].shape == (0,)
    dw = torch.full((64,), 7.0, device="cuda")
    assert torch.equal(m.add_norm_bwd(x, x, w, out={"dw": dw})["dw"], torch.zeros_like(dw))
    assert m.quant_rows(x)[0].shape == (0, 64)


def test_values_that_are_not_finite_stay_in_their_rows(m):
    x, w = rn(1, 6, 520), rn(2, 520)
    ref = m.add_norm_fwd(x, None, w)[0]
    codes = m.quant_rows(x)[0].float()
    bad = x.clone()
    bad[1, 3], bad[2, 5], bad[3] = float("inf"), float("nan"), 0.0
    y = m.add_norm_fwd(bad, None, w)[0]
    assert torch.isnan(y[1, 3]) and (y[1, :3] == 0).all() and torch.isnan(y[2]).all() and (y[3] == 0).all()
    rest = [0, 4, 5]
    assert torch.equal(y[rest], ref[rest])
    assert torch.isnan(m.add_norm_fwd(bad, None, w, 0.0)[0][3]).all()  # a zero row without eps
    q, s = m.quant_rows(bad)
    assert torch.isinf(s[1]) and torch.isnan(q[1, 3].float()) and torch.isnan(s[2]) and s[3] == 0
    assert torch.isnan(q[2].float()).all() and (q[3].float() == 0).all()
    assert torch.equal(q[rest].float(), codes[rest])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 1e-37, 3e37])
@pytest.mark.parametrize("M,D", [(1, 8), (64, 5632), (37, 72), (3, 8200), (2, 40000), (500, 1024), (5, 65536)])
def test_quant_rows(m, M, D, scale, dtype):
    """Bit for bit the codes of torch's fp32 quotients, ties (which quotients of
    bf16 values meet) to even."""
    x = (rn(1, M, D, dtype=dtype).float() * rn(2, M, D, dtype=dtype).float() * scale).clamp(-3e38, 3e38).to(TD[dtype])
    q, s = m.quant_rows(x)
    top = x.float().abs().amax(-1)
    ref = top / torch.full_like(top, 448.0)
    assert torch.equal(s, ref)
    codes = torch.where(ref[:, None] > 0, x.float() / ref[:, None], torch.zeros_like(x, dtype=torch.float32))
    assert torch.equal(q.view(torch.uint8) & 0x7F, codes.to(torch.float8_e4m3fn).view(torch.uint8) & 0x7F)
    assert torch.equal(q.float(), codes.to(torch.float8_e4m3fn).float())
    wide = torch.zeros(M, D + 16, dtype=x.dtype, device="cuda")
    wide[:, 8:8 + D] = x
    qw, sw = m.quant_rows(wide[:, 8:8 + D])
    assert torch.equal(qw.view(torch.uint8), q.view(torch.uint8)) and torch.equal(sw, s)


def test_far_rows(m):
    """Rows 2^31 elements apart in all: offsets in 64 bits."""
    if torch.cuda.get_device_properties(0).total_memory < 32 << 30:
        pytest.skip("needs 9 GB of device memory")
    M, D, row = 34, 256, (1 << 26) + 64
    buf = torch.empty(M * row, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((M, D), (row, 1))
    xc, w, dy = rn(1, M, D), rn(2, D), rn(3, M, D)
    x.copy_(xc)
    assert (M - 1) * row > 1 << 31
    assert torch.equal(m.add_norm_fwd(x, x, w)[0], m.add_norm_fwd(xc, xc, w)[0])
    a, b = m.add_norm_bwd(x, dy, w), m.add_norm_bwd(xc, dy, w)
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dw"], b["dw"])
    assert torch.equal(m.quant_rows(x)[0].view(torch.uint8), m.quant_rows(xc)[0].view(torch.uint8))
