"""The gated feed-forward products (glu_fwd, glu_bwd) against a plain
implementation in 64 bits on the same inputs.

Tolerances, derived, elementwise.  Let S(a, b) be the product of the absolute
values of a and b.  A step of the tensor core (16 k) may cut off one place of
its sum, 2^-23 of at most S, and what is added in fp32 after it rounds by 2^-24:
  bf16: D / 16 steps: e(g) = (D / 16 + 20) 2^-23 S(x, wg), for few tokens too (there
    the steps are split over eight warps);
  fp32: the dropped products of terms are 2^-26 of S, a chain has 16 leading steps
    and five times as many small ones of 2^-8 S each, chunks of 256 k (and parts) are added with
    rounding: e(g) = (24 + D / 256) 2^-23 S(x, wg).
act' is at most 1.13 and act'' at most 1.2 for both activations; the activation itself is
off by 2^-20 (bf16, special-function unit; |g| 2^-22 of the sigmoid's argument) or 2^-21
(fp32, expf and a division).  h is rounded once (half a step H: 2^-8, 2^-24).
dg = dh u act'(g), du = dh act(g): with bf16 inputs rounded to bf16 (2^-8), up to M D F = 2^30 to
two terms (2^-16), exact terms with fp32; their errors enter dx, dwg and dwu through S.
"""
import pytest
import torch
import torch.nn.functional as nnf

pytestmark = pytest.mark.gpu

TD = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    from non_linear_matrix_gb300 import m2rnn
    m2rnn.use_library("normal")
    return m2rnn


def rn(seed, *s, dtype="bf16", scale=1.0):
    return (torch.randn(*s, generator=torch.Generator().manual_seed(seed)) * scale).to(TD[dtype]).cuda()


def act64(g, act):
    return nnf.silu(g) if act == "silu" else nnf.gelu(g, approximate="tanh")


def chain(K, dtype):
    """Error of a sum over K, as a share of the sum of absolute products."""
    return (K / 16 + 20) * 2.0 ** -23 if dtype == "bf16" else (24 + K / 256) * 2.0 ** -23


def within(got, ref, tol, label):
    assert got.shape == ref.shape
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (label, int(bad.sum()), ((got.double() - ref).abs() / tol.clamp_min(1e-300)).max().item())


class Case:
    """Inputs and the 64-bit results with their bounds."""

    def __init__(self, M, D, F, dtype, act, seed=0):
        self.x = rn(seed + 1, M, D, dtype=dtype)
        self.wg, self.wu = (rn(seed + s, F, D, dtype=dtype, scale=D ** -0.5) for s in (2, 3))
        self.dh = rn(seed + 4, M, F, dtype=dtype)
        self.act, self.dtype = act, dtype
        self.X, self.G, self.U = (t.double() for t in (self.x, self.wg, self.wu))
        g, u = self.X @ self.G.T, self.X @ self.U.T
        sx = self.X.abs()
        e = chain(D, dtype)
        self.eg, self.eu = e * (sx @ self.G.abs().T), e * (sx @ self.U.abs().T)
        leaf = g.clone().requires_grad_()
        a = act64(leaf, act)
        da, = torch.autograd.grad(a.sum(), leaf)
        a = a.detach()
        self.g, self.u, self.a, self.da = g, u, a, da
        unit = 2.0 ** -20 if dtype == "bf16" else 2.0 ** -21
        self.ea = unit * (a.abs() + g.abs() * 2.0 ** -2)  # the activation's own error
        self.h = a * u
        self.h_tol = (1.13 * self.eg + self.ea) * u.abs() + a.abs() * self.eu + self.h.abs() * HALF[dtype] * 1.01 + 1e-30

    def gradients(self):
        dh = self.dh.double()
        dg, du = dh * self.u * self.da, dh * self.a
        small = self.g.numel() * self.X.shape[1] <= 1 << 30
        half = 2.0 ** -22 if self.dtype == "f32" else 2.0 ** -16 if small else HALF["bf16"] * 1.01
        unit = 2.0 ** -19
        egd = dh.abs() * (self.eu * self.da.abs() + self.u.abs() * (1.2 * self.eg + unit)) + dg.abs() * half
        eud = dh.abs() * (1.13 * self.eg + self.ea) + du.abs() * half
        M, F = dg.shape
        h = HALF[self.dtype] * 1.01
        G, U, X = self.G.abs(), self.U.abs(), self.X.abs()
        dx = dg @ self.G + du @ self.U
        c = chain(2 * F, self.dtype)
        out = {"dx": (dx, (egd + c * dg.abs()) @ G + (eud + c * du.abs()) @ U + h * dx.abs() + 1e-30)}
        c = chain(M, self.dtype) + 64 * 2.0 ** -24  # (and the parts of a last wave)
        for n, d, ed in (("dwg", dg, egd), ("dwu", du, eud)):
            dw = d.T @ self.X
            out[n] = (dw, (ed + c * d.abs()).T @ X + h * dw.abs() + 1e-30)
        return out


# tokens from one to several tiles, both sides of the few-token rule (16; fp32 64), widths that
# end inside a vector's, a K tile's and a tile's extent, whole waves and cut ones
SIZES = [(1, 8, 8), (1, 1024, 512), (3, 40, 24), (8, 512, 72), (9, 264, 200), (16, 1032, 136), (17, 104, 56), (33, 72, 264),
         (64, 520, 312), (65, 64, 64), (128, 128, 128), (129, 136, 8), (200, 8, 264), (255, 1000, 72), (257, 64, 1032),
         (513, 2056, 520), (1554, 520, 1400), (2500, 264, 2048), (70, 2000, 136), (169, 4104, 72)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,D,F", SIZES)
def test_forward_and_gradients(m, M, D, F, act, dtype):
    c = Case(M, D, F, dtype, act)
    within(m.glu_fwd(c.x, c.wg, c.wu, act=act), c.h, c.h_tol, "h")
    got = m.glu_bwd(c.x, c.wg, c.wu, c.dh, act=act)
    for n, (ref, tol) in c.gradients().items():
        assert got[n].dtype is c.x.dtype
        within(got[n], ref, tol, n)
    assert m.device_status() == (0, 0)


@pytest.mark.parametrize("M,D,F", [(5000, 512, 2816), (20000, 264, 1416), (4097, 1024, 4104)])
def test_pairs_of_ctas_and_many_waves(m, M, D, F):
    """The 256 x 256 tiles, bf16 (several waves of every product)."""
    c = Case(M, D, F, "bf16", "silu", seed=10)
    within(m.glu_fwd(c.x, c.wg, c.wu), c.h, c.h_tol, "h")
    got = m.glu_bwd(c.x, c.wg, c.wu, c.dh)
    for n, (ref, tol) in c.gradients().items():
        within(got[n], ref, tol, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [5, 40, 300])
def test_rows_of_a_wider_buffer(m, M, dtype):
    B, D, F = 3, 136, 200
    buf = rn(1, B, M, D + 32, dtype=dtype)
    wg, wu = (rn(s, F, D, dtype=dtype, scale=0.1) for s in (2, 3))
    dh = rn(4, B, M, F, dtype=dtype)
    x = buf[..., 16:16 + D]
    h = m.glu_fwd(x, wg, wu)
    assert h.shape == (B, M, F) and torch.equal(h, m.glu_fwd(x.contiguous(), wg, wu))
    a, b = m.glu_bwd(x, wg, wu, dh), m.glu_bwd(x.contiguous(), wg, wu, dh)
    assert all(torch.equal(a[n], b[n]) for n in a)
    with pytest.raises(ValueError):
        m.glu_fwd(rn(5, B, M + 1, D, dtype=dtype)[:, :M], wg, wu)  # rows not evenly spaced


@pytest.mark.parametrize("M,D,F", [(3, 432, 96), (300, 136, 264), (1500, 264, 1416)])
def test_small_products_round_their_gradients_once(m, M, D, F):
    """Up to M D F = 2^30.  Of values whose mantissas are spread evenly over an octave, one rounding
    to bf16 leaves a relative 2-norm of about 1.66e-3, two
    independent ones 2.35e-3; the bound lies between them (outputs of these sizes
    scatter by less than a tenth)."""
    c = Case(M, D, F, "bf16", "silu", seed=30)
    got = m.glu_bwd(c.x, c.wg, c.wu, c.dh)
    for n, (ref, _) in c.gradients().items():
        assert (got[n].double() - ref).norm() <= 1.95e-3 * ref.norm(), n


def test_long_sums_do_not_drift(m):
    """Gradients of the weights over 300,000 tokens of one sign: the mean relative error of 4,096
    sums is that of their chains (at most 2,048 steps that each cut off 3.1 2^-24 of a
    growing sum, half of it: 1.9e-4) and of 4,096 roundings (2^-8 / 3^(1/2) / 64 = 3.5e-5 in the
    mean's standard deviation, three of them 1.1e-4)."""
    M, D, F = 300_000, 64, 64
    x, dh = rn(1, M, D).abs(), rn(2, M, F).abs()
    wg, wu = rn(3, F, D).abs() * 0.1, rn(4, F, D).abs() * 0.1
    got = m.glu_bwd(x, wg, wu, dh, want_dx=False)
    X, G, U = x.double(), wg.double(), wu.double()
    g, u = X @ G.T, X @ U.T
    s = torch.sigmoid(g)
    for n, d in (("dwg", dh.double() * u * (s + g * s * (1 - s))), ("dwu", dh.double() * g * s)):
        ref = d.T @ X
        assert abs(((got[n].double() - ref) / ref).mean().item()) <= 3e-4
        assert ((got[n].double() - ref).abs() <= ref * (2.0 ** -8 + 3e-4)).all()


def test_what_is_wanted(m):
    c = Case(300, 136, 200, "bf16", "silu")
    whole = m.glu_bwd(c.x, c.wg, c.wu, c.dh)
    only = m.glu_bwd(c.x, c.wg, c.wu, c.dh, want_dw=False)
    assert only["dwg"] is None and only["dwu"] is None and torch.equal(only["dx"], whole["dx"])
    only = m.glu_bwd(c.x, c.wg, c.wu, c.dh, want_dx=False)
    assert only["dx"] is None and torch.equal(only["dwg"], whole["dwg"]) and torch.equal(only["dwu"], whole["dwu"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_tokens(m, dtype):
    x, wg, dh = rn(1, 0, 64, dtype=dtype), rn(2, 72, 64, dtype=dtype), rn(3, 0, 72, dtype=dtype)
    assert m.glu_fwd(x, wg, wg).shape == (0, 72)
    out = {n: torch.full_like(wg, 7.0) for n in ("dwg", "dwu")}
    g = m.glu_bwd(x, wg, wg, dh, out=out)
    assert g["dx"].shape == (0, 64) and not g["dwg"].any() and not g["dwu"].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [12, 300])
def test_values_that_are_not_finite_stay_in_their_rows(m, M, dtype):
    """A token's values reach no other token's outputs; a weight's row only its column."""
    c = Case(M, 136, 200, dtype, "silu")
    ref = m.glu_fwd(c.x, c.wg, c.wu)
    x, wu = c.x.clone(), c.wu.clone()
    x[3, 7], x[5] = float("nan"), float("inf")
    h = m.glu_fwd(x, c.wg, c.wu)
    keep = [i for i in range(M) if i not in (3, 5)]
    assert torch.isnan(h[3]).all() and not torch.isfinite(h[5]).all() and torch.equal(h[keep], ref[keep])
    wu[11, 2] = float("nan")
    h = m.glu_fwd(c.x, c.wg, wu)
    cols = [i for i in range(200) if i != 11]
    assert torch.isnan(h[:, 11]).all() and torch.equal(h[:, cols], ref[:, cols])


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_arguments_of_the_activation(m, act, dtype):
    """g from -1e4 to 1e4 (and 1e30): the activation goes to 0 and g, its derivative to 0 and 1,
    with no NaN.  x is a unit vector per token, so g and u are single products."""
    vals = [-1e30, -1e4, -300.0, -100.0, -88.0, -20.0, 0.0, 20.0, 88.0, 300.0, 1e4]
    M, D = 80, 16
    x = torch.zeros(M, D, dtype=TD[dtype], device="cuda")
    x[:, 0] = 1
    F = 16
    wg = torch.zeros(F, D, dtype=TD[dtype], device="cuda")
    wg[:len(vals), 0] = torch.tensor(vals, device="cuda").to(TD[dtype])
    wu = torch.zeros_like(wg)
    wu[:, 0] = 1
    dh = torch.ones(M, F, dtype=TD[dtype], device="cuda")
    for rows in (slice(0, 4), slice(0, M)):
        h = m.glu_fwd(x[rows], wg, wu, act=act).double()
        ref = act64(wg[:, 0].double(), act).expand_as(h)
        assert ((h - ref).abs() <= ref.abs() * (HALF[dtype] + 2.0 ** -18) + 1e-6).all()
    g = m.glu_bwd(x, wg, wu, dh, act=act)
    leaf = wg[:, 0].double().requires_grad_()
    da, = torch.autograd.grad(act64(leaf, act).sum(), leaf)
    da = torch.where(leaf < -50, torch.zeros_like(da), da)  # (NaN in 64 bits at -1e30)
    dw = g["dwg"][:, 0].double()
    assert ((dw - M * da).abs() <= M * (da.abs() * 2.0 ** -6 + 1e-6)).all()


@pytest.mark.parametrize("M", [9, 100])
def test_fp32_values_at_the_end_of_the_range(m, M):
    """fp32 operands up to the largest value (which bf16's rounding would pass) and down to
    2^-100, one product to a sum, are held whole: u = x w within four roundings."""
    top = torch.finfo(torch.float32).max
    vals = torch.tensor([top, -top, 3.3953e38, 1e30, 1.0, 2.0 ** -60 * 1.2345678, 2.0 ** -100 * 1.7654321, 0.0], device="cuda")
    D = F = 16
    x = torch.zeros(M, D, device="cuda")
    x[:, 0] = 1.0
    wu = torch.zeros(F, D, device="cuda")
    wu[:8, 0] = vals
    wg = torch.zeros(F, D, device="cuda")
    wg[:, 0] = 1.25
    h = m.glu_fwd(x, wg, wu)
    ref = (torch.nn.functional.silu(torch.tensor(1.25, dtype=torch.float64)).item() * wu[:, 0].double()).expand(M, F)
    fits = ref.abs() <= top
    assert ((h.double() - ref).abs()[fits] <= ref.abs()[fits] * 2.0 ** -20).all() and torch.isinf(h[~fits]).all()


def test_against_differences(m):
    """fp32: the slope of sum(h dh) along a direction of all leaves, central differences
    with step 2^-7: third derivatives of the sum along the unit-scale direction are below
    the sum of |h dh| (2^-14 / 6 of it), rounding is 2^-22 of that sum over the step."""
    M, D, F = 70, 72, 56
    t = {n: rn(i, *s, dtype="f32", scale=c) for i, (n, s, c) in enumerate(
        (("x", (M, D), 1.0), ("wg", (F, D), D ** -0.5), ("wu", (F, D), D ** -0.5)))}
    d = {n: rn(10 + i, *v.shape, dtype="f32", scale=v.abs().mean().item()) for i, (n, v) in enumerate(t.items())}
    dh = rn(20, M, F, dtype="f32")
    step = 2.0 ** -7

    def at(k):
        h = m.glu_fwd(*(t[n] + k * step * d[n] for n in t)).double()
        return (h * dh.double()).sum(), (h * dh.double()).abs().sum()
    (up, size), (down, _) = at(1), at(-1)
    g = m.glu_bwd(t["x"], t["wg"], t["wu"], dh)
    want = sum((g["d" + n].double() * d[n].double()).sum() for n in t)
    assert abs((up - down) / (2 * step) - want) <= size * (2.0 ** -22 / step + 2.0 ** -10)


def test_far_rows(m):
    """Rows of x 2^31 elements apart in all."""
    if torch.cuda.get_device_properties(0).total_memory < 32 << 30:
        pytest.skip("needs 9 GB of device memory")
    M, D, F = 70, 136, 72
    row = (1 << 25) + 64
    buf = torch.empty(M * row, dtype=torch.bfloat16, device="cuda")
    x, xc = buf.as_strided((M, D), (row, 1)), rn(1, M, D)
    x.copy_(xc)
    wg, wu, dh = rn(2, F, D), rn(3, F, D), rn(4, M, F)
    assert (M - 1) * row > 1 << 31
    assert torch.equal(m.glu_fwd(x, wg, wu), m.glu_fwd(xc, wg, wu))
    assert torch.equal(m.glu_fwd(x[:9], wg, wu), m.glu_fwd(xc[:9], wg, wu))
    a, b = m.glu_bwd(x, wg, wu, dh), m.glu_bwd(xc, wg, wu, dh)
    assert all(torch.equal(a[n], b[n]) for n in a)
