"""Codes of add_norm_q8: the nearest e4m3 values of y / scale, ties to even, where
y = w (.) r s and scale = max|y| / 448.

The row's factor s leaves the quotient: y / scale = 448 w r / max|w r|.  With bf16 inputs w r has
16 bits and 448 w r 19, so the 64-bit quotient below meets the middle between two codes
exactly where the formula does (quotients of such numbers that are not on a middle are 2^-21 and
more of their size away from it, so that their way through fp32 decides nothing), and about one
code in 10^4 of normal rows lies there.  The codes have to be the formula's, all of them.

With fp32 inputs w r is rounded (2^-24) and so is the quotient: a code may differ
only where the 64-bit quotient is within 2^-22 of its size of a middle.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

TD = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    from non_linear_matrix_gb300 import m2rnn
    m2rnn.use_library("normal")
    return m2rnn


def rn(seed, *s, dtype="bf16", scale=1.0):
    return (torch.randn(*s, generator=torch.Generator().manual_seed(seed)) * scale).to(TD[dtype]).cuda()


def quotients(r, w):
    p = r.double() if w is None else r.double() * w.double()
    return p * 448 / p.abs().amax(-1, keepdim=True)


def nearest(t):
    return t.float().to(torch.float8_e4m3fn)


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


SIZES = [(1, 8), (3, 72), (305, 264), (12001, 2000), (4096, 1024), (700, 4096), (301, 8200), (33, 16384)]


@pytest.mark.parametrize("M,D", SIZES)
def test_codes_are_the_formulas(m, M, D):
    x, res, w = rn(1, M, D), rn(2, M, D, scale=2), (1 + 0.1 * rn(3, D).float()).bfloat16()
    for weight in (w, None, -w):
        q, scale, r = m.add_norm_q8(x, res, weight)
        assert torch.equal(q.float(), nearest(quotients(r, weight)).float())  # (a zero is one value, -0 or 0)
        q2, scale2, _ = m.add_norm_q8(r, None, weight)  # the norm alone
        assert same(q2, q) and torch.equal(scale2, scale)
    stream = res.clone()  # the stream in place
    assert same(m.add_norm_q8(x, stream, None, out={"r": stream})[0], m.add_norm_q8(x, res, None)[0])


@pytest.mark.parametrize("M,D", SIZES)
def test_fp32(m, M, D):
    r, w = rn(4, M, D, dtype="f32"), rn(5, D, dtype="f32")
    q = m.add_norm_q8(r, None, w)[0]
    t = quotients(r, w)
    other = q.float() != nearest(t).float()
    near = nearest(t * (1 + 2.0 ** -22)).float() != nearest(t * (1 - 2.0 ** -22)).float()
    assert not (other & ~near).any() and (other.sum() <= 8 + 2e-6 * t.numel())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [72, 520, 2000, 8200])
@pytest.mark.parametrize("rows", [5, 400])
def test_rows_of_far_sizes(m, rows, D, dtype):
    """Rows of one size each, from where the squares are below fp32's smallest (eps decides
    the root) to near its largest, with weights from 1e-12 to 1e12 between: each code is off by half a
    step of y / scale at most, and where products or squares pass fp32's range y is what fp32 gives:
    zeros or values that are not finite, never a finite code of something else."""
    sizes = [1e-35, 1e-25, 1e-15, 1e-3, 1.0, 1e5, 1e10, 1e15, 1e17]
    base = rn(6, rows, D, dtype=dtype).clamp(-3, 3)
    r = torch.stack([(base[i].float() * sizes[i % len(sizes)]) for i in range(rows)]).to(TD[dtype])
    for power in (-12, 0, 12):
        w = (rn(7, D, dtype=dtype).float().clamp(-3, 3) * 10.0 ** power).to(TD[dtype])
        q, scale, _ = m.add_norm_q8(r, None, w, 1e-6)
        y = r.double() * (r.double().square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w.double()
        s = scale.double()[:, None]
        # fp32's smallest numbers: y below 2^-126 loses bits in the scale
        ok = y.abs().amax(-1) > 1e-33
        tol = y.abs() * (2.0 ** -4 + 2.0 ** -18) + s * 2.0 ** -10 * (1 + 2.0 ** -18)
        assert (((q.double() * s - y).abs() <= tol) | ~ok[:, None]).all()
        assert torch.isfinite(q.float()).all() and torch.isfinite(scale).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [72, 2000])
def test_rows_of_zeros_and_not_finite(m, D, dtype):
    r, w = rn(8, 9, D, dtype=dtype), rn(9, D, dtype=dtype)
    want, ws, _ = m.add_norm_q8(r, None, w)
    bad = r.clone()
    bad[1] = 0
    bad[3, 7], bad[5, 2] = float("nan"), float("inf")
    bad[6] = 3e19  # the squares pass fp32's largest: y is 0 there
    q, s, _ = m.add_norm_q8(bad, None, w)
    assert s[1] == 0 and not q[1].float().any()
    assert s[6] == 0 and not q[6].float().any()
    for i in (3, 5):
        assert torch.isnan(s[i]) and torch.isnan(q[i].float()).all()
    rest = [0, 2, 4, 7, 8]
    assert same(q[rest], want[rest]) and torch.equal(s[rest], ws[rest])
    q, s, _ = m.add_norm_q8(bad, None, w, 0.0)  # a zero row without eps
    assert torch.isnan(s[1]) and torch.isnan(q[1].float()).all()
    w2 = w.clone()
    w2[3] = float("nan")
    q, s, _ = m.add_norm_q8(r, None, w2)
    assert torch.isnan(s).all() and torch.isnan(q.float()).all()
    zero = m.add_norm_q8(r, None, torch.zeros_like(w))
    assert not zero[0].float().any() and not zero[1].any()
    huge = torch.full_like(w, 3e38)  # w r passes fp32's largest where r is above 1, y does not have to
    q, s, _ = m.add_norm_q8(torch.full_like(r, 1e3), None, huge)
    assert (s == s[0]).all() and (q.float() == 448).all() and abs(s[0].item() * 448 / 3e38 - 1) < 2.0 ** -8
    assert m.device_status() == (0, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D", [(5, 72), (9, 2000), (400, 520), (7, 8200)])
def test_far_rows_under_the_index_checks(m, M, D, dtype):
    """Rows that leave fp32's range, with the sum in place, alone and as slices of a wider
    buffer: the checked build finds no index outside, and both builds agree."""
    from non_linear_matrix_gb300 import build as b
    b.build(checked=True)
    sizes = torch.tensor([1e-30, 1.0, 1e19, 1e25], device="cuda")[torch.arange(M, device="cuda") % 4]
    wide = (rn(10, M, D + 16, dtype="f32") * sizes[:, None]).to(TD[dtype])
    x, res, w = wide[:, 8:8 + D], rn(11, M, D, dtype=dtype), (rn(12, D, dtype="f32") * 1e12).to(TD[dtype])
    got = {}
    for which in ("normal", "checked"):
        m.use_library(which)
        try:
            m.device_status(clear=True)
            stream = res.clone()
            got[which] = [*m.add_norm_q8(x, stream, w, out={"r": stream}), *m.add_norm_q8(x, None, w)[:2],
                          *m.add_norm_q8(x, res, w)]
            assert m.device_status(clear=True) == (0, 0)
        finally:
            m.use_library("normal")
    raw = [[t.view(torch.uint8) for t in g] for g in got.values()]
    assert all(torch.equal(a, b) for a, b in zip(*raw))
    g = got["normal"]
    assert torch.equal(g[0].view(torch.uint8), g[5].view(torch.uint8)) and torch.equal(g[2], g[7])
