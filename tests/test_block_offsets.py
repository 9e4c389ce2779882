"""Inputs whose batch items lie more than 2^31 elements apart (a slice of a
long buffer): offsets are formed in 64 bits.  Results equal those of a
contiguous copy bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu

FAR = (1 << 31) + 4096  # elements of bf16: 4.3 GB


@pytest.fixture(scope="module")
def far():
    """A buffer of 2 x FAR bf16 elements."""
    import __graft_entry__
    __graft_entry__.build()
    from non_linear_matrix_gb300 import m2rnn as m
    m.use_library("normal")
    if torch.cuda.get_device_properties(0).total_memory < 32 << 30:
        pytest.skip("needs 9 GB of device memory")
    return m, torch.empty(2, FAR, dtype=torch.bfloat16, device="cuda")


def place(buf, shape, at, seed):
    """A random [2, ...] tensor in buf, items FAR elements apart, and a copy."""
    n = torch.Size(shape[1:]).numel()
    x = torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
    view = buf[:, at:at + n].view(shape)
    view.copy_(x)
    assert view.stride(0) == FAR
    return view, x


def test_conv(far):
    m, buf = far
    x, xc = place(buf, (2, 37, 72), FAR - 37 * 72 - 8, 1)
    w = torch.randn(72, 4, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    for a, b in zip(m.conv_fwd(x, w), m.conv_fwd(xc, w)):
        assert torch.equal(a, b)
    g, gc = m.conv_bwd(x, w, xc), m.conv_bwd(xc, w, xc)
    assert torch.equal(g["dx"], gc["dx"]) and torch.equal(g["dw"], gc["dw"])
    st = torch.zeros(2, 3, 72, device="cuda").bfloat16()
    assert torch.equal(m.conv_step(x[:, 5], w, st)[0], m.conv_step(xc[:, 5], w, st)[0])


def test_qk_norm(far):
    m, buf = far
    q, qc = place(buf, (2, 9, 3, 64), FAR - 4096, 3)
    k, kc = place(buf, (2, 9, 1, 64), 64, 4)
    for a, b in zip(m.qk_norm_fwd(q, k), m.qk_norm_fwd(qc, kc)):
        assert torch.equal(a, b)
    g, gc = m.qk_norm_bwd(q, k, None, None, qc, kc), m.qk_norm_bwd(qc, kc, None, None, qc, kc)
    assert torch.equal(g["dq"], gc["dq"]) and torch.equal(g["dk"], gc["dk"])


def test_scan(far):
    m, buf = far
    q, qc = place(buf, (2, 130, 1, 32), 0, 5)
    k, kc = place(buf, (2, 130, 1, 32), 8192, 6)
    v, vc = place(buf, (2, 130, 3, 16), FAR - 8192, 7)
    a, ac = place(buf, (2, 130, 3), 16384 + 8, 8)
    par = [torch.full((3,), x, device="cuda").bfloat16() for x in (1.0, -2.0)]
    for x, y in zip(m.scan_fwd(q, k, v, a, *par)[:2], m.scan_fwd(qc, kc, vc, ac, *par)[:2]):
        assert torch.equal(x, y)
    dy = torch.ones_like(vc)
    g, gc = m.scan_bwd(q, k, v, a, *par, dy), m.scan_bwd(qc, kc, vc, ac, *par, dy)
    for n in ("dq", "dk", "dv", "da", "dalpha", "dbeta"):
        assert torch.equal(g[n], gc[n]), n
    H = torch.zeros(2, 3, 32, 16, device="cuda")
    s, sc = [[t[:, 3] for t in x] for x in ((q, k, v, a), (qc, kc, vc, ac))]
    for x, y in zip(m.scan_step(*s, *par, H), m.scan_step(*sc, *par, H)):
        assert torch.equal(x, y)
