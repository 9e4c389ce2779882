"""Norm of queries and keys with the position rotation (qk_norm_fwd,
qk_norm_bwd) against a plain implementation in 64 bits.

Tolerances, derived: bf16 outputs: half an ulp of the result (2^-9) plus
fp32 arithmetic; the rotation adds two products that may cancel, whose
rounding is relative to the row's scale: elementwise 2^-8 of (|exact| + rms).
fp32: rsqrtf (2 ulp), K squares summed in fp32 over lanes (K 2^-24 at most,
K <= 256), five products: 2^-17 of (|exact| + rms).  Parameter gradients:
sums of n rows in runs of fp32: 1e-5 relative L2.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

TD = {"bf16": torch.bfloat16, "f32": torch.float32}
ELEM = {"bf16": 2.0 ** -8, "f32": 2.0 ** -17}
PARAM_REL = 1e-5
EPS = 1e-6


@pytest.fixture(scope="module")
def m2rnn():
    import __graft_entry__
    __graft_entry__.build()
    from non_linear_matrix_gb300 import m2rnn as m
    m.use_library("normal")
    return m


def make(B, T, Nq, Nk, K, R, dtype, seed, P=None, slices=True):
    g = torch.Generator().manual_seed(seed)
    td = TD[dtype]

    def rn(*s):
        return torch.randn(*s, generator=g).cuda()
    buf = (3 * rn(B, T, (Nq + Nk) * K + 16)).to(td)
    d = {"q": buf[..., :Nq * K].view(B, T, Nq, K) if slices else buf[..., :Nq * K].reshape(B, T, Nq, K),
         "k": buf[..., Nq * K:(Nq + Nk) * K].unflatten(-1, (Nk, K)) if Nk else None,
         "wq": (1 + 0.2 * rn(K)).to(td), "wk": (1 + 0.2 * rn(K)).to(td) if Nk else None,
         "dqo": rn(B, T, Nq, K).to(td), "dko": rn(B, T, Nk, K).to(td) if Nk else None}
    P = P or max(T, 50)
    if R:
        ang = torch.randn(P, R // 2, generator=g).cuda() * 3
        d.update(cos=ang.cos(), sin=ang.sin(),
                 pos=torch.randint(0, P, (B, T), generator=g).int().cuda())
    else:
        d.update(cos=None, sin=None, pos=None)
    return d


def plain(x, w, cos, sin, pos, inter, eps=EPS, dy=None):
    x64 = x.double().requires_grad_(dy is not None)
    w64 = None if w is None else w.double().requires_grad_(dy is not None)
    u = x64 * (x64.square().mean(-1, keepdim=True) + eps).rsqrt()
    if w64 is not None:
        u = u * w64
    if cos is not None:
        R = 2 * cos.shape[1]
        c, s = cos.double()[pos.long()][:, :, None], sin.double()[pos.long()][:, :, None]
        a, b = (u[..., 0:R:2], u[..., 1:R:2]) if inter else (u[..., :R // 2], u[..., R // 2:R])
        ra, rb = a * c - b * s, b * c + a * s
        rot = torch.stack([ra, rb], -1).flatten(-2) if inter else torch.cat([ra, rb], -1)
        u = torch.cat([rot, u[..., R:]], -1)
    if dy is None:
        return u.detach()
    use = [t for t in (x64, w64) if t is not None]
    gr = torch.autograd.grad(u, use, dy.double())
    return gr[0], gr[1] if w64 is not None else None


def close(got, ref, tol, label):
    if ref.numel() == 0:
        return
    scale = ref.abs() + ref.square().mean().sqrt()
    err = ((got.double() - ref).abs() / scale).max().item()
    assert err <= tol, (label, err)


def rel(got, ref):
    return ((got.double() - ref).norm() / ref.norm().clamp_min(1e-30)).item()


SHAPES = [(1, 1, 1, 1, 16, 16), (2, 3, 1, 1, 64, 64), (1, 5, 3, 1, 128, 32), (2, 7, 8, 2, 64, 0),
          (3, 17, 4, 4, 16, 8), (1, 33, 6, 3, 32, 16), (2, 9, 2, 1, 96, 64), (1, 4, 5, 0, 80, 16),
          (1, 40, 2, 2, 256, 256), (1, 300, 16, 16, 64, 48), (2, 2, 1, 1, 8, 8), (1, 6, 3, 2, 64, 24), (1, 3, 2, 1, 104, 40)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,Nq,Nk,K,R", SHAPES)
def test_forward(m2rnn, B, T, Nq, Nk, K, R, dtype):
    for inter in ([False, True] if R else [False]):
        d = make(B, T, Nq, Nk, K, R, dtype, 7 * T + K)
        rot = dict(cos=d["cos"], sin=d["sin"], pos=d["pos"], interleaved=inter)
        qo, ko = m2rnn.qk_norm_fwd(d["q"], d["k"], d["wq"], d["wk"], EPS, **rot)
        p = (d["cos"], d["sin"], d["pos"], inter)
        close(qo, plain(d["q"], d["wq"], *p), ELEM[dtype], "q")
        if Nk:
            close(ko, plain(d["k"], d["wk"], *p), ELEM[dtype], "k")
        else:
            assert ko is None


@pytest.mark.parametrize("dtype,gdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("B,T,Nq,Nk,K,R", SHAPES)
def test_backward(m2rnn, B, T, Nq, Nk, K, R, dtype, gdtype):
    for inter in ([False, True] if R else [False]):
        d = make(B, T, Nq, Nk, K, R, dtype, 9 * T + K)
        rot = dict(cos=d["cos"], sin=d["sin"], pos=d["pos"], interleaved=inter)
        dqo = d["dqo"].to(TD[gdtype])
        dko = d["dko"].to(TD[gdtype]) if Nk else None
        g = m2rnn.qk_norm_bwd(d["q"], d["k"], d["wq"], d["wk"], dqo, dko, EPS, **rot)
        p = (d["cos"], d["sin"], d["pos"], inter)
        rq, rwq = plain(d["q"], d["wq"], *p, dy=dqo)
        close(g["dq"], rq, ELEM[dtype], "dq")
        assert rel(g["dwq"], rwq) <= PARAM_REL
        if Nk:
            rk, rwk = plain(d["k"], d["wk"], *p, dy=dko)
            close(g["dk"], rk, ELEM[dtype], "dk")
            assert rel(g["dwk"], rwk) <= PARAM_REL


def test_gradient_by_differences(m2rnn):
    """Against central differences of the forward kernel (fp32, h = 2^-7:
    truncation ~ h^2, rounding 2^-22 / h ~ 3e-5 of the loss's scale)."""
    d = make(1, 2, 2, 1, 16, 16, "f32", 4, slices=False)
    rot = dict(cos=d["cos"], sin=d["sin"], pos=d["pos"])
    d["k"] = d["k"].contiguous()
    g = m2rnn.qk_norm_bwd(d["q"], d["k"], d["wq"], d["wk"], d["dqo"], d["dko"], EPS, **rot)

    def loss(**kw):
        a = {**d, **kw}
        qo, ko = m2rnn.qk_norm_fwd(a["q"], a["k"], a["wq"], a["wk"], EPS, **rot)
        return ((qo.double() * d["dqo"]).sum() + (ko.double() * d["dko"]).sum()).item()

    h = 2.0 ** -7
    for name in ("q", "k", "wq", "wk"):
        t, gr = d[name], g["d" + name].reshape(-1)
        for i in range(0, t.numel(), max(1, t.numel() // 8)):
            up, dn = t.clone(), t.clone()
            up.view(-1)[i] += h
            dn.view(-1)[i] -= h
            num = (loss(**{name: up}) - loss(**{name: dn})) / (2 * h)
            assert abs(num - gr[i].item()) <= 2e-3 * (1 + abs(num)), (name, i)


def test_weights_absent_and_default_positions(m2rnn):
    """No weight is a weight of ones; no positions are 0, 1, 2, ..."""
    d = make(2, 12, 2, 1, 64, 64, "bf16", 11)
    ones = torch.ones(64, device="cuda").bfloat16()
    pos = torch.arange(12, device="cuda", dtype=torch.int32).expand(2, 12).contiguous()
    a = m2rnn.qk_norm_fwd(d["q"], d["k"], None, None, EPS, cos=d["cos"], sin=d["sin"])
    b = m2rnn.qk_norm_fwd(d["q"], d["k"], ones, ones, EPS, cos=d["cos"], sin=d["sin"], pos=pos)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    g = m2rnn.qk_norm_bwd(d["q"], d["k"], None, None, d["dqo"], d["dko"], EPS, cos=d["cos"],
                          sin=d["sin"])
    assert g["dwq"] is None and g["dwk"] is None


def test_l2_norm_of_the_recurrence(m2rnn):
    """w = K^(-1/2), eps = 0 is the L2 norm that the recurrence's workloads
    put on q and k."""
    d = make(2, 5, 1, 1, 64, 0, "f32", 12)
    w = torch.full((64,), 0.125, device="cuda")
    qo, _ = m2rnn.qk_norm_fwd(d["q"], d["k"], w, w, 0.0)
    close(qo, d["q"].double() / d["q"].double().norm(dim=-1, keepdim=True), ELEM["f32"], "q")


def test_zero_rows(m2rnn):
    """A zero row: 0 with eps > 0 (and a finite gradient), NaN in that row
    alone with eps = 0."""
    d = make(1, 4, 2, 1, 64, 64, "f32", 13)
    q = d["q"].clone()
    q[0, 1, 0] = 0
    rot = dict(cos=d["cos"], sin=d["sin"], pos=d["pos"])
    qo, _ = m2rnn.qk_norm_fwd(q, d["k"], d["wq"], d["wk"], EPS, **rot)
    assert not qo[0, 1, 0].any() and qo.isfinite().all()
    g = m2rnn.qk_norm_bwd(q, d["k"], d["wq"], d["wk"], d["dqo"], d["dko"], EPS, **rot)
    assert g["dq"].isfinite().all() and g["dwq"].isfinite().all()
    qo, _ = m2rnn.qk_norm_fwd(q, d["k"], d["wq"], d["wk"], 0.0, **rot)
    assert qo[0, 1, 0].isnan().all() and qo.isnan().sum() == 64


def test_position_outside_the_table(m2rnn):
    """NaN in that token's rotated features, M2RNN_ERR_BOUNDS in the status
    word, everything else as without it."""
    d = make(1, 6, 2, 1, 64, 32, "f32", 14, P=50)
    rot = dict(cos=d["cos"], sin=d["sin"])
    ref, _ = m2rnn.qk_norm_fwd(d["q"], d["k"], d["wq"], d["wk"], EPS, pos=d["pos"], **rot)
    m2rnn.device_status(clear=True)
    for bad in (50, -1):
        pos = d["pos"].clone()
        pos[0, 2] = bad
        qo, _ = m2rnn.qk_norm_fwd(d["q"], d["k"], d["wq"], d["wk"], EPS, pos=pos, **rot)
        st, _ = m2rnn.device_status(clear=True)
        assert st == -8
        assert qo[0, 2, :, :32].isnan().all() and torch.equal(qo[0, 2, :, 32:], ref[0, 2, :, 32:])
        assert torch.equal(qo[0, 3:], ref[0, 3:]) and torch.equal(qo[0, :2], ref[0, :2])


def test_single_tokens_equal_the_prompt(m2rnn):
    d = make(1, 20, 4, 2, 64, 64, "bf16", 15)
    rot = dict(cos=d["cos"], sin=d["sin"])
    qo, ko = m2rnn.qk_norm_fwd(d["q"], d["k"], d["wq"], d["wk"], EPS, pos=d["pos"], **rot)
    q1, k1 = d["q"].transpose(0, 1).contiguous(), d["k"].transpose(0, 1).contiguous()
    a, b = m2rnn.qk_norm_fwd(q1, k1, d["wq"], d["wk"], EPS,
                             pos=d["pos"].transpose(0, 1).contiguous(), **rot)
    assert torch.equal(a.transpose(0, 1), qo) and torch.equal(b.transpose(0, 1), ko)


def test_empty_deterministic_stream(m2rnn):
    d = make(2, 0, 2, 1, 64, 64, "bf16", 16, P=8)
    rot = dict(cos=d["cos"], sin=d["sin"], pos=d["pos"])
    qo, ko = m2rnn.qk_norm_fwd(d["q"], d["k"], d["wq"], d["wk"], EPS, **rot)
    assert qo.shape == (2, 0, 2, 64)
    g = m2rnn.qk_norm_bwd(d["q"], d["k"], d["wq"], d["wk"], d["dqo"], d["dko"], EPS, **rot)
    assert not g["dwq"].any() and not g["dwk"].any()
    d = make(4, 500, 8, 2, 64, 64, "bf16", 17)
    rot = dict(cos=d["cos"], sin=d["sin"], pos=d["pos"])
    args = (d["q"], d["k"], d["wq"], d["wk"], d["dqo"], d["dko"], EPS)
    ref = m2rnn.qk_norm_bwd(*args, **rot)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    again = m2rnn.qk_norm_bwd(*args, **rot, stream=st)
    st.synchronize()
    for n in ("dq", "dk", "dwq", "dwk"):
        assert torch.equal(ref[n], again[n]), n


def test_refusals(m2rnn):
    d = make(2, 6, 2, 1, 64, 32, "bf16", 18)
    rot = dict(cos=d["cos"], sin=d["sin"], pos=d["pos"])
    a = (d["q"], d["k"], d["wq"], d["wk"])

    def code(f):
        with pytest.raises(m2rnn.M2RNNError) as e:
            f()
        return e.value.code

    assert code(lambda: m2rnn.qk_norm_fwd(*a, -1.0, **rot)) == -1
    assert code(lambda: m2rnn.qk_norm_fwd(*a, float("nan"), **rot)) == -1
    c12 = torch.ones(50, 10, device="cuda")                       # R = 20
    assert code(lambda: m2rnn.qk_norm_fwd(*a, EPS, cos=c12, sin=c12, pos=d["pos"])) == -2
    c64 = torch.ones(50, 64, device="cuda")                       # R > K
    assert code(lambda: m2rnn.qk_norm_fwd(*a, EPS, cos=c64, sin=c64, pos=d["pos"])) == -2
    short = d["cos"][:4].contiguous()                             # 6 tokens, 4 positions
    assert code(lambda: m2rnn.qk_norm_fwd(*a, EPS, cos=short, sin=short)) == -1
    x = torch.zeros(1, 2, 1, 20, device="cuda").bfloat16()
    assert code(lambda: m2rnn.qk_norm_fwd(x, None, None, None, EPS)) == -2
    assert code(lambda: m2rnn.qk_norm_bwd(*a, d["dqo"], d["dko"], EPS, **rot,
                                          workspace=torch.zeros(16, device="cuda").byte())) == -5
    with pytest.raises(TypeError):
        m2rnn.qk_norm_fwd(d["q"], d["k"].float(), d["wq"], d["wk"], EPS, **rot)
    with pytest.raises(ValueError):
        m2rnn.qk_norm_fwd(*a, EPS, cos=d["cos"], pos=d["pos"])
    with pytest.raises(ValueError):
        m2rnn.qk_norm_fwd(d["q"].transpose(2, 3), d["k"].transpose(2, 3), None, None, EPS)
    with pytest.raises(TypeError):
        m2rnn.qk_norm_fwd(*a, EPS, cos=d["cos"], sin=d["sin"], pos=d["pos"].long())
