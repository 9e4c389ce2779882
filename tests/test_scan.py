"""The selective scan (scan_fwd, scan_bwd, scan_step) against the recurrence
token by token in 64 bits, and its chain rule in reverse.

Tolerances, derived.  bf16 outputs (relative L2): half an ulp of the output
(2^-9 at most, 2^-9.8 rms) and one rounding of each weight q.k 2^S dt to bf16
(the same size, independent): 2^-9 sqrt(2) < 4e-3 at most.  States and
parameter gradients of bf16 inputs: decayed operands in two bf16 terms (2^-18
at most each), powers of two to 2^-22, fp32 sums: 1e-5.  fp32 inputs: three
terms (the whole fp32 value), decays to a few 2^-24 of |log2 decay| (< 2^6
here): 1e-5.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TD = {"bf16": torch.bfloat16, "f32": torch.float32}
OUT_REL = {"bf16": 4e-3, "f32": 1e-5}
FP32_REL = 1e-5


@pytest.fixture(scope="module")
def m2rnn():
    import __graft_entry__
    __graft_entry__.build()
    from non_linear_matrix_gb300 import m2rnn as m
    m.use_library("normal")
    return m


def make(B, T, N, K, V, Nq, dtype, seed, sliced=False, state=True):
    """Step sizes of 1e-3 to 0.1 at a = 0, decay rates of 1 to 16."""
    g = torch.Generator().manual_seed(seed)
    td = TD[dtype]

    def rn(*s):
        return torch.randn(*s, generator=g)
    d = {}
    if sliced:  # rows of one [B,T,C] projection, the heads' gate inputs behind them
        wide = 2 * Nq * K + N * V + N + 8
        wide += -wide % 8
        buf = rn(B, T, wide).to(td).cuda()
        d["q"] = buf[..., :Nq * K].unflatten(-1, (Nq, K))
        d["k"] = buf[..., Nq * K:2 * Nq * K].unflatten(-1, (Nq, K))
        d["v"] = buf[..., 2 * Nq * K:2 * Nq * K + N * V].unflatten(-1, (N, V))
        d["a"] = buf[..., 2 * Nq * K + N * V:2 * Nq * K + N * V + N]
    else:
        for n in ("q", "k"):
            x = rn(B, T, Nq, K)
            d[n] = (x / x.norm(dim=-1, keepdim=True)).to(td).cuda()
        d["v"] = rn(B, T, N, V).to(td).cuda()
        d["a"] = rn(B, T, N).to(td).cuda()
    dt = torch.exp(torch.rand(N, generator=g) * math.log(100) + math.log(1e-3))
    d["beta"] = (dt + torch.log(-torch.expm1(-dt))).to(td).cuda()
    d["alpha"] = (1 + 15 * torch.rand(N, generator=g)).to(td).cuda()
    d["w_r"] = rn(N, V).to(td).cuda()
    d["H0"] = (0.1 * rn(B, N, K, V)).cuda() if state else None
    d["dy"] = rn(B, T, N, V).to(td).cuda()
    d["dHT"] = (0.1 * rn(B, N, K, V)).cuda() if state else None
    return d


def plain(d, backward=False):
    """Token by token in 64 bits; q, k [B,T,Nq,K]."""
    x = {n: t.double() if t is not None else None for n, t in d.items()}
    B, T, N, V = x["v"].shape
    Nq, K = x["q"].shape[2:]
    r = N // Nq
    q, k = x["q"].repeat_interleave(r, 2), x["k"].repeat_interleave(r, 2)
    w_r = x["w_r"] if x["w_r"] is not None else torch.zeros(N, V, dtype=torch.float64, device=q.device)
    z = x["a"] + x["beta"]
    dt = torch.logaddexp(z, torch.zeros_like(z))
    f = torch.exp(-x["alpha"] * dt)
    H = x["H0"] if x["H0"] is not None else x["v"].new_zeros(B, N, K, V)
    ys, hist = [], []
    for t in range(T):
        hist.append(H)
        H = f[:, t, :, None, None] * H + dt[:, t, :, None, None] * k[:, t, :, :, None] * x["v"][:, t, :, None]
        ys.append((H * q[:, t, :, :, None]).sum(2))
    y = torch.stack(ys, 1) if T else x["v"].clone()
    out = {"y": y + w_r * x["v"], "HT": H}
    if not backward:
        return out
    dy = x["dy"]
    C = x["dHT"] if x["dHT"] is not None else torch.zeros_like(H)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(x["v"])
    ddt, df = torch.zeros_like(dt), torch.zeros_like(dt)
    hist.append(H)
    for t in reversed(range(T)):
        C = C + q[:, t, :, :, None] * dy[:, t, :, None]
        dq[:, t] = (hist[t + 1] * dy[:, t, :, None]).sum(-1)
        Cv = (C * x["v"][:, t, :, None]).sum(-1)
        dk[:, t] = dt[:, t, :, None] * Cv
        dv[:, t] = dt[:, t, :, None] * (C * k[:, t, :, :, None]).sum(2)
        ddt[:, t] = (k[:, t] * Cv).sum(-1)
        df[:, t] = (C * hist[t]).sum((-1, -2))
        C = f[:, t, :, None, None] * C
    da = (ddt - x["alpha"] * f * df) * torch.sigmoid(z)
    out.update(dq=dq.unflatten(2, (Nq, r)).sum(3), dk=dk.unflatten(2, (Nq, r)).sum(3),
               dv=dv + w_r * dy, da=da, dalpha=(-dt * f * df).sum((0, 1)), dbeta=da.sum((0, 1)),
               dw_r=(dy * x["v"]).sum((0, 1)), dH0=C)
    return out


def rel(got, ref):
    return ((got.double() - ref).norm() / ref.norm().clamp_min(1e-30)).item() if ref.numel() else 0.0


def args(d):
    return d["q"], d["k"], d["v"], d["a"], d["alpha"], d["beta"]


# B, T, N, K, V, Nq
SHAPES = [(1, 1, 1, 16, 16, 1), (2, 5, 3, 32, 16, 1), (1, 63, 4, 64, 16, 1), (2, 64, 4, 64, 32, 2),
          (1, 65, 5, 64, 16, 5), (3, 130, 6, 128, 32, 3), (1, 200, 9, 16, 32, 1),
          (2, 333, 7, 128, 16, 7), (1, 1027, 32, 64, 16, 1), (40, 70, 4, 32, 32, 4)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,N,K,V,Nq", SHAPES)
def test_forward(m2rnn, B, T, N, K, V, Nq, dtype):
    for sliced, state in [(False, True), (True, False)]:
        d = make(B, T, N, K, V, Nq, dtype, T + K, sliced, state)
        y, HT, saved = m2rnn.scan_fwd(*args(d), d["w_r"], d["H0"])
        ref = plain(d)
        assert saved is None
        assert rel(y, ref["y"]) <= OUT_REL[dtype], ("y", sliced, rel(y, ref["y"]))
        assert rel(HT, ref["HT"]) <= FP32_REL, ("HT", sliced, rel(HT, ref["HT"]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_options(m2rnn, dtype):
    """No w_r, no H_T, [B,T,K] queries, saved or not: the same y."""
    d = make(2, 100, 4, 64, 16, 1, dtype, 3)
    d["w_r"] = None
    y, HT, _ = m2rnn.scan_fwd(*args(d), None, d["H0"], want_HT=False)
    assert HT is None and rel(y, plain(d)["y"]) <= OUT_REL[dtype]
    y2, _, saved = m2rnn.scan_fwd(d["q"][:, :, 0], d["k"][:, :, 0], *args(d)[2:], None, d["H0"],
                                  save=True)
    assert torch.equal(y, y2) and saved is not None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,K,V,Nq", [(1, 1, 16, 16, 1), (3, 5, 64, 16, 1), (2, 6, 128, 32, 3),
                                        (70, 4, 32, 32, 1)])
def test_steps_against_the_recurrence(m2rnn, B, N, K, V, Nq, dtype):
    """Single tokens, the state in place and apart, on slices."""
    T = 4
    d = make(B, T, N, K, V, Nq, dtype, 5, sliced=True)
    ref = plain(d)
    H = d["H0"].clone()
    for t in range(T):
        y1, H1 = m2rnn.scan_step(d["q"][:, t], d["k"][:, t], d["v"][:, t], d["a"][:, t],
                                 d["alpha"], d["beta"], H, d["w_r"])
        y, H2 = m2rnn.scan_step(d["q"][:, t], d["k"][:, t], d["v"][:, t], d["a"][:, t],
                                d["alpha"], d["beta"], H, d["w_r"], H_out=H)
        assert H2 is H and torch.equal(H1, H) and torch.equal(y, y1)
        assert rel(y, ref["y"][:, t]) <= OUT_REL[dtype]
    assert rel(H, ref["HT"]) <= FP32_REL


GRADS_OUT, GRADS_FP32 = ("dq", "dk", "dv", "da"), ("dalpha", "dbeta", "dw_r", "dH0")


def check_grads(g, ref, dtype, names=GRADS_OUT + GRADS_FP32):
    bad = {n: rel(g[n], ref[n]) for n in names
           if not rel(g[n], ref[n]) <= (OUT_REL[dtype] if n in GRADS_OUT else FP32_REL)}
    assert not bad, bad


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,N,K,V,Nq", SHAPES)
def test_backward(m2rnn, B, T, N, K, V, Nq, dtype):
    for sliced, state, save in [(False, True, True), (True, False, False)]:
        d = make(B, T, N, K, V, Nq, dtype, T + K + 1, sliced, state)
        saved = m2rnn.scan_fwd(*args(d), d["w_r"], d["H0"], save=True)[2] if save else None
        g = m2rnn.scan_bwd(*args(d), d["dy"], d["w_r"], d["H0"], d["dHT"], saved=saved, want_dH0=True)
        check_grads(g, plain(d, backward=True), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_options(m2rnn, dtype):
    """No w_r; saved or recomputed: the same bits; another stream too."""
    d = make(2, 150, 4, 64, 16, 1, dtype, 30)
    d["w_r"] = None
    saved = m2rnn.scan_fwd(*args(d), None, d["H0"], save=True)[2]
    g = m2rnn.scan_bwd(*args(d), d["dy"], None, d["H0"], d["dHT"], saved=saved)
    assert g["dw_r"] is None and "dH0" not in g
    check_grads(g, plain(d, backward=True), dtype, GRADS_OUT + ("dalpha", "dbeta"))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    g2 = m2rnn.scan_bwd(*args(d), d["dy"], None, d["H0"], d["dHT"], stream=st)
    st.synchronize()
    for n in GRADS_OUT + ("dalpha", "dbeta"):
        assert torch.equal(g[n], g2[n]), n


def test_gradient_by_differences(m2rnn):
    """Every input's gradient against central differences of the forward
    kernel (fp32, h = 2^-7: truncation ~ h^2 of the third derivative, rounding
    2^-20 of the loss / h: 1e-3 of the gradient's scale covers both)."""
    d = make(1, 70, 2, 16, 16, 1, "f32", 31)
    g = m2rnn.scan_bwd(*args(d), d["dy"], d["w_r"], d["H0"], d["dHT"], want_dH0=True)

    def loss(**kw):
        a = {**d, **kw}
        y, HT, _ = m2rnn.scan_fwd(*args(a), a["w_r"], a["H0"])
        return ((y.double() * d["dy"].double()).sum() + (HT.double() * d["dHT"].double()).sum()).item()

    h = 2.0 ** -7
    for name in ("q", "k", "v", "a", "alpha", "beta", "w_r", "H0"):
        t, gr = d[name], g["d" + name].reshape(-1)
        scale = gr.abs().max().item()
        for i in range(0, t.numel(), max(1, t.numel() // 9)):
            up, dn = t.clone(), t.clone()
            up.view(-1)[i] += h
            dn.view(-1)[i] -= h
            num = (loss(**{name: up}) - loss(**{name: dn})) / (2 * h)
            assert abs(num - gr[i].item()) <= 2e-2 * scale + 1e-4, (name, i, num, gr[i].item())


def test_shared_head_gradients(m2rnn):
    """dq, dk of a shared group are the sums of those with a group per head."""
    d = make(2, 100, 6, 32, 16, 1, "f32", 32)
    g = m2rnn.scan_bwd(*args(d), d["dy"], d["w_r"], d["H0"], d["dHT"])
    e = dict(d, q=d["q"].expand(-1, -1, 6, -1).contiguous(), k=d["k"].expand(-1, -1, 6, -1).contiguous())
    g6 = m2rnn.scan_bwd(*args(e), d["dy"], d["w_r"], d["H0"], d["dHT"])
    for n in ("dq", "dk"):
        assert rel(g[n][:, :, 0], g6[n].double().sum(2)) <= 1e-5, n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [-120.0, -80.0, 30.0, 200.0])
def test_backward_extreme_gates(m2rnn, dtype, shift):
    d = make(1, 150, 4, 64, 16, 1, dtype, 33)
    d["a"] = (d["a"].float() + shift).to(d["a"].dtype)
    d["a"][:, 50:60] = -math.inf  # padding: da = 0 there
    g = m2rnn.scan_bwd(*args(d), d["dy"], d["w_r"], d["H0"], d["dHT"], want_dH0=True)
    ref = plain(d, backward=True)
    assert all(t.isfinite().all() for t in g.values())
    assert not g["da"][:, 50:60].any()
    names = ("dq", "dv", "dw_r", "dH0") if shift < -100 else GRADS_OUT[:3] + ("dw_r", "dH0")
    check_grads(g, ref, dtype, names)  # (dt < 1e-38 has no normal fp32 value)


def test_padding_tokens_leave_the_state(m2rnn):
    """a = -inf: dt = 0, so the state passes through and y reads it."""
    d = make(1, 90, 4, 64, 16, 1, "f32", 6)
    d["a"][:, 40:80] = -math.inf
    y, HT, _ = m2rnn.scan_fwd(*args(d), d["w_r"], d["H0"])
    cut = {n: (t[:, list(range(40)) + list(range(80, 90))] if n in ("q", "k", "v", "a", "dy") else t)
           for n, t in d.items()}
    ref = plain(cut)
    assert rel(HT, ref["HT"]) <= FP32_REL and rel(y[:, 80:], ref["y"][:, 40:]) <= OUT_REL["f32"]
    assert y.isfinite().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [-80.0, 30.0, 200.0])
def test_extreme_gates(m2rnn, dtype, shift):
    """dt from 1e-30 to 200: no decay at all, and decays that vanish at once
    (the sum over a chunk reaches 10^5)."""
    d = make(1, 150, 4, 64, 16, 1, dtype, 7)
    d["a"] = (d["a"].float() + shift).to(d["a"].dtype)
    y, HT, _ = m2rnn.scan_fwd(*args(d), d["w_r"], d["H0"])
    ref = plain(d)
    assert y.isfinite().all() and HT.isfinite().all()
    assert rel(y, ref["y"]) <= OUT_REL[dtype] and rel(HT, ref["HT"]) <= FP32_REL


def test_split_sequence(m2rnn):
    """A sequence in two calls, the state carried."""
    d = make(2, 300, 4, 64, 32, 1, "f32", 8)
    y, HT, _ = m2rnn.scan_fwd(*args(d), d["w_r"], d["H0"])
    cut = 137
    y1, H1, _ = m2rnn.scan_fwd(*[t[:, :cut] for t in args(d)[:4]], *args(d)[4:], d["w_r"], d["H0"])
    y2, H2, _ = m2rnn.scan_fwd(*[t[:, cut:] for t in args(d)[:4]], *args(d)[4:], d["w_r"], H1)
    assert rel(torch.cat([y1, y2], 1), y.double()) <= 1e-5 and rel(H2, HT.double()) <= 1e-5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_sequence(m2rnn, dtype):
    """T = 20,000 with long retention (dt alpha ~ 1e-3): segments joined."""
    d = make(1, 20000, 2, 64, 16, 1, dtype, 9)
    d["alpha"] = torch.full_like(d["alpha"], 0.125)
    y, HT, _ = m2rnn.scan_fwd(*args(d), d["w_r"], d["H0"])
    ref = plain(d)
    assert rel(y, ref["y"]) <= OUT_REL[dtype] and rel(HT, ref["HT"]) <= FP32_REL


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sums_do_not_drift(m2rnn, dtype):
    """A state that hardly decays is a plain sum of many positive parts, where a
    rounding that always goes one way would add up.  912 head blocks: the whole
    sequence is one chain of chunks.

    Tolerance: a part (16 tokens' products, or with bf16 inputs a chunk's) is off
    by half of the last place 12 times at most, 12 * 2^-24 of itself; adding the
    T/16 = 32 parts rounds the sum so far, on average half of the final one, by
    2^-24 each time, in either direction: sqrt(32) / 2 * 2^-24.  Together < 15 * 2^-24 <
    9e-7; the step sizes' and decays' own errors (2^-22 of a step, in either
    direction over 512 tokens) add 2e-8."""
    B, T, N, K, V = 912, 512, 2, 16, 32
    g = torch.Generator(device="cuda").manual_seed(9)

    def ru(*s):
        return torch.rand(*s, generator=g, device="cuda").to(TD[dtype])
    q, k, v, a = ru(B, T, 1, K), ru(B, T, 1, K), ru(B, T, N, V), ru(B, T, N)
    alpha = torch.full((N,), 1e-3, device="cuda").to(TD[dtype])
    beta = torch.full((N,), -4.0, device="cuda").to(TD[dtype])
    H = m2rnn.scan_fwd(q, k, v, a, alpha, beta)[1]
    z = a.double() + beta.double()
    dt = torch.logaddexp(z, torch.zeros_like(z))
    tail = (dt.sum(1, keepdim=True) - dt.cumsum(1)) * -alpha.double()
    ref = torch.einsum("btn,btk,btnv->bnkv", torch.exp(tail) * dt, k[:, :, 0].double(), v.double())
    assert rel(H, ref) < 9e-7


def test_empty_sequence(m2rnn):
    d = make(2, 0, 4, 64, 16, 1, "bf16", 10)
    y, HT, _ = m2rnn.scan_fwd(*args(d), d["w_r"], d["H0"])
    assert y.shape == (2, 0, 4, 16) and torch.equal(HT, d["H0"])
    _, HT, _ = m2rnn.scan_fwd(*args(d), d["w_r"])
    assert not HT.any()
    g = m2rnn.scan_bwd(*args(d), d["dy"], d["w_r"], d["H0"], d["dHT"], want_dH0=True)
    assert torch.equal(g["dH0"], d["dHT"]) and not g["dalpha"].any() and not g["dw_r"].any()


def test_refusals(m2rnn):
    d = make(2, 8, 4, 64, 16, 1, "bf16", 11)

    def code(f):
        with pytest.raises(m2rnn.M2RNNError) as e:
            f()
        return e.value.code

    v24 = torch.zeros(2, 8, 4, 24, device="cuda").bfloat16()
    assert code(lambda: m2rnn.scan_fwd(d["q"], d["k"], v24, *args(d)[3:])) == -2
    odd = torch.zeros(2, 8, 1, 68, device="cuda").bfloat16()[..., :64]
    assert code(lambda: m2rnn.scan_fwd(odd, *args(d)[1:])) == -3
    assert code(lambda: m2rnn.scan_fwd(*args(d), workspace=torch.zeros(16, device="cuda").byte())) == -5
    big = torch.zeros(2, 4, 64, 16, device="cuda")
    s = [t[:, 0] for t in args(d)[:4]] + list(args(d)[4:])
    flat = torch.zeros(2 * 4 * 64 * 16 + 4, device="cuda")
    assert code(lambda: m2rnn.scan_step(*s, flat[:-4].view(2, 4, 64, 16),
                                        H_out=flat[4:].view(2, 4, 64, 16))) == -1
    with pytest.raises(TypeError):
        m2rnn.scan_fwd(d["q"].float(), *args(d)[1:])
    with pytest.raises(TypeError):
        m2rnn.scan_step(*s, big.bfloat16())
    with pytest.raises(ValueError):
        m2rnn.scan_fwd(d["q"].transpose(2, 3), *args(d)[1:])
    with pytest.raises(ValueError):
        m2rnn.scan_fwd(*args(d)[:3], d["a"][..., :3], *args(d)[4:])
