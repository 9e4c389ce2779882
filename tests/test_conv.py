"""The short causal convolution with SiLU (conv_fwd, conv_bwd, conv_step)
against a plain implementation in 64 bits on the same inputs.

Tolerances, derived: outputs in bf16 differ from the exact value by half an
ulp (2^-9 relative) plus the fp32 arithmetic before it; elementwise 2^-8 of
|exact| + 2^-8 of the row's scale covers values that cancel.  fp32: W + 1
fused multiply-adds (2^-24 each of the largest partial sum, at most the sum
of |terms|), expf (2 ulp) and one division: 2^-20 of the sum of |terms|.
Parameter gradients: n products summed in runs of fp32 (32 to 4,096 terms
each in order) and then over parts: 1e-5 relative L2.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

TD = {"bf16": torch.bfloat16, "f32": torch.float32}
ELEM = {"bf16": 2.0 ** -8, "f32": 2.0 ** -19}
PARAM_REL = 1e-5


@pytest.fixture(scope="module")
def m2rnn():
    import __graft_entry__
    __graft_entry__.build()
    from non_linear_matrix_gb300 import m2rnn as m
    m.use_library("normal")
    return m


def make(B, T, C, W, dtype, seed, pad=0):
    """Inputs; pad > 0 makes x a slice of rows C + pad wide."""
    g = torch.Generator().manual_seed(seed)
    td = TD[dtype]

    def rn(*s):
        return torch.randn(*s, generator=g).to(td).cuda()
    buf = rn(B, T, C + pad)
    return dict(x=buf[..., pad // 2:pad // 2 + C], w=rn(C, W), bias=rn(C), state=rn(B, W - 1, C),
                dy=rn(B, T, C), ds=rn(B, W - 1, C))


def plain(x, w, bias, state, silu, dy=None, ds=None):
    """64-bit forward, and gradients by torch's differentiation."""
    W, T = w.shape[1], x.shape[1]
    leaves = [t.double().requires_grad_(dy is not None) if t is not None else None
              for t in (x, w, bias, state)]
    x, w, bias, state = leaves
    if state is None:
        state = x.new_zeros(x.shape[0], W - 1, x.shape[2])
    f = torch.cat([state, x], 1)
    z = sum(w[:, i] * f[:, i:i + T] for i in range(W))
    if bias is not None:
        z = z + bias
    y = z * torch.sigmoid(z) if silu else z
    out = {"y": y, "state": f[:, T:]}
    if dy is not None:
        use = [t for t in leaves if t is not None]
        total = (y * dy.double()).sum()
        if ds is not None:
            total = total + (f[:, T:] * ds.double()).sum()
        gr = iter(torch.autograd.grad(total, use, allow_unused=True))
        for n, t in zip(("dx", "dw", "dbias", "dstate"), leaves):
            if t is not None:
                gg = next(gr)
                out[n] = torch.zeros_like(t) if gg is None else gg
    return {n: t.detach() for n, t in out.items()}


def close(got, ref, tol, label):
    if ref.numel() == 0:
        return
    scale = ref.abs() + ref.square().mean().sqrt()
    err = ((got.double() - ref).abs() / scale.clamp_min(1e-30)).max().item()
    assert err <= tol, (label, err)


def rel(got, ref):
    return ((got.double() - ref).norm() / ref.norm().clamp_min(1e-30)).item()


SHAPES = [(1, 1, 8, 4), (2, 2, 64, 4), (3, 3, 40, 4), (1, 5, 128, 2), (2, 33, 136, 3),
          (5, 127, 640, 4), (1, 700, 72, 4), (2, 64, 1152, 3)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,W", SHAPES)
def test_forward(m2rnn, B, T, C, W, dtype):
    for k, (silu, with_state, with_bias) in enumerate([(True, True, True), (False, True, False),
                                                       (True, False, True)]):
        d = make(B, T, C, W, dtype, 10 * T + k, pad=16 * k)
        bias = d["bias"] if with_bias else None
        state = d["state"] if with_state else None
        y, so = m2rnn.conv_fwd(d["x"], d["w"], bias, state, silu=silu)
        ref = plain(d["x"], d["w"], bias, state, silu)
        close(y, ref["y"], ELEM[dtype], "y")
        assert torch.equal(so.double(), ref["state"])  # copies of inputs


@pytest.mark.parametrize("dtype,gdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("B,T,C,W", SHAPES)
def test_backward(m2rnn, B, T, C, W, dtype, gdtype):
    for k, (silu, with_state, with_ds) in enumerate([(True, True, True), (False, False, False)]):
        d = make(B, T, C, W, dtype, 20 * T + k, pad=32 * k)
        state = d["state"] if with_state else None
        ds = d["ds"] if with_ds else None
        dy = d["dy"].to(TD[gdtype])
        g = m2rnn.conv_bwd(d["x"], d["w"], dy, d["bias"], state, ds, silu=silu,
                           want_dstate=with_state)
        ref = plain(d["x"], d["w"], d["bias"], state, silu, dy, ds)
        close(g["dx"], ref["dx"], ELEM[dtype], "dx")
        if with_state:
            close(g["dstate"], ref["dstate"], ELEM[dtype], "dstate")
        # bf16: the fast sigmoid's 2^-21 per product
        assert rel(g["dw"], ref["dw"]) <= PARAM_REL
        assert rel(g["dbias"], ref["dbias"]) <= PARAM_REL


def test_gradient_by_differences(m2rnn):
    """dx, dw, dbias, dstate of sum(y dy) + sum(state_out ds) against central
    differences of the forward kernel (fp32, step 2^-6: truncation
    h^2/6 |f'''| ~ 1e-4 of the derivative's scale, rounding 2^-22 / h ~ 2e-5)."""
    B, T, C, W = 2, 6, 8, 4
    d = make(B, T, C, W, "f32", 3)
    g = m2rnn.conv_bwd(d["x"], d["w"], d["dy"], d["bias"], d["state"], d["ds"], want_dstate=True)

    def loss(**kw):
        a = {**d, **kw}
        y, so = m2rnn.conv_fwd(a["x"].contiguous(), a["w"], a["bias"], a["state"])
        return ((y.double() * d["dy"].double()).sum() + (so.double() * d["ds"].double()).sum()).item()

    h = 2.0 ** -6
    for name, gname in (("x", "dx"), ("w", "dw"), ("bias", "dbias"), ("state", "dstate")):
        t, gr = d[name].contiguous(), g[gname].reshape(-1)
        for i in range(0, t.numel(), max(1, t.numel() // 12)):
            up, dn = t.clone(), t.clone()
            up.view(-1)[i] += h
            dn.view(-1)[i] -= h
            num = (loss(**{name: up}) - loss(**{name: dn})) / (2 * h)
            assert abs(num - gr[i].item()) <= 2e-3 * (1 + abs(num)), (name, i)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_steps_reproduce_the_prompt(m2rnn, W, dtype):
    """T single tokens, in place, give the prompt's y and state bit for bit
    (the same operations in the same order)."""
    B, T, C = 3, 9, 72
    d = make(B, T, C, W, dtype, 5)
    y, so = m2rnn.conv_fwd(d["x"], d["w"], d["bias"], d["state"])
    st = d["state"].clone()
    for t in range(T):
        yt, st2 = m2rnn.conv_step(d["x"][:, t], d["w"], st, d["bias"], state_out=st)
        assert st2 is st
        assert torch.equal(yt, y[:, t])
    assert torch.equal(st, so)


def test_split_sequence_equals_whole(m2rnn):
    d = make(2, 50, 64, 4, "bf16", 6)
    y, so = m2rnn.conv_fwd(d["x"], d["w"], d["bias"], d["state"])
    y1, s1 = m2rnn.conv_fwd(d["x"][:, :2], d["w"], d["bias"], d["state"])
    y2, s2 = m2rnn.conv_fwd(d["x"][:, 2:], d["w"], d["bias"], s1)
    assert torch.equal(torch.cat([y1, y2], 1), y) and torch.equal(s2, so)


def test_extremes(m2rnn):
    """SiLU at z = +-1e4 (exp overflows on one side): 0 and z; NaN stays in
    the rows that see it; the gradient there is 0 and 1."""
    C, W = 8, 2
    x = torch.zeros(1, 6, C, device="cuda")
    x[0, 1], x[0, 2] = -1e4, 1e4
    w = torch.tensor([[0.0, 1.0]] * C, device="cuda")
    y, _ = m2rnn.conv_fwd(x, w)
    assert torch.equal(y[0, 1].abs(), torch.zeros(C, device="cuda"))
    assert torch.equal(y[0, 2], x[0, 2])
    g = m2rnn.conv_bwd(x, w, torch.ones_like(x))
    assert torch.equal(g["dx"][0, 1].abs(), torch.zeros(C, device="cuda"))
    assert torch.equal(g["dx"][0, 2], torch.ones(C, device="cuda"))
    x[0, 3, 0] = float("nan")
    w[:, 0] = 0.5
    y, _ = m2rnn.conv_fwd(x, w)
    assert y[0, 3:5, 0].isnan().all() and not y[0, :3].isnan().any() and not y[0, 5].isnan().any()


def test_empty_sequence(m2rnn):
    B, C, W = 2, 16, 4
    d = make(B, 0, C, W, "f32", 7)
    y, so = m2rnn.conv_fwd(d["x"], d["w"], d["bias"], d["state"])
    assert y.shape == (B, 0, C) and torch.equal(so, d["state"])
    g = m2rnn.conv_bwd(d["x"], d["w"], d["dy"], d["bias"], d["state"], d["ds"], want_dstate=True)
    assert torch.equal(g["dstate"], d["ds"]) and not g["dw"].any() and not g["dbias"].any()


def test_deterministic_and_on_another_stream(m2rnn):
    d = make(4, 300, 640, 4, "bf16", 8)
    ref = m2rnn.conv_bwd(d["x"], d["w"], d["dy"], d["bias"], d["state"])
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    again = m2rnn.conv_bwd(d["x"], d["w"], d["dy"], d["bias"], d["state"], stream=st)
    st.synchronize()
    for n in ("dx", "dw", "dbias"):
        assert torch.equal(ref[n], again[n]), n


def test_refusals(m2rnn):
    d = make(2, 8, 64, 4, "bf16", 9)
    E = m2rnn.M2RNNError

    def code(f):
        with pytest.raises(E) as e:
            f()
        return e.value.code

    assert code(lambda: m2rnn.conv_fwd(d["x"][..., :12], d["w"][:12])) == -2        # C % 8
    assert code(lambda: m2rnn.conv_fwd(d["x"], torch.zeros(64, 5, device="cuda").bfloat16())) == -2
    assert code(lambda: m2rnn.conv_fwd(d["x"][..., 4:60], d["w"][:56])) == -3       # 8-byte offset
    odd = torch.zeros(2, 8, 68, device="cuda").bfloat16()[..., :64]                 # 136-byte rows
    assert code(lambda: m2rnn.conv_fwd(odd, d["w"])) == -3
    assert code(lambda: m2rnn.conv_fwd(d["x"], d["w"], state=d["state"],
                                       out={"state": d["state"]})) == -1            # overlap
    assert code(lambda: m2rnn.conv_bwd(d["x"], d["w"], d["dy"],
                                       workspace=torch.zeros(16, device="cuda").byte())) == -5
    with pytest.raises(TypeError):
        m2rnn.conv_fwd(d["x"], d["w"].float())
    with pytest.raises(TypeError):
        m2rnn.conv_bwd(d["x"], d["w"], d["dy"].half())
    with pytest.raises(ValueError):
        m2rnn.conv_fwd(d["x"].transpose(1, 2), torch.zeros(8, 4, device="cuda").bfloat16())
    with pytest.raises(ValueError):
        m2rnn.conv_fwd(d["x"].cpu(), d["w"])
