"""The block operators under the checked build (every computed global index
tested against its array) and between guard regions: on ragged shapes the
status word stays clean, the results are the normal build's bit for bit, no
guard and no input changes."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

GUARD, SENTINEL = 64, -7.25e33


@pytest.fixture(scope="module")
def m2rnn():
    import __graft_entry__
    __graft_entry__.build()
    from non_linear_matrix_gb300 import build as b
    b.build(checked=True)
    from non_linear_matrix_gb300 import m2rnn as m
    m.use_library("normal")
    yield m
    m.use_library("normal")


class Guarded:
    """Buffers with sentinel values before and behind."""

    def __init__(self):
        self.bufs = []

    def __call__(self, shape, dtype=torch.float32):
        n = math.prod(shape)
        g = GUARD * 4 // torch.tensor([], dtype=dtype).element_size()
        buf = torch.full((n + 2 * g,), SENTINEL if dtype != torch.uint8 else 165, dtype=dtype,
                         device="cuda")
        self.bufs.append((buf, g, n))
        return buf[g:g + n].view(*shape)

    def check(self):
        torch.cuda.synchronize()
        for buf, g, n in self.bufs:
            assert torch.equal(buf[:g], torch.full_like(buf[:g], buf[0].item()))
            assert torch.equal(buf[g + n:], torch.full_like(buf[g + n:], buf[0].item()))
            assert buf[0].item() == (torch.tensor(SENTINEL, dtype=buf.dtype).item()
                                     if buf.dtype != torch.uint8 else 165)


def _both(m2rnn, inputs, run):
    """run(Guarded) -> dict under both builds."""
    copies = {n: t.clone() for n, t in inputs.items() if t is not None}
    res = []
    for which in ("normal", "checked"):
        m2rnn.use_library(which)
        try:
            assert m2rnn.lib().m2rnn_checked() == (which == "checked")
            m2rnn.device_status(clear=True)
            gd = Guarded()
            res.append(run(gd))
            gd.check()
            assert m2rnn.device_status(clear=True) == (0, 0)
        finally:
            m2rnn.use_library("normal")
    for n, t in copies.items():
        assert torch.equal(t, inputs[n]), n
    for n, t in res[0].items():
        if t is not None:
            assert torch.equal(t, res[1][n]), n


TD = {"bf16": torch.bfloat16, "f32": torch.float32}


def _rn(seed, td):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g).to(td).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,W", [(1, 1, 8, 4), (3, 37, 136, 4), (2, 5, 40, 2), (1, 301, 200, 3)])
def test_conv(m2rnn, B, T, C, W, dtype):
    td = TD[dtype]
    rn = _rn(T + C, td)
    buf = rn(B, T, C + 16)
    d = dict(buf=buf, w=rn(C, W), bias=rn(C), state=rn(B, W - 1, C), dy=rn(B, T, C), ds=rn(B, W - 1, C))
    x = buf[..., 8:8 + C]

    def run(gd):
        y, so = m2rnn.conv_fwd(x, d["w"], d["bias"], d["state"],
                               out={"y": gd((B, T, C), td), "state": gd((B, W - 1, C), td)})
        out = {"dx": gd((B, T, C), td), "dw": gd((C, W)), "dbias": gd((C,)),
               "dstate": gd((B, W - 1, C), td)}
        ws = gd((1 << 22,), torch.uint8)
        g = m2rnn.conv_bwd(x, d["w"], d["dy"], d["bias"], d["state"], d["ds"], out=out, workspace=ws)
        y1, s1 = m2rnn.conv_step(x[:, 0], d["w"], d["state"], d["bias"], y=gd((B, C), td),
                                 state_out=gd((B, W - 1, C), td))
        return {"y": y, "so": so, **g, "y1": y1, "s1": s1}

    _both(m2rnn, d, run)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,Nq,Nk,K,R", [(1, 1, 1, 1, 16, 16), (2, 37, 3, 2, 64, 32), (1, 9, 5, 0, 104, 24),
                                           (3, 21, 2, 1, 256, 256)])
def test_qk_norm(m2rnn, B, T, Nq, Nk, K, R, dtype):
    td = TD[dtype]
    rn = _rn(T + K, td)
    buf = rn(B, T, (Nq + Nk) * K + 8)
    d = dict(buf=buf, wq=rn(K), wk=rn(K) if Nk else None, dqo=rn(B, T, Nq, K),
             dko=rn(B, T, Nk, K) if Nk else None, cos=rn(40, R // 2).float(), sin=rn(40, R // 2).float(),
             pos=torch.randint(0, 40, (B, T), dtype=torch.int32).cuda())
    q = buf[..., :Nq * K].unflatten(-1, (Nq, K))
    k = buf[..., Nq * K:(Nq + Nk) * K].unflatten(-1, (Nk, K)) if Nk else None

    def run(gd):
        rot = dict(cos=d["cos"], sin=d["sin"], pos=d["pos"], interleaved=T % 2 == 0)
        out = {"q": gd((B, T, Nq, K), td)}
        grads = {"dq": gd((B, T, Nq, K), td), "dwq": gd((K,))}
        if Nk:
            out["k"] = gd((B, T, Nk, K), td)
            grads.update(dk=gd((B, T, Nk, K), td), dwk=gd((K,)))
        qo, ko = m2rnn.qk_norm_fwd(q, k, d["wq"], d["wk"], 1e-6, out=out, **rot)
        g = m2rnn.qk_norm_bwd(q, k, d["wq"], d["wk"], d["dqo"], d["dko"], 1e-6, out=grads,
                              workspace=gd((1 << 22,), torch.uint8), **rot)
        return {"q": qo, "k": ko, **g}

    _both(m2rnn, d, run)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,N,K,V,Nq", [(1, 1, 1, 16, 16, 1), (2, 130, 5, 64, 16, 1), (1, 333, 6, 128, 32, 2),
                                          (3, 64, 7, 32, 16, 7), (1, 700, 2, 64, 32, 1)])
def test_scan(m2rnn, B, T, N, K, V, Nq, dtype):
    td = TD[dtype]
    rn = _rn(T + K, td)
    wide = 2 * Nq * K + N * V
    buf = rn(B, T, wide + 8)
    d = dict(buf=buf, a=rn(B, T, N), alpha=rn(N).abs(), beta=rn(N) - 3, w_r=rn(N, V),
             dy=rn(B, T, N, V), H0=rn(B, N, K, V).float(), dHT=rn(B, N, K, V).float())
    q = buf[..., :Nq * K].unflatten(-1, (Nq, K))
    k = buf[..., Nq * K:2 * Nq * K].unflatten(-1, (Nq, K))
    v = buf[..., 2 * Nq * K:wide].unflatten(-1, (N, V))
    args = (q, k, v, d["a"], d["alpha"], d["beta"])
    st = (B, N, K, V)

    def run(gd):
        ws = gd((64 << 20,), torch.uint8)
        y, HT, saved = m2rnn.scan_fwd(*args, d["w_r"], d["H0"], workspace=ws,
                                      out={"y": gd((B, T, N, V), td), "HT": gd(st),
                                           "saved": gd((32 << 20,), torch.uint8)})
        res = {"y": y, "HT": HT}
        for n, kept in (("a", saved), ("b", None)):
            out = {"dq": gd((B, T, Nq, K), td), "dk": gd((B, T, Nq, K), td), "dv": gd((B, T, N, V), td),
                   "da": gd((B, T, N), td), "dalpha": gd((N,)), "dbeta": gd((N,)), "dw_r": gd((N, V)),
                   "dH0": gd(st)}
            g = m2rnn.scan_bwd(*args, d["dy"], d["w_r"], d["H0"], d["dHT"], saved=kept, out=out,
                               workspace=ws)
            res.update({n + m: t for m, t in g.items()})
        y1, H1 = m2rnn.scan_step(*[t[:, 0] for t in args[:4]], *args[4:], d["H0"], d["w_r"],
                                 H_out=gd(st), y=gd((B, N, V), td))
        return {**res, "y1": y1, "H1": H1}

    _both(m2rnn, d, run)
