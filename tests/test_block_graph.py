"""The block operators recorded into a CUDA graph: a replay on new inputs gives
the bits of the plain calls."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    from non_linear_matrix_gb300 import m2rnn
    m2rnn.use_library("normal")
    return m2rnn


def rn(*s, seed=0, dtype=torch.bfloat16):
    return torch.randn(*s, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def outputs(r):
    r = r.values() if isinstance(r, dict) else r
    return [t for t in r if torch.is_tensor(t)]


def bits(t):
    return t.view(torch.int16 if t.dtype is torch.bfloat16 else torch.int32)


def recorded(call, inputs, fresh):
    """call() with `inputs` filled from `fresh`: by itself, then by a graph that was
    recorded on other values."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = outputs(call())
    for x, y in zip(inputs, fresh):
        x.copy_(y)
    want = [t.clone() for t in outputs(call())]
    graph.replay()
    torch.cuda.synchronize()
    assert len(got) == len(want) > 0
    for a, b in zip(got, want):
        assert torch.equal(bits(a), bits(b))


def test_single_token(m):
    B, N, K, V, W = 5, 4, 64, 16, 4
    C = 2 * K + N * V
    w, state = rn(C, W, seed=1), rn(B, W - 1, C, seed=2)
    par = [rn(N, seed=s) for s in (3, 4)]
    ang = rn(32, K // 2, seed=5, dtype=torch.float32)
    cos, sin = ang.cos(), ang.sin()
    pos = torch.full((B, 1), 7, dtype=torch.int32, device="cuda")
    x, a, H = rn(B, C, seed=6), rn(B, N, seed=7), rn(B, N, K, V, seed=8, dtype=torch.float32)

    def token():
        y, st = m.conv_step(x, w, state)
        q, k = m.qk_norm_fwd(y[:, None, None, :K], y[:, None, None, K:2 * K], cos=cos, sin=sin, pos=pos)
        return m.scan_step(q[:, 0], k[:, 0], y[:, 2 * K:].unflatten(1, (N, V)), a, *par, H) + (st,)
    recorded(token, (x, a, H), (rn(B, C, seed=9), rn(B, N, seed=10), H * 0.5))


def test_sequence_and_gradients(m):
    B, T, N, K, V, W = 2, 150, 4, 64, 16, 4
    x, w, dx = rn(B, T, 72, seed=1), rn(72, W, seed=2), rn(B, T, 72, seed=3)
    q, k, v = rn(B, T, 1, K, seed=4), rn(B, T, 1, K, seed=5), rn(B, T, N, V, seed=6)
    a, dy, w_r = rn(B, T, N, seed=7), rn(B, T, N, V, seed=8), rn(N, V, seed=9)
    par = [rn(N, seed=s) for s in (10, 11)]

    def conv():
        return outputs(m.conv_fwd(x, w)) + outputs(m.conv_bwd(x, w, dx))

    def norm():
        return outputs(m.qk_norm_fwd(q, k)) + outputs(m.qk_norm_bwd(q, k, None, None, q, k))

    def scan():
        y, HT, saved = m.scan_fwd(q * 0.1, k * 0.1, v, a, *par, w_r)
        return [y, HT] + outputs(m.scan_bwd(q * 0.1, k * 0.1, v, a, *par, dy, w_r))
    fresh = lambda t, s: rn(*t.shape, seed=s)  # noqa: E731
    recorded(conv, (x, dx), (fresh(x, 20), fresh(dx, 21)))
    recorded(norm, (q, k), (fresh(q, 22), fresh(k, 23)))
    recorded(scan, (v, a, dy), (fresh(v, 24), fresh(a, 25), fresh(dy, 26)))
