"""How the feed-forward operators are called: on another stream, captured into CUDA graphs
(two that share a workspace among them), back to back through the same scratch, and together
as examples/layer.py uses them."""
import contextlib
import importlib.util
import os
import types

import pytest
import torch

from non_linear_matrix_gb300 import m2rnn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ---- on the CPU: whose memory a call with stream= takes ------------------------------


class FakeTensor:
    """A contiguous CUDA tensor as far as the binding looks at one."""

    def __init__(self, shape, dtype, pool=None):
        self.shape, self.dtype, self.pool, self.used_on = torch.Size(shape), dtype, pool, []
        self.is_cuda, self.device = True, "cuda:0"

    def numel(self):
        return max(1, self.shape.numel())

    def dim(self):
        return len(self.shape)

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def get_device(self):
        return 0

    def record_stream(self, s):
        self.used_on.append(s)


class FakeStream:
    cuda_stream, device = 7, "cuda:0"


class FakeLib:
    def __getattr__(self, name):
        return lambda *a: 1 << 16 if name.endswith("_size") else 0


def calls():
    t = lambda *s, dtype=torch.bfloat16: FakeTensor(s, dtype)  # noqa: E731
    q = lambda *s: FakeTensor(s, torch.float8_e4m3fn)  # noqa: E731
    f = lambda *s: FakeTensor(s, torch.float32)  # noqa: E731
    x, w, W, h = t(2, 8, 64), t(64), t(72, 64), t(2, 8, 72)
    return {"add_norm_fwd": (x, x, w), "add_norm_q8": (x, x, w), "add_norm_bwd": (x, x, w, x), "quant_rows": (x,),
            "glu_fwd": (f(2, 8, 64), f(72, 64), f(72, 64)), "glu_bwd": (x, W, W, h),
            "glu_q8": (q(2, 8, 64), f(2, 8), q(72, 64), f(72), q(72, 64), f(72)),
            "linear_q8": (q(2, 8, 64), f(2, 8), q(72, 64), f(72), h)}


@pytest.mark.parametrize("name", sorted(calls()))
def test_allocations_are_the_launching_streams(monkeypatch, name):
    current, side, made = FakeStream(), FakeStream(), []
    now = [current]

    @contextlib.contextmanager
    def on(s):
        now.append(s)
        yield
        now.pop()

    def empty(*s, device=None, dtype=None):
        s = s[0] if len(s) == 1 and not isinstance(s[0], int) else s
        made.append(FakeTensor((s,) if isinstance(s, int) else s, dtype, now[-1]))
        return made[-1]
    monkeypatch.setattr(m2rnn, "lib", lambda: FakeLib())
    monkeypatch.setattr(m2rnn, "torch", types.SimpleNamespace(
        empty=empty, empty_like=lambda x: empty(x.shape, dtype=x.dtype), float32=torch.float32,
        bfloat16=torch.bfloat16, uint8=torch.uint8, int32=torch.int32, float8_e4m3fn=torch.float8_e4m3fn,
        cuda=types.SimpleNamespace(stream=on, current_stream=lambda *a: now[-1])))
    got = getattr(m2rnn, name)(*calls()[name], stream=side)
    assert made and all(x.pool is side for x in made)
    got = got.values() if isinstance(got, dict) else got if isinstance(got, tuple) else (got,)
    for x in got:
        assert x is None or x.used_on == [current]


# ---- on the GPU ------------------------------------------------------------------


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    m2rnn.use_library("normal")
    return m2rnn


def rn(seed, *s, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*s, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


def outputs(r):
    r = r.values() if isinstance(r, dict) else r if isinstance(r, (tuple, list)) else (r,)
    return [t for t in r if torch.is_tensor(t)]


def same(a, b):
    return len(a) == len(b) > 0 and all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


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
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [3, 300])
def test_captured(m, M, dtype):
    D, F = 136, 264
    x, res, w = rn(1, M, D, dtype=dtype), rn(2, M, D, dtype=dtype), rn(3, D, dtype=dtype)
    wg, wu, dh = rn(4, F, D, dtype=dtype), rn(5, F, D, dtype=dtype), rn(6, M, F, dtype=dtype)

    def call():
        y, r = m.add_norm_fwd(x, res, w)
        h = m.glu_fwd(y, wg, wu)
        g = m.glu_bwd(y, wg, wu, dh)
        n = m.add_norm_bwd(r, g["dx"], w, res)
        return [y, r, h] + outputs(g) + outputs(n)
    recorded(call, (x, res, dh), [rn(10 + i, *t.shape, dtype=dtype) for i, t in enumerate((x, res, dh))])


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 300])
def test_captured_in_8_bits(m, M):
    D, F = 144, 272
    (wg, gs), (wu, us), (wd, ds) = (m.quant_rows(rn(s, *sh)) for s, sh in ((1, (F, D)), (2, (F, D)), (3, (D, F))))
    x, res = rn(4, M, D), rn(5, M, D)

    def call():
        q, qs, r = m.add_norm_q8(x, res)
        hq, hs = m.quant_rows(m.glu_q8(q, qs, wg, gs, wu, us))
        return [q, qs, r, hq, hs, m.linear_q8(hq, hs, wd, ds, r)]
    recorded(call, (x, res), (rn(6, M, D), rn(7, M, D)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_two_graphs_share_a_workspace(m, dtype):
    """Replayed one after the other and interleaved with plain calls on one stream."""
    M, D, F = 300, 136, 264
    wg, wu = rn(1, F, D, dtype=dtype), rn(2, F, D, dtype=dtype)
    ins = [(rn(3 + i, M, D, dtype=dtype), rn(6 + i, M, F, dtype=dtype)) for i in range(2)]
    want = [outputs(m.glu_bwd(x, wg, wu, dh)) for x, dh in ins]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graphs, got = [], []
    for x, dh in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(outputs(m.glu_bwd(x, wg, wu, dh, workspace=ws)))
        graphs.append(g)
    for i in (0, 1, 1, 0, 0, 1):
        for t in got[i]:
            t.fill_(7)
        graphs[i].replay()
        plain = outputs(m.glu_bwd(*ins[1 - i][:1], wg, wu, ins[1 - i][1], workspace=ws))
        torch.cuda.synchronize()
        assert same(got[i], want[i]) and same(plain, want[1 - i])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_back_to_back_through_one_workspace(m, dtype):
    D, F = 264, 392
    wg, wu = rn(1, F, D, dtype=dtype), rn(2, F, D, dtype=dtype)
    w = rn(3, D, dtype=dtype)
    ins = [(rn(10 + i, M, D, dtype=dtype), rn(20 + i, M, F, dtype=dtype)) for i, M in enumerate((700, 80, 1300, 17, 300))]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def one(x, dh, **k):
        return outputs(m.glu_bwd(x, wg, wu, dh, **k)) + [m.glu_fwd(x, wg, wu, **k)] + outputs(m.add_norm_bwd(x, x, w, **k))
    want = []
    for x, dh in ins:
        want.append(one(x, dh))
        torch.cuda.synchronize()
    got = [one(x, dh, workspace=ws) for x, dh in ins]
    assert all(same(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_two_streams_at_once(m):
    """Calls on two streams that overlap: each kernel's waits are within its own grid."""
    D, F = 512, 1400
    wg, wu, w = rn(1, F, D, scale=0.05), rn(2, F, D, scale=0.05), rn(3, D)
    ins = [(rn(4 + i, 2500, D), rn(6 + i, 2500, F)) for i in range(2)]

    def one(x, dh, **k):
        y, r = m.add_norm_fwd(x, x, w, **k)
        return [y, r, m.glu_fwd(x, wg, wu, **k)] + outputs(m.glu_bwd(x, wg, wu, dh, **k)) + outputs(m.add_norm_bwd(x, x, w, **k))
    want = [one(*i) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [one(*i, stream=s) for i, s in zip(ins, streams)]
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))
    assert m.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["glu_fwd", "glu_bwd", "add_norm_bwd"])
def test_scratch_is_not_given_away(m, name):
    """The side stream waits (some milliseconds) in front of the call, so the call is still to
    run while the current stream fills new buffers of all sizes that the call may have had."""
    x, wg, dh, w = (rn(s, *sh, dtype=torch.float32) for s, sh in ((1, (300, 136)), (2, (264, 136)), (3, (300, 264)), (4, (136,))))
    call = {"glu_fwd": lambda **k: m.glu_fwd(x, wg, wg, **k), "glu_bwd": lambda **k: m.glu_bwd(x, wg, wg, dh, **k),
            "add_norm_bwd": lambda **k: m.add_norm_bwd(x, x, w, **k)}[name]
    want = outputs(call())
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)  # about 20 ms
    got = outputs(call(stream=side))
    fill = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in
            (1 << 12, 1 << 16, 1 << 18, 1 << 20, 1 << 21, 3 << 20, 1 << 22, 5 << 20, 1 << 23)]
    torch.cuda.synchronize()
    assert len(fill) == 9 and same(got, want)


# ---- the operators together ----------------------------------------------------------


@pytest.fixture(scope="module")
def layer(m):
    spec = importlib.util.spec_from_file_location("layer", os.path.join(ROOT, "examples", "layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.gpu
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("tokens", [1, 70])
def test_single_tokens_continue_a_prompt(layer, tokens, q8):
    """Two ways to the same outputs; between them lie the roundings of the mixer's
    output (2^-6 of its scale, as in the mixer's own test), of the sum, the norm and h to bf16,
    each at most a half step of another value's: four of them at once, and in 8 bits codes that
    fall on the other side of a step: 2^-4 of single terms of the products, of which D or F are
    summed (2^-4 of the outputs' scale)."""
    net = layer.Layer("scan", d=64, F=176, q8=q8, N=8, K=32, V=16, Nq=2)
    x = torch.randn(3, tokens + 3, 64, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    whole, _, _ = net.prompt(x)
    _, state, _ = net.prompt(x[:, :tokens])
    for i in range(3):
        out = net.step(x[:, tokens + i], state)
        ref = whole[:, tokens + i].float()
        assert (out.float() - ref).abs().max() <= 2.0 ** (-2 if q8 else -4) * (1 + ref.abs().max())


@pytest.mark.gpu
def test_gradients_against_differences(layer):
    """fp32: the slope of the loss along a direction of every weight of the feed-forward half
    (and of the mixer's output projection, which it reaches through the norm), by
    central differences of step 2^-7.  Rounding: 2^-20 of the sum of |out c| over the step; the
    third derivative along a direction a fifth of each weight's size: 2^-10 of that sum."""
    net = layer.Layer("scan", d=64, F=176, N=4, K=32, V=16, dtype=torch.float32)
    g = torch.Generator().manual_seed(3)
    x, c = torch.randn(2, 40, 64, generator=g).cuda(), torch.randn(2, 40, 64, generator=g).cuda()
    out, _, kept = net.prompt(x, save=True)
    grads = net.backward(kept, c)
    weights = net.weights()
    step = 2.0 ** -7
    for n in ("norm", "wg", "wu", "wd", "mixer.out"):
        w = weights[n]
        d = torch.randn(*w.shape, generator=g).cuda() * w.abs().mean() * 0.2
        at, old = [], w.clone()
        for k in (step, -step):
            w.copy_(old + k * d)
            at.append((net.prompt(x)[0].double() * c.double()).sum())
        w.copy_(old)
        size = (out.double() * c.double()).abs().sum()
        want = (grads[n].double() * d.double()).sum()
        assert abs((at[0] - at[1]) / (2 * step) - want) <= size * (2.0 ** -20 / step + 2.0 ** -10), n
