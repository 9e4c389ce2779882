"""How often glu_bwd rounds: once at every size, or, where the caller asks for it, the
gradients of g and u too.

Of values whose mantissas are spread evenly over an octave one rounding to bf16 leaves a
relative 2-norm of about 1.66e-3, two independent ones 2.35e-3.  Outputs of the sizes here
scatter by less than a tenth, and the sums' own errors are below 1e-4: 1.95e-3 tells the two apart,
and 2.6e-3 is a tenth above the latter."""
import ctypes

import pytest
import torch

from non_linear_matrix_gb300 import build as nb

ROUND = 16  # M2RNN_GLU_ROUND


@pytest.fixture(scope="module")
def m():
    nb.build()
    from non_linear_matrix_gb300 import m2rnn
    m2rnn.use_library("normal")
    return m2rnn


def shape(m, *s):
    return ctypes.byref(m.GluShape(*s))


def test_the_flag(m):
    """Sizes and refusals, on the host."""
    L = m.lib()
    A = [ctypes.c_void_p((i + 1) << 40) for i in range(8)]
    bwd = lambda s: L.m2rnn_glu_bwd(s, A[0], 72, A[1], A[2], A[3], A[4], A[5], A[6], A[7], 1 << 50, None)  # noqa: E731
    assert m.M2RNN_GLU_ROUND == ROUND
    for act in (ROUND, ROUND | 1):
        assert bwd(shape(m, 4, 72, 64, 0, act)) == -1  # fp32
    for act in (2, ROUND | 2, 2 * ROUND, -1):
        assert bwd(shape(m, 4, 72, 64, 1, act)) == -1
    # two planes or one of each gradient, of M x F (rows of whole 128 bytes), at any size
    size = lambda *s: L.m2rnn_glu_bwd_workspace_size(shape(m, *s))  # noqa: E731
    for M, D, F in ((40, 72, 64), (1024, 1024, 1024), (1025, 1024, 1024), (32768, 1024, 2816)):
        one, two = size(M, D, F, 1, ROUND), size(M, D, F, 1, 0)
        assert one >= 4 * M * F and two >= 8 * M * F and two - one >= 4 * M * F - (64 << 20)
        assert size(M, D, F, 0, ROUND) == 0
        assert L.m2rnn_glu_fwd_workspace_size(shape(m, M, D, F, 1, ROUND)) == 0


def rn(seed, *s, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*s, generator=g, device="cuda") * scale).bfloat16()


def case(M, D, F, act="silu"):
    x, wg, wu, dh = rn(1, M, D), rn(2, F, D, scale=D ** -0.5), rn(3, F, D, scale=D ** -0.5), rn(4, M, F)
    ref = {"dx": [], "dwg": 0, "dwu": 0}
    G, U = wg.double(), wu.double()
    for i in range(0, M, 8192):
        X, H = x[i:i + 8192].double(), dh[i:i + 8192].double()
        g, u = X @ G.T, X @ U.T
        leaf = g.requires_grad_()
        a = torch.nn.functional.silu(leaf) if act == "silu" else torch.nn.functional.gelu(leaf, approximate="tanh")
        da, = torch.autograd.grad(a.sum(), leaf)
        dg, du = H * u * da, H * a.detach()
        ref["dx"].append(dg @ G + du @ U)
        ref["dwg"], ref["dwu"] = ref["dwg"] + dg.T @ X, ref["dwu"] + du.T @ X
    ref["dx"] = torch.cat(ref["dx"])
    return (x, wg, wu, dh), ref


def off(got, ref):
    return {n: ((got[n].double() - ref[n]).norm() / ref[n].norm()).item() for n in ref}


# both sides of M D F = 2^30, chains of sums over 512 K tiles in dw (M) and dx (F), odd sizes
SIZES = [(3, 432, 96), (1023, 1024, 1024), (1024, 1024, 1024), (1025, 1024, 1024), (20000, 264, 1416), (4097, 1024, 4104),
         (40001, 264, 520), (601, 264, 9000)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,D,F", SIZES)
def test_gradients_are_rounded_once_at_every_size(m, M, D, F):
    args, ref = case(M, D, F)
    for n, e in off(m.glu_bwd(*args), ref).items():
        assert e <= 1.95e-3, (n, e)
    assert m.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,D,F", [(3, 432, 96), (1500, 264, 1416), (20000, 264, 1416), (40001, 264, 520)])
def test_rounded_between_where_the_caller_asks(m, M, D, F, act):
    args, ref = case(M, D, F, act)
    got = m.glu_bwd(*args, act=act, round_between=True)
    for n, e in off(got, ref).items():
        assert e <= 2.6e-3, (n, e)
    need = m.lib().m2rnn_glu_bwd_workspace_size(shape(m, M, D, F, 1, ROUND | (act == "gelu")))
    ws = torch.full((need + 512,), 165, dtype=torch.uint8, device="cuda")  # exactly what is asked for, and a guard
    again = m.glu_bwd(*args, act=act, round_between=True, workspace=ws[:need])
    assert all(torch.equal(again[n], got[n]) for n in got) and (ws[need:] == 165).all()
    with pytest.raises(m.M2RNNError) as e:
        m.glu_bwd(*args, act=act, round_between=True, workspace=ws[:need - 1])
    assert e.value.code == -5
    with pytest.raises(m.M2RNNError) as e:
        m.glu_bwd(*(t.float() for t in args), act=act, round_between=True)
    assert e.value.code == -1
    assert m.device_status() == (0, 0)
