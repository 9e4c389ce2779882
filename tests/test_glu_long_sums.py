"""Long sums of the gated products' gradients with fp32 operands.

Sums of one sign over hundreds of thousands of tokens.  Within a chunk of 256 the tensor core cuts
its sums off, which takes about the same share of every sum; that share is not what is looked at
here.  What differs from sum to sum, the spread of the relative errors, comes from the
roundings to fp32 with which chunks are added.  One rounding is uniform in half a step, at most
2^-24: a standard deviation of 2^-24 / 3^(1/2) = 3.4e-8 of the running sum, which grows evenly:
  n adds in one run: (n / 3)^(1/2) 3.4e-8;  2,344 of them (600,000 tokens): 9.6e-7;
  runs of 128 that are added apart (19 of them): 2.2e-7 / 19^(1/2) and (19 / 3)^(1/2) 3.4e-8: 1.0e-7.
Chunks' own spread is that of 16 cut-off steps, below a third of the latter over so many chunks.
The bound, 3e-7, lies between the two."""
import ctypes

import pytest
import torch

from non_linear_matrix_gb300 import build as nb


@pytest.fixture(scope="module")
def m():
    nb.build()
    from non_linear_matrix_gb300 import m2rnn
    m2rnn.use_library("normal")
    return m2rnn


def test_few_tiles_are_cut_as_before(m):
    """Scratch of fp32 gradients: short sums and those of few tiles need what they needed, 600,000
    tokens at least 18 parts more of 80 tiles of 256 x 128."""
    need = lambda *s: m.lib().m2rnn_glu_bwd_workspace_size(ctypes.byref(m.GluShape(*s)))  # noqa: E731

    def fixed(M, D, F):  # terms of x, wg and wu, and of the gradients of g and u
        up = lambda n: (n + 255) // 256 * 256  # noqa: E731
        d, f = (D + 63) // 64 * 64, (F + 63) // 64 * 64
        return up(6 * M * d) + 2 * up(6 * F * d) + up(12 * M * f)
    assert need(1554, 520, 1400, 0, 0) - fixed(1554, 520, 1400) <= 76 * 2 * 256 * 128 * 4
    assert need(300_000, 64, 64, 0, 0) - fixed(300_000, 64, 64) <= 152 * 256 * 128 * 4
    assert need(600_000, 1280, 1024, 0, 0) - fixed(600_000, 1280, 1024) >= 19 * 80 * 256 * 128 * 4


@pytest.mark.gpu
@pytest.mark.parametrize("M,D,F", [(600_000, 1280, 1024), (600_000, 64, 72)])
def test_long_sums_in_fp32_do_not_drift(m, M, D, F):
    if torch.cuda.get_device_properties(0).total_memory < 64 << 30:
        pytest.skip("needs 30 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").abs_()  # noqa: E731
    x, dh, wg, wu = rn(M, D), rn(M, F), rn(F, D) * 0.05 * D ** -0.5, rn(F, D) * 0.05 * D ** -0.5
    got = m.glu_bwd(x, wg, wu, dh, want_dx=False)
    some = torch.arange(0, F, max(1, F // 16), device="cuda")  # of the features
    G, U = wg[some].double(), wu[some].double()
    ref = {"dwg": 0, "dwu": 0}
    for i in range(0, M, 50_000):
        X, H = x[i:i + 50_000].double(), dh[i:i + 50_000][:, some].double()
        a, u = X @ G.T, X @ U.T
        s = torch.sigmoid(a)
        ref["dwg"] = ref["dwg"] + (H * u * (s + a * s * (1 - s))).T @ X
        ref["dwu"] = ref["dwu"] + (H * a * s).T @ X
    for n in ref:
        e = (got[n][some].double() - ref[n]) / ref[n]
        assert e.std().item() <= 3e-7, (n, e.std().item(), e.mean().item())
        assert abs(e.mean().item()) <= 1.5e-6  # 16 steps that cut off 3.1 2^-24 of a growing sum, half of it
    assert m.device_status() == (0, 0)
