"""Features that the rotation leaves alone (the first R of K turn): an infinity
there stays in its own feature."""
import math

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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("feature", [17, 30])
def test_infinity_behind_the_rotated_features(m, dtype, interleaved, feature):
    """x = inf: r = 0, so the row is 0 but for the feature itself (0 times inf)."""
    g = torch.Generator().manual_seed(1)
    q = torch.randn(2, 3, 2, 32, generator=g).to(dtype).cuda()
    q[1, 1, 1, feature] = math.inf
    ang = torch.randn(8, 8, generator=g).cuda()
    qo, _ = m.qk_norm_fwd(q, None, cos=ang.cos(), sin=ang.sin(), interleaved=interleaved)
    row = qo[1, 1, 1]
    rest = torch.arange(32, device="cuda") != feature
    assert row[feature].isnan() and not row[rest].any()
    assert qo[0].isfinite().all() and qo[1, 0].isfinite().all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_weight_gradients_keep_to_their_feature(m, dtype, interleaved):
    """An infinite gradient of one feature that does not turn: dw is not finite there,
    and finite for every other feature."""
    g = torch.Generator().manual_seed(2)
    q, d = (torch.randn(1, 3, 2, 32, generator=g).to(dtype).cuda() for _ in range(2))
    d[0, 1, 0, 20] = math.inf
    w = torch.ones(32, dtype=dtype, device="cuda")
    ang = torch.randn(8, 8, generator=g).cuda()
    dw = m.qk_norm_bwd(q, None, w, None, d, None, cos=ang.cos(), sin=ang.sin(),
                       interleaved=interleaved)["dwq"]
    rest = torch.arange(32, device="cuda") != 20
    assert not dw[20].isfinite() and dw[rest].isfinite().all()
