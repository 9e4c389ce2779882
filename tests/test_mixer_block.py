"""The block operators together, as examples/mixer_block.py uses them: single
tokens continue a prompt, and a training step's gradients follow the loss."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def mixer():
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location(
        "mixer_block", os.path.join(ROOT, "examples", "mixer_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.m2rnn.use_library("normal")
    return mod


@pytest.mark.parametrize("layer", ["scan", "m2rnn"])
@pytest.mark.parametrize("tokens", [1, 3, 70])
def test_single_tokens_continue_a_prompt(mixer, layer, tokens):
    """Two ways to the same outputs.  Between them lie the roundings of z, q',
    k' and y to bf16 (equal on both ways: the same operations) and of the
    scan's chunk weights (2^-9 of each); out sums N V = 128 such terms:
    2^-6 of the outputs' scale is four of them at once."""
    block = mixer.MixerBlock(layer, d=64, N=8, K=32, V=16, Nq=2)
    x = torch.randn(3, tokens + 4, 64, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    whole, _, _ = block.prompt(x)
    _, state, _ = block.prompt(x[:, :tokens])
    for i in range(4):
        out = block.step(x[:, tokens + i], state)
        ref = whole[:, tokens + i].float()
        assert (out.float() - ref).abs().max() <= 2.0 ** -6 * (1 + ref.abs().max())


@pytest.mark.parametrize("layer", ["scan", "m2rnn"])
def test_training_lowers_the_loss(mixer, layer):
    """Ten small steps along the gradients in fp32: the loss falls every time,
    and the first step's fall is the gradient's prediction within a quarter
    (second order in the step)."""
    block = mixer.MixerBlock(layer, d=64, N=4, K=32, V=16, dtype=torch.float32)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2, 90, 64, generator=g).cuda()
    target = torch.randn(2, 90, 64, generator=g).cuda()
    losses, predicted = [], None
    for i in range(10):
        out, _, kept = block.prompt(x, save=True)
        err = (out - target).double()
        losses.append(err.square().mean().item())
        grads = block.backward(kept, (2 * err / err.numel()).float())
        lr = 0.02
        if predicted is None:
            predicted = lr * sum(gr.double().square().sum().item() for gr in grads.values())
        for n, gr in grads.items():
            block.w[n].sub_(gr, alpha=lr)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    fall = losses[0] - losses[1]
    assert abs(fall - predicted) <= 0.25 * predicted, (fall, predicted)
