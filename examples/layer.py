"""One layer on the package's operators: a mixer block (examples/mixer_block.py) and the
feed-forward half behind it, with the residual stream between them: a prompt, single
tokens that continue it, a training step, and the feed-forward half in 8 bits.

    o = mixer(x)
    y, r = add_norm(o, x)                 the stream r = x + o, and its norm
    h = act(y wg^T) (.) (y wu^T)          glu_fwd
    out = h wd^T + r

In 8 bits (q8=True, no gradients) y and h are e4m3 codes with a scale per token, the weights
codes with a scale per row: add_norm_q8, glu_q8, quant_rows, linear_q8, which adds r.

    python examples/layer.py [--layer scan|m2rnn] [--q8] [--tokens T] [--steps S]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from mixer_block import EPS, MixerBlock  # noqa: E402

from non_linear_matrix_gb300 import m2rnn  # noqa: E402


class Layer:
    """``layer``, and what a MixerBlock takes besides; F the feed-forward's width."""

    def __init__(self, layer="scan", d=512, F=1408, q8=False, dtype=torch.bfloat16, seed=0, **mixer):
        self.mixer = MixerBlock(layer, d=d, dtype=dtype, seed=seed, **mixer)
        g = torch.Generator().manual_seed(seed + 1)

        def rn(*s):
            return (torch.randn(*s, generator=g) * s[-1] ** -0.5).to(dtype).cuda()
        self.w = {"norm": torch.ones(d).to(dtype).cuda(), "wg": rn(F, d), "wu": rn(F, d), "wd": rn(d, F)}
        # laid out once: codes and scales of the weights' rows
        self.w8 = {n: m2rnn.quant_rows(self.w[n]) for n in ("wg", "wu", "wd")} if q8 else None

    def weights(self):
        return {**self.w, **{"mixer." + n: t for n, t in self.mixer.w.items()}}

    def half(self, o, x):
        """The feed-forward half: (out, what backward needs)."""
        if self.w8:
            q, s, r = m2rnn.add_norm_q8(o, x, self.w["norm"], EPS)
            h, hs = m2rnn.quant_rows(m2rnn.glu_q8(q, s, *self.w8["wg"], *self.w8["wu"]))
            return m2rnn.linear_q8(h, hs, *self.w8["wd"], r, out={"y": r}), None  # the stream in place
        y, r = m2rnn.add_norm_fwd(o, x, self.w["norm"], EPS)
        h = m2rnn.glu_fwd(y, self.w["wg"], self.w["wu"])
        return h @ self.w["wd"].T + r, (y, r, h)

    def prompt(self, x, save=False):
        """x [B,T,d] -> (out [B,T,d], decode state, what backward needs)."""
        o, state, kept = self.mixer.prompt(x, save=save)
        out, mine = self.half(o, x)
        return out, state, (kept, mine)

    def step(self, x, state):
        """One token: x [B,d] -> out [B,d]; the state is updated in place."""
        return self.half(self.mixer.step(x, state), x)[0]

    def backward(self, kept, dout):
        """Gradients of every weight for dL/dout, from what ``prompt(save=True)`` kept."""
        w, (mixer, (y, r, h)) = self.w, kept
        g = m2rnn.glu_bwd(y, w["wg"], w["wu"], dout @ w["wd"])
        n = m2rnn.add_norm_bwd(r, g["dx"], w["norm"], dout, EPS)  # dout reaches r past the norm too
        grads = {"mixer." + k: t for k, t in self.mixer.backward(mixer, n["dx"]).items()}
        grads.update(norm=n["dw"], wg=g["dwg"], wu=g["dwu"],
                     wd=dout.flatten(0, -2).T @ h.flatten(0, -2))
        return grads


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layer", choices=("scan", "m2rnn"), default="scan")
    ap.add_argument("--q8", action="store_true")
    ap.add_argument("--batch", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    net = Layer(a.layer, q8=a.q8)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(a.batch, a.tokens + a.steps, 512, generator=g).bfloat16().cuda()
    whole, _, _ = net.prompt(x)
    _, state, _ = net.prompt(x[:, :a.tokens])
    worst = 0.0
    for i in range(a.steps):
        out = net.step(x[:, a.tokens + i], state)
        worst = max(worst, (out.float() - whole[:, a.tokens + i].float()).abs().max().item())
    print(f"{a.layer}: {a.tokens}-token prompt, {a.steps} single tokens; against one prompt of "
          f"{a.tokens + a.steps}: max difference {worst:.3g}")
    if not a.q8:
        target = torch.randn(a.batch, a.tokens, 512, generator=g).bfloat16().cuda()
        weights = net.weights()
        for i in range(3):
            out, _, kept = net.prompt(x[:, :a.tokens], save=True)
            err = out.float() - target.float()
            for n, gr in net.backward(kept, (2 * err / err.numel()).bfloat16()).items():
                weights[n].sub_(gr.to(weights[n].dtype), alpha=1.0)
            print(f"training step {i}: loss {err.square().mean().item():.5f}")
    st, detail = m2rnn.device_status()
    assert st == 0, (st, detail)


if __name__ == "__main__":
    main()
