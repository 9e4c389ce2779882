"""One mixer block on the package's operators: a prompt, single tokens that
continue it, and a training step.

    x -> projection -> [q | k | v] -> short causal convolution + SiLU (conv_*)
      -> norm of q and k with the position rotation (qk_norm_*)
      -> the layer: the selective scan (scan_*) or the M2RNN recurrence
         (fwd_gated, decode_gated, bwd_gated)
      -> projection back

q, k and v stay slices of one [B,T,C] buffer: the operators take row strides.

    python examples/mixer_block.py [--layer scan|m2rnn] [--tokens T] [--steps S]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from non_linear_matrix_gb300 import m2rnn  # noqa: E402

EPS = 1e-6


class MixerBlock:
    """Weights and the two ways through the block.  ``layer`` is "scan" or
    "m2rnn"; d model width, N value heads of V columns sharing Nq query/key
    groups of K features, W taps."""

    def __init__(self, layer="scan", d=512, N=32, K=64, V=16, Nq=1, W=4, positions=4096,
                 dtype=torch.bfloat16, seed=0):
        g = torch.Generator().manual_seed(seed)

        def rn(*s, scale=1.0):
            return (torch.randn(*s, generator=g) * scale).to(dtype).cuda()
        self.layer, self.N, self.K, self.V, self.Nq, self.W = layer, N, K, V, Nq, W
        self.C = 2 * Nq * K + N * V  # convolved channels: q | k | v
        self.w = {
            "in": rn(d, self.C, scale=d ** -0.5), "gate": rn(d, N, scale=d ** -0.5),
            "out": rn(N * V, d, scale=(N * V) ** -0.5),
            "conv": rn(self.C, W, scale=W ** -0.5), "conv_bias": rn(self.C, scale=0.1),
            # the L2 norm: RMS norm times K^-1/2
            "wq": torch.full((K,), K ** -0.5).to(dtype).cuda(),
            "wk": torch.full((K,), K ** -0.5).to(dtype).cuda(),
            "alpha": (torch.rand(N, generator=g) * 3 + 0.5).to(dtype).cuda(),
            "beta": rn(N, scale=0.5) - 3.0, "w_r": rn(N, V),
            "W": rn(N, V, V, scale=V ** -0.5),
        }
        inv = 10000.0 ** (-torch.arange(0, K, 2, dtype=torch.float64) / K)
        ang = torch.arange(positions, dtype=torch.float64)[:, None] * inv
        self.cos, self.sin = ang.cos().float().cuda(), ang.sin().float().cuda()

    def split(self, z):
        """[..., C] -> q, k [..., Nq, K] and v [..., N, V], as views."""
        n = self.Nq * self.K
        return (z[..., :n].unflatten(-1, (self.Nq, self.K)),
                z[..., n:2 * n].unflatten(-1, (self.Nq, self.K)),
                z[..., 2 * n:].unflatten(-1, (self.N, self.V)))

    def prompt(self, x, save=False):
        """x [B,T,d] -> (out [B,T,d], decode state, what backward needs)."""
        w = self.w
        p, a = x @ w["in"], x @ w["gate"]
        z, conv_state = m2rnn.conv_fwd(p, w["conv"], w["conv_bias"])
        q, k, v = self.split(z)
        qn, kn = m2rnn.qk_norm_fwd(q, k, w["wq"], w["wk"], EPS, cos=self.cos, sin=self.sin)
        if self.layer == "scan":
            y, H, saved = m2rnn.scan_fwd(qn, kn, v, a, w["alpha"], w["beta"], w["w_r"], save=save)
        else:
            v = v.contiguous()
            y, H, saved = m2rnn.fwd_gated(qn, kn, v, a, w["alpha"], w["beta"], w["W"], w["w_r"],
                                          ckpt_every=64 if save else 0)
        out = y.flatten(2) @ w["out"]
        return out, {"conv": conv_state, "H": H, "pos": x.shape[1]}, (x, p, a, z, qn, kn, v, y, saved)

    def step(self, x, state):
        """One token: x [B,d] -> out [B,d]; the state is updated in place."""
        w = self.w
        p, a = x @ w["in"], x @ w["gate"]
        z, _ = m2rnn.conv_step(p, w["conv"], state["conv"], w["conv_bias"], state_out=state["conv"])
        q, k, v = self.split(z)
        pos = torch.full((x.shape[0], 1), state["pos"], dtype=torch.int32, device=x.device)
        qn, kn = m2rnn.qk_norm_fwd(q[:, None], k[:, None], w["wq"], w["wk"], EPS, cos=self.cos,
                                   sin=self.sin, pos=pos)
        if self.layer == "scan":
            y, _ = m2rnn.scan_step(qn[:, 0], kn[:, 0], v, a, w["alpha"], w["beta"], state["H"],
                                   w["w_r"], H_out=state["H"])
        else:
            y, _ = m2rnn.decode_gated(qn[:, 0].contiguous(), kn[:, 0].contiguous(), v.contiguous(), a,
                                      w["alpha"], w["beta"], w["W"], w["w_r"], state["H"],
                                      H_out=state["H"])
        state["pos"] += 1
        return y.flatten(1) @ w["out"]

    def backward(self, kept, dout):
        """Gradients of every weight for dL/dout, from what ``prompt(save=True)`` kept."""
        w, (x, p, a, z, qn, kn, v, y, saved) = self.w, kept
        td = x.dtype
        q, k, vz = self.split(z)
        dy = (dout @ w["out"].T).unflatten(-1, (self.N, self.V)).contiguous()
        if self.layer == "scan":
            g = m2rnn.scan_bwd(qn, kn, vz, a, w["alpha"], w["beta"], dy, w["w_r"], saved=saved)
        else:
            g = m2rnn.bwd_gated(qn, kn, v, a, w["alpha"], w["beta"], w["W"], w["w_r"], dy, ckpt=saved,
                                ckpt_every=64)
        n = m2rnn.qk_norm_bwd(q, k, w["wq"], w["wk"], g["dq"], g["dk"], EPS, cos=self.cos,
                              sin=self.sin)
        dz = torch.cat([n["dq"].flatten(2), n["dk"].flatten(2), g["dv"].flatten(2).to(td)], -1)
        c = m2rnn.conv_bwd(p, w["conv"], dz, w["conv_bias"])
        grads = {"in": x.flatten(0, 1).T @ c["dx"].flatten(0, 1),
                 "gate": x.flatten(0, 1).T @ g["da"].flatten(0, 1).to(td),
                 "out": y.flatten(2).flatten(0, 1).T @ dout.flatten(0, 1),
                 "conv": c["dw"], "conv_bias": c["dbias"], "wq": n["dwq"], "wk": n["dwk"],
                 "alpha": g["dalpha"], "beta": g["dbeta"], "w_r": g["dw_r"]}
        if self.layer == "m2rnn":
            grads["W"] = g["dW"]
        return grads


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layer", choices=("scan", "m2rnn"), default="scan")
    ap.add_argument("--batch", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    block = MixerBlock(a.layer)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(a.batch, a.tokens + a.steps, 512, generator=g).bfloat16().cuda()
    whole, _, _ = block.prompt(x)
    _, state, _ = block.prompt(x[:, :a.tokens])
    worst = 0.0
    for i in range(a.steps):
        out = block.step(x[:, a.tokens + i], state)
        worst = max(worst, (out.float() - whole[:, a.tokens + i].float()).abs().max().item())
    print(f"{a.layer}: {a.tokens}-token prompt, {a.steps} single tokens; against one prompt of "
          f"{a.tokens + a.steps}: max difference {worst:.3g}")
    target = torch.randn(a.batch, a.tokens, 512, generator=g).bfloat16().cuda()
    for i in range(3):
        out, _, kept = block.prompt(x[:, :a.tokens], save=True)
        err = out.float() - target.float()
        grads = block.backward(kept, (2 * err / err.numel()).bfloat16())
        for n, gr in grads.items():
            block.w[n].sub_(gr.to(block.w[n].dtype), alpha=20.0)
        print(f"training step {i}: loss {err.square().mean().item():.5f}")
    st, detail = m2rnn.device_status()
    assert st == 0, (st, detail)


if __name__ == "__main__":
    main()
