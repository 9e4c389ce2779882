"""What the feed-forward half of a layer is measured on: the residual's addition
with the RMS norm behind it (add_norm), the gated feed-forward products (glu)
and the 8-bit product with scales (linear_q8), each for single tokens and for
prompts, the first two for training steps too.

``own`` false: the operators in plain torch, in 32 bits, rounded once at the
end (gradients by torch's differentiation of these elementary operations).
``own`` true: the calls a user makes of ``non_linear_matrix_gb300.m2rnn``.

Sizes follow the package's workloads (T=2048, 4096 and 65536, B=1, 8 and 64,
a model width of 512 in the example's block, N*V = 512 and 1,024 features per
token in the benchmark); a feed-forward's width is 2.75 or 4 times the model's.

8 bits are e4m3 with one fp32 scale per row (a token, or a row of a weight):
scale = max|row| / 448, code = the nearest e4m3 value of row / scale.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
EPS = 1e-6


def listed():
    return [
        # one token for 64 sequences, between a block and the next: latency
        dict(name="add_norm_step_b64", op="add_norm", mode="step", dtype="bf16", M=64, D=1024),
        # one long prompt of a small model
        dict(name="add_norm_prompt_t65536", op="add_norm", mode="prompt", dtype="bf16", M=65536,
             D=1024),
        # a training step, forward and backward
        dict(name="add_norm_train_b8_t4096", op="add_norm", mode="train", dtype="bf16", M=32768,
             D=2048),
        # a ragged prompt batch in front of an 8-bit product
        dict(name="add_norm_q8_t12001", op="add_norm", mode="q8", dtype="bf16", M=12001, D=2000),
        # one token for 8 sequences: the weights' traffic
        dict(name="glu_step_b8", op="glu", mode="step", dtype="bf16", M=8, D=1024, F=2816),
        # an ordinary prompt batch
        dict(name="glu_prompt_b8_t2048", op="glu", mode="prompt", dtype="bf16", M=16384, D=1024,
             F=4096),
        # a training step, forward and backward
        dict(name="glu_train_b8_t4096", op="glu", mode="train", dtype="bf16", M=32768, D=1024,
             F=2816),
        # fp32 operands, ragged sizes
        dict(name="glu_train_f32_t777", op="glu", mode="train", dtype="f32", M=1554, D=520,
             F=1400),
        # one token for 64 sequences in 8 bits
        dict(name="glu_q8_step_b64", op="glu", mode="q8", dtype="bf16", M=64, D=2048, F=5632),
        # a large prompt batch in 8 bits: the most operations
        dict(name="glu_q8_prompt_b8_t2048", op="glu", mode="q8", dtype="bf16", M=16384, D=2048,
             F=5632),
        # the way back from the feed-forward's width, added to the residual: one token ...
        dict(name="linear_q8_step_b8", op="linear_q8", mode="q8", dtype="bf16", M=8, D=5632,
             F=2048),
        # ... and a prompt batch
        dict(name="linear_q8_prompt_b8_t2048", op="linear_q8", mode="q8", dtype="bf16", M=16384,
             D=5632, F=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges: any operator, direction and type, odd sizes,
    at most the work of the largest listed case of its kind."""
    op = rng.choice(["add_norm", "glu", "glu", "linear_q8"])
    mode = "q8" if op == "linear_q8" else rng.choice(["step", "prompt", "train", "q8"])
    dtype = "bf16" if mode == "q8" and op != "add_norm" else rng.choice(["bf16", "bf16", "f32"])
    c = dict(op=op, mode=mode, dtype=dtype)
    c["M"] = _log(rng, 1, 64) if mode == "step" else _log(rng, 1, 32768)
    if op == "add_norm":
        c["D"] = 8 * _log(rng, 8, 1024)
        most = 65536 * 1024
        c["M"] = max(1, min(c["M"], most // c["D"]))
        return c
    unit = 16 if mode == "q8" else 8
    c["D"] = unit * _log(rng, 64 // unit, 4096 // unit)
    c["F"] = unit * _log(rng, 64 // unit, 8192 // unit)
    most = 16384 * 1024 * 4096
    if mode == "q8":
        most = 16384 * 2048 * 5632
    if dtype == "f32":
        most //= 16
    c["M"] = max(1, min(c["M"], most // (c["D"] * c["F"])))
    return c


# ---- inputs -----------------------------------------------------------------


def _codes(x):
    """x [..., D] -> e4m3 codes and scales [...]."""
    x = x.float()
    amax = x.abs().amax(-1)
    scale = amax / torch.full_like(amax, 448.0)
    q = torch.where(scale[..., None] > 0, x / scale[..., None], torch.zeros_like(x))
    return q.to(E4M3), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dev, td = "cuda", DT[case["dtype"]]
    M, D = case["M"], case["D"]

    def randn(*s):
        return torch.randn(*s, generator=g, device=dev)

    s = dict(case)
    if case["op"] == "add_norm":
        # a block's output, the stream that it is added to and the norm's weight
        s["x"] = randn(M, D).to(td)
        s["res"] = (2 * randn(M, D)).to(td)
        s["w"] = (1 + 0.1 * randn(D)).to(td)
        if case["mode"] == "train":
            s["dy"] = randn(M, D).to(td)
            s["dr"] = randn(M, D).to(td)  # what reaches the sum past the norm
        return s
    F = case["F"]
    if case["op"] == "linear_q8":
        s["x"] = (randn(M, D) * randn(M, D)).to(td)  # a product of two, as the gated products leave it
        s["res"] = randn(M, F).to(td)
        s["w8"], s["ws"] = _codes(randn(F, D) * D ** -0.5)
        return s
    # a normed stream, and weights that keep its scale
    x = randn(M, D) * (1 + 0.1 * randn(D))
    wg, wu = randn(F, D) * D ** -0.5, randn(F, D) * D ** -0.5
    if case["mode"] == "q8":
        s["x8"], s["xs"] = _codes(x)
        s["wg8"], s["wgs"] = _codes(wg)
        s["wu8"], s["wus"] = _codes(wu)
        return s
    s["x"], s["wg"], s["wu"] = x.to(td), wg.to(td), wu.to(td)
    if case["mode"] == "train":
        s["dh"] = randn(M, F).to(td)
    return s


# ---- one pass ---------------------------------------------------------------


def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_add_norm(s):
    from non_linear_matrix_gb300 import m2rnn
    if s["mode"] == "q8":
        q, scale, r = m2rnn.add_norm_q8(s["x"], s["res"], s["w"], EPS)
        return {"q": q, "scale": scale, "r": r}
    y, r = m2rnn.add_norm_fwd(s["x"], s["res"], s["w"], EPS)
    if s["mode"] != "train":
        return {"y": y, "r": r}
    g = m2rnn.add_norm_bwd(r, s["dy"], s["w"], s["dr"], EPS)
    return {"y": y, "r": r, "dx": g["dx"], "dw": g["dw"]}


def _own_glu(s):
    from non_linear_matrix_gb300 import m2rnn
    if s["mode"] == "q8":
        return {"h": m2rnn.glu_q8(s["x8"], s["xs"], s["wg8"], s["wgs"], s["wu8"], s["wus"])}
    h = m2rnn.glu_fwd(s["x"], s["wg"], s["wu"])
    if s["mode"] != "train":
        return {"h": h}
    g = m2rnn.glu_bwd(s["x"], s["wg"], s["wu"], s["dh"])
    return {"h": h, "dx": g["dx"], "dwg": g["dwg"], "dwu": g["dwu"]}


def _own_linear_q8(s):
    from non_linear_matrix_gb300 import m2rnn
    q, scale = m2rnn.quant_rows(s["x"])
    return {"y": m2rnn.linear_q8(q, scale, s["w8"], s["ws"], s["res"]), "q": q, "scale": scale}


_own = {"add_norm": _own_add_norm, "glu": _own_glu, "linear_q8": _own_linear_q8}


def _norm_f32(r, w):
    return r / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS) * w


def _plain_add_norm(s):
    td, train = DT[s["dtype"]], s["mode"] == "train"
    # the sum is an output of its own: the norm takes it as it is stored
    stored = (s["x"].float() + s["res"].float()).to(td)
    r = stored.float().requires_grad_(train)
    w = s["w"].float().requires_grad_(train)
    y = _norm_f32(r, w)
    if s["mode"] == "q8":
        q, scale = _codes(y)
        return {"q": q, "scale": scale, "r": stored}
    if not train:
        return {"y": y.to(td), "r": stored}
    dr, dw = torch.autograd.grad(y, (r, w), s["dy"].float())
    return {"y": y.detach().to(td), "r": stored, "dx": (dr + s["dr"].float()).to(td), "dw": dw}


def _glu_f32(x, wg, wu):
    g, u = x @ wg.T, x @ wu.T
    return g / (1 + torch.exp(-g)) * u


def _plain_glu(s):
    td, train = DT[s["dtype"]], s["mode"] == "train"
    if s["mode"] == "q8":
        x, wg, wu = (s[n + "8"].float() * s[n + "s"][:, None] for n in ("x", "wg", "wu"))
        return {"h": _glu_f32(x, wg, wu).to(td)}
    x, wg, wu = (s[n].float().detach().requires_grad_(train) for n in ("x", "wg", "wu"))
    h = _glu_f32(x, wg, wu)
    if not train:
        return {"h": h.to(td)}
    dx, dwg, dwu = torch.autograd.grad(h, (x, wg, wu), s["dh"].float())
    return {"h": h.detach().to(td), "dx": dx.to(td), "dwg": dwg.to(td), "dwu": dwu.to(td)}


def _plain_linear_q8(s):
    q, scale = _codes(s["x"])
    x, w = q.float() * scale[:, None], s["w8"].float() * s["ws"][:, None]
    return {"y": (x @ w.T + s["res"].float()).to(DT[s["dtype"]]), "q": q, "scale": scale}


_plain = {"add_norm": _plain_add_norm, "glu": _plain_glu, "linear_q8": _plain_linear_q8}


# ---- what a pass cannot do without ---------------------------------------------


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    M, D = case["M"], case["D"]
    if case["op"] == "add_norm":
        n = M * D
        if case["mode"] == "q8":  # x and the stream in; the sum, the codes and their scales out
            return {"bytes": n * (3 * e + 1) + 4 * M + e * D, "flops": 7 * n}
        if case["mode"] != "train":
            return {"bytes": 4 * n * e + e * D, "flops": 5 * n}
        # the sum again, dy and dr in, dx and dw out
        return {"bytes": 8 * n * e + 2 * e * D + 4 * D, "flops": 15 * n}
    F = case["F"]
    if case["op"] == "linear_q8":  # x twice (its maximum, its codes), its codes out and in
        return {"bytes": M * D * (e + 1) + F * D + 4 * (M + F) + 2 * M * F * e,
                "flops": 2 * M * D * F + 3 * M * D}
    if case["mode"] == "q8":
        return {"bytes": M * D + 2 * F * D + 4 * (M + 2 * F) + M * F * e, "flops": 4 * M * D * F}
    b, f = e * (M * D + 2 * F * D + M * F), 4 * M * D * F
    if case["mode"] == "train":  # x, the weights and dh in, dx and the weights' gradients out
        b += e * (2 * M * D + 4 * F * D + M * F)
        f += 8 * M * D * F
    return {"bytes": b, "flops": f}


# ---- the definitions in 64 bits --------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    d = {n: x.double() if torch.is_tensor(x) else x for n, x in s.items()}
    return _exact[case["op"]](d)


def _row_codes(x):
    """Scales, and what the codes stand for before they are rounded."""
    scale = x.abs().max(dim=-1).values / 448
    return torch.nan_to_num(x / scale.unsqueeze(-1), nan=0.0), scale


def _exact_add_norm(s):
    td = DT[s["dtype"]]
    # the stored sum is part of the definition
    r = (s["x"] + s["res"]).to(td).double()
    inv = (r.square().sum(-1, keepdim=True) / r.shape[-1] + EPS).rsqrt()
    n = r * inv
    y = n * s["w"]
    out = {"r": s["x"] + s["res"]}
    if s["mode"] == "q8":
        out["q"], out["scale"] = _row_codes(y)
        return out
    out["y"] = y
    if s["mode"] == "train":
        p = s["dy"] * s["w"]
        out["dx"] = s["dr"] + inv * (p - n * (p * n).mean(-1, keepdim=True))
        out["dw"] = torch.einsum("md,md->d", s["dy"], n)
    return out


def _exact_glu(s):
    if s["mode"] == "q8":
        x, wg, wu = (torch.einsum("r,rd->rd", s[n + "s"], s[n + "8"]) for n in ("x", "wg", "wu"))
    else:
        x, wg, wu = s["x"], s["wg"], s["wu"]
    g = torch.einsum("md,fd->mf", x, wg)
    u = torch.einsum("md,fd->mf", x, wu)
    sg = torch.sigmoid(g)
    a = g * sg
    out = {"h": a * u}
    if s["mode"] == "train":
        du = s["dh"] * a
        dg = s["dh"] * u * (sg + a * (1 - sg))
        out["dx"] = torch.einsum("mf,fd->md", dg, wg) + torch.einsum("mf,fd->md", du, wu)
        out["dwg"] = torch.einsum("mf,md->fd", dg, x)
        out["dwu"] = torch.einsum("mf,md->fd", du, x)
    return out


def _exact_linear_q8(s):
    # the product is of the codes: their rounding is part of the definition
    v, scale = _row_codes(s["x"])
    x = v.float().to(E4M3).double() * scale[:, None]
    w = s["w8"] * s["ws"][:, None]
    return {"y": torch.einsum("md,fd->mf", x, w) + s["res"], "q": v, "scale": scale}


_exact = {"add_norm": _exact_add_norm, "glu": _exact_glu, "linear_q8": _exact_linear_q8}
