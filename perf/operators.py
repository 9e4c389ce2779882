"""What the mixer block's operators are measured on: the short causal
convolution (conv), the per-head norm of queries and keys with the position
rotation (qk_norm) and the selective scan (scan), each for prompts, for
training steps and for single tokens.

``own`` false: the operators in plain torch, in 32 bits, rounded once at the
end (gradients by torch's differentiation of these elementary operations).
``own`` true: the calls a user makes of ``non_linear_matrix_gb300.m2rnn``.

Sizes follow the package's workloads (K=64, V=16 per value head, N=32 or 64
heads sharing q and k, T=2048, 4096 and 65536, B=1, 8 and 2048); a
convolution's channels are the concatenated q|k|v projection, 2*Nq*K + N*V.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
CHUNK = 64  # tokens per block of the plain scan


def listed():
    return [
        # one token for 64 sequences behind the q|k|v projection: latency
        dict(name="conv_step_b64", op="conv", mode="step", dtype="bf16", B=64, T=1, C=640, W=4),
        # a long prompt, N=64 heads: 2*64 + 64*16 channels, a single sequence
        dict(name="conv_prompt_t65536", op="conv", mode="prompt", dtype="bf16", B=1, T=65536,
             C=1152, W=4),
        # a training step's convolution, forward and backward
        dict(name="conv_train_b8_t4096", op="conv", mode="train", dtype="bf16", B=8, T=4096,
             C=640, W=4),
        # one token for 64 sequences, each at its own position
        dict(name="qk_norm_step_b64", op="qk_norm", mode="step", dtype="bf16", B=64, T=1, Nq=8,
             Nk=8, K=64, R=64),
        # a prompt batch with a query/key group for every head
        dict(name="qk_norm_prompt_b8_t2048", op="qk_norm", mode="prompt", dtype="bf16", B=8,
             T=2048, Nq=32, Nk=32, K=64, R=64),
        # a training step: grouped heads, a quarter of the features rotated
        dict(name="qk_norm_train_b8_t4096", op="qk_norm", mode="train", dtype="bf16", B=8, T=4096,
             Nq=8, Nk=2, K=128, R=32),
        # one token for 8 sequences: latency
        dict(name="scan_step_b8", op="scan", mode="step", dtype="bf16", B=8, T=1, N=32, Nq=1,
             K=64, V=16),
        # one token for 2048 sequences: the state's traffic
        dict(name="scan_step_b2048", op="scan", mode="step", dtype="bf16", B=2048, T=1, N=32,
             Nq=1, K=64, V=16),
        # an ordinary prompt batch
        dict(name="scan_prompt_b8_t2048", op="scan", mode="prompt", dtype="bf16", B=8, T=2048,
             N=32, Nq=1, K=64, V=16),
        # one long sequence: few rows, a long axis
        dict(name="scan_prompt_t65536", op="scan", mode="prompt", dtype="bf16", B=1, T=65536,
             N=64, Nq=1, K=64, V=16),
        # a training step, forward and backward
        dict(name="scan_train_b8_t4096", op="scan", mode="train", dtype="bf16", B=8, T=4096, N=32,
             Nq=1, K=64, V=16),
        # fp32 operands, ragged length, grouped q/k, the largest state
        dict(name="scan_train_f32_t777", op="scan", mode="train", dtype="f32", B=2, T=777, N=8,
             Nq=2, K=128, V=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges: any operator, direction and type, odd sizes,
    at most the work of the largest listed case of its kind."""
    op = rng.choice(["conv", "qk_norm", "scan", "scan"])
    mode = rng.choice(["step", "prompt", "train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    c = dict(op=op, mode=mode, dtype=dtype)
    if mode == "step":
        c["B"], c["T"] = _log(rng, 1, 1024 if op == "scan" else 2048), 1
    else:
        c["B"] = _log(rng, 1, 16)
        c["T"] = _log(rng, 1, 16384)
    tokens = c["B"] * c["T"]
    if op == "conv":
        c["C"] = 8 * _log(rng, 8, 320)
        c["W"] = rng.choice([2, 3, 4, 4])
        most = 8 * 4096 * 640
        if tokens * c["C"] > most:
            c["T"] = max(1, most // (c["B"] * c["C"]))
    elif op == "qk_norm":
        c["K"] = rng.choice([16, 32, 64, 128])
        c["Nk"] = rng.choice([1, 2, 4, 8])
        c["Nq"] = c["Nk"] * rng.choice([1, 1, 2, 3])
        c["R"] = rng.choice([0, c["K"] // 2, c["K"]])
        c["interleaved"] = rng.choice([False, True])
        row, most = (c["Nq"] + c["Nk"]) * c["K"], 8 * 4096 * 1280
        if tokens * row > most:
            c["T"] = max(1, most // (c["B"] * row))
    else:
        c["K"] = rng.choice([16, 32, 64, 128])
        c["V"] = rng.choice([16, 32])
        c["Nq"] = rng.choice([1, 1, 2])
        c["N"] = c["Nq"] * _log(rng, 1, 32)
        row, most = c["N"] * c["K"] * c["V"], 8 * 4096 * 32 * 1024
        if dtype == "f32":
            most //= 8
        if tokens * row > most:
            c["T"] = max(1, most // (c["B"] * row))
            c["B"] = max(1, min(c["B"], most // row))
    return c


# ---- inputs -----------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dev, td = "cuda", DT[case["dtype"]]
    B, T, step = case["B"], case["T"], case["mode"] == "step"

    def randn(*s):
        return torch.randn(*s, generator=g, device=dev)

    def rand(*s):
        return torch.rand(*s, generator=g, device=dev)

    s = dict(case)
    if case["op"] == "conv":
        C, W = case["C"], case["W"]
        s["w"] = ((rand(C, W) * 2 - 1) / math.sqrt(W)).to(td)
        s["bias"] = ((rand(C) * 2 - 1) / math.sqrt(W)).to(td)
        # the last W - 1 inputs before this call
        s["state"] = randn(B, W - 1, C).to(td)
        s["x"] = randn(*((B, C) if step else (B, T, C))).to(td)
        if case["mode"] == "train":
            s["dy"] = randn(B, T, C).to(td)
        if step:
            s["state_out"] = torch.empty_like(s["state"])
    elif case["op"] == "qk_norm":
        K, R = case["K"], case["R"]
        # q and k as they leave a projection: rows of one buffer
        n = case["Nq"] + case["Nk"]
        buf = (randn(B, T, n * K) * 2).to(td)
        s["q"] = buf[..., :case["Nq"] * K].view(B, T, case["Nq"], K)
        s["k"] = buf[..., case["Nq"] * K:].view(B, T, case["Nk"], K)
        s["wq"] = (1 + 0.1 * randn(K)).to(td)
        s["wk"] = (1 + 0.1 * randn(K)).to(td)
        s["cos"] = s["sin"] = s["pos"] = None
        if R:
            P = max(T, 4096)
            inv = 10000.0 ** (-torch.arange(0, R, 2, device=dev, dtype=torch.float64) / R)
            ang = torch.arange(P, device=dev, dtype=torch.float64)[:, None] * inv
            s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
            if step:
                s["pos"] = torch.randint(0, P, (B, 1), generator=g, device=dev, dtype=torch.int32)
            else:
                s["pos"] = torch.arange(T, device=dev, dtype=torch.int32).expand(B, T).contiguous()
        if case["mode"] == "train":
            s["dqo"] = randn(B, T, case["Nq"], K).to(td)
            s["dko"] = randn(B, T, case["Nk"], K).to(td)
    else:
        N, Nq, K, V = case["N"], case["Nq"], case["K"], case["V"]
        lead = (B,) if step else (B, T)
        for n in ("q", "k"):
            x = randn(*lead, Nq, K)
            s[n] = (x / x.norm(dim=-1, keepdim=True)).to(td)
        s["v"] = randn(*lead, N, V).to(td)
        s["a"] = randn(*lead, N).to(td)
        # step sizes between 1e-3 and 0.1 at a = 0, decay rates between 1 and 16
        dt = torch.exp(rand(N) * math.log(100.0) + math.log(1e-3))
        s["beta"] = (dt + torch.log(-torch.expm1(-dt))).to(td)
        s["alpha"] = (1 + 15 * rand(N)).to(td)
        s["w_r"] = randn(N, V).to(td)
        s["H0"] = 0.1 * randn(B, N, K, V)
        if case["mode"] == "train":
            s["dy"] = randn(B, T, N, V).to(td)
            s["dHT"] = 0.1 * randn(B, N, K, V)
        if step:
            s["H_out"] = torch.empty_like(s["H0"])
    return s


# ---- one pass ---------------------------------------------------------------


def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_conv(s):
    from non_linear_matrix_gb300 import m2rnn
    if s["mode"] == "step":
        y, st = m2rnn.conv_step(s["x"], s["w"], s["state"], s["bias"], state_out=s["state_out"])
        return {"y": y, "state": st}
    y, st = m2rnn.conv_fwd(s["x"], s["w"], s["bias"], s["state"])
    if s["mode"] == "prompt":
        return {"y": y, "state": st}
    g = m2rnn.conv_bwd(s["x"], s["w"], s["dy"], s["bias"], s["state"])
    return {"y": y, "dx": g["dx"], "dw": g["dw"], "dbias": g["dbias"]}


def _own_qk_norm(s):
    from non_linear_matrix_gb300 import m2rnn
    rot = dict(cos=s["cos"], sin=s["sin"], pos=s["pos"], interleaved=s.get("interleaved", False))
    qo, ko = m2rnn.qk_norm_fwd(s["q"], s["k"], s["wq"], s["wk"], EPS, **rot)
    if s["mode"] != "train":
        return {"q": qo, "k": ko}
    g = m2rnn.qk_norm_bwd(s["q"], s["k"], s["wq"], s["wk"], s["dqo"], s["dko"], EPS, **rot)
    return {"q": qo, "k": ko, "dq": g["dq"], "dk": g["dk"], "dwq": g["dwq"], "dwk": g["dwk"]}


def _own_scan(s):
    from non_linear_matrix_gb300 import m2rnn
    args = (s["q"], s["k"], s["v"], s["a"], s["alpha"], s["beta"])
    if s["mode"] == "step":
        y, H = m2rnn.scan_step(*args, s["H0"], s["w_r"], H_out=s["H_out"])
        return {"y": y, "H": H}
    y, HT, saved = m2rnn.scan_fwd(*args, s["w_r"], s["H0"], save=s["mode"] == "train")
    if s["mode"] == "prompt":
        return {"y": y, "H": HT}
    g = m2rnn.scan_bwd(*args, s["dy"], s["w_r"], s["H0"], s["dHT"], saved=saved, want_dH0=True)
    return {"y": y, "H": HT, **{n: g[n] for n in ("dq", "dk", "dv", "da", "dalpha", "dbeta",
                                                 "dw_r", "dH0")}}


_own = {"conv": _own_conv, "qk_norm": _own_qk_norm, "scan": _own_scan}


def _leaves(s, names, train):
    return [s[n].float().detach().requires_grad_(train) for n in names]


def _conv_f32(x, w, bias, state):
    """x [B,T,C] -> y [B,T,C], all fp32."""
    T, W = x.shape[1], w.shape[1]
    xs = torch.cat([state, x], 1)
    z = bias.expand_as(x)
    z = z + sum(w[:, i] * xs[:, i:i + T] for i in range(W))
    return z / (1 + torch.exp(-z))


def _plain_conv(s):
    td, train = DT[s["dtype"]], s["mode"] == "train"
    x, w, bias = _leaves(s, ("x", "w", "bias"), train)
    step = s["mode"] == "step"
    x3 = x[:, None] if step else x
    y = _conv_f32(x3, w, bias, s["state"].float())
    state = torch.cat([s["state"], s["x"][:, None] if step else s["x"]], 1)
    state = state[:, state.shape[1] - (s["W"] - 1):].contiguous()
    if not train:
        return {"y": (y[:, 0] if step else y).to(td), "state": state}
    dx, dw, db = torch.autograd.grad(y, (x, w, bias), s["dy"].float())
    return {"y": y.detach().to(td), "dx": dx.to(td), "dw": dw, "dbias": db}


def _rot_f32(u, cos, sin, inter):
    """Rotates the first 2*cos.shape[-1] features of u [B,T,H,K]."""
    R = 2 * cos.shape[-1]
    if inter:
        x1, x2 = u[..., 0:R:2], u[..., 1:R:2]
    else:
        x1, x2 = u[..., :R // 2], u[..., R // 2:R]
    c, n = cos[:, :, None], sin[:, :, None]
    y1, y2 = x1 * c - x2 * n, x2 * c + x1 * n
    r = torch.stack([y1, y2], -1).flatten(-2) if inter else torch.cat([y1, y2], -1)
    return torch.cat([r, u[..., R:]], -1)


def _plain_qk_norm(s):
    td, train = DT[s["dtype"]], s["mode"] == "train"
    q, k, wq, wk = _leaves(s, ("q", "k", "wq", "wk"), train)
    out = []
    for x, w in ((q, wq), (k, wk)):
        u = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        if s["R"]:
            p = s["pos"].long()
            u = _rot_f32(u, s["cos"][p], s["sin"][p], s.get("interleaved", False))
        out.append(u)
    if not train:
        return {"q": out[0].to(td), "k": out[1].to(td)}
    dq, dk, dwq, dwk = torch.autograd.grad(out, (q, k, wq, wk), (s["dqo"].float(), s["dko"].float()))
    return {"q": out[0].detach().to(td), "k": out[1].detach().to(td), "dq": dq.to(td),
            "dk": dk.to(td), "dwq": dwq, "dwk": dwk}


def _softplus(x):
    return torch.where(x > 20, x, torch.log1p(torch.exp(torch.clamp_max(x, 20))))


def _segsum(x):
    """x [..., L] -> [..., L, L]: sum of x over (j, i] for i >= j, -inf above."""
    L = x.shape[-1]
    i = torch.arange(L, device=x.device)
    m = x[..., :, None].expand(*x.shape, L).masked_fill(i[:, None] <= i[None, :], 0)
    return torch.cumsum(m, -2).masked_fill(i[:, None] < i[None, :], -math.inf)


def _scan_f32(q, k, v, a, alpha, beta, w_r, H0):
    """The scan over blocks of CHUNK tokens: inside a block as a masked
    matrix product, between blocks by the products of the blocks' decays."""
    B, T, N, V = v.shape
    Nq, K = q.shape[2], q.shape[3]
    r = N // Nq
    n = -(-T // CHUNK)
    pad = n * CHUNK - T
    dt = _softplus(a + beta)
    ld = -alpha * dt
    if pad:
        q, k, v, dt, ld = (torch.cat([x, x.new_zeros(B, pad, *x.shape[2:])], 1)
                           for x in (q, k, v, dt, ld))
    q, k = (x.view(B, n, CHUNK, Nq, K).permute(0, 3, 1, 2, 4)[:, :, None] for x in (q, k))
    vv = v.view(B, n, CHUNK, Nq, r, V).permute(0, 3, 4, 1, 2, 5)           # B Nq r n L V
    dt, ld = (x.view(B, n, CHUNK, Nq, r).permute(0, 3, 4, 1, 2) for x in (dt, ld))
    seg = _segsum(ld)                                                      # B Nq r n L L
    u = vv * dt[..., None]
    y = (torch.matmul(q, k.transpose(-1, -2)) * torch.exp(seg)) @ u
    total = ld.sum(-1)                                                     # B Nq r n
    tail = torch.exp(seg[..., -1, :])                                      # to the block's end
    S = torch.matmul(k.transpose(-1, -2), u * tail[..., None])             # B Nq r n K V
    S = torch.cat([H0.view(B, Nq, r, 1, K, V), S], 3)
    D = torch.exp(_segsum(torch.cat([torch.zeros_like(total[..., :1]), total], -1)))
    H = torch.matmul(D, S.flatten(-2)).view(B, Nq, r, n + 1, K, V)         # after each block
    head = torch.exp(ld.cumsum(-1))
    y = y + torch.matmul(q, H[..., :-1, :, :]) * head[..., None]
    y = y.permute(0, 3, 4, 1, 2, 5).reshape(B, n * CHUNK, N, V)[:, :T] + w_r * v[:, :T]
    return y, H[..., -1, :, :].reshape(B, N, K, V)


def _plain_scan(s):
    td, train, step = DT[s["dtype"]], s["mode"] == "train", s["mode"] == "step"
    leaves = _leaves(s, ("q", "k", "v", "a", "alpha", "beta", "w_r", "H0"), train)
    q, k, v, a, alpha, beta, w_r, H0 = leaves
    if step:
        r = s["N"] // s["Nq"]
        dt = _softplus(a + beta)
        kk, qq = (x.repeat_interleave(r, 1)[..., None] for x in (k, q))
        H = torch.exp(-alpha * dt)[..., None, None] * H0 + (dt[..., None, None] * kk) * v[:, :, None]
        return {"y": ((H * qq).sum(2) + w_r * v).to(td), "H": H}
    y, HT = _scan_f32(q, k, v, a, alpha, beta, w_r, H0)
    if not train:
        return {"y": y.to(td), "H": HT}
    g = torch.autograd.grad((y, HT), leaves, (s["dy"].float(), s["dHT"]))
    dq, dk, dv, da, dalpha, dbeta, dw_r, dH0 = g
    return {"y": y.detach().to(td), "H": HT.detach(), "dq": dq.to(td), "dk": dk.to(td),
            "dv": dv.to(td), "da": da.to(td), "dalpha": dalpha, "dbeta": dbeta, "dw_r": dw_r,
            "dH0": dH0}


_plain = {"conv": _plain_conv, "qk_norm": _plain_qk_norm, "scan": _plain_scan}


# ---- what a pass cannot do without ---------------------------------------------


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, T = case["B"], case["T"]
    train, step = case["mode"] == "train", case["mode"] == "step"
    if case["op"] == "conv":
        C, W = case["C"], case["W"]
        n, state = B * T * C, B * (W - 1) * C
        par = C * (W + 1)
        b = e * (2 * n + par + 2 * state)
        f = n * (2 * W + 4)
        if train:  # x and dy again, dx; dw, dbias in 32 bits
            b = e * (2 * n + par + state) + e * (3 * n + par + state) + 4 * par
            f += n * (6 * W + 10)
    elif case["op"] == "qk_norm":
        n = B * T * (case["Nq"] + case["Nk"]) * case["K"]
        par = 2 * case["K"] * e
        tab = B * T * case["R"] * 4 if step else T * case["R"] * 4
        b, f = 2 * n * e + par + tab, n * 8
        if train:
            b += 3 * n * e + par + tab + 2 * case["K"] * 4
            f += n * 16
    else:
        N, Nq, K, V = case["N"], case["Nq"], case["K"], case["V"]
        th, state = B * T * N, 4 * B * N * K * V
        qk = 2 * B * T * Nq * K * e
        par = e * N * (2 + V)
        b = qk + th * e * (2 * V + 1) + par + 2 * state
        f = th * (6 * K * V)
        if train:  # q, k, v, a, dy in, dq, dk, dv, da out; dHT in, dH0 out, H0 again
            b += 2 * qk + th * e * (3 * V + 2) + par + 4 * N * (2 + V) + 3 * state
            f += th * (14 * K * V)
    return {"bytes": b, "flops": f}


# ---- the definitions in 64 bits --------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    d = {n: x.double() if torch.is_tensor(x) and x.is_floating_point() else x for n, x in s.items()}
    return _exact[case["op"]](d)


def _exact_conv(s):
    W = s["W"]
    if s["mode"] == "step":
        rows = [s["state"][:, i] for i in range(W - 1)] + [s["x"]]
        z = s["bias"] + sum(s["w"][:, i] * rows[i] for i in range(W))
        return {"y": z * torch.sigmoid(z), "state": torch.stack(rows[1:], 1)}
    x = s["x"]
    B, T, C = x.shape
    full = torch.zeros(B, T + W - 1, C, dtype=torch.float64, device=x.device)
    full[:, :W - 1] = s["state"]
    full[:, W - 1:] = x
    win = full.unfold(1, W, 1)                       # B T C W
    z = torch.einsum("btcw,cw->btc", win, s["w"]) + s["bias"]
    sg = torch.sigmoid(z)
    y = z * sg
    if s["mode"] == "prompt":
        return {"y": y, "state": full[:, T:].clone()}
    dz = s["dy"] * (sg + y * (1 - sg))
    dfull = torch.zeros_like(full)
    for i in range(W):
        dfull[:, i:i + T] += dz * s["w"][:, i]
    return {"y": y, "dx": dfull[:, W - 1:], "dw": torch.einsum("btcw,btc->cw", win, dz),
            "dbias": dz.sum((0, 1))}


def _exact_qk_norm(s):
    K, R, out, grads = s["K"], s["R"], {}, {}
    if R:  # the whole rotation as one K x K matrix per token
        h = R // 2
        i = torch.arange(h, device=s["q"].device)
        i1, i2 = (2 * i, 2 * i + 1) if s.get("interleaved", False) else (i, i + h)
        c, n = s["cos"][s["pos"].long()], s["sin"][s["pos"].long()]
    for name in ("q", "k"):
        x, w = s[name], s["w" + name]
        rstd = (x.square().sum(-1, keepdim=True) / K + EPS).rsqrt()
        xh = x * rstd
        u = xh * w

        def turn(t, sign):
            if not R:
                return t
            t = t.clone()
            a, b = t[..., i1], t[..., i2]
            t[..., i1] = a * c[:, :, None] - sign * b * n[:, :, None]
            t[..., i2] = b * c[:, :, None] + sign * a * n[:, :, None]
            return t

        out[name] = turn(u, 1)
        if s["mode"] == "train":
            du = turn(s["d" + name + "o"], -1)
            grads["dw" + name] = (du * xh).sum((0, 1, 2))
            g = du * w
            grads["d" + name] = rstd * (g - xh * (g * xh).sum(-1, keepdim=True) / K)
    return {**out, **grads}


def _exact_scan(s):
    """The recurrence token by token, and its chain rule in reverse."""
    N, Nq, T, mode = s["N"], s["Nq"], s["T"], s["mode"]
    step = mode == "step"
    q, k, v, a = (x[:, None] if step else x for x in (s["q"], s["k"], s["v"], s["a"]))
    if mode == "train" and s["H0"].numel() * T > 4e9:
        return None
    q, k = (x.repeat_interleave(N // Nq, 2) for x in (q, k))
    x = a + s["beta"]
    dt = torch.logaddexp(x, torch.zeros_like(x))
    f = torch.exp(-s["alpha"] * dt)
    H, ys, hist = s["H0"], torch.empty_like(v), []
    kd = k * dt[..., None]
    fx = f[..., None, None]
    for t in range(T):
        if mode == "train":
            hist.append(H)
        H = H * fx[:, t]
        H += kd[:, t, :, :, None] * v[:, t, :, None, :]
        ys[:, t] = torch.matmul(q[:, t, :, None, :], H)[:, :, 0]
    y = ys + s["w_r"] * v
    if step:
        return {"y": y[:, 0], "H": H}
    out = {"y": y, "H": H}
    if mode == "prompt":
        return out
    dy = s["dy"]
    C, HT = s["dHT"], H                        # C: dL/dH_t from the steps after t
    dqh, dkh, dvv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    df, ddt = torch.empty_like(f), torch.empty_like(f)
    after = HT
    for t in range(T - 1, -1, -1):
        before = hist.pop()
        C = C + q[:, t, :, :, None] * dy[:, t, :, None, :]
        dqh[:, t] = torch.matmul(after, dy[:, t, :, :, None])[..., 0]
        Cv = torch.matmul(C, v[:, t, :, :, None])[..., 0]
        dkh[:, t] = dt[:, t, :, None] * Cv
        dvv[:, t] = dt[:, t, :, None] * torch.matmul(k[:, t, :, None, :], C)[:, :, 0]
        ddt[:, t] = (k[:, t] * Cv).sum(-1)
        df[:, t] = (C * before).sum((-1, -2))
        C = C * fx[:, t]
        after = before
    ddt = ddt - s["alpha"] * f * df
    da = ddt * torch.sigmoid(x)
    B, r = s["B"], N // Nq
    out.update(dq=dqh.view(B, T, Nq, r, -1).sum(3), dk=dkh.view(B, T, Nq, r, -1).sum(3),
               dv=dvv + s["w_r"] * dy, da=da, dalpha=(-dt * f * df).sum((0, 1)),
               dbeta=da.sum((0, 1)), dw_r=(dy * v).sum((0, 1)), dH0=C)
    return out


_exact = {"conv": _exact_conv, "qk_norm": _exact_qk_norm, "scan": _exact_scan}
