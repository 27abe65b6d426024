"""The operators of an adapter's training step beside its linears, as cases to be measured:
block norms with their gate and residual scale (forward and backward), the token
log-probabilities and the paired preference loss over a vocabulary (loss and gradient of the
logits), and the global gradient norm with clipping and the clipped optimizer step.

`run` computes a case in plain form (elementary torch operations in FP32, rounded once at
the end) where `own` is false, and calls this repository's entry points where it is true.
"""

import math
import random

import torch

own = False

DEV = "cuda"
# d_out, d_in of the seven adapted linears of the 8B-shaped layer (rank 16: A [16, d_in], B [d_out, 16])
LAYER = [(4096, 4096), (1024, 4096), (1024, 4096), (4096, 4096), (14336, 4096), (14336, 4096), (4096, 14336)]
RANK = 16
ADAMW = dict(step=10, lr=2e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decoded token passes a block's boundary: latency counts
        dict(name="norm fwd 1x4096", op="norm_fwd", M=1, d=4096, stream="bf16", post=True, gate="channel", rows=0),
        # a training batch at the 8B layer's width: post-norm, per-channel gate, next pre-norm
        dict(name="norm fwd 8192x4096", op="norm_fwd", M=8192, d=4096, stream="bf16", post=True, gate="channel", rows=0),
        # a ragged batch on an FP32 residual stream of odd width, one gate row per sequence
        dict(name="norm fwd 1777x2051 f32", op="norm_fwd", M=1777, d=2051, stream="f32", post=True, gate="sequence", rows=300),
        # the backward of a training batch at the 70B layer's width, every gradient wanted
        dict(name="norm bwd 4096x8192", op="norm_bwd", M=4096, d=8192, stream="bf16", post=True, gate="channel", rows=0),
        # the backward of a short batch of sequences, each with its own gate row; FP32 stream, odd width
        dict(name="norm bwd 999x1535 f32", op="norm_bwd", M=999, d=1535, stream="f32", post=True, gate="sequence", rows=111),
        # the reference model's pass: log-probabilities of the labels, no gradient
        dict(name="token logps 4096x32768", op="logps", pairs=4, S=512, V=32768, dtype="bf16"),
        # one short pair over a small odd vocabulary, FP32 logits: latency counts
        dict(name="preference 1x33x1003 f32", op="pref", pairs=1, S=33, V=1003, dtype="f32", smoothing=0.1),
        # a preference batch: prompts and padding masked
        dict(name="preference 4x512x32768", op="pref", pairs=4, S=512, V=32768, dtype="bf16", smoothing=0.0),
        # long answers over a large vocabulary
        dict(name="preference 2x1024x131072", op="pref", pairs=2, S=1024, V=131072, dtype="bf16", smoothing=0.0),
        # the adapters of one layer: 14 small gradient tensors, latency counts
        dict(name="grad norm 14 tensors", op="grad_norm", tensors=14, elements=0, dtype="bf16"),
        # all adapters of 32 such layers: FP32 accumulated gradients clipped into the optimizer's BF16 gradients
        dict(name="grad clip 448 tensors f32", op="grad_clip", tensors=448, elements=0, dtype="f32"),
        # the same parameters' optimizer step with the clipping folded in
        dict(name="clipped adamw 41.9M", op="adamw", tensors=448, elements=0, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width of [lo, hi]: odd, or a model's (4, 5 or 7 times a power of two)."""
    n = _log(rng, lo, hi)
    if rng.random() < 0.5:
        return min(n | 1, hi)
    return min((m << k for m in (4, 5, 7) for k in range(16) if lo <= m << k <= hi), key=lambda w: abs(w - n))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "norm_bwd", "logps", "pref", "pref", "grad_norm", "grad_clip", "adamw"])
    if op in ("norm_fwd", "norm_bwd"):
        d = _width(rng, 64, 8192)
        M = _log(rng, 1, max(1, min(8192, (1 << 25) // d)))
        gate = rng.choice(["none", "channel", "sequence", "element"])
        rows = rng.randint(2, max(2, M // 2)) if gate == "sequence" else 0
        return dict(op=op, M=M, d=d, stream=rng.choice(["bf16", "f32"]), post=rng.random() < 0.75, gate=gate, rows=rows)
    if op in ("logps", "pref"):
        V = _width(rng, 512, 131072)
        pairs = _log(rng, 1, 8)
        S = _log(rng, 1, max(1, min(1024, (1 << 28) // (2 * pairs * V))))
        c = dict(op=op, pairs=pairs, S=S, V=V, dtype=rng.choice(["bf16", "bf16", "f32"]))
        return c if op == "logps" else dict(c, smoothing=rng.choice([0.0, 0.1]))
    tensors = _log(rng, 1, 448)
    return dict(op=op, tensors=tensors, elements=_log(rng, max(64, tensors), 1 << 25), dtype="bf16" if op == "adamw" else rng.choice(["bf16", "f32"]))


def _sizes(case):
    """Elements of each gradient tensor: adapters of whole layers, or a ragged set of that many in all."""
    n = case["tensors"]
    if not case["elements"]:
        layer = [k for d_out, d_in in LAYER for k in (RANK * d_in, RANK * d_out)]
        return (layer * (n // len(layer) + 1))[:n]
    rng = random.Random(n * 1000003 + case["elements"])
    share = [rng.random() ** 2 + 0.01 for _ in range(n)]
    return [max(1, int(case["elements"] * s / sum(share))) for s in share]


def _answers(case):
    """[first, last) answer token of each sequence: prompts before it and padding after it are masked."""
    S, rng = case["S"], random.Random(case["pairs"] * 7919 + case["S"])
    out = []
    for _ in range(case["pairs"]):
        first = rng.randint(0, S // 3)  # the two answers share their prompt
        out.append((first, rng.randint(first + (S - first) // 2, S)))
        out.append((first, rng.randint(first + (S - first) // 2, S)))
    return out[0::2] + out[1::2]


def _randn(gen, shape, std=1.0, mean=0.0, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device=DEV, dtype=dtype).mul_(std).add_(mean)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case=case)
    if case["op"] in ("norm_fwd", "norm_bwd"):
        M, d = case["M"], case["d"]
        stream, bf16 = DTYPE[case["stream"]], torch.bfloat16
        s["x"] = _randn(gen, (M, d), 2.0).to(stream)  # the residual stream: M tokens
        s["y"] = _randn(gen, (M, d), 0.5).to(bf16)  # what the block gave for them
        s["w_post"] = _randn(gen, (d,), 0.2, 1.0).to(bf16) if case["post"] else None
        s["w_pre"] = _randn(gen, (d,), 0.2, 1.0).to(bf16)
        s["gate_rows"] = {"none": 0, "channel": M, "sequence": case["rows"], "element": 1}[case["gate"]]
        groups = -(-M // s["gate_rows"]) if s["gate_rows"] else 0
        s["gate"] = _randn(gen, (groups, d), 0.3, 0.5).to(bf16) if groups else None
        s["scale"], s["eps"] = 0.9, 1e-5
        if case["op"] == "norm_bwd":
            s["dx_out"] = _randn(gen, (M, d), 0.1).to(stream)
            s["dh"] = _randn(gen, (M, d), 0.1).to(bf16)
    elif case["op"] in ("logps", "pref"):
        n, S, V = 2 * case["pairs"], case["S"], case["V"]
        s["logits"] = _randn(gen, (n, S, V), 2.0, 0.0, DTYPE[case["dtype"]])
        labels = torch.randint(0, V, (n, S), generator=gen, device=DEV)
        lift = torch.full((n, S, 1), math.log(V) + 1.0, device=DEV, dtype=s["logits"].dtype)
        s["logits"].scatter_add_(2, labels[:, :, None], lift)  # a model gives its text a fair share
        spans = torch.tensor(_answers(case), device=DEV)
        at = torch.arange(S, device=DEV)[None]
        s["labels"] = torch.where((at >= spans[:, :1]) & (at < spans[:, 1:]), labels, torch.full_like(labels, -100))
        if case["op"] == "pref":
            near = s["logits"].gather(2, labels[:, :, None])[:, :, 0].float() - math.log(V) - 2.5
            s["ref_logps"] = near + _randn(gen, (n, S), 0.1)  # the reference model is near the policy
            s["beta"], s["smoothing"] = 0.1, case["smoothing"]
    else:
        sizes = _sizes(case)
        n = sum(sizes)
        flat = _randn(gen, (n,), 1e-3).to(DTYPE[case["dtype"]])
        s["max_norm"] = 0.3 * 1e-3 * math.sqrt(n)
        if case["op"] == "adamw":
            s["grad"] = flat
            s["master"] = _randn(gen, (n,), 0.02)
            s["m"] = _randn(gen, (n,), 1e-3)
            s["v"] = torch.rand(n, generator=gen, device=DEV) * 1e-6
            s["param"] = torch.empty(n, device=DEV, dtype=torch.bfloat16)
            s["grads"] = [flat]
            clipped = None
        else:
            s["grads"] = list(flat.split(sizes))
            s["clipped"] = torch.empty(n, device=DEV, dtype=torch.bfloat16)
            clipped = list(s["clipped"].split(sizes)) if case["op"] == "grad_clip" else None
        if own:
            import bit_nf4_quantized_dq_amd as Q

            s["list"] = Q.GradList(s["grads"], out=clipped)
    return s


def _plain_rms(v, eps):
    return torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)


def _plain_gate(s):
    if s["gate"] is None:
        return None
    return s["gate"].float().repeat_interleave(s["gate_rows"], 0)[: s["case"]["M"]]


def _plain_norm_fwd(s):
    x, n = s["x"].float(), s["y"].float()
    if s["w_post"] is not None:
        n = n * _plain_rms(n, s["eps"]) * s["w_post"].float()
    gate = _plain_gate(s)
    if gate is not None:
        n = n * gate
    x = s["scale"] * x + n
    h = x * _plain_rms(x, s["eps"]) * s["w_pre"].float()
    return x.to(s["x"].dtype), h.to(torch.bfloat16)


def _plain_rms_bwd(dn, v, w, eps):
    """Input gradient and per-row weight gradient of v * rms(v) * w."""
    r = _plain_rms(v, eps)
    u = v * r
    g = dn * w
    return r * (g - u * (g * u).mean(-1, keepdim=True)), dn * u


def _plain_norm_bwd(s):
    # s["x"] is the forward's residual output here
    bf16 = torch.bfloat16
    x, y = s["x"].float(), s["y"].float()
    through, dw = _plain_rms_bwd(s["dh"].float(), x, s["w_pre"].float(), s["eps"])
    total = s["dx_out"].float() + through
    out = dict(dx=(s["scale"] * total).to(s["x"].dtype), dw_pre=dw.sum(0).to(bf16))
    n = y
    if s["w_post"] is not None:
        n = y * _plain_rms(y, s["eps"]) * s["w_post"].float()
    gate = _plain_gate(s)
    dn = total
    if gate is not None:
        dn = total * gate
        per = total * n
        rows, (M, d) = s["gate_rows"], x.shape
        groups = s["gate"].shape[0]
        per = torch.cat([per, per.new_zeros(groups * rows - M, d)])
        out["dgate"] = per.view(groups, rows, d).sum(1).to(bf16)
    if s["w_post"] is not None:
        dn, dw = _plain_rms_bwd(dn, y, s["w_post"].float(), s["eps"])
        out["dw_post"] = dw.sum(0).to(bf16)
    out["dy"] = dn.to(bf16)
    return out


def _plain_logps(logits, labels):
    x = logits.float()
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    counted = (labels >= 0) & (labels < x.shape[-1])
    at = torch.where(counted, labels, torch.zeros_like(labels))[..., None]
    lp = (x.gather(-1, at) - m - torch.log(z))[..., 0]
    return torch.where(counted, lp, torch.zeros_like(lp)), counted, at, e, z


def _plain_pref(s):
    P, beta, eps = s["case"]["pairs"], s["beta"], s["smoothing"]
    lp, counted, at, e, z = _plain_logps(s["logits"], s["labels"])
    ratio = torch.where(counted, lp - s["ref_logps"], torch.zeros_like(lp)).sum(1)
    t = beta * (ratio[:P] - ratio[P:])
    tail = torch.log1p(torch.exp(-t.abs()))
    loss = ((1 - eps) * (tail + torch.clamp(-t, min=0)) + eps * (tail + torch.clamp(t, min=0))).mean()
    g = (eps - 1 + torch.sigmoid(t)) * (beta / P)
    d = e.div_(z).neg_()
    d.scatter_add_(2, at, torch.ones_like(d[:, :, :1]))
    d.mul_(torch.cat([g, -g])[:, None, None])
    d = torch.where(counted[..., None], d, torch.zeros_like(d[:1, :1, :1]))
    return dict(loss=loss.reshape(1), log_ratios=ratio, logps=lp, dlogits=d.to(s["logits"].dtype))


def _plain_norm(s):
    flat = torch.cat([g.reshape(-1) for g in s["grads"]]).float()
    return flat, (flat * flat).sum().sqrt().reshape(1)


def _plain_adamw(s):
    flat, norm = _plain_norm(s)
    g = flat * torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    a = ADAMW
    theta, m, v = s["master"], s["m"], s["v"]
    theta.mul_(1 - a["lr"] * a["weight_decay"])
    m.mul_(a["beta1"]).add_(g, alpha=1 - a["beta1"])
    v.mul_(a["beta2"]).add_(g * g, alpha=1 - a["beta2"])
    den = v.sqrt().div_(math.sqrt(1 - a["beta2"] ** a["step"])).add_(a["eps"])
    theta.sub_(m / den * (a["lr"] / (1 - a["beta1"] ** a["step"])))
    s["param"].copy_(theta)
    return dict(norm=norm, master=theta, m=m, v=v, param=s["param"])


def _plain(s):
    op = s["case"]["op"]
    if op == "norm_fwd":
        return _plain_norm_fwd(s)
    if op == "norm_bwd":
        return _plain_norm_bwd(s)
    if op == "logps":
        return _plain_logps(s["logits"], s["labels"])[0]
    if op == "pref":
        return _plain_pref(s)
    if op == "grad_norm":
        return _plain_norm(s)[1]
    if op == "grad_clip":
        flat, norm = _plain_norm(s)
        s["clipped"].copy_(flat * torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0))
        return dict(norm=norm, clipped=s["clipped"])
    return _plain_adamw(s)


def _kernels(s):
    import bit_nf4_quantized_dq_amd as Q

    op = s["case"]["op"]
    if op == "norm_fwd":
        return Q.norm_residual_fwd(s["x"], s["y"], w_post=s["w_post"], post_norm=s["case"]["post"], gate=s["gate"],
                                   gate_rows=s["gate_rows"], w_pre=s["w_pre"], res_scale=s["scale"], eps=s["eps"])
    if op == "norm_bwd":
        dx, dy, dw_post, dgate, dw_pre = Q.norm_residual_bwd(
            s["x"], s["y"], s["dh"], s["dx_out"], w_post=s["w_post"], post_norm=s["case"]["post"], gate=s["gate"],
            gate_rows=s["gate_rows"], w_pre=s["w_pre"], res_scale=s["scale"], eps=s["eps"])
        out = dict(dx=dx, dy=dy, dw_pre=dw_pre)
        if dgate is not None:
            out["dgate"] = dgate
        if dw_post is not None:
            out["dw_post"] = dw_post
        return out
    if op == "logps":
        return Q.token_logps(s["logits"], s["labels"])
    if op == "pref":
        loss, log_ratios, logps, dlogits = Q.preference_loss(s["logits"], s["labels"], s["ref_logps"], s["beta"],
                                                             label_smoothing=s["smoothing"])
        return dict(loss=loss, log_ratios=log_ratios, logps=logps, dlogits=dlogits)
    if op == "grad_norm":
        return Q.grad_norm(s["list"])
    if op == "grad_clip":
        return dict(norm=Q.grad_clip(s["list"], s["max_norm"]), clipped=s["clipped"])
    norm = Q.grad_norm(s["list"])
    Q.adamw_step_clipped(s["master"], s["m"], s["v"], s["grad"], norm, s["max_norm"], param=s["param"], **ADAMW)
    return dict(norm=norm, master=s["master"], m=s["m"], v=s["v"], param=s["param"])


def run(state):
    return _kernels(state) if own else _plain(state)


def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        n, e = case["M"] * case["d"], 2 if case["stream"] == "bf16" else 4
        groups = {"none": 0, "channel": 1, "sequence": -(-case["M"] // max(1, case["rows"])), "element": case["M"]}[case["gate"]]
        small = 2 * case["d"] * (1 + int(case["post"]) + groups)
        if op == "norm_fwd":  # x, y in; x, h out
            return dict(bytes=n * (2 * e + 4) + small, flops=12 * n)
        return dict(bytes=n * (3 * e + 6) + 2 * small, flops=30 * n)  # x, y, dh, dx in; dx, dy out
    if op in ("logps", "pref"):
        rows = 2 * case["pairs"] * case["S"]
        counted = sum(last - first for first, last in _answers(case))
        e = 2 if case["dtype"] == "bf16" else 4
        if op == "logps":  # the logits of the counted rows, the labels; the log-probabilities
            return dict(bytes=counted * case["V"] * e + rows * 12, flops=4 * counted * case["V"])
        return dict(bytes=(counted + rows) * case["V"] * e + rows * 16, flops=8 * counted * case["V"])
    n, e = sum(_sizes(case)), 2 if case["dtype"] == "bf16" else 4
    if op == "grad_norm":
        return dict(bytes=n * e, flops=2 * n)
    if op == "grad_clip":
        return dict(bytes=n * (e + 2), flops=3 * n)
    return dict(bytes=n * 28, flops=16 * n)


def exact(case, seed):
    """The operators' definitions in FP64, row block by row block where the whole would be large."""
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op in ("norm_fwd", "norm_bwd"):
        M, d = case["M"], case["d"]
        x, y = s["x"].to(f64), s["y"].to(f64)
        gamma = torch.ones(M, d, device=DEV, dtype=f64)
        if s["gate"] is not None:
            owner = torch.arange(M, device=DEV) // s["gate_rows"]
            gamma = s["gate"].to(f64)[owner]
        w_pre = s["w_pre"].to(f64)
        w_post = s["w_post"].to(f64) if case["post"] else None
        norm_y = (y.square().sum(1, keepdim=True) / d + s["eps"]).sqrt() if case["post"] else None
        inner = y / norm_y * w_post if case["post"] else y
        if op == "norm_fwd":
            x1 = x * s["scale"] + gamma * inner
            return x1, x1 / (x1.square().sum(1, keepdim=True) / d + s["eps"]).sqrt() * w_pre
        norm_x = (x.square().sum(1, keepdim=True) / d + s["eps"]).sqrt()
        dh = s["dh"].to(f64)
        a = dh * w_pre
        t = s["dx_out"].to(f64) + a / norm_x - x * ((a * x).sum(1, keepdim=True) / (d * norm_x**3))
        out = dict(dx=t * s["scale"], dw_pre=(dh * x / norm_x).sum(0))
        if s["gate"] is not None:
            out["dgate"] = torch.zeros_like(s["gate"], dtype=f64).index_add_(0, owner, t * inner)
        b = t * gamma
        if case["post"]:
            out["dw_post"] = (b * y / norm_y).sum(0)
            b = b * w_post
            b = b / norm_y - y * ((b * y).sum(1, keepdim=True) / (d * norm_y**3))
        out["dy"] = b
        return out
    if op in ("logps", "pref"):
        n, S, V = s["logits"].shape
        labels = s["labels"].reshape(-1)
        x = s["logits"].reshape(n * S, V)
        counted = labels >= 0
        block = max(1, (1 << 26) // V)
        lse = torch.cat([torch.logsumexp(x[i:i + block].to(f64), 1) for i in range(0, n * S, block)])
        got = x.gather(1, labels.clamp(min=0)[:, None])[:, 0].to(f64)
        lp = (got - lse) * counted
        if op == "logps":
            return lp.reshape(n, S)
        P, eps = case["pairs"], s["smoothing"]
        ratio = ((lp - s["ref_logps"].reshape(-1).to(f64)) * counted).reshape(n, S).sum(1)
        t = s["beta"] * (ratio[:P] - ratio[P:])
        log_win, log_lose = torch.nn.functional.logsigmoid(t), torch.nn.functional.logsigmoid(-t)
        loss = -((1 - eps) * log_win + eps * log_lose).mean()
        slope = s["beta"] / P * (eps * log_win.exp() - (1 - eps) * log_lose.exp())
        per_row = torch.cat([slope, -slope]).repeat_interleave(S) * counted
        d = torch.empty(n * S, V, device=DEV, dtype=f64)
        for i in range(0, n * S, block):
            p = torch.exp(x[i:i + block].to(f64) - lse[i:i + block, None])
            d[i:i + block] = -p * per_row[i:i + block, None]
        d.scatter_add_(1, labels.clamp(min=0)[:, None], per_row[:, None])
        return dict(loss=loss.reshape(1), log_ratios=ratio, logps=lp.reshape(n, S), dlogits=d.reshape(n, S, V))
    g = torch.cat([t.to(f64) for t in s["grads"]])
    norm = g.square().sum().sqrt().reshape(1)
    if op == "grad_norm":
        return norm
    g = g * min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    if op == "grad_clip":
        return dict(norm=norm, clipped=g)
    a = ADAMW
    m = a["beta1"] * s["m"].to(f64) + (1 - a["beta1"]) * g
    v = a["beta2"] * s["v"].to(f64) + (1 - a["beta2"]) * g.square()
    m_hat, v_hat = m / (1 - a["beta1"] ** a["step"]), v / (1 - a["beta2"] ** a["step"])
    theta = s["master"].to(f64) * (1 - a["lr"] * a["weight_decay"]) - a["lr"] * m_hat / (v_hat.sqrt() + a["eps"])
    return dict(norm=norm, master=theta, m=m, v=v, param=theta)
