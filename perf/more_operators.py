"""The operators of a frozen 4-bit linear that many low-rank adapters share, as cases to be
measured: its forward for rows that each name their adapter (requests being served, sequences
of several tasks in one training batch), its backward with every adapter's gradients, both
with the adapters' input dropout, and the dropout of a residual stream.  Dropout masks come
from a counter-based generator (Philox4x32-10, Salmon et al. 2011) and are never stored.

`run` computes a case in plain form (elementary torch operations in FP32, rounded once at
the end) where `own` is false, and calls this repository's entry points where it is true.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
# FP32 levels of the 4-bit NormalFloat codes
NF4 = [-1.0, -0.728114128112793, -0.5598623156547546, -0.4367327392101288, -0.33419176936149597, -0.24312838912010193,
       -0.15887711942195892, -0.07853864878416061, 0.0, 0.1078658401966095, 0.2182035744190216, 0.33391520380973816,
       0.4589826464653015, 0.5998135805130005, 0.7689210772514343, 1.0]
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _linear(op, M, d_out, d_in, adapters, rank, mixed, rows, p=0.0, saved=True, **name):
    """rows: "one" (all rows adapter 0), "tokens" (each row its own request, some without an
    adapter) or "sequences" (ragged runs of rows).  mixed: ranks from 1 up to `rank`.  p: dropout
    of the adapters' input.  saved: the backward has the forward's T = drop(X) A^T at hand."""
    return dict(op=op, M=M, d_out=d_out, d_in=d_in, adapters=adapters, rank=rank, mixed=mixed, rows=rows, p=p, saved=saved, **name)


def listed():
    return [
        # one decoded token of one request, eight adapters loaded: latency counts
        _linear("fwd", 1, 4096, 4096, 8, 16, False, "tokens", name="serve 1 of 8 adapters 4096x4096"),
        # a decode batch of requests over adapters of mixed ranks, some rows without any; wide projection
        _linear("fwd", 37, 14336, 4096, 24, 64, True, "tokens", name="serve 37 of 24 adapters 14336x4096"),
        # a large decode batch, many adapters, down projection
        _linear("fwd", 256, 4096, 14336, 48, 16, False, "tokens", name="serve 256 of 48 adapters 4096x14336"),
        # prompts of several requests in one pass, key projection
        _linear("fwd", 1999, 1024, 4096, 12, 32, True, "sequences", name="prompts 1999 of 12 adapters 1024x4096"),
        # a short odd training batch on a small layer
        _linear("train_fwd", 33, 1040, 320, 3, 8, True, "sequences", p=0.1, name="train fwd 33 of 3 adapters 1040x320"),
        # a training batch, one adapter of rank 64 with dropout on its input
        _linear("train_fwd", 8192, 4096, 4096, 1, 64, False, "one", p=0.05, name="train fwd 8192 dropout 4096x4096"),
        # a ragged batch of several tasks, mixed ranks, dropout, T recomputed (checkpointing)
        _linear("bwd", 555, 1040, 4096, 6, 40, True, "sequences", p=0.1, saved=False, name="train bwd 555 of 6 adapters 1040x4096"),
        # one adapter of rank 64 with dropout on its input
        _linear("bwd", 4096, 4096, 4096, 1, 64, False, "one", p=0.05, name="train bwd 4096 dropout 4096x4096"),
        # four tasks trained at once on the gate projection
        _linear("bwd", 8192, 14336, 4096, 4, 16, False, "sequences", name="train bwd 8192 of 4 adapters 14336x4096"),
        # one decoded token's activations while a model is sampled with dropout on: latency counts
        dict(op="dropout", M=1, d=4096, x="bf16", out="bf16", residual=False, p=0.1, name="dropout 1x4096"),
        # a block's output dropped and added to the residual stream
        dict(op="dropout", M=8192, d=4096, x="bf16", out="bf16", residual=True, p=0.1, name="dropout add 8192x4096"),
        # the gradient of an FP32 stream of odd width on its way back into a BF16 block
        dict(op="dropout", M=1777, d=2051, x="f32", out="bf16", residual=False, p=0.5, name="dropout 1777x2051 f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, unit, lo, hi):
    """A multiple of `unit` in [lo, hi]: any, or a model's (4, 5 or 7 times a power of two)."""
    n = _log(rng, lo, hi)
    if rng.random() < 0.5:
        return max(lo, n // unit * unit)
    return min((m << k for m in (4, 5, 7) for k in range(4, 16) if lo <= m << k <= hi and not (m << k) % unit), key=lambda w: abs(w - n))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "fwd", "train_fwd", "train_fwd", "bwd", "bwd", "bwd", "dropout"])
    if op == "dropout":
        d = _log(rng, 64, 16384)
        residual = rng.random() < 0.5
        return dict(op=op, M=_log(rng, 1, max(1, min(16384, (1 << 26) // d))), d=d, x=rng.choice(["bf16", "f32"]),
                    out=rng.choice(["bf16", "f32"]), residual=residual, p=rng.choice([0.05, 0.1, 0.3, 0.5]))
    d_out, d_in = _width(rng, 16, 64, 16384), _width(rng, 64, 64, 16384)
    M = _log(rng, 1, max(1, min(8192, (1 << 38) // (d_out * d_in))))
    adapters = _log(rng, 1, 64)
    rows = rng.choice(["tokens", "sequences"] if M <= 512 else ["sequences"])
    if op != "fwd" and rng.random() < 0.4:
        adapters, rows = 1, "one"
    return _linear(op, M, d_out, d_in, adapters, _log(rng, 4, 128), rng.random() < 0.5, rows,
                   0.0 if op == "fwd" else rng.choice([0.0, 0.05, 0.1]), rng.random() < 0.5)


def _ranks(case):
    n, r = case["adapters"], case["rank"]
    if not case["mixed"]:
        return [r] * n
    rng = random.Random(n * 7919 + r)
    return [r] + [rng.choice([r, max(1, r // 2), max(1, r // 4), rng.randint(1, r)]) for _ in range(n - 1)]


def _ids(case):
    """The adapter of each row, -1 for none."""
    M, n, rng = case["M"], case["adapters"], random.Random(case["M"] * 31 + case["adapters"])
    if case["rows"] == "one":
        return [0] * M
    if case["rows"] == "tokens":  # requests in the order of their arrival
        return [-1 if M > 8 and rng.random() < 0.05 else rng.randrange(n) for _ in range(M)]
    ids, turn = [], rng.sample(range(n), n)
    while len(ids) < M:  # sequences of uneven lengths, the adapters in turn
        ids += [turn[0]] * max(1, int(M / max(4, n) * (0.4 + 1.2 * rng.random())))
        turn = turn[1:] + turn[:1]
    return ids[:M]


def _randn(gen, shape, std=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device=DEV).mul_(std).to(dtype)


def _quantized(gen, d_out, d_in):
    """A weight as it is stored: codes, 8-bit block constants, their scales and mean."""
    level = torch.tensor(NF4, device=DEV)
    w = _randn(gen, (d_out * d_in // 64, 64), 0.02)
    c1 = w.abs().amax(1)
    code = torch.bucketize(w / c1[:, None], (level[1:] + level[:-1]) / 2).to(torch.uint8).view(-1, 8)
    mu = c1.double().mean().float().reshape(1)
    d = torch.nn.functional.pad(c1 - mu, (0, -len(c1) % 256)).view(-1, 256)
    c2s = d.abs().amax(1) / 448
    code8 = (d / c2s[:, None].clamp(min=1e-30)).to(torch.float8_e4m3fn).view(torch.uint8).view(-1)[: len(c1)]
    return dict(codes=(code[:, :4] | code[:, 4:] << 4).reshape(-1), code8=code8.contiguous(), c2s=c2s, mu=mu)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    bf16 = torch.bfloat16
    s = dict(case=case, rng=torch.randint(0, 1 << 62, (2,), generator=gen, device=DEV))  # the generator's seed and offset
    if case["op"] == "dropout":
        shape = (case["M"], case["d"])
        s["x"] = _randn(gen, shape, 1.0, DTYPE[case["x"]])
        s["residual"] = _randn(gen, shape, 2.0, DTYPE[case["out"]]) if case["residual"] else None
        s["out"] = torch.empty(shape, device=DEV, dtype=DTYPE[case["out"]])
        return s
    M, d_out, d_in = case["M"], case["d_out"], case["d_in"]
    s["ranks"] = _ranks(case)
    s["weight"] = _quantized(gen, d_out, d_in)
    s["A"] = [_randn(gen, (r, d_in), d_in**-0.5, bf16) for r in s["ranks"]]
    s["B"] = [_randn(gen, (d_out, r), 0.1, bf16) for r in s["ranks"]]
    s["alpha"] = [float(max(8, r)) for r in s["ranks"]]
    s["X"] = _randn(gen, (M, d_in), 1.0, bf16)
    s["ids"] = None if case["rows"] == "one" else torch.tensor(_ids(case), device=DEV, dtype=torch.int32)
    width = -(-max(s["ranks"]) // 8) * 8
    s["T"] = None
    if case["op"] == "train_fwd":
        s["T"] = torch.empty(M, width, device=DEV)
    elif case["op"] == "bwd":
        s["dY"] = _randn(gen, (M, d_out), 0.01, bf16)
        # the optimizer's flat gradients
        s["dA"] = torch.empty(sum(s["ranks"]) * d_in, device=DEV, dtype=bf16)
        s["dB"] = torch.empty(sum(s["ranks"]) * d_out, device=DEV, dtype=bf16)
        if case["saved"]:  # as the forward left it: zeros past the row's rank, and for rows without an adapter
            ids = torch.zeros(M, dtype=torch.int64, device=DEV) if s["ids"] is None else s["ids"].long()
            rank = torch.tensor(s["ranks"] + [0], device=DEV)[ids]
            s["T"] = _randn(gen, (M, width)) * (torch.arange(width, device=DEV) < rank[:, None])
    if own:
        import bit_nf4_quantized_dq_amd as Q

        w = s["weight"]
        s["q"] = Q.QuantizedWeight(w["codes"], w["code8"], w["c2s"], w["mu"], d_out, d_in)
        grads = {}
        if case["op"] == "bwd":
            grads = dict(dA=[t.view(-1, d_in) for t in s["dA"].split([r * d_in for r in s["ranks"]])],
                         dB=[t.view(d_out, -1) for t in s["dB"].split([r * d_out for r in s["ranks"]])])
        s["adapters"] = Q.AdapterSet(s["A"], s["B"], s["alpha"], **grads)
    return s


def _threshold(p):
    return int(p * 65536 + 0.5)


def _kept(rng, p, n):
    """Which of n elements stay: element e has half e % 8 of the block that counter (e // 8, offset) gives."""
    low = 0xFFFFFFFF
    at = torch.arange(-(-n // 8), device=DEV)
    seed, offset = rng[0], rng[1]
    a, b, c, d = at & low, at >> 32, offset & low, (offset >> 32) & low
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        x, y = a * 0xD2511F53, c * 0xCD9E8D57  # 64-bit products (modulo 2^64)
        a, b, c, d = ((y >> 32) & low) ^ b ^ k0, y & low, ((x >> 32) & low) ^ d ^ k1, x & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([a, b, c, d], 1)
    halves = torch.stack([words & 0xFFFF, words >> 16], 2).view(-1)[:n]
    return halves >= _threshold(p)


def _decoded(w, d_out, d_in):
    """The weight in BF16's values: level times recovered block constant, each FP32 step rounded."""
    b = w["codes"].view(-1, 4)
    q = torch.tensor(NF4, device=DEV)[torch.cat([b & 15, b >> 4], 1).long()]
    c2s = w["c2s"].repeat_interleave(256)[: len(w["code8"])]
    c1 = w["code8"].view(torch.float8_e4m3fn).float() * c2s + w["mu"]
    return (q.view(-1, 64) * c1[:, None]).bfloat16().float().view(d_out, d_in)


def _plain_linear(s):
    case = s["case"]
    M, d_out, d_in = case["M"], case["d_out"], case["d_in"]
    w = _decoded(s["weight"], d_out, d_in)
    X = s["X"].float()
    # all adapters side by side: a row keeps the columns of its own one
    A, B = torch.cat(s["A"]).float(), torch.cat(s["B"], 1).float()
    ranks = torch.tensor(s["ranks"], device=DEV)
    owner = torch.repeat_interleave(torch.arange(len(s["ranks"]), device=DEV), ranks, output_size=sum(s["ranks"]))
    scale = (torch.tensor(s["alpha"], device=DEV) / ranks)[owner]
    ids = torch.zeros(M, dtype=torch.int64, device=DEV) if s["ids"] is None else s["ids"].long()
    mine = (owner == ids[:, None]).float()
    Xd, keep = X, None
    if case["p"]:
        thr = _threshold(case["p"])
        keep = _kept(s["rng"], case["p"], M * d_in).view(M, d_in).float() * (65536 / (65536 - thr))
        Xd = X * keep
    width = -(-max(s["ranks"]) // 8) * 8
    first = torch.cumsum(ranks, 0) - ranks
    column = torch.arange(width, device=DEV) + first[ids.clamp(min=0)][:, None]  # where a row's own columns lie
    has = (torch.arange(width, device=DEV) < ranks[ids.clamp(min=0)][:, None]) & (ids >= 0)[:, None]
    column = column.clamp(max=len(owner) - 1)
    if case["op"] != "bwd":
        T = (Xd @ A.T) * mine
        Y = (X @ w.T + (T * scale) @ B.T).bfloat16()
        return Y if case["op"] == "fwd" else dict(Y=Y, T=torch.where(has, T.gather(1, column), 0.0))
    if s["T"] is None:
        T = (Xd @ A.T) * mine
    else:
        T = torch.zeros_like(mine).scatter_add_(1, column, torch.where(has, s["T"], 0.0))
    dY = s["dY"].float()
    G = (dY @ B) * mine * scale
    back = G @ A
    dX = (dY @ w + (back if keep is None else back * keep)).bfloat16()
    dA = (G.T @ Xd).bfloat16().view(-1)
    dB = (dY.T @ T) * scale  # [d_out, all ranks], flat adapter by adapter
    dB = torch.cat([t.reshape(-1) for t in dB.split(s["ranks"], 1)]).bfloat16()
    return dict(dX=dX, dA=dA, dB=dB)


def _plain_dropout(s):
    case, x = s["case"], s["x"].float()
    keep = _kept(s["rng"], case["p"], x.numel()).view(x.shape)
    y = torch.where(keep, x * (65536 / (65536 - _threshold(case["p"]))), 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["out"].dtype)


def _kernels(s):
    import bit_nf4_quantized_dq_amd as Q

    case = s["case"]
    if case["op"] == "dropout":
        return Q.dropout(s["x"], case["p"], s["rng"], residual=s["residual"], out=s["out"])
    if case["op"] == "fwd":
        return Q.linear_adapters_fwd(s["q"], s["adapters"], s["X"], s["ids"])
    if case["op"] == "train_fwd":
        Y = Q.linear_adapters_fwd(s["q"], s["adapters"], s["X"], s["ids"], dropout=case["p"], rng=s["rng"], T_save=s["T"])
        return dict(Y=Y, T=s["T"])
    dX = Q.linear_adapters_bwd(s["q"], s["adapters"], s["X"], s["dY"], s["ids"], dropout=case["p"], rng=s["rng"], T_saved=s["T"])
    return dict(dX=dX, dA=s["dA"], dB=s["dB"])


def run(state):
    if own:
        return _kernels(state)
    return _plain_dropout(state) if state["case"]["op"] == "dropout" else _plain_linear(state)


def work(case):
    if case["op"] == "dropout":
        n = case["M"] * case["d"]
        size = {"bf16": 2, "f32": 4}
        return dict(bytes=n * (size[case["x"]] + size[case["out"]] * (1 + case["residual"])), flops=2 * n)
    M, N, K = case["M"], case["d_out"], case["d_in"]
    ranks, ids = _ranks(case), _ids(case)
    used = sum(ranks[a] for a in set(ids) if a >= 0)  # ranks of the adapters that some row names
    rows = sum(ranks[a] for a in ids if a >= 0)  # ranks over all rows
    weight = N * K // 2 + N * K // 64
    width = -(-max(ranks) // 8) * 8
    if case["op"] != "bwd":
        T = 4 * M * width if case["op"] == "train_fwd" else 0
        return dict(bytes=weight + 2 * M * (N + K) + 2 * used * (N + K) + T + 4 * M, flops=2 * M * N * K + 2 * rows * (N + K))
    T = 4 * M * width if case["saved"] else 0
    return dict(bytes=weight + 2 * M * (N + 2 * K) + 2 * (used + sum(ranks)) * (N + K) + T + 4 * M,
                flops=2 * M * N * K + rows * (4 * N + 4 * K + (0 if case["saved"] else 2 * K)))


def _exact_kept(rng, p, n):
    """The same mask, from unsigned 64-bit integers on the host."""
    seed, offset = (int(v) & (2**64 - 1) for v in rng.tolist())
    u32, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    blocks = np.arange((n + 7) // 8, dtype=np.uint64)
    ctr = [blocks & u32, blocks >> half, np.full_like(blocks, offset & 0xFFFFFFFF), np.full_like(blocks, offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p0, p1 = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(p1 >> half) ^ ctr[1] ^ np.uint64(key[0]), p1 & u32, (p0 >> half) ^ ctr[3] ^ np.uint64(key[1]), p0 & u32]
        key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
    words = np.stack(ctr, 1).astype("<u4")
    return torch.from_numpy((words.view("<u2").reshape(-1)[:n] >= _threshold(p))).to(DEV)


def exact(case, seed):
    """The operators' definitions in FP64, adapter by adapter."""
    s = prepare(case, seed)
    f64 = torch.float64
    keep_scale = 65536.0 / (65536.0 - _threshold(case["p"]))
    if case["op"] == "dropout":
        y = s["x"].to(f64) * keep_scale
        y[~_exact_kept(s["rng"], case["p"], y.numel()).view(y.shape)] = 0.0
        return y if s["residual"] is None else y + s["residual"].to(f64)
    M, d_out, d_in = case["M"], case["d_out"], case["d_in"]
    w = s["weight"]
    byte = w["codes"].view(-1, 4, 1).expand(-1, 4, 2)
    code = (byte >> torch.tensor([0, 4], device=DEV, dtype=torch.uint8)) & 15  # [word, byte, nibble]
    level = torch.tensor(NF4, device=DEV)[code.transpose(1, 2).reshape(d_out, -1, 64).long()]  # low nibbles first
    group = torch.arange(len(w["code8"]), device=DEV) // 256
    c1 = w["code8"].view(torch.float8_e4m3fn).to(torch.float32).mul(w["c2s"][group]).add(w["mu"])
    weight = (level * c1.view(d_out, -1, 1)).to(torch.bfloat16).to(f64).view(d_out, d_in)
    X = s["X"].to(f64)
    Xd, gate = X, None
    if case["p"]:
        gate = _exact_kept(s["rng"], case["p"], M * d_in).view(M, d_in).to(f64) * keep_scale
        Xd = X * gate
    ids = torch.tensor(_ids(case), device=DEV)
    members = [(a, (ids == a).nonzero()[:, 0], s["A"][a].to(f64), s["B"][a].to(f64), s["alpha"][a] / s["ranks"][a])
               for a in range(case["adapters"])]
    if case["op"] != "bwd":
        Y = X @ weight.T
        T = torch.zeros(M, -(-max(s["ranks"]) // 8) * 8, device=DEV, dtype=f64)
        for a, at, A, B, scale in members:
            t = Xd[at] @ A.T
            T[at, : s["ranks"][a]] = t
            Y[at] += scale * (t @ B.T)
        return Y if case["op"] == "fwd" else dict(Y=Y, T=T)
    dY = s["dY"].to(f64)
    dX, dA, dB = dY @ weight, [], []
    for a, at, A, B, scale in members:
        g = scale * (dY[at] @ B)
        t = Xd[at] @ A.T if s["T"] is None else s["T"][at, : s["ranks"][a]].to(f64)
        dX[at] += g @ A if gate is None else (g @ A) * gate[at]
        dA.append((g.T @ Xd[at]).reshape(-1))
        dB.append((scale * (dY[at].T @ t)).reshape(-1))
    return dict(dX=dX, dA=torch.cat(dA), dB=torch.cat(dB))
