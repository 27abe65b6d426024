"""The plain oracle of the frozen linear with many adapters and of dropout, in FP64 (torch, on
whatever device the operands are), with the sums of absolute terms that the tests' tolerances
are made of.  Test infrastructure only."""

from __future__ import annotations

import numpy as np
import torch

F64 = torch.float64


def philox(counter, key):
    """Philox4x32-10 (Salmon et al. 2011) of uint32 words: counter [n, 4], key (k0, k1) -> uint32 [n, 4]."""
    m = np.uint64(0xFFFFFFFF)
    c = [np.asarray(counter, dtype=np.uint64)[:, i].copy() for i in range(4)]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [((p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0)) & m, p1 & m, ((p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1)) & m, p0 & m]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, 1).astype(np.uint32)


def threshold(p: float) -> int:
    return int(np.floor(float(np.float32(p)) * 65536 + 0.5))


def keep_mask(n: int, p: float, seed: int, offset: int) -> np.ndarray:
    """bool [n]: which elements stay."""
    t = threshold(p)
    if t == 0:
        return np.ones(n, dtype=bool)
    words = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF, offset & 0xFFFFFFFF, (offset >> 32) & 0xFFFFFFFF]
    block = np.arange((n + 7) // 8, dtype=np.uint64)
    ctr = np.stack([block & np.uint64(0xFFFFFFFF), block >> np.uint64(32), np.full_like(block, words[2]),
                    np.full_like(block, words[3])], 1)
    w = philox(ctr, words[:2])
    halves = np.stack([w & 0xFFFF, w >> 16], 2).reshape(-1)
    return halves[:n] >= t


def scale(p: float) -> float:
    return 65536.0 / (65536.0 - threshold(p))


def _masked(X, p, rng):
    """(drop(X), mask times scale or None)."""
    if threshold(p) == 0:
        return X, None
    keep = torch.from_numpy(keep_mask(X.numel(), p, *rng)).to(X.device).view(X.shape)
    return torch.where(keep, X * scale(p), 0.0), keep.to(F64) * scale(p)


def _members(ids, count, M):
    ids = torch.zeros(M, dtype=torch.int64) if ids is None else ids.cpu().long()
    return [(ids == a).nonzero()[:, 0] for a in range(count)]


def fwd(what, A, B, alpha, X, ids=None, p=0.0, rng=(0, 0)):
    """Y, T and the absolute sums of Y's base term, of its adapters' term and of T.  what: the decoded
    weight; operands of any float type."""
    what, X = what.to(F64), X.to(F64)
    M, width = X.shape[0], -(-max(a.shape[0] for a in A) // 8) * 8
    Xd, _ = _masked(X, p, rng)
    Y, base = X @ what.T, X.abs() @ what.abs().T
    T = torch.zeros(M, width, dtype=F64, device=X.device)
    Tm, branch = torch.zeros_like(T), torch.zeros_like(Y)
    for a, at in enumerate(_members(ids, len(A), M)):
        at = at.to(X.device)
        if not len(at):
            continue
        Aa, Ba, r = A[a].to(F64), B[a].to(F64), A[a].shape[0]
        T[at, :r], Tm[at, :r] = Xd[at] @ Aa.T, Xd[at].abs() @ Aa.abs().T
        Y[at] += alpha[a] / r * (T[at, :r] @ Ba.T)
        branch[at] = abs(alpha[a] / r) * (Tm[at, :r] @ Ba.abs().T)
    return dict(Y=Y, T=T, Y_base=base, Y_branch=branch, T_sum=Tm)


def bwd(what, A, B, alpha, X, dY, ids=None, p=0.0, rng=(0, 0), T=None):
    """dX, dA, dB (lists) and their absolute sums."""
    what, X, dY = what.to(F64), X.to(F64), dY.to(F64)
    M = X.shape[0]
    Xd, gate = _masked(X, p, rng)
    dX, base, branch = dY @ what, dY.abs() @ what.abs(), torch.zeros_like(X)
    out = dict(dX=dX, dX_base=base, dX_branch=branch, dA=[], dB=[], dA_sum=[], dB_sum=[])
    for a, at in enumerate(_members(ids, len(A), M)):
        at = at.to(X.device)
        Aa, Ba, r = A[a].to(F64), B[a].to(F64), A[a].shape[0]
        s = alpha[a] / r
        G, Gm = dY[at] @ Ba, dY[at].abs() @ Ba.abs()
        back, backm = s * (G @ Aa), abs(s) * (Gm @ Aa.abs())
        dX[at] += back if gate is None else torch.where(gate[at] > 0, back * gate[at], 0.0)
        branch[at] = backm if gate is None else torch.where(gate[at] > 0, backm * gate[at], 0.0)
        t = Xd[at] @ Aa.T if T is None else T[at, :r].to(F64)
        tm = Xd[at].abs() @ Aa.abs().T if T is None else t.abs()
        out["dA"].append(s * (G.T @ Xd[at]))
        out["dA_sum"].append(abs(s) * (Gm.T @ Xd[at].abs()))
        out["dB"].append(s * (dY[at].T @ t))
        out["dB_sum"].append(abs(s) * (dY[at].abs().T @ tm))
    return out


def dropout(x, p, rng, residual=None):
    y, _ = _masked(x.to(F64).reshape(-1), p, rng)
    y = y.view(x.shape)
    return y if residual is None else y + residual.to(F64)
