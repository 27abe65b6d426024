"""Preference tuning of one adapted block, end to end on the library's operators.

A frozen NF4 model of one MLP block and a vocabulary projection, with LoRA adapters on all
four linears and a trained residual gate, learns to prefer the chosen answer of each pair:

    h  = norm(x);  y = mlp(h);  x' = x + gate * norm(y), h' = norm(x');  logits = head(h')

Each step runs the forward (norm_residual_fwd, mlp_fwd, linear_fwd), the loss against the
frozen base's log-probabilities (token_logps once, preference_loss), the backward
(linear_bwd, norm_residual_bwd, mlp_bwd), the clipping of all gradients into one flat buffer
(GradList, grad_clip), and AdamW over it (adamw_step).  Synthetic data; no files are read.

    python examples/preference_step.py [steps]
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_nf4_quantized_dq_amd as Q  # noqa: E402

BF16 = torch.bfloat16


class Model:
    """Frozen NF4 weights, and the trained parameters as views of one flat BF16 working copy."""

    def __init__(self, d=512, f=1024, vocab=2048, r=16, alpha=32.0, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s, std=1.0: torch.randn(*s, generator=gen, device=device) * std  # noqa: E731
        shapes = [(f, d), (f, d), (d, f), (vocab, d)]  # gate, up, down, head
        self.w = [Q.quantize(rand(n, k, std=k**-0.5)) for n, k in shapes]
        self.embed = rand(vocab, d).to(BF16)
        self.norms = [(1 + rand(d, std=0.1)).to(BF16) for _ in range(3)]  # before, after, last
        self.alpha = alpha
        init = [rand(r, k, std=k**-0.5) for _, k in shapes] + [torch.zeros(n, r, device=device) for n, _ in shapes]
        init.append(torch.ones(1, d, device=device))  # the block's gate
        sizes = [t.numel() for t in init]
        self.master = torch.cat([t.reshape(-1) for t in init])
        self.m, self.v = torch.zeros_like(self.master), torch.zeros_like(self.master)
        self.param = self.master.to(BF16)
        self.grad = torch.zeros_like(self.param)
        view = lambda flat: [p.view(t.shape) for p, t in zip(flat.split(sizes), init)]  # noqa: E731
        params = view(self.param)
        self.A, self.B, self.gate = params[:4], params[4:8], params[8]
        self.grad_views = view(self.grad)
        self.t = 0

    def forward(self, tokens, adapted=True):
        """Logits [n, S, vocab], and what the backward needs."""
        A, B, gate = self.A, self.B, self.gate
        if not adapted:
            B, gate = [torch.zeros_like(b) for b in B], torch.ones_like(gate)
        x = self.embed[tokens.reshape(-1)]
        M = x.shape[0]
        _, h = Q.norm_residual_fwd(x, w_pre=self.norms[0])
        y = Q.mlp_fwd(self.w[:3], h, A[:3], B[:3], self.alpha)
        xo, last = Q.norm_residual_fwd(x, y, post_norm=True, w_post=self.norms[1], gate=gate, gate_rows=M,
                                       w_pre=self.norms[2])
        logits = Q.linear_fwd(self.w[3], last, A[3], B[3], self.alpha)
        return logits.view(*tokens.shape, -1), (h, y, xo, last)

    def backward(self, dlogits, saved):
        """Gradients in the parameters' order."""
        h, y, xo, last = saved
        M = h.shape[0]
        dlast, dA3, dB3 = Q.linear_bwd(self.w[3], last, dlogits.view(M, -1), self.A[3], self.B[3], self.alpha)
        _, dy, _, dgate, _ = Q.norm_residual_bwd(xo, y, dlast, post_norm=True, w_post=self.norms[1], gate=self.gate,
                                                 gate_rows=M, w_pre=self.norms[2], need_weights=False)
        _, dA, dB = Q.mlp_bwd(self.w[:3], h, dy, self.A[:3], self.B[:3], self.alpha)
        return [*dA, dA3, *dB, dB3, dgate]

    def update(self, grads, max_norm, lr):
        """Clips the gradients into the flat buffer and steps; returns their norm."""
        norm = Q.grad_clip(Q.GradList(grads, out=self.grad_views), max_norm)
        self.t += 1
        Q.adamw_step(self.master, self.m, self.v, self.grad, self.t, lr, param=self.param)
        return norm


def batch(model, pairs=4, S=48, prompt=16, seed=1):
    """Pairs that share a prompt: the chosen answers use the lower half of the vocabulary, the
    rejected ones the upper half.  Labels are the next tokens; prompts and padding are masked."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    vocab = model.embed.shape[0]
    pick = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=gen, device="cuda")  # noqa: E731
    text = pick(0, vocab, pairs, prompt).repeat(2, 1)
    answers = torch.cat([pick(0, vocab // 2, pairs, S + 1 - prompt), pick(vocab // 2, vocab, pairs, S + 1 - prompt)])
    tokens = torch.cat([text, answers], 1)
    labels = tokens[:, 1:].clone()
    labels[:, : prompt - 1] = -100
    length = pick(S // 2, S + 1, 2 * pairs, 1)
    labels[torch.arange(S, device="cuda")[None] >= length] = -100
    return tokens[:, :-1].contiguous(), labels


def train(steps=20, beta=0.1, max_norm=1.0, lr=1e-3, report=print):
    model = Model()
    tokens, labels = batch(model)
    ref = Q.token_logps(model.forward(tokens, adapted=False)[0], labels)
    losses, norms = [], []
    for step in range(steps):
        logits, saved = model.forward(tokens)
        loss, ratios, _, dlogits = Q.preference_loss(logits, labels, ref, beta, dlogits=logits)
        norm = model.update(model.backward(dlogits, saved), max_norm, lr)
        losses.append(float(loss))
        norms.append(float(norm))
        half = len(ratios) // 2
        report(f"step {step}: loss {losses[-1]:.4f}, margin {float((ratios[:half] - ratios[half:]).mean()):+.2f}, "
               f"gradient norm {norms[-1]:.3f}")
    return losses, norms


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 20)
