"""A layer of linear attention with a decay for each head, served and trained.

    n = norm(x);  q, k, v = n Uq^T, n Uk^T, n Uv^T;  o = attention(q, k, v)
    y = x + norm_per_head(o) Uo^T

Runs a prompt, then its last tokens one at a time from the carried state, and
compares the two; then one backward pass of the norms and the attention, compared
with a difference quotient.  Needs the GPU:

    python examples/linear_attention_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from persistent_rnn_fwd_amd import Handle  # noqa: E402


class Layer:
    """Width heads * size; projections fp16, as the library's own take them."""

    def __init__(self, handle, heads, kv_heads, size, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        width, kv = heads * size, kv_heads * size

        def weights(n, m):
            return (torch.randn((n, m), generator=g, device="cuda") * m ** -0.5).half()

        self.handle, self.heads, self.kv_heads, self.size = handle, heads, kv_heads, size
        self.Uq, self.Uk, self.Uv, self.Uo = weights(width, width), weights(kv, width), weights(kv, width), weights(width, width)
        self.norm = [torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")]
        self.head_norm = [torch.ones(size, device="cuda"), torch.zeros(size, device="cuda")]
        # half-lives from a few tokens to some hundred
        self.log_decay = torch.log1p(-torch.exp2(-3 - 6 * torch.arange(heads, device="cuda") / heads))

    def project(self, n):
        lead = n.shape[:-1]
        q, k, v = (self.handle.project(U, n) for U in (self.Uq, self.Uk, self.Uv))
        return (q.view(*lead, self.heads, self.size), k.view(*lead, self.kv_heads, self.size),
                v.view(*lead, self.kv_heads, self.size))

    def output(self, x, o):
        o = self.handle.layer_norm(o, *self.head_norm)
        return x + self.handle.project(self.Uo, o.flatten(-2))

    def prompt(self, x, state):
        """x [T, B, width]; state [B, heads, size, size] is carried on in place."""
        q, k, v = self.project(self.handle.layer_norm(x, *self.norm))
        return self.output(x, self.handle.linear_attention(q, k, v, self.log_decay, initial_state=state, final_state=state))

    def step(self, x, state):
        """One token of each sequence, x [B, width]."""
        q, k, v = self.project(self.handle.layer_norm(x, *self.norm))
        return self.output(x, self.handle.linear_attention_step(q, k, v, self.log_decay, state))

    def gradients(self, q, k, v, dy):
        """Of the sum of dy * norm_per_head(attention(q, k, v)): dq, dk, dv and the
        norm's dweight, dbias."""
        h = self.handle
        o = h.linear_attention(q, k, v, self.log_decay)
        mean, rstd = (torch.empty(o.shape[:-1], device="cuda") for _ in range(2))
        h.layer_norm(o, *self.head_norm, mean=mean, rstd=rstd)
        do, dw, db = h.layer_norm_backward(dy, o, mean, rstd, self.head_norm[0])
        return (*h.linear_attention_backward(q, k, v, self.log_decay, do), dw, db)

    def loss(self, q, k, v, dy):
        o = self.handle.layer_norm(self.handle.linear_attention(q, k, v, self.log_decay), *self.head_norm)
        return float((o.double() * dy.double()).sum())


def main(T=200, B=3, heads=4, kv_heads=2, size=64, steps=8):
    g = torch.Generator(device="cuda").manual_seed(1)
    with Handle() as h:
        layer = Layer(h, heads, kv_heads, size)
        x = torch.randn((T, B, heads * size), generator=g, device="cuda")
        whole = layer.prompt(x, torch.zeros((B, heads, size, size), device="cuda"))

        state = torch.zeros((B, heads, size, size), device="cuda")
        parts = [layer.prompt(x[:T - steps], state)] + [layer.step(x[t], state)[None] for t in range(T - steps, T)]
        apart = float((torch.cat(parts) - whole).abs().max() / whole.abs().max())
        print(f"prompt of {T} tokens against {T - steps} and {steps} single ones: {apart:.1e} apart")

        q, k, v = layer.project(h.layer_norm(x, *layer.norm))
        dy = torch.randn((T, B, heads, size), generator=g, device="cuda")
        dq, dk, dv, dw, db = layer.gradients(q, k, v, dy)
        along = [torch.randn(t.shape, generator=g, device="cuda") for t in (q, k, v)]
        slope = sum(float((a.double() * d.double()).sum()) for a, d in zip(along, (dq, dk, dv)))
        eps = 1e-2
        up, down = (layer.loss(*(t + s * a for t, a in zip((q, k, v), along)), dy) for s in (eps, -eps))
        off = abs((up - down) / (2 * eps) - slope) / sum(float((a.double() * d.double()).square().sum()) for a, d in
                                                           zip(along, (dq, dk, dv))) ** 0.5
        print(f"slope {slope:.4f}, from differences {(up - down) / (2 * eps):.4f} ({off:.1e} of its spread apart)")
        h.synchronize()
    return apart, off


if __name__ == "__main__":
    apart, off = main()
    sys.exit(0 if apart < 1e-4 and off < 1e-2 else 1)
