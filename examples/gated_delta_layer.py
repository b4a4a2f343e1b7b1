"""A layer of the gated delta rule between rms norms, served and trained.

    s = x + r;  n = norm(s);  q, k, v = n Uq^T, n Uk^T, n Uv^T;  k of each head of unit length, q too
    decay = exp(-softplus(n Ud^T)), beta = sigmoid(n Ub^T)
    r' = norm_per_head(rule(q, k, v, decay, beta)) Uo^T;  n' = norm(s + r') in 8 bits with scales

Runs a prompt, then its last tokens one at a time from the carried state, and
compares the two; compares the 8-bit rows with the same rows in fp32; then one
backward pass of the norms and the rule, compared with a difference quotient.
Needs the GPU:

    python examples/gated_delta_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from persistent_rnn_fwd_amd import Handle  # noqa: E402


class Layer:
    """Width heads * size; projections fp16, as the library's own take them."""

    def __init__(self, handle, heads, key_heads, size, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        width, keys = heads * size, key_heads * size

        def weights(n, m):
            return (torch.randn((n, m), generator=g, device="cuda") * m ** -0.5).half()

        self.handle, self.heads, self.key_heads, self.size = handle, heads, key_heads, size
        self.Uq, self.Uk, self.Uv, self.Uo = weights(keys, width), weights(keys, width), weights(width, width), weights(width, width)
        self.Ud, self.Ub = weights(heads, width), weights(heads, width)
        self.norm = torch.ones(width, device="cuda")
        self.head_norm = torch.ones(size, device="cuda")
        # the root of the mean square is the length over size ** 0.5
        self.unit = torch.full((size,), size ** -0.5, device="cuda")

    def project(self, n):
        """q, k and v of the heads (q and k not yet of unit length), log decay and beta."""
        lead, p = n.shape[:-1], self.handle.project
        return (p(self.Uq, n).view(*lead, self.key_heads, self.size), p(self.Uk, n).view(*lead, self.key_heads, self.size),
                p(self.Uv, n).view(*lead, self.heads, self.size), -torch.nn.functional.softplus(p(self.Ud, n)),
                torch.sigmoid(p(self.Ub, n)))

    def units(self, x, rstd=None):
        return self.handle.rms_norm(x, self.unit, 1e-12, rstd=rstd)

    def layer(self, x, r, rule):
        """Of x and what the layer before adds to it: the sum, and what this one adds."""
        s = torch.empty_like(x)
        q, k, v, log_decay, beta = self.project(self.handle.rms_norm(x, self.norm, residual=r, sum_out=s))
        o = rule(self.units(q), self.units(k), v, log_decay, beta)
        return s, self.handle.project(self.Uo, self.handle.rms_norm(o, self.head_norm).flatten(-2))

    def prompt(self, x, r, state):
        """x and r [T, B, width]; state [B, heads, size, size] is carried on in place."""
        return self.layer(x, r, lambda *a: self.handle.gated_delta_rule(*a, initial_state=state, final_state=state))

    def step(self, x, r, state):
        """One token of each sequence, x and r [B, width]."""
        return self.layer(x, r, lambda *a: self.handle.gated_delta_rule_step(*a, state))

    def outputs(self, q, k, v, log_decay, beta, keep=None):
        """norm_per_head(rule(unit(q), unit(k), v, ..)); keep gets what the gradients need."""
        h = self.handle
        rq, rk, ro = (torch.empty(t.shape[:-1], device="cuda") for t in (q, k, v))
        qn, kn = self.units(q, rq), self.units(k, rk)
        o = h.gated_delta_rule(qn, kn, v, log_decay, beta)
        if keep is not None:
            keep += [qn, kn, o, rq, rk, ro]
        return h.rms_norm(o, self.head_norm, rstd=ro)

    def gradients(self, q, k, v, log_decay, beta, dy):
        """Of the sum of dy * outputs: dq, dk, dv, dlog_decay, dbeta and the head norm's dweight."""
        h, keep = self.handle, []
        self.outputs(q, k, v, log_decay, beta, keep)
        qn, kn, o, rq, rk, ro = keep
        do, dw = h.rms_norm_backward(dy, o, ro, self.head_norm)
        dqn, dkn, dv, dg, db = h.gated_delta_rule_backward(qn, kn, v, log_decay, beta, do)
        dq, _ = h.rms_norm_backward(dqn, q, rq, self.unit)
        dk, _ = h.rms_norm_backward(dkn, k, rk, self.unit)
        return dq, dk, dv, dg, db, dw


def main(T=200, B=3, heads=4, key_heads=2, size=64, steps=8):
    g = torch.Generator(device="cuda").manual_seed(1)
    with Handle() as h:
        layer = Layer(h, heads, key_heads, size)
        x, r = (torch.randn((T, B, heads * size), generator=g, device="cuda") for _ in range(2))
        s, whole = layer.prompt(x, r, torch.zeros((B, heads, size, size), device="cuda"))

        state = torch.zeros((B, heads, size, size), device="cuda")
        parts = [layer.prompt(x[:T - steps], r[:T - steps], state)[1]]
        parts += [layer.step(x[t], r[t], state)[1][None] for t in range(T - steps, T)]
        apart = float((torch.cat(parts) - whole).abs().max() / whole.abs().max())
        print(f"prompt of {T} tokens against {T - steps} and {steps} single ones: {apart:.1e} apart")

        eight, scales = h.rms_norm_e4m3(s, layer.norm, residual=whole, group=128)
        n = h.rms_norm(s, layer.norm, residual=whole)
        width = n.shape[-1]
        back = eight.float() * scales.repeat_interleave(128, -1)[..., :width]
        # of a normal number half a step is at most 2^-4 of it; below 2^-6 a step is 2^-9
        step = torch.maximum(n.abs() * 2 ** -4, scales.repeat_interleave(128, -1)[..., :width] * 2.0 ** -10)
        eighth = float(((back - n).abs() / step).max())
        print(f"8-bit rows: {eighth:.3f} half steps from the rows in fp32")

        inputs = layer.project(n)
        dy = torch.randn((T, B, heads, size), generator=g, device="cuda")
        grads = layer.gradients(*inputs, dy)[:5]
        along = [0.2 * torch.randn(t.shape, generator=g, device="cuda") for t in inputs]
        along[3], along[4] = along[3] * inputs[3], along[4] * inputs[4]  # decays stay below 1
        each = [float((a.double() * d.double()).sum()) for a, d in zip(along, grads)]
        eps = 1e-2
        up, down = (float((layer.outputs(*(t + e * a for t, a in zip(inputs, along))).double() * dy.double()).sum()) for e in (eps, -eps))
        spread = sum(float((a.double() * d.double()).square().sum()) for a, d in zip(along, grads)) ** 0.5
        off = abs((up - down) / (2 * eps) - sum(each)) / spread
        print(f"slope {sum(each):.4f}, from differences {(up - down) / (2 * eps):.4f} ({off:.1e} of its spread apart)")
        h.synchronize()
    return apart, eighth, off


if __name__ == "__main__":
    apart, eighth, off = main()
    sys.exit(0 if apart < 1e-4 and eighth < 1.001 and off < 1e-2 else 1)
