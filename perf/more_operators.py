"""What the gated delta rule (a prompt, its backward pass, one new token) and rms
norm (with the residual's addition and an 8-bit output, and its backward pass)
are measured on.

Each case is computed in its plain form (elementary torch operations in 32
bits) or, with ``own`` set, by the library's kernels.  Definitions, t the token
of a sequence and h the head (head h of v, o, the decay and beta uses head
h // (H // Hk) of q and k):

  gated delta rule  S[t] = a S[t-1] + beta k[t] (v[t] - a S[t-1]^T k[t])^T,   a = exp(log_decay[t]),
                    S[-1] = initial state or 0,   o[t] = scale * S[t]^T q[t]
  rms norm          s = x + residual,   y = s * rstd * weight,   rstd = 1 / sqrt(mean(s^2) + eps)
      in 8 bits     scale = max(max |y| / 448, 2^-126) over a row or 128 of its columns, and y / scale as e4m3

Tensors are laid out as everywhere in this library, time first: q, k [T, B, Hk,
Dk], v [T, B, H, Dv], log_decay and beta [T, B, H]; packed sequences drop B and
follow each other along the tokens, sequence b being rows offsets[b] ..
offsets[b + 1] - 1.
"""
from __future__ import annotations

import math
import random

import torch

own = False

EPS = 1e-6
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
CHUNK = 64  # tokens the plain form takes at once
GROUP = 128  # columns that share a scale where a row has several
E4M3_MAX = 448.0


# -- cases ---------------------------------------------------------------------------------------------------

def _delta(name, op, type, B, T, H, Hk, Dk, Dv, packed=False, state=False):
    case = {"op": op, "type": type, "B": B, "T": T, "H": H, "Hk": Hk, "Dk": Dk, "Dv": Dv}
    if op != "step":
        case.update(packed=packed, state=state)
    return {"name": name, **case} if name else case


def _norm(name, op, type, params, M, N, residual=False, out=None):
    """out: None (x's type), "row" or "group" (e4m3 with a scale for each row, or for each 128 of its columns)."""
    case = {"op": op, "type": type, "params": params, "M": M, "N": N, "residual": residual}
    if op == "norm":
        case["out"] = out or "same"
    return {"name": name, **case} if name else case


def listed():
    return [
        # One token of one request through a layer of width 1792 (14 heads of 128): latency.
        _delta("delta_step_one", "step", "f16", 1, 1, 14, 14, 128, 128),
        # One token of 64 requests served together, each head of q and k used by two heads of v: the
        # state's bandwidth.
        _delta("delta_step_batch", "step", "bf16", 64, 1, 32, 16, 128, 128),
        # Seven prompts of unequal length (one empty, one of a single token) packed into one call, with
        # carried states, as a server fills a batch.
        _delta("delta_prompt_packed", "forward", "f16", 7, 3001, 16, 4, 64, 64, packed=True, state=True),
        # A layer of width 1792 at the library's own batch and sequence (B = 4, T = 256), in fp32 as its
        # projections leave it.
        _delta("delta_prompt_layer", "forward", "f32", 4, 256, 14, 14, 128, 128),
        # One long prompt: few rows, a long axis.
        _delta("delta_prompt_long", "forward", "bf16", 1, 32768, 32, 16, 128, 128, state=True),
        # Backward of a layer of width 1152 in fp32 at B = 4, T = 256, two heads of 64 on each head of q and k.
        _delta("delta_grad_layer", "backward", "f32", 4, 256, 18, 9, 64, 64),
        # Backward with head sizes that fill no tile and a length that ends inside one.
        _delta("delta_grad_odd", "backward", "f16", 3, 1531, 6, 6, 96, 80, state=True),
        # Backward of one training batch.
        _delta("delta_grad_batch", "backward", "bf16", 8, 2048, 16, 16, 128, 128),
        # The four rows of one timestep at width 1792, with the residual: latency.
        _norm("rms_step", "norm", "f32", "f32", 4, 1792, residual=True),
        # The tokens of a batch at width 5760, the residual added, for a projection in 8 bits.
        _norm("rms_tokens_8bit", "norm", "bf16", "bf16", 16384, 5760, residual=True, out="row"),
        # A width that no vector load divides, 8 bits with a scale for each 128 columns.
        _norm("rms_odd_8bit", "norm", "f16", "f32", 4099, 1153, out="group"),
        # Backward of a training batch at width 5760, fp32 parameters, the residual's gradient added.
        _norm("rms_grad_tokens", "norm_backward", "bf16", "f32", 16384, 5760, residual=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _head_size(rng):
    if rng.random() < 0.25:
        return rng.randint(9, 255)
    return rng.choice((32, 48, 64, 80, 96, 112, 128, 128, 160, 192, 256))


def draw(rng):
    op = rng.choice(("step", "forward", "forward", "backward", "backward", "norm", "norm_backward"))
    limit = max((work(c) for c in listed() if c["op"] == op), key=lambda w: w["bytes"])
    while True:
        type = rng.choice(("f32", "f16", "bf16"))
        if op in ("norm", "norm_backward"):
            case = _norm(None, op, type, rng.choice(("f32", type)), _log_int(rng, 1, 400000), _log_int(rng, 32, 12000),
                         residual=rng.random() < 0.5, out=rng.choice((None, "row", "group")))
        else:
            Hk = rng.choice((1, 2, 3, 4, 5, 8, 12, 16))
            H = Hk * rng.choice((1, 1, 2, 3, 4))
            Dk = _head_size(rng)
            Dv = Dk if rng.random() < 0.6 else _head_size(rng)
            if op == "step":
                case = _delta(None, op, type, _log_int(rng, 1, 256), 1, H, Hk, Dk, Dv)
            else:
                case = _delta(None, op, type, _log_int(rng, 1, 32), _log_int(rng, 1, 32768), H, Hk, Dk, Dv,
                              packed=rng.random() < 0.3, state=rng.random() < 0.4)
        w = work(case)
        if w["bytes"] <= limit["bytes"] and w["flops"] <= limit["flops"]:
            return case


def _offsets(case):
    """Where the packed sequences of a case start: B of them in T tokens, the
    first empty where there are three or more, the second of one token."""
    B, T = case["B"], case["T"]
    rng = random.Random(1000 * T + B)
    fixed = [0, 1] if B >= 3 and T >= 2 else []
    rest = B - len(fixed)
    left = T - sum(fixed)
    cuts = sorted(rng.randint(0, left) for _ in range(rest - 1))
    lengths = fixed + [b - a for a, b in zip([0] + cuts, cuts + [left])]
    offsets = [0]
    for n in lengths:
        offsets.append(offsets[-1] + n)
    return offsets


def _tokens(case):
    return case["T"] if case.get("packed") else case["B"] * case["T"]


def work(case):
    """Inputs once, outputs once, and the multiply-adds of the recurrence
    itself: three products of the state with a vector and its decay a token; for
    the gradients also those of the adjoint recurrence, with the state's two
    again."""
    e = SIZE[case["type"]]
    if case["op"] in ("norm", "norm_backward"):
        M, N = case["M"], case["N"]
        p = SIZE[case["params"]]
        if case["op"] == "norm":
            out = {"same": e * N, "row": N + 4, "group": N + 4 * -(-N // GROUP)}[case["out"]]
            rows = (3 if case["residual"] else 1) * N * e + out + 4
            return {"bytes": M * rows + N * p, "flops": (6 if case["out"] == "same" else 9) * M * N}
        return {"bytes": (4 if case["residual"] else 3) * M * N * e + 2 * N * p + 4 * M, "flops": 11 * M * N}
    B, H, Hk, Dk, Dv = (case[x] for x in ("B", "H", "Hk", "Dk", "Dv"))
    n = _tokens(case)
    state = 4 * B * H * Dk * Dv
    qk, vo, scalars = n * Hk * 2 * Dk * e, n * H * Dv * e, n * H * 8
    if case["op"] == "step":
        return {"bytes": qk + 2 * vo + scalars + 2 * state, "flops": 7 * n * H * Dk * Dv}
    extra = 4 * (B + 1) if case["packed"] else 0
    if case["op"] == "forward":
        return {"bytes": qk + 2 * vo + scalars + extra + (2 * state if case["state"] else 0),
                "flops": 7 * n * H * Dk * Dv}
    return {"bytes": 2 * qk + 3 * vo + 2 * scalars + extra + (3 * state if case["state"] else 0),
            "flops": 20 * n * H * Dk * Dv}


# -- inputs --------------------------------------------------------------------------------------------------

def _inputs(case, seed):
    """Seeded inputs on the GPU.  Queries and keys are what a layer makes of its
    projections, silu and then unit length, so that keys of one head resemble
    each other; decays are -rate softplus(.), the rates from 2 down to 0.002
    along the heads; beta is a sigmoid."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    if case["op"] in ("norm", "norm_backward"):
        M, N = case["M"], case["N"]
        pt = TYPES[case["params"]]
        x = (normal(M, N) * (0.5 + 2.0 * torch.rand((M, 1), generator=g, device="cuda"))).to(dt)
        s = {"x": x, "weight": (1.0 + 0.1 * normal(N)).to(pt)}
        if case["op"] == "norm":
            s["residual"] = (2.0 * normal(M, N)).to(dt) if case["residual"] else None
            return s
        s["grad_out"] = normal(M, N).to(dt)
        s["grad_sum"] = normal(M, N).to(dt) if case["residual"] else None
        xd = x.double() if M * N <= 1 << 24 else x.float()  # the statistics the forward pass has left
        s["rstd"] = torch.rsqrt(xd.square().mean(1) + EPS).float()
        return s
    B, T, H, Hk, Dk, Dv = (case[x] for x in ("B", "T", "H", "Hk", "Dk", "Dv"))
    rows = (T,) if case.get("packed") else (B,) if case["op"] == "step" else (T, B)

    def unit(*shape):
        x = normal(*shape)
        x = x * torch.sigmoid(x)
        return (x / x.square().sum(-1, keepdim=True).add(1e-12).sqrt()).to(dt)

    s = {"q": unit(*rows, Hk, Dk), "k": unit(*rows, Hk, Dk), "v": normal(*rows, H, Dv).to(dt)}
    rate = 2.0 * torch.pow(10.0, -3.0 * torch.arange(H, device="cuda", dtype=torch.float32) / H)
    s["log_decay"] = -rate * torch.log1p(torch.exp(normal(*rows, H)))
    s["beta"] = torch.sigmoid(normal(*rows, H))
    s["scale"] = Dk ** -0.5
    if case["op"] == "step":
        s["state"] = normal(B, H, Dk, Dv)
        s["new_state"] = torch.empty_like(s["state"])
        return s
    s["offsets"] = None
    s["initial_state"] = normal(B, H, Dk, Dv) if case["state"] else None
    if case["packed"]:
        s["offsets"] = torch.tensor(_offsets(case), device="cuda", dtype=torch.int32)
        s["max_len"] = max(b - a for a, b in zip(_offsets(case), _offsets(case)[1:]))
        s["lengths_on_host"] = _offsets(case)
    if case["op"] == "backward":
        s["grad_out"] = normal(*rows, H, Dv).to(dt)
        s["grad_final_state"] = normal(B, H, Dk, Dv) if case["state"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        from persistent_rnn_fwd_amd import default_handle
        s["handle"] = default_handle()
    if case["op"] == "forward" and case["state"]:
        s["final_state"] = torch.empty_like(s["initial_state"])
    if case["op"] == "backward" and case["state"]:
        s["grad_initial_state"] = torch.empty_like(s["initial_state"])
    return s


# -- the library's calls -------------------------------------------------------------------------------------

def _run_own(s):
    h, case = s["handle"], s["case"]
    op = case["op"]
    if op == "norm":
        x = s["x"]
        rstd = torch.empty(x.shape[0], device=x.device)
        total = torch.empty_like(x) if case["residual"] else None
        kind = {"eps": EPS, "residual": s["residual"], "sum_out": total, "rstd": rstd}
        if case["out"] == "same":
            y = (h.rms_norm(x, s["weight"], **kind),)
        else:
            y = h.rms_norm_e4m3(x, s["weight"], group=GROUP if case["out"] == "group" else None, **kind)
        return (*y, rstd, total) if case["residual"] else (*y, rstd)
    if op == "norm_backward":
        return h.rms_norm_backward(s["grad_out"], s["x"], s["rstd"], s["weight"], grad_sum=s["grad_sum"])
    inputs = s["q"], s["k"], s["v"], s["log_decay"], s["beta"]
    if op == "step":
        return h.gated_delta_rule_step(*inputs, s["state"], scale=s["scale"], new_state=s["new_state"]), s["new_state"]
    seq = {"scale": s["scale"], "initial_state": s["initial_state"]}
    if s["offsets"] is not None:
        seq.update(offsets=s["offsets"], max_len=s["max_len"])
    if op == "forward":
        if not case["state"]:
            return h.gated_delta_rule(*inputs, **seq)
        return h.gated_delta_rule(*inputs, final_state=s["final_state"], **seq), s["final_state"]
    if not case["state"]:
        return h.gated_delta_rule_backward(*inputs, s["grad_out"], **seq)
    grads = h.gated_delta_rule_backward(*inputs, s["grad_out"], grad_final_state=s["grad_final_state"],
                                        grad_initial_state=s["grad_initial_state"], **seq)
    return (*grads, s["grad_initial_state"])


# -- the plain form ------------------------------------------------------------------------------------------

class _Chunks:
    """The inputs of one batch of sequences in chunks, [B, H, chunks, C, ...] in
    fp32, and what the chunks need of each other's pairs.  With G the sums of
    the log decays inside a chunk (64 bits) and d(i, j) = exp(G_i - G_j):

        inverse = (I + A)^-1,   A_ij = d(i, j) k_i.k_j beta_j  (j < i)
        pairs = scale d(i, j) q_i.k_j beta_j  (j <= i)

    x = inverse (v - exp(G) k S) are the corrected values and beta x what enters
    the state."""

    def __init__(self, q, k, v, a, beta, scale):
        T, B, H, _ = v.shape
        self.T, self.H, self.Hk, self.scale = T, H, q.shape[2], scale
        self.n = max(1, -(-T // CHUNK))
        self.q, self.k, self.v = (self.cut(x) for x in (q, k, v))
        self.beta = self.cut(beta[..., None])[..., 0]
        G = self.cut(a.double()[..., None])[..., 0].cumsum(-1)
        self.up = torch.exp(G).float()  # from the chunk's start through token i
        self.down = torch.exp(G[..., -1:] - G).float()  # from token i to the chunk's end
        self.whole = self.up[..., -1]
        lower = torch.ones((CHUNK, CHUNK), device=q.device, dtype=torch.bool).tril()
        self.decays = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~lower, -math.inf)).float()
        kk = torch.matmul(self.k, self.k.transpose(-1, -2))
        self.strict = self.decays * lower.tril(-1)
        self.inverse = self._inverse(kk * self.strict * self.beta[..., None, :])
        self.pairs = torch.matmul(self.q, self.k.transpose(-1, -2)) * self.decays * (scale * self.beta[..., None, :])

    def cut(self, x):
        """[T, B, h, D] -> [B, H, chunks, C, D], zeros behind the last token."""
        T, B, h, D = x.shape
        x = x if x.dtype == torch.float64 else x.float()
        x = torch.cat([x, x.new_zeros((self.n * CHUNK - T, B, h, D))]).permute(1, 2, 0, 3)
        return x.repeat_interleave(self.H // h, 1).reshape(B, self.H, self.n, CHUNK, D)

    def join(self, x, heads=None):
        """... and back, summed over the heads that share one."""
        B, H, n, C, D = x.shape
        x = x.reshape(B, H, n * C, D)[:, :, :self.T]
        if heads is not None:
            x = x.reshape(B, heads, H // heads, self.T, D).sum(2)
        return x.permute(2, 0, 1, 3)

    @staticmethod
    def _inverse(A):
        """(I + A)^-1 of strictly lower triangular blocks, from blocks of half the
        size: [[P, 0], [-Q A21 P, Q]]."""
        size, inv = 1, torch.ones((*A.shape[:-2], CHUNK, 1, 1), device=A.device)
        while size < CHUNK:
            blocks = A.unflatten(-1, (-1, 2 * size)).unflatten(-3, (-1, 2 * size))
            at = torch.arange(CHUNK // (2 * size), device=A.device)
            low = blocks[..., at, size:, at, :size].movedim(0, -3)
            first, second = inv[..., 0::2, :, :], inv[..., 1::2, :, :]
            corner = -torch.matmul(torch.matmul(second, low), first)
            inv = torch.cat([torch.cat([first, torch.zeros_like(corner)], -1), torch.cat([corner, second], -1)], -2)
            size *= 2
        return inv[..., 0, :, :]

    def forward(self, S):
        """The states that the chunks start from, x, and the last state."""
        x0 = torch.matmul(self.inverse, self.v)
        W = torch.matmul(self.inverse, self.k * self.up[..., None])
        into = (self.k * (self.down * self.beta)[..., None]).transpose(-1, -2)
        states, xs = [], []
        for c in range(self.n):
            states.append(S)
            xs.append(x0[:, :, c] - torch.matmul(W[:, :, c], S))
            S = S * self.whole[:, :, c, None, None] + torch.matmul(into[:, :, c], xs[-1])
        return torch.stack(states, 2), torch.stack(xs, 2), S


def _state_or_zeros(S, v, Dk):
    return S if S is not None else torch.zeros((v.shape[1], v.shape[2], Dk, v.shape[3]), device=v.device)


def _plain_forward(q, k, v, a, beta, scale, initial):
    c = _Chunks(q, k, v, a, beta, scale)
    states, x, S = c.forward(_state_or_zeros(initial, v, q.shape[3]))
    o = torch.matmul(c.q * (scale * c.up)[..., None], states) + torch.matmul(c.pairs, x)
    return c.join(o).to(q.dtype).contiguous(), S


def _plain_backward(q, k, v, a, beta, scale, initial, do, dfinal):
    c = _Chunks(q, k, v, a, beta, scale)
    S, x, _ = c.forward(_state_or_zeros(initial, v, q.shape[3]))
    do = c.cut(do)
    up, down, beta = c.up[..., None], c.down[..., None], c.beta[..., None]
    # backwards along the chunks: R the gradient of the state behind a chunk, w that of v
    from_out = torch.matmul(c.pairs.transpose(-1, -2), do)
    into = torch.matmul((c.q * (scale * up)).transpose(-1, -2), do)
    kb, ku, inverse = c.k * (down * beta), (c.k * up).transpose(-1, -2), c.inverse.transpose(-1, -2)
    R, Rs, ws = _state_or_zeros(dfinal, v, q.shape[3]), [], []
    for i in reversed(range(c.n)):
        Rs.append(R)
        ws.append(torch.matmul(inverse[:, :, i], from_out[:, :, i] + torch.matmul(kb[:, :, i], R)))
        R = R * c.whole[:, :, i, None, None] + into[:, :, i] - torch.matmul(ku[:, :, i], ws[-1])
    dS0, R, w = R, torch.stack(Rs[::-1], 2), torch.stack(ws[::-1], 2)
    xt = x.transpose(-1, -2)
    Y = torch.matmul(do, xt) * (scale * c.decays)
    Z = torch.matmul(w, xt) * c.strict
    kb = c.k * beta
    dq = torch.matmul(do, S.transpose(-1, -2)) * (scale * up) + torch.matmul(Y, kb)
    row = -(torch.matmul(w, S.transpose(-1, -2)) * up + torch.matmul(Z, kb))
    ends = torch.matmul(x, R.transpose(-1, -2)) * down
    col = ends + torch.matmul(Y.transpose(-1, -2), c.q) - torch.matmul(Z.transpose(-1, -2), c.k)
    dbeta = (c.k * col).sum(-1)
    dG = (c.q * dq).sum(-1) + (c.k * row).sum(-1) - c.beta * dbeta
    behind = c.whole * (R * S).sum((-1, -2)) + (c.beta * (c.k * ends).sum(-1)).sum(-1)
    da = behind[..., None] + dG.double().flip(-1).cumsum(-1).flip(-1)
    if initial is None:
        da[:, :, 0, 0] = 0.0  # nothing there to decay before the first token

    def scalars(x):
        return c.join(x[..., None])[..., 0].float().contiguous()

    def back(x, heads=None):
        return c.join(x, heads).to(q.dtype).contiguous()

    return back(dq, c.Hk), back(row + beta * col, c.Hk), back(w), scalars(da), scalars(dbeta), dS0


def _by_sequence(s, one):
    """Calls one(lo, hi, b) for every packed sequence and joins the results:
    tokens along dimension 0, states along the batch."""
    bounds = s["lengths_on_host"]
    parts = [one(lo, hi, b) for b, (lo, hi) in enumerate(zip(bounds, bounds[1:]))]
    joined = [torch.cat([p[i] for p in parts]) for i in range(len(parts[0]))]
    return [x.squeeze(1) for x in joined[:-1]] + [joined[-1]]


def _plain_norm(s):
    x, case = s["x"], s["case"]
    total = x.float() + s["residual"].float() if case["residual"] else x.float()
    rstd = torch.rsqrt(total.square().mean(1) + EPS)
    y = total * rstd[:, None] * s["weight"].float()
    M, N = y.shape
    if case["out"] == "same":
        out = (y.to(x.dtype),)
    else:
        width = N if case["out"] == "row" else GROUP
        groups = -(-N // width)
        parts = torch.nn.functional.pad(y, (0, groups * width - N)).reshape(M, groups, width)
        scale = (parts.abs().amax(-1) / E4M3_MAX).clamp(min=2.0 ** -126)
        q = (parts / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).reshape(M, groups * width)[:, :N]
        out = (q.to(torch.float8_e4m3fn).contiguous(), scale if case["out"] == "group" else scale[:, 0])
    return (*out, rstd, total.to(x.dtype)) if case["residual"] else (*out, rstd)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_backward":
        dy = s["grad_out"].float()
        n = s["x"].float() * s["rstd"][:, None]
        dw = (dy * n).sum(0)
        g = dy * s["weight"].float()
        dx = (g - n * (g * n).mean(1, keepdim=True)) * s["rstd"][:, None]
        dx = dx + s["grad_sum"].float() if case["residual"] else dx
        return dx.to(s["x"].dtype), dw.to(s["weight"].dtype)
    q, k, v, a, beta, scale = (s[x] for x in ("q", "k", "v", "log_decay", "beta", "scale"))
    if op == "step":
        group = case["H"] // case["Hk"]
        qf, kf = (x.float().repeat_interleave(group, 1) for x in (q, k))
        S = s["state"] * torch.exp(a)[..., None, None]
        u = beta[..., None] * (v.float() - (S * kf[..., :, None]).sum(2))
        S = S + kf[..., :, None] * u[..., None, :]
        return ((qf[..., :, None] * S).sum(2) * scale).to(q.dtype), S
    init = s["initial_state"]

    def part(lo, hi, b):
        seq = [x[lo:hi, None] for x in (q, k, v, a, beta)] + [scale, init[b:b + 1] if init is not None else None]
        if op == "forward":
            return _plain_forward(*seq)
        dfinal = s["grad_final_state"]
        return _plain_backward(*seq, s["grad_out"][lo:hi, None], dfinal[b:b + 1] if dfinal is not None else None)

    if case["packed"]:
        out = _by_sequence(s, part)
    elif op == "forward":
        out = _plain_forward(q, k, v, a, beta, scale, init)
    else:
        out = _plain_backward(q, k, v, a, beta, scale, init, s["grad_out"], s["grad_final_state"])
    if case["state"]:
        return tuple(out)
    return out[0] if op == "forward" else tuple(out[:-1])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -- 64 bits -------------------------------------------------------------------------------------------------

def _exact_token(S, k, v, a, beta):
    """One token: the decayed state, what the key finds missing in it, the new state."""
    Sd = S * a[..., None, None].exp()
    missing = v - torch.sum(Sd * k.unsqueeze(-1), -2)
    return Sd, missing, Sd + k.unsqueeze(-1) * (beta[..., None] * missing).unsqueeze(-2)


def _exact_sequence(q, k, v, a, beta, scale, S, do=None, dS=None):
    """The recurrence token by token in 64 bits; q and k already repeated for
    their groups.  With do also its gradients, by the reversed recurrence, the
    states of 32 tokens at a time computed again from those kept."""
    T = q.shape[0]
    o = torch.empty_like(v)
    kept = {}
    for t in range(T):
        if do is not None and t % 32 == 0:
            kept[t] = S
        S = _exact_token(S, k[t], v[t], a[t], beta[t])[2]
        if do is None:
            torch.sum(q[t].unsqueeze(-1) * S, -2, out=o[t])
    if do is None:
        return o * scale, S
    dq, dk, dv, da, db = (torch.empty_like(x) for x in (q, k, v, a, beta))
    R = dS
    for t0 in sorted(kept, reverse=True):
        S, run_of = kept.pop(t0), []
        for t in range(t0, min(T, t0 + 32)):
            Sd, missing, S = _exact_token(S, k[t], v[t], a[t], beta[t])
            run_of.append((Sd, missing, S))
        for t in range(min(T, t0 + 32) - 1, t0 - 1, -1):
            Sd, missing, S = run_of.pop()
            dq[t] = scale * torch.sum(S * do[t].unsqueeze(-2), -1)
            R = R + scale * q[t].unsqueeze(-1) * do[t].unsqueeze(-2)
            du = torch.sum(R * k[t].unsqueeze(-1), -2)
            db[t] = torch.sum(du * missing, -1)
            dv[t] = beta[t][..., None] * du
            dk[t] = torch.sum(R * (beta[t][..., None] * missing).unsqueeze(-2), -1) - torch.sum(Sd * dv[t].unsqueeze(-2), -1)
            R = R - k[t].unsqueeze(-1) * dv[t].unsqueeze(-2)
            da[t] = torch.sum(R * Sd, (-1, -2))
            R = R * a[t][..., None, None].exp()
    return dq, dk, dv, da, db, R


def _exact_norm(s, case):
    x = s["x"]
    M, N = x.shape
    total = x + s["residual"] if case["residual"] else x
    rstd = (total.pow(2).sum(1) / N + EPS) ** -0.5
    y = total * rstd[:, None] * s["weight"]
    if case["out"] == "same":
        out = (y,)
    else:
        width = N if case["out"] == "row" else GROUP
        q, scales = torch.empty_like(y), []
        for lo in range(0, N, width):
            part = y[:, lo:lo + width]
            scales.append(torch.maximum(part.max(1).values, -part.min(1).values) / E4M3_MAX)
            q[:, lo:lo + width] = (part / scales[-1][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        scale = torch.stack(scales, 1)
        out = (q.to(torch.float8_e4m3fn).double(), scale if case["out"] == "group" else scale[:, 0])
    return (*out, rstd, total) if case["residual"] else (*out, rstd)


def exact(case, seed):
    s = {n: x.double() if isinstance(x, torch.Tensor) and x.is_floating_point() else x
         for n, x in _inputs(case, seed).items()}
    op = case["op"]
    if op == "norm":
        return _exact_norm(s, case)
    if op == "norm_backward":
        x, dy = s["x"], s["grad_out"]
        rstd = s["rstd"][:, None]
        n = x * rstd
        g = dy * s["weight"]
        dx = rstd * (g - n * ((g * n).sum(1, keepdim=True) / x.shape[1]))
        return dx + s["grad_sum"] if case["residual"] else dx, (dy * n).sum(0)
    B, H, Hk, Dk, Dv = (case[x] for x in ("B", "H", "Hk", "Dk", "Dv"))
    wide = torch.arange(H, device="cuda") // (H // Hk)  # each head's head of q and k
    q, k, v, a, beta, scale = (s["q"].index_select(-2, wide), s["k"].index_select(-2, wide), s["v"], s["log_decay"],
                               s["beta"], s["scale"])
    if op == "step":
        S = _exact_token(s["state"], k, v, a, beta)[2]
        return torch.sum(q.unsqueeze(-1) * S, -2) * scale, S
    if _tokens(case) * H * Dk * Dv * (1 if op == "forward" else 4) > 1 << 37 or case["T"] > (1 << 16 if op == "forward" else 1 << 14):
        return None
    zero = torch.zeros((B, H, Dk, Dv), device="cuda", dtype=torch.float64)
    S0 = s["initial_state"] if case["state"] else zero
    back = op == "backward"
    do = s["grad_out"] if back else None
    dS = (s["grad_final_state"] if case["state"] else zero) if back else None
    if case["packed"]:
        bounds = _offsets(case)
        parts = [_exact_sequence(q[lo:hi], k[lo:hi], v[lo:hi], a[lo:hi], beta[lo:hi], scale, S0[b],
                                 do[lo:hi] if back else None, dS[b] if back else None)
                 for b, (lo, hi) in enumerate(zip(bounds, bounds[1:]))]
        out = [torch.cat([p[i] for p in parts]) for i in range(len(parts[0]) - 1)]
        out.append(torch.stack([p[-1] for p in parts]))
    else:
        out = list(_exact_sequence(q, k, v, a, beta, scale, S0, do, dS))
    if back:  # a shared head's gradient is the sum over its group
        out[:2] = [x.unflatten(-2, (Hk, H // Hk)).sum(-2) for x in out[:2]]
    if not case["state"]:
        out.pop()
    return tuple(out) if len(out) > 1 else out[0]
