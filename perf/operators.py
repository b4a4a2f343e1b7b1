"""What the sequence operators are measured on: linear attention with a decay
for each head (a prompt, its backward pass, one new token) and layer norm
(forward and backward).

Each case is computed in its plain form (elementary torch operations in 32
bits) or, with ``own`` set, by the library's kernels.  Definitions, t the token
of a sequence and h the head (head h of q, o and the decay uses head
h // (H / Hkv) of k and v):

  linear attention  S[t] = exp(a[h]) S[t-1] + k[t] v[t]^T,   S[-1] = initial state or 0
                    o[t] = scale * S[t]^T q[t]
  layer norm        y = (x - mean) * rstd * weight + bias,   rstd = 1 / sqrt(var + eps)

Tensors are laid out as everywhere in this library, time first: q [T, B, H, Dk],
k [T, B, Hkv, Dk], v [T, B, Hkv, Dv]; packed sequences drop B and follow each
other along the tokens, sequence b being rows offsets[b] .. offsets[b + 1] - 1.
"""
from __future__ import annotations

import math
import random

import torch

own = False

EPS = 1e-5
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
CHUNK = 128  # tokens the plain form takes at once


# -- cases ---------------------------------------------------------------------------------------------------

def _attention(name, op, type, B, T, H, Hkv, Dk, Dv, packed=False, state=False):
    case = {"op": op, "type": type, "B": B, "T": T, "H": H, "Hkv": Hkv, "Dk": Dk, "Dv": Dv}
    if op != "step":
        case.update(packed=packed, state=state)
    return {"name": name, **case} if name else case


def _norm(name, op, type, params, M, N):
    case = {"op": op, "type": type, "params": params, "M": M, "N": N}
    return {"name": name, **case} if name else case


def listed():
    return [
        # One token of one request through a layer of width 1792 (14 heads of 128): latency.
        _attention("step_one", "step", "f16", 1, 1, 14, 14, 128, 128),
        # One token of 64 requests served together, 8 key-value heads shared by 32: the state's bandwidth.
        _attention("step_batch", "step", "bf16", 64, 1, 32, 8, 128, 128),
        # Seven prompts of unequal length (one empty, one of a single token) packed into one call, with
        # carried states, as a server fills a batch.
        _attention("prompt_packed", "forward", "f16", 7, 3001, 16, 4, 64, 64, packed=True, state=True),
        # A layer of width 1792 at the library's own batch and sequence (B = 4, T = 256), fed by the fp32
        # input projection.
        _attention("prompt_layer", "forward", "f32", 4, 256, 14, 14, 128, 128),
        # One long prompt: few rows, a long axis.
        _attention("prompt_long", "forward", "bf16", 1, 32768, 32, 32, 128, 128, state=True),
        # Backward of a layer of width 1152 in fp32 at B = 4, T = 256, two heads of 64 on each key-value head.
        _attention("grad_layer", "backward", "f32", 4, 256, 18, 9, 64, 64),
        # Backward with head sizes that fill no tile and a length that ends inside one.
        _attention("grad_odd", "backward", "f16", 3, 1531, 6, 6, 96, 80, state=True),
        # Backward of one training batch.
        _attention("grad_batch", "backward", "bf16", 8, 2048, 16, 16, 128, 128),
        # The four rows of one timestep at width 1792: latency.
        _norm("norm_step", "norm", "f32", "f32", 4, 1792),
        # The tokens of a batch at width 5760.
        _norm("norm_tokens", "norm", "bf16", "bf16", 16384, 5760),
        # A width that no vector load divides.
        _norm("norm_grad_odd", "norm_backward", "f32", "f32", 4099, 1153),
        # Backward of a training batch at width 5760, fp32 parameters.
        _norm("norm_grad_tokens", "norm_backward", "bf16", "f32", 16384, 5760),
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
            case = _norm(None, op, type, rng.choice(("f32", type)), _log_int(rng, 1, 400000), _log_int(rng, 32, 12000))
        else:
            Hkv = rng.choice((1, 2, 3, 4, 5, 8, 12, 16))
            H = Hkv * rng.choice((1, 1, 2, 3, 4))
            Dk = _head_size(rng)
            Dv = Dk if rng.random() < 0.6 else _head_size(rng)
            if op == "step":
                case = _attention(None, op, type, _log_int(rng, 1, 256), 1, H, Hkv, Dk, Dv)
            else:
                case = _attention(None, op, type, _log_int(rng, 1, 32), _log_int(rng, 1, 32768), H, Hkv, Dk, Dv,
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
    itself (or of the products over pairs of tokens, where those are fewer)."""
    e = SIZE[case["type"]]
    if case["op"] in ("norm", "norm_backward"):
        M, N = case["M"], case["N"]
        p = SIZE[case["params"]]
        if case["op"] == "norm":
            return {"bytes": 2 * M * N * e + 2 * N * p + 8 * M, "flops": 8 * M * N}
        return {"bytes": 3 * M * N * e + 3 * N * p + 8 * M, "flops": 14 * M * N}
    B, H, Hkv, Dk, Dv = (case[x] for x in ("B", "H", "Hkv", "Dk", "Dv"))
    n = _tokens(case)
    state = 4 * B * H * Dk * Dv
    qo, kv = n * H * e, n * Hkv * (Dk + Dv) * e
    if case["op"] == "step":
        return {"bytes": qo * (Dk + Dv) + kv + 2 * state + 4 * H, "flops": 4 * n * H * Dk * Dv}
    lengths = [b - a for a, b in zip(_offsets(case), _offsets(case)[1:])] if case["packed"] else [case["T"]] * B
    extra = (4 * (B + 1) if case["packed"] else 0) + 4 * H
    if case["op"] == "forward":
        flops = H * sum(min(4 * t * Dk * Dv, t * (t + 1) * (Dk + Dv)) for t in lengths)
        if case["state"]:
            flops += 2 * n * H * Dk * Dv
        return {"bytes": qo * (Dk + Dv) + kv + extra + (2 * state if case["state"] else 0), "flops": flops}
    flops = H * sum(min(10 * t * Dk * Dv, t * (t + 1) * (3 * Dk + 2 * Dv)) for t in lengths)
    return {"bytes": qo * (2 * Dk + Dv) + 2 * kv + extra + (3 * state if case["state"] else 0), "flops": flops}


# -- inputs --------------------------------------------------------------------------------------------------

def _inputs(case, seed):
    """Seeded inputs on the GPU.  Decays follow the usual ladder of retentive
    layers, 1 - 2^-(3 + 6 h / H), each moved a little by the seed."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    if case["op"] in ("norm", "norm_backward"):
        M, N = case["M"], case["N"]
        pt = TYPES[case["params"]]
        x = (normal(M, N) * (0.5 + 2.0 * torch.rand((M, 1), generator=g, device="cuda")) + 0.5 * normal(M, 1)).to(dt)
        s = {"x": x, "weight": (1.0 + 0.1 * normal(N)).to(pt), "bias": (0.1 * normal(N)).to(pt)}
        if case["op"] == "norm_backward":
            s["grad_out"] = normal(M, N).to(dt)
            xd = x.double() if M * N <= 1 << 24 else x.float()  # the statistics the forward pass has left
            mean = xd.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = torch.rsqrt((xd - mean[:, None]).square().mean(1) + EPS).float()
        return s
    B, T, H, Hkv, Dk, Dv = (case[x] for x in ("B", "T", "H", "Hkv", "Dk", "Dv"))
    rows = (T,) if case.get("packed") else (B,) if case["op"] == "step" else (T, B)
    s = {"q": normal(*rows, H, Dk).to(dt), "k": normal(*rows, Hkv, Dk).to(dt), "v": normal(*rows, Hkv, Dv).to(dt)}
    ladder = 3.0 + 6.0 * torch.arange(H, device="cuda", dtype=torch.float32) / H
    s["log_decay"] = torch.log1p(-torch.exp2(-ladder)) * (0.8 + 0.4 * torch.rand(H, generator=g, device="cuda"))
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
    h, op = s["handle"], s["case"]["op"]
    if op == "norm":
        x = s["x"]
        mean = torch.empty(x.shape[0], device=x.device)
        rstd = torch.empty(x.shape[0], device=x.device)
        return h.layer_norm(x, s["weight"], s["bias"], EPS, mean=mean, rstd=rstd), mean, rstd
    if op == "norm_backward":
        return h.layer_norm_backward(s["grad_out"], s["x"], s["mean"], s["rstd"], s["weight"])
    qkv = s["q"], s["k"], s["v"], s["log_decay"]
    if op == "step":
        return h.linear_attention_step(*qkv, s["state"], scale=s["scale"], new_state=s["new_state"]), s["new_state"]
    seq = {"scale": s["scale"], "initial_state": s["initial_state"]}
    if s["offsets"] is not None:
        seq.update(offsets=s["offsets"], max_len=s["max_len"])
    if op == "forward":
        if not s["case"]["state"]:
            return h.linear_attention(*qkv, **seq)
        return h.linear_attention(*qkv, final_state=s["final_state"], **seq), s["final_state"]
    if not s["case"]["state"]:
        return h.linear_attention_backward(*qkv, s["grad_out"], **seq)
    grads = h.linear_attention_backward(*qkv, s["grad_out"], grad_final_state=s["grad_final_state"],
                                        grad_initial_state=s["grad_initial_state"], **seq)
    return (*grads, s["grad_initial_state"])


# -- the plain form ------------------------------------------------------------------------------------------

def _heads_first(x, heads):
    """[T, B, h, D] -> fp32 [B, heads, T, D], each of the h heads repeated for its group."""
    x = x.float().permute(1, 2, 0, 3)
    return x.repeat_interleave(heads // x.shape[1], 1).contiguous()


def _decays(a, n):
    """exp(a m) for m = 0 .. n, [H, n + 1], the exponents in 64 bits."""
    m = torch.arange(n + 1, device=a.device, dtype=torch.float64)
    return torch.exp(a.double()[:, None] * m).float()


def _pair_decays(w, n):
    """exp(a (i - j)) for j <= i < n, else 0: [H, n, n]."""
    i = torch.arange(n, device=w.device)
    d = i[:, None] - i[None, :]
    return torch.where(d >= 0, w[:, d.clamp(min=0)], torch.zeros((), device=w.device))


def _plain_forward(q, k, v, a, scale, initial):
    T, B, H, Dk = q.shape
    Dv = v.shape[3]
    qf, kf, vf = (_heads_first(x, H) for x in (q, k, v))
    S = initial.clone() if initial is not None else torch.zeros((B, H, Dk, Dv), device=q.device)
    o = torch.empty((B, H, T, Dv), device=q.device)
    w = _decays(a, CHUNK)
    pairs = _pair_decays(w, CHUNK)
    for t in range(0, T, CHUNK):
        n = min(CHUNK, T - t)
        qc, kc, vc = (x[:, :, t:t + n] for x in (qf, kf, vf))
        inside = torch.matmul(qc, kc.transpose(-1, -2)) * pairs[:, :n, :n]
        o[:, :, t:t + n] = torch.matmul(inside, vc) + torch.matmul(qc * w[:, 1:n + 1, None], S)
        S = S * w[:, n, None, None] + torch.matmul((kc * w[:, :n, None].flip(1)).transpose(-1, -2), vc)
    return (o * scale).permute(2, 0, 1, 3).to(q.dtype).contiguous(), S


def _plain_backward(q, k, v, a, scale, initial, do, dfinal):
    T, B, H, Dk = q.shape
    Dv, Hkv = v.shape[3], k.shape[2]
    qf, kf, vf, df = (_heads_first(x, H) for x in (q, k, v, do))
    df = df * scale
    w = _decays(a, CHUNK)
    pairs = _pair_decays(w, CHUNK)
    starts = list(range(0, T, CHUNK))
    zero = torch.zeros((B, H, Dk, Dv), device=q.device)
    states, S = [], initial if initial is not None else zero
    for t in starts:
        n = min(CHUNK, T - t)
        states.append(S)
        S = S * w[:, n, None, None] + torch.matmul((kf[:, :, t:t + n] * w[:, :n, None].flip(1)).transpose(-1, -2),
                                                   vf[:, :, t:t + n])
    dq, dk, dv = torch.empty_like(qf), torch.empty_like(kf), torch.empty_like(vf)
    dS = dfinal if dfinal is not None else zero
    for t, S in zip(reversed(starts), reversed(states)):
        n = min(CHUNK, T - t)
        qc, kc, vc, dc = (x[:, :, t:t + n] for x in (qf, kf, vf, df))
        m = pairs[:, :n, :n]
        up, down = w[:, 1:n + 1, None], w[:, :n, None].flip(1)
        dp = torch.matmul(dc, vc.transpose(-1, -2)) * m
        p = torch.matmul(qc, kc.transpose(-1, -2)) * m
        dq[:, :, t:t + n] = torch.matmul(dp, kc) + torch.matmul(dc * up, S.transpose(-1, -2))
        dk[:, :, t:t + n] = torch.matmul(dp.transpose(-1, -2), qc) + torch.matmul(vc * down, dS.transpose(-1, -2))
        dv[:, :, t:t + n] = torch.matmul(p.transpose(-1, -2), dc) + torch.matmul(kc * down, dS)
        dS = dS * w[:, n, None, None] + torch.matmul((qc * up).transpose(-1, -2), dc)

    def back(x, heads):
        x = x.reshape(B, heads, H // heads, T, x.shape[3]).sum(2)
        return x.permute(2, 0, 1, 3).to(q.dtype).contiguous()

    return back(dq, H), back(dk, Hkv), back(dv, Hkv), dS


def _by_sequence(s, one):
    """Calls one(lo, hi, b) for every packed sequence and joins the results:
    tokens along dimension 0, states along the batch."""
    bounds = s["lengths_on_host"]
    parts = [one(lo, hi, b) for b, (lo, hi) in enumerate(zip(bounds, bounds[1:]))]
    joined = [torch.cat([p[i] for p in parts]) for i in range(len(parts[0]))]
    return [x.squeeze(1) for x in joined[:-1]] + [joined[-1]]


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(1)
        x = x - mean[:, None]
        rstd = torch.rsqrt(x.square().mean(1) + EPS)
        y = x * rstd[:, None] * s["weight"].float() + s["bias"].float()
        return y.to(s["x"].dtype), mean, rstd
    if op == "norm_backward":
        dy = s["grad_out"].float()
        n = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        db, dw = dy.sum(0), (dy * n).sum(0)
        dn = dy * s["weight"].float()
        dx = (dn - dn.mean(1, keepdim=True) - n * (dn * n).mean(1, keepdim=True)) * s["rstd"][:, None]
        return dx.to(s["x"].dtype), dw.to(s["weight"].dtype), db.to(s["weight"].dtype)
    q, k, v, a, scale = (s[x] for x in ("q", "k", "v", "log_decay", "scale"))
    if op == "step":
        group = case["H"] // case["Hkv"]
        kf, vf = (x.float().repeat_interleave(group, 1) for x in (k, v))
        S = s["state"] * torch.exp(a)[:, None, None] + kf[..., :, None] * vf[..., None, :]
        o = (q.float()[..., :, None] * S).sum(2) * scale
        return o.to(q.dtype), S
    init = s["initial_state"]
    if op == "forward":
        def forward(lo, hi, b):
            return _plain_forward(q[lo:hi, None], k[lo:hi, None], v[lo:hi, None], a, scale,
                                  init[b:b + 1] if init is not None else None)
        o, S = _by_sequence(s, forward) if case["packed"] else _plain_forward(q, k, v, a, scale, init)
        return (o, S) if case["state"] else o
    do, dfinal = s["grad_out"], s["grad_final_state"]

    def backward(lo, hi, b):
        return _plain_backward(q[lo:hi, None], k[lo:hi, None], v[lo:hi, None], a, scale,
                               init[b:b + 1] if init is not None else None, do[lo:hi, None],
                               dfinal[b:b + 1] if dfinal is not None else None)
    grads = _by_sequence(s, backward) if case["packed"] else _plain_backward(q, k, v, a, scale, init, do, dfinal)
    return tuple(grads) if case["state"] else tuple(grads[:3])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -- 64 bits -------------------------------------------------------------------------------------------------

def _exact_sequence(q, k, v, decay, scale, S, do=None, dS=None):
    """The recurrence token by token in 64 bits; k and v already repeated for
    their groups.  With do also its gradients, by the reversed recurrence."""
    T = q.shape[0]
    o, dq = torch.empty_like(v), torch.empty_like(q)
    for t in range(T):
        S = S * decay + k[t].unsqueeze(-1) * v[t].unsqueeze(-2)
        if do is None:
            torch.sum(q[t].unsqueeze(-1) * S, -2, out=o[t])
        else:
            torch.sum(S * do[t].unsqueeze(-2), -1, out=dq[t])
    if do is None:
        return o * scale, S
    dk, dv = torch.empty_like(k), torch.empty_like(v)
    for t in range(T - 1, -1, -1):
        dS = dS + q[t].unsqueeze(-1) * (do[t] * scale).unsqueeze(-2)
        torch.sum(dS * v[t].unsqueeze(-2), -1, out=dk[t])
        torch.sum(dS * k[t].unsqueeze(-1), -2, out=dv[t])
        dS = dS * decay
    return dq * scale, dk, dv, dS


def exact(case, seed):
    s = {n: x.double() if isinstance(x, torch.Tensor) and x.is_floating_point() else x
         for n, x in _inputs(case, seed).items()}
    op = case["op"]
    if op in ("norm", "norm_backward"):
        x = s["x"]
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        rstd = (var + EPS) ** -0.5
        n = (x - mean) * rstd
        if op == "norm":
            return torch.addcmul(s["bias"], n, s["weight"]), mean[:, 0], rstd[:, 0]
        dy = s["grad_out"]
        g = dy * s["weight"]
        along = (g * n).sum(1, keepdim=True) / x.shape[1]
        return rstd * (g - g.sum(1, keepdim=True) / x.shape[1] - n * along), (dy * n).sum(0), dy.sum(0)
    B, H, Hkv, Dk, Dv = (case[x] for x in ("B", "H", "Hkv", "Dk", "Dv"))
    decay = s["log_decay"].exp()[:, None, None]
    wide = torch.arange(H, device="cuda") // (H // Hkv)  # each head's key-value head
    q, k, v, scale = s["q"], s["k"].index_select(-2, wide), s["v"].index_select(-2, wide), s["scale"]
    if op == "step":
        S = s["state"] * decay + k.unsqueeze(-1) * v.unsqueeze(-2)
        return torch.sum(q.unsqueeze(-1) * S, -2) * scale, S
    if _tokens(case) * H * Dk * Dv * (1 if op == "forward" else 4) > 1 << 38 or case["T"] > 1 << 17:
        return None
    zero = torch.zeros((B, H, Dk, Dv), device="cuda", dtype=torch.float64)
    S0 = s["initial_state"] if case["state"] else zero
    back = op == "backward"
    do = s["grad_out"] if back else None
    dS = (s["grad_final_state"] if case["state"] else zero) if back else None
    if case["packed"]:
        bounds = _offsets(case)
        parts = [_exact_sequence(q[lo:hi], k[lo:hi], v[lo:hi], decay, scale, S0[b],
                                 do[lo:hi] if back else None, dS[b] if back else None)
                 for b, (lo, hi) in enumerate(zip(bounds, bounds[1:]))]
        out = [torch.cat([p[i] for p in parts]) for i in range(len(parts[0]) - 1)]
        out.append(torch.stack([p[-1] for p in parts]))
    else:
        out = list(_exact_sequence(q, k, v, decay, scale, S0, do, dS))
    if back:  # a shared head's gradient is the sum over its group
        out[1:3] = [x.unflatten(-2, (Hkv, H // Hkv)).sum(-2) for x in out[1:3]]
    if not case["state"]:
        out.pop()
    return tuple(out) if len(out) > 1 else out[0]
