"""GPU parity of linear attention with a decay for each head and of layer norm
(through the C ABI) against the fp64 oracle.

Tolerances come from the arithmetic.  Linear attention: with A the same result
computed from absolute values, an output differs from the exact one by half a
step of its type, plus, in fp32, two roundings of the state a token, the sum
over Dk rows and a few single roundings (each at most 2^-24 of A), plus, for
16-bit operands, the score or the state (2^-16) and the decayed operand of
the state (2^-16).  Layer norm: sums of at most 96 sequential roundings
(registers, lanes, waves), so statistics and outputs to 128 * 2^-24 of their
absolute terms, plus half a step of the output's type.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from persistent_rnn_fwd_amd import Handle, PrnnError, binding

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def handle(gpu):
    h = Handle()
    yield h
    h.close()


def host(t):
    return t.detach().double().cpu().numpy()


def half_step(dtype, ref):
    f = torch.finfo(dtype)
    return f.eps / 2 * np.abs(ref) + f.smallest_normal * f.eps / 2


# -- linear attention --------------------------------------------------------------------------------------

def attention_problem(seed, type, T, B, H, Hkv, Dk, Dv, decay=None):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[type]
    p = {"q": torch.randn((T, B, H, Dk), generator=g).to(dt).cuda(),
         "k": torch.randn((T, B, Hkv, Dk), generator=g).to(dt).cuda(),
         "v": torch.randn((T, B, Hkv, Dv), generator=g).to(dt).cuda()}
    a = -torch.exp2(-8.0 * torch.rand(H, generator=g)) if decay is None else torch.tensor(decay, dtype=torch.float32)
    p["log_decay"] = a.float().cuda()
    extra = {"S0": torch.randn((B, H, Dk, Dv), generator=g).cuda(),
             "do": torch.randn((T, B, H, Dv), generator=g).to(dt).cuda(),
             "dS1": torch.randn((B, H, Dk, Dv), generator=g).cuda()}
    return p, extra


def absolute(p):
    return {n: (np.abs(x) if n != "log_decay" else x) for n, x in p.items()}


def attention_rounding(dtype, T, D):
    return U * (2 * T + D + 16) + (2.0 ** -15 if dtype != torch.float32 else 0.0)


def close(name, got, ref, A, dtype, c):
    got = host(got)
    tol = half_step(dtype, ref) + c * A
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (name, int(bad.sum()), float(np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300))))


def check_forward(o, S, p, scale, S0=None, lengths=None):
    n = {x: host(y) for x, y in p.items()}
    s0 = host(S0) if S0 is not None else None
    ref, refS = oracle.linear_attention(**n, scale=scale, S0=s0, lengths=lengths)
    A, AS = oracle.linear_attention(**absolute(n), scale=abs(scale), S0=np.abs(s0) if s0 is not None else None,
                                    lengths=lengths)
    c = attention_rounding(p["q"].dtype, ref.shape[0], n["q"].shape[3])
    close("o", o, ref, A, p["q"].dtype, c)
    if S is not None:
        close("S", S, refS, AS, torch.float32, c)


def check_backward(grads, dS0, p, do, scale, S0=None, dS1=None, lengths=None):
    n = {x: host(y) for x, y in p.items()}
    s = {"do": host(do), "S0": host(S0) if S0 is not None else None, "dS1": host(dS1) if dS1 is not None else None}
    ref = oracle.linear_attention_backward(**n, **s, scale=scale, lengths=lengths)
    A = oracle.linear_attention_backward(**absolute(n), **{x: (np.abs(y) if y is not None else None) for x, y in s.items()},
                                         scale=abs(scale), lengths=lengths)
    T, B, H, Dk = n["q"].shape
    c = attention_rounding(p["q"].dtype, T, max(Dk, n["v"].shape[3])) + U * (H // n["k"].shape[2])
    for name, g, r, a in zip(("dq", "dk", "dv"), grads, ref, A):
        close(name, g, r, a, p["q"].dtype, c)
    if dS0 is not None:
        close("dS0", dS0, ref[3], A[3], torch.float32, c)


# (T, B, H, Hkv, Dk, Dv): one token; lengths around and across chunks of 32 and
# 64; heads that fill, do not fill and exceed a tile; shared heads; odd sizes.
SHAPES = [(1, 1, 1, 1, 1, 1), (1, 3, 4, 2, 64, 64), (5, 2, 2, 1, 8, 16), (31, 1, 2, 2, 32, 32), (63, 1, 2, 2, 64, 64),
          (64, 2, 4, 2, 64, 64), (65, 1, 3, 3, 128, 128), (130, 2, 3, 1, 96, 80), (200, 1, 2, 2, 128, 64),
          (97, 1, 1, 1, 37, 53), (70, 1, 1, 1, 256, 256), (129, 1, 2, 2, 64, 200), (150, 1, 1, 1, 255, 9)]


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_attention_forward(handle, type, shape):
    p, x = attention_problem(sum(shape), type, *shape)
    S = torch.full_like(x["S0"], float("nan"))
    o = handle.linear_attention(**p, scale=0.3, initial_state=x["S0"], final_state=S)
    check_forward(o, S, p, 0.3, x["S0"])
    o = handle.linear_attention(**p)
    check_forward(o, None, p, shape[4] ** -0.5)


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_attention_backward(handle, type, shape):
    p, x = attention_problem(1 + sum(shape), type, *shape)
    dS0 = torch.full_like(x["S0"], float("nan"))
    grads = handle.linear_attention_backward(**p, grad_out=x["do"], scale=0.3, initial_state=x["S0"],
                                             grad_final_state=x["dS1"], grad_initial_state=dS0)
    check_backward(grads, dS0, p, x["do"], 0.3, x["S0"], x["dS1"])
    grads = handle.linear_attention_backward(**p, grad_out=x["do"])
    check_backward(grads, None, p, x["do"], shape[4] ** -0.5)


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("T", [700, 2500])
def test_attention_long_sequence_of_one_head(handle, type, T):
    """One state only: the sequence is split over workgroups and joined."""
    p, x = attention_problem(T, type, T, 1, 1, 1, 64, 48, decay=[-0.003])
    S, dS0 = torch.empty_like(x["S0"]), torch.empty_like(x["S0"])
    o = handle.linear_attention(**p, scale=0.1, initial_state=x["S0"], final_state=S)
    check_forward(o, S, p, 0.1, x["S0"])
    grads = handle.linear_attention_backward(**p, grad_out=x["do"], scale=0.1, initial_state=x["S0"],
                                             grad_final_state=x["dS1"], grad_initial_state=dS0)
    check_backward(grads, dS0, p, x["do"], 0.1, x["S0"], x["dS1"])


@pytest.mark.parametrize("type", sorted(TYPES))
def test_attention_decays(handle, type):
    """No decay, total decay (minus infinity), fast and slow ones, and growth."""
    decay = [0.0, -float("inf"), -40.0, -1e-6, -2.0, 0.01]
    p, x = attention_problem(5, type, 150, 1, 6, 6, 32, 32, decay=decay)
    S, dS0 = torch.empty_like(x["S0"]), torch.empty_like(x["S0"])
    o = handle.linear_attention(**p, scale=0.2, initial_state=x["S0"], final_state=S)
    check_forward(o, S, p, 0.2, x["S0"])
    grads = handle.linear_attention_backward(**p, grad_out=x["do"], scale=0.2, initial_state=x["S0"],
                                             grad_final_state=x["dS1"], grad_initial_state=dS0)
    check_backward(grads, dS0, p, x["do"], 0.2, x["S0"], x["dS1"])


@pytest.mark.parametrize("type", sorted(TYPES))
def test_attention_lengths(handle, type):
    """A padded batch with an empty sequence, one token, a full one, lengths
    out of range; what the padding holds (NaN here) reaches nothing."""
    lengths = [0, 1, 90, 64, 200, -3]
    used = [0, 1, 90, 64, 90, 0]
    p, x = attention_problem(6, type, 90, 6, 2, 1, 64, 32)
    for b, n in enumerate(used):
        for t in (p["q"], p["k"], p["v"], x["do"]):
            t[n:, b] = float("nan")
    S, dS0 = torch.empty_like(x["S0"]), torch.empty_like(x["S0"])
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o = handle.linear_attention(**p, scale=0.2, initial_state=x["S0"], final_state=S, lengths=n)
    grads = handle.linear_attention_backward(**p, grad_out=x["do"], scale=0.2, initial_state=x["S0"],
                                             grad_final_state=x["dS1"], grad_initial_state=dS0, lengths=n)
    clean = {m: torch.nan_to_num(t) if m != "log_decay" else t for m, t in p.items()}
    check_forward(o, S, clean, 0.2, x["S0"], used)
    check_backward(grads, dS0, clean, torch.nan_to_num(x["do"]), 0.2, x["S0"], x["dS1"], used)
    for b, m in enumerate(used):
        for t in (o, *grads):
            assert not t[m:, b].any()


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("max_len", [None, 100])
def test_attention_packed(handle, type, max_len):
    """Packed sequences, empty ones among them; rows that belong to none keep
    what the outputs held."""
    offsets = [2, 2, 3, 103, 103, 140, 141]
    rows = 143
    B, H, Hkv = 6, 4, 2
    p, x = attention_problem(7, type, rows, 1, H, Hkv, 48, 64)
    S0 = torch.randn((B, H, 48, 64), device="cuda")
    packed = {m: (t[:, 0].contiguous() if m != "log_decay" else t) for m, t in p.items()}
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    S, dS0 = torch.empty_like(S0), torch.empty_like(S0)
    out = torch.full((rows, H, 64), 7.0, dtype=TYPES[type], device="cuda")
    seq = {"scale": 0.2, "offsets": off, "max_len": max_len, "initial_state": S0}
    handle.linear_attention(**packed, final_state=S, out=out, **seq)
    grads = handle.linear_attention_backward(**packed, grad_out=x["do"][:, 0].contiguous(), grad_final_state=S0 + 1,
                                             grad_initial_state=dS0, grad_k=torch.full_like(packed["k"], 7.0), **seq)
    for b, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        one = {m: (t[lo:hi] if m != "log_decay" else t) for m, t in p.items()}
        check_forward(out[lo:hi, None], S[b:b + 1], one, 0.2, S0[b:b + 1])
        check_backward([g[lo:hi, None] for g in grads], dS0[b:b + 1], one, x["do"][lo:hi], 0.2, S0[b:b + 1],
                       S0[b:b + 1] + 1)
    for t in (out, grads[1]):
        assert (t[:2] == 7).all() and (t[141:] == 7).all()


def test_attention_offsets_out_of_range_stay_inside(handle):
    """Offsets are clamped to the rows there are, and to max_len."""
    p, _ = attention_problem(8, "f32", 40, 1, 1, 1, 16, 16)
    packed = {m: (t[:, 0].contiguous() if m != "log_decay" else t) for m, t in p.items()}
    off = torch.tensor([-5, 10, 4, 1000, 12], dtype=torch.int32, device="cuda")
    S = torch.empty((4, 1, 16, 16), device="cuda")
    out = torch.zeros((40, 1, 16), device="cuda")
    handle.linear_attention(**packed, scale=1.0, offsets=off, max_len=30, final_state=S, out=out)
    for b, (lo, hi) in enumerate(((0, 10), (10, 10), (4, 34), (40, 40))):
        one = {m: (t[lo:hi] if m != "log_decay" else t) for m, t in p.items()}
        _, ref = oracle.linear_attention(**{m: host(t) for m, t in one.items()}, scale=1.0)
        np.testing.assert_allclose(host(S[b:b + 1]), ref, rtol=1e-3, atol=1e-4)
    assert not out[34:].any()


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("layout", ["batch first", "fused", "unaligned", "repeated"])
def test_attention_strides(handle, type, layout):
    T, B, H, Hkv, D = 70, 2, 4, 2, 64
    p, x = attention_problem(9, type, T, B, H, Hkv, D, D)
    out = grads = None
    if layout == "batch first":
        move = lambda t: t.permute(1, 2, 0, 3).contiguous().permute(2, 0, 1, 3)
        p = {m: (move(t) if m != "log_decay" else t) for m, t in p.items()}
        x["do"] = move(x["do"])
        out = torch.empty((B, H, T, D), dtype=TYPES[type], device="cuda").permute(2, 0, 1, 3)
    elif layout == "fused":
        fused = torch.cat([p["q"].flatten(2), p["k"].flatten(2), p["v"].flatten(2)], dim=2)
        q, k, v = fused.split([H * D, Hkv * D, Hkv * D], dim=2)
        p.update(q=q.unflatten(2, (H, D)), k=k.unflatten(2, (Hkv, D)), v=v.unflatten(2, (Hkv, D)))
        q, k, v = torch.empty_like(fused).split([H * D, Hkv * D, Hkv * D], dim=2)
        grads = {"grad_q": q.unflatten(2, (H, D)), "grad_k": k.unflatten(2, (Hkv, D)), "grad_v": v.unflatten(2, (Hkv, D))}
    elif layout == "unaligned":
        def shift(t):
            buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
            buf[1:].view(t.shape).copy_(t)
            return buf[1:].view(t.shape)
        p = {m: shift(t) for m, t in p.items()}
        x["do"] = shift(x["do"])
        out = shift(torch.zeros((T, B, H, D), dtype=TYPES[type], device="cuda"))
    else:
        p["k"] = p["k"][:, :1, :1].expand(T, B, Hkv, D)
        p["q"] = p["q"][:1].expand(T, B, H, D)
    S = torch.empty_like(x["S0"])
    o = handle.linear_attention(**p, scale=0.2, initial_state=x["S0"], final_state=S, out=out)
    check_forward(o, S, p, 0.2, x["S0"])
    got = handle.linear_attention_backward(**p, grad_out=x["do"], scale=0.2, **(grads or {}))
    check_backward(got, None, p, x["do"], 0.2)


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("where", ["q", "k", "v"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_attention_later_tokens_reach_no_earlier_row(handle, type, where, value):
    """A NaN or infinity at one token: the rows before it are as if it were not
    there; the rows from it on have the recurrence's infinities and NaN."""
    T, t = 150, 75
    p, x = attention_problem(10, type, T, 1, 2, 2, 64, 64, decay=[-0.01, -0.5])
    p[where][t, 0, 0, 5] = value
    S = torch.empty_like(x["S0"])
    o = handle.linear_attention(**p, scale=0.2, initial_state=x["S0"], final_state=S)
    before = {m: (y[:t] if m != "log_decay" else y) for m, y in p.items()}
    check_forward(o[:t], None, before, 0.2, x["S0"])
    with np.errstate(invalid="ignore"):
        ref, refS = oracle.linear_attention(**{m: host(y) for m, y in p.items()}, scale=0.2, S0=host(x["S0"]))
    for got, want in ((host(o), ref), (host(S), refS)):
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])


def test_attention_large_values_of_fp16(handle):
    """Scores and states beyond fp16's range, outputs inside it."""
    p, x = attention_problem(11, "f16", 100, 1, 1, 1, 64, 64)
    p["q"], p["k"] = p["q"] * 100, p["k"] * 100
    p["v"] = p["v"] * 50
    S = torch.empty_like(x["S0"])
    o = handle.linear_attention(**p, scale=1e-4, final_state=S)
    check_forward(o, S, p, 1e-4)
    small = {m: (y * 1e-3 if m != "log_decay" else y) for m, y in attention_problem(12, "f16", 100, 1, 1, 1, 64, 64)[0].items()}
    o = handle.linear_attention(**small, scale=1e6, final_state=S)
    check_forward(o, S, small, 1e6)


def test_attention_row_offsets_past_32_bits(handle):
    T, D, stride = 300, 64, 1 << 23
    buf = torch.empty(T * stride, dtype=torch.float16, device="cuda")  # 5 GB
    p, x = attention_problem(13, "f16", T, 1, 1, 1, D, D)
    views = {}
    for i, m in enumerate(("q", "k", "v", "o")):
        views[m] = buf.as_strided((T, 1, 1, D), (stride, D, D, 1), 100 * i * 64)
        if m != "o":
            views[m].copy_(p[m])
    o = handle.linear_attention(views["q"], views["k"], views["v"], p["log_decay"], scale=0.2, out=views["o"])
    check_forward(o.contiguous(), None, p, 0.2)


def test_attention_gradients_match_differences(handle):
    """o is linear in q, in k and in v, so the difference of two calls is the
    gradient along a direction, to the rounding of the two sums."""
    p, x = attention_problem(14, "f32", 100, 2, 4, 2, 32, 48)
    do, dS1 = x["do"], x["dS1"]
    dS0 = torch.empty_like(x["S0"])
    grads = handle.linear_attention_backward(**p, grad_out=do, scale=0.3, initial_state=x["S0"], grad_final_state=dS1,
                                             grad_initial_state=dS0)

    def loss(p, S0):
        S = torch.empty_like(S0)
        o = handle.linear_attention(**p, scale=0.3, initial_state=S0, final_state=S)
        return (o.double() * do.double()).sum() + (S.double() * dS1.double()).sum(), \
            (o.double() * do.double()).abs().sum() + (S.double() * dS1.double()).abs().sum()

    g = torch.Generator().manual_seed(0)
    for name, grad in zip(("q", "k", "v", "S0"), (*grads, dS0)):
        at = x["S0"] if name == "S0" else p[name]
        d = torch.randn(at.shape, generator=g).cuda()
        (hi, a1), (lo, a2) = (loss(p, at + s) if name == "S0" else loss({**p, name: at + s}, x["S0"]) for s in (d, -d))
        want = (grad.double() * d.double()).sum()
        assert abs((hi - lo) / 2 - want) <= 2e-5 * (a1 + a2), name


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1), (1, 14, 14, 128, 128), (5, 4, 2, 64, 80), (3, 6, 3, 37, 53),
                                   (2, 2, 1, 256, 255)], ids=str)
def test_attention_step(handle, type, shape):
    """Steps one after another, in place and into another state, are the prompt."""
    B, H, Hkv, Dk, Dv = shape
    p, x = attention_problem(15, type, 4, B, H, Hkv, Dk, Dv)
    state, outs = x["S0"].clone(), []
    for t in range(4):
        kept = state.clone()
        new = torch.empty_like(state) if t % 2 else None
        outs.append(handle.linear_attention_step(p["q"][t], p["k"][t], p["v"][t], p["log_decay"], state, scale=0.3,
                                                 new_state=new))
        if new is not None:
            assert torch.equal(state, kept)
            state = new
    check_forward(torch.stack(outs), state, p, 0.3, x["S0"])


def test_attention_step_strides(handle):
    """q, k, v as slices of one token's fused projection; a head size that
    vectors do not divide, at an odd element."""
    B, H, D = 3, 4, 33
    g = torch.Generator().manual_seed(3)
    fused = torch.randn((B, 3 * H * D + 1), generator=g).cuda()[:, 1:]
    q, k, v = (y.unflatten(1, (H, D)) for y in fused.split(H * D, dim=1))
    a = -torch.rand(H, generator=g).cuda()
    S0 = torch.randn((B, H, D, D), generator=g).cuda()
    S = S0.clone()
    o = handle.linear_attention_step(q, k, v, a, S)
    p = {"q": q[None], "k": k[None], "v": v[None], "log_decay": a}
    check_forward(o[None], S, p, D ** -0.5, S0)


def test_attention_without_tokens(handle):
    p, x = attention_problem(16, "f32", 0, 2, 2, 2, 16, 16)
    S = torch.empty_like(x["S0"])
    o = handle.linear_attention(**p, initial_state=x["S0"], final_state=S)
    assert o.shape == (0, 2, 2, 16) and torch.equal(S, x["S0"])
    handle.linear_attention(**p, final_state=S)
    assert not S.any()
    dS0 = torch.empty_like(S)
    handle.linear_attention_backward(**p, grad_out=o, grad_final_state=x["dS1"], grad_initial_state=dS0)
    assert torch.equal(dS0, x["dS1"])


def test_attention_state_in_place_and_repeatable(handle):
    p, x = attention_problem(17, "bf16", 700, 1, 2, 2, 64, 64)
    S = torch.empty_like(x["S0"])
    o = handle.linear_attention(**p, initial_state=x["S0"], final_state=S)
    state = x["S0"].clone()
    again = handle.linear_attention(**p, initial_state=state, final_state=state)
    assert torch.equal(o, again) and torch.equal(S, state)
    one = handle.linear_attention_backward(**p, grad_out=x["do"])
    two = handle.linear_attention_backward(**p, grad_out=x["do"])
    assert all(torch.equal(m, n) for m, n in zip(one, two))


def test_attention_binding_refusals(handle):
    p, x = attention_problem(18, "f32", 4, 2, 4, 2, 16, 16)
    ok = dict(p)
    with pytest.raises(TypeError):
        handle.linear_attention(**{**ok, "q": p["q"].double()})
    with pytest.raises(TypeError):
        handle.linear_attention(**{**ok, "k": p["k"].half()})
    with pytest.raises(ValueError):
        handle.linear_attention(**{**ok, "v": p["v"].cpu()})
    with pytest.raises(ValueError):
        handle.linear_attention(**{**ok, "k": p["k"][:3]})
    with pytest.raises(ValueError):
        handle.linear_attention(**{**ok, "q": p["q"].transpose(2, 3)})
    with pytest.raises(ValueError):
        handle.linear_attention(**ok, initial_state=x["S0"][:1])
    with pytest.raises(ValueError):
        handle.linear_attention(**ok, final_state=x["S0"].transpose(2, 3))
    with pytest.raises(ValueError):
        handle.linear_attention(**ok, lengths=torch.zeros(2, dtype=torch.int32, device="cuda"),
                                offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(PrnnError) as e:  # 3 heads of 2 key-value heads
        handle.linear_attention(p["q"][:, :, :3], p["k"], p["v"], p["log_decay"][:3].contiguous())
    assert e.value.status == binding.BAD_PARAM
    with pytest.raises(PrnnError) as e:
        handle.linear_attention(**ok, out=p["q"])
    assert e.value.status == binding.BAD_PARAM
    big = torch.zeros((2, 1, 1, 257), device="cuda")
    with pytest.raises(PrnnError) as e:
        handle.linear_attention(big, big, big, p["log_decay"][:1].contiguous())
    assert e.value.status == binding.BAD_PARAM


# -- layer norm ----------------------------------------------------------------------------------------------

def norm_problem(seed, type, M, N, params="same", offset=0.5):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[type]
    pt = dt if params == "same" else torch.float32
    x = (torch.randn((M, N), generator=g) * 2 + offset).to(dt).cuda()
    w = (1 + 0.3 * torch.randn(N, generator=g)).to(pt).cuda()
    b = (0.3 * torch.randn(N, generator=g)).to(pt).cuda()
    dy = torch.randn((M, N), generator=g).to(dt).cuda()
    return x, w, b, dy


def check_norm(y, mean, rstd, x, w, b, eps=1e-5):
    xn = host(x)
    wn, bn = (host(t) if t is not None else None for t in (w, b))
    ref, rm, rr = oracle.layer_norm(xn, wn, bn, eps)
    size = np.abs(xn).mean(-1)
    W = np.abs(wn) if wn is not None else 1.0
    A = np.abs(ref if bn is None else ref - bn) + (np.abs(bn) if bn is not None else 0.0) + \
        W * rr[..., None] * (np.abs(xn) + size[..., None])
    tol = half_step(y.dtype, ref) + 128 * U * A
    assert (np.abs(host(y) - ref) <= tol).all(), float((np.abs(host(y) - ref) / tol).max())
    if mean is not None:
        assert (np.abs(host(mean) - rm) <= 128 * U * size + 1e-38).all()
    if rstd is not None:
        # a mean off by 128 U size moves the variance by less than twice that times the deviation
        assert (np.abs(host(rstd) / rr - 1) <= 128 * U * (1 + 2 * size * rr)).all()


def check_norm_backward(dx, dw, db, dy, x, w, mean, rstd):
    dyn, xn = host(dy), host(x)
    wn = host(w) if w is not None else None
    rdx, rdw, rdb = oracle.layer_norm_backward(dyn, xn, wn)
    _, m, r = oracle.layer_norm(xn)
    m, r = m[..., None], r[..., None]
    n = np.abs((xn - m) * r)
    en = n + r * (np.abs(xn) + np.abs(m))   # what an error of U in the statistics does to n, over U
    g = np.abs(dyn if wn is None else dyn * wn)
    A = r * (g + g.mean(-1, keepdims=True) + (n + en) * (g * (n + en)).mean(-1, keepdims=True))
    if dx is not None:
        tol = half_step(dx.dtype, rdx) + 128 * U * A
        assert (np.abs(host(dx) - rdx) <= tol).all(), float((np.abs(host(dx) - rdx) / tol).max())
    M = xn.shape[0]
    if dw is not None:
        tol = half_step(dw.dtype, rdw) + (M + 16) * U * np.abs(dyn * en).sum(0)
        assert (np.abs(host(dw) - rdw) <= tol).all(), float((np.abs(host(dw) - rdw) / tol).max())
    if db is not None:
        tol = half_step(db.dtype, rdb) + (M + 16) * U * np.abs(dyn).sum(0)
        assert (np.abs(host(db) - rdb) <= tol).all(), float((np.abs(host(db) - rdb) / tol).max())


# every number of threads and vectors a row can take, widths that vectors do not divide, wider rows
NORM_SHAPES = [(1, 1), (3, 2), (5, 7), (300, 64), (70, 128), (33, 130), (9, 256), (17, 512), (4, 1000), (6, 1152),
               (4, 1792), (3, 2047), (3, 2304), (700, 257), (5, 4000), (3, 5760), (2, 7999), (3, 8000), (2, 12000),
               (2, 16384), (2, 12289), (3, 20001)]


@pytest.mark.parametrize("params", ["same", "f32"])
@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_norm(handle, type, params, shape):
    x, w, b, dy = norm_problem(sum(shape), type, *shape, params)
    mean = torch.empty(shape[0], device="cuda")
    rstd = torch.empty(shape[0], device="cuda")
    y = handle.layer_norm(x, w, b, mean=mean, rstd=rstd)
    check_norm(y, mean, rstd, x, w, b)
    dx, dw, db = handle.layer_norm_backward(dy, x, mean, rstd, w)
    check_norm_backward(dx, dw, db, dy, x, w, mean, rstd)


@pytest.mark.parametrize("type", sorted(TYPES))
def test_norm_without_parameters_and_in_place(handle, type):
    x, w, b, dy = norm_problem(1, type, 40, 192)
    mean, rstd = torch.empty(40, device="cuda"), torch.empty(40, device="cuda")
    check_norm(handle.layer_norm(x), None, None, x, None, None)
    check_norm(handle.layer_norm(x, w), None, None, x, w, None)
    check_norm(handle.layer_norm(x, None, b, mean=mean, rstd=rstd), mean, rstd, x, None, b)
    dx, dw, db = handle.layer_norm_backward(dy, x, mean, rstd)
    assert dw is None and db is None
    check_norm_backward(dx, None, None, dy, x, None, mean, rstd)
    dw = torch.empty(192, device="cuda")
    _, got, none = handle.layer_norm_backward(dy, x, mean, rstd, grad_weight=dw)
    assert got is dw and none is None
    check_norm_backward(None, dw, None, dy, x, None, mean, rstd)
    over = dy.clone()
    assert torch.equal(handle.layer_norm_backward(over, x, mean, rstd, grad_x=over)[0], dx)
    over = x.clone()
    assert torch.equal(handle.layer_norm_backward(dy, over, mean, rstd, grad_x=over)[0], dx)
    over = x.clone()
    y = handle.layer_norm(x, w, b)
    assert handle.layer_norm(over, w, b, out=over) is over and torch.equal(over, y)


@pytest.mark.parametrize("N", [96, 20000])
def test_norm_in_place_of_wide_rows_and_of_strided_ones(handle, N):
    x, w, b, dy = norm_problem(2, "f32", 6, 2 * N)
    xs, dys = x[:, N:], dy[:, :N]  # halves of wider rows
    w, b = w[:N].contiguous(), b[:N].contiguous()
    mean, rstd = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    y = torch.full((6, 2 * N), 3.0, device="cuda")
    handle.layer_norm(xs, w, b, out=y[:, :N], mean=mean, rstd=rstd)
    check_norm(y[:, :N], mean, rstd, xs, w, b)
    assert (y[:, N:] == 3).all()
    dx, dw, db = handle.layer_norm_backward(dys, xs, mean, rstd, w)
    check_norm_backward(dx, dw, db, dys, xs, w, mean, rstd)
    over = x.clone()
    dx2, dw2, _ = handle.layer_norm_backward(dys, over[:, N:], mean, rstd, w, grad_x=over[:, N:])
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw) and torch.equal(over[:, :N], x[:, :N])


def test_norm_leading_axes_and_unaligned_rows(handle):
    x, w, b, dy = norm_problem(3, "bf16", 6 * 5, 64)
    buf = torch.empty(6 * 5 * 64 + 1, dtype=torch.bfloat16, device="cuda")
    odd = buf[1:].view(6, 5, 64)
    odd.copy_(x.view(6, 5, 64))
    mean, rstd = torch.empty((6, 5), device="cuda"), torch.empty((6, 5), device="cuda")
    y = handle.layer_norm(odd, w, b, mean=mean, rstd=rstd)
    check_norm(y.view(30, 64), mean.view(30), rstd.view(30), x, w, b)
    with pytest.raises(ValueError):
        handle.layer_norm(torch.empty((4, 6, 64), device="cuda")[:, :5], None, None)


@pytest.mark.parametrize("type", sorted(TYPES))
def test_norm_of_constant_and_of_far_rows(handle, type):
    """Rows without variance give the bias; rows far from zero keep the digits
    their type holds."""
    x, w, b, _ = norm_problem(4, type, 8, 256)
    x[:4] = torch.tensor([0.0, 1.0, -3.0, 100.0], device="cuda")[:, None].to(x.dtype)
    y = handle.layer_norm(x, w, b)
    check_norm(y, None, None, x, w, b)
    far = norm_problem(5, "f32", 8, 1000, offset=1000.0)[0].to(TYPES[type])
    mean, rstd = torch.empty(8, device="cuda"), torch.empty(8, device="cuda")
    check_norm(handle.layer_norm(far, mean=mean, rstd=rstd), mean, rstd, far, None, None)


def test_norm_of_many_rows(handle):
    """More rows than the backward grid: the rows' sums run over several rounds."""
    for type, M, N in (("bf16", 20000, 64), ("f32", 5000, 520), ("f16", 3000, 1030)):
        x, w, b, dy = norm_problem(6, type, M, N, "f32")
        mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        y = handle.layer_norm(x, w, b, mean=mean, rstd=rstd)
        check_norm(y, mean, rstd, x, w, b)
        one = handle.layer_norm_backward(dy, x, mean, rstd, w)
        check_norm_backward(*one, dy, x, w, mean, rstd)
        two = handle.layer_norm_backward(dy, x, mean, rstd, w)
        assert all(torch.equal(p, q) for p, q in zip(one, two))


def test_norm_without_rows(handle):
    x = torch.empty((0, 64), device="cuda")
    none = torch.empty(0, device="cuda")
    w = torch.ones(64, device="cuda")
    assert handle.layer_norm(x, w).shape == (0, 64)
    dx, dw, db = handle.layer_norm_backward(x, x, none, none, w)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_norm_binding_refusals(handle):
    x, w, b, dy = norm_problem(7, "f16", 4, 64)
    with pytest.raises(TypeError):
        handle.layer_norm(x, w.bfloat16())
    with pytest.raises(TypeError):
        handle.layer_norm(x, w, b.float())
    with pytest.raises(ValueError):
        handle.layer_norm(x, w[:32].contiguous())
    with pytest.raises(TypeError):
        handle.layer_norm(x.double())
    with pytest.raises(ValueError):
        handle.layer_norm(x, out=torch.empty((4, 128), dtype=x.dtype, device="cuda")[:, ::2])
    with pytest.raises(PrnnError) as e:
        handle.layer_norm(x, eps=-1.0)
    assert e.value.status == binding.BAD_PARAM
    with pytest.raises(PrnnError) as e:
        handle.layer_norm(x, out=x.view(-1)[:4 * 63 + 1].as_strided((4, 64), (63, 1)))
    assert e.value.status == binding.BAD_PARAM


# -- streams and graphs ----------------------------------------------------------------------------------------

def layer(h, p, x, w, b, do, bufs, stream=None):
    """Norm, attention, their gradients and one step, into fixed buffers."""
    h.layer_norm(x, w, b, out=bufs["y"], mean=bufs["mean"], rstd=bufs["rstd"], stream=stream)
    q = bufs["y"].view(p["q"].shape)
    h.linear_attention(q, p["k"], p["v"], p["log_decay"], final_state=bufs["S"], out=bufs["o"], stream=stream)
    h.linear_attention_backward(q, p["k"], p["v"], p["log_decay"], do, grad_q=bufs["dq"], grad_k=bufs["dk"],
                                grad_v=bufs["dv"], stream=stream)
    h.layer_norm_backward(bufs["dq"].view(x.shape), x, bufs["mean"], bufs["rstd"], w, grad_x=bufs["dx"],
                          grad_weight=bufs["dw"], grad_bias=bufs["db"], stream=stream)
    h.linear_attention_step(q[0], p["k"][0], p["v"][0], p["log_decay"], bufs["S"], out=bufs["o1"],
                            new_state=bufs["S1"], stream=stream)


def layer_problem(seed):
    T, B, H, D = 300, 1, 2, 64
    p, e = attention_problem(seed, "bf16", T, B, H, 1, D, D)
    x, w, b, _ = norm_problem(seed, "bf16", T * B, H * D)
    like = lambda t: torch.empty_like(t)
    bufs = {"y": like(x), "mean": torch.empty(T * B, device="cuda"), "rstd": torch.empty(T * B, device="cuda"),
            "S": like(e["S0"]), "S1": like(e["S0"]), "o": like(e["do"]), "o1": like(e["do"][0]), "dq": like(p["q"]),
            "dk": like(p["k"]), "dv": like(p["v"]), "dx": like(x), "dw": like(w), "db": like(w)}
    return p, x, w, b, e["do"], bufs


def test_calls_follow_their_stream(gpu):
    p, x, w, b, do, bufs = layer_problem(20)
    with Handle() as h:
        layer(h, p, x, w, b, do, bufs)
        want = {n: t.clone() for n, t in bufs.items()}
        for t in bufs.values():
            t.fill_(float("nan"))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        layer(h, p, x, w, b, do, bufs, stream=side)
        alone = h.layer_norm(x, w, b, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
    for n, t in bufs.items():
        assert torch.equal(t, want[n]), n
    assert torch.equal(alone, want["y"])


def test_calls_in_a_graph(gpu):
    p, x, w, b, do, bufs = layer_problem(21)
    with Handle() as h:
        layer(h, p, x, w, b, do, bufs)  # the workspace grows here
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer(h, p, x, w, b, do, bufs)
        for seed in (22, 23, 24):
            p2, x2, _, _, do2, other = layer_problem(seed)
            layer(h, p2, x2, w, b, do2, other)  # eager, between replays, same sizes
            big = attention_problem(seed, "bf16", 500, 2, 4, 2, 64, 64)
            h.linear_attention_backward(**big[0], grad_out=big[1]["do"])  # eager; may need a larger workspace
            for to, of in ((p["q"], p2["q"]), (p["k"], p2["k"]), (p["v"], p2["v"]), (p["log_decay"], p2["log_decay"]),
                           (x, x2), (do, do2)):
                to.copy_(of)
            for t in bufs.values():
                t.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            for n, t in bufs.items():
                assert torch.equal(t, other[n]), n
        del graph


def test_growth_while_capturing_is_refused(gpu):
    x, w, b, dy = norm_problem(25, "f32", 64, 512)
    mean, rstd = torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    with Handle() as h:
        y = h.layer_norm(x, w, b, mean=mean, rstd=rstd)
        grads = [torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            h.layer_norm(x, w, b, out=y)
            with pytest.raises(PrnnError) as e:
                h.layer_norm_backward(dy, x, mean, rstd, w, grad_x=grads[0], grad_weight=grads[1], grad_bias=grads[2])
            assert e.value.status == binding.NOT_SUPPORTED
        graph.replay()
        torch.cuda.synchronize()
        check_norm(y, None, None, x, w, b)
