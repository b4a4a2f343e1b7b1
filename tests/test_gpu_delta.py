"""GPU parity of the gated delta rule (through the C ABI) against the fp64 oracle.

Tolerances come from the arithmetic.  The transition of a token, exp(log_decay)
(I - beta k k^T), has a 2-norm of at most 1 here (unit keys, beta in [0, 2],
decays <= 1, unless a test says otherwise), so a rounding error in a column of
the state is never enlarged by what follows.  A column meets about T + Dk + 64
roundings of at most 2^-24 of its 2-norm (or of the value it is compared with)
each: one or two a token in chunks, the sum over Dk rows, and the pairs of 32
tokens.  They add up as independent ones: c = 16 * 2^-24 sqrt(T + Dk + 64) bounds
the sum at many standard deviations.  By Cauchy-Schwarz an error of 2-norm d in
a column moves o by at most scale |q| d; the gradients' bounds are products of
2-norms in the same way (oracle.gated_delta_rule_backward returns them), with
3 c for the three passes.  Rounding to the type adds half a step of it.
"""
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
    return None if t is None else t.detach().double().cpu().numpy()


def half_step(dtype, ref):
    f = torch.finfo(dtype)
    return f.eps / 2 * np.abs(ref) + f.smallest_normal * f.eps / 2


def problem(seed, type, T, B, H, Hk, Dk, Dv, decay=None, beta=None):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[type]

    def unit(*shape):
        x = torch.randn(shape, generator=g) + 0.5
        x = x / x.square().sum(-1, keepdim=True).sqrt()
        return (x * (1 - 2.0 ** -7)).to(dt).cuda()  # (of a length of at most 1 after its rounding)

    p = {"q": unit(T, B, Hk, Dk), "k": unit(T, B, Hk, Dk), "v": torch.randn((T, B, H, Dv), generator=g).to(dt).cuda()}
    a = -torch.exp2(-8.0 * torch.rand((T, B, H), generator=g)) if decay is None else torch.tensor(decay).float().expand(T, B, H)
    b = torch.rand((T, B, H), generator=g) if beta is None else torch.tensor(beta).float().expand(T, B, H)
    p["log_decay"], p["beta"] = a.contiguous().cuda(), b.contiguous().cuda()
    extra = {"S0": torch.randn((B, H, Dk, Dv), generator=g).cuda(),
             "do": torch.randn((T, B, H, Dv), generator=g).to(dt).cuda(),
             "dS1": torch.randn((B, H, Dk, Dv), generator=g).cuda()}
    return p, extra


def close(name, got, ref, bound, dtype):
    got = host(got)
    tol = half_step(dtype, ref) + bound
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (name, int(bad.sum()), float(np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300))))


def rounding(T, Dk):
    return 16 * U * np.sqrt(T + Dk + 64)


def check_forward(o, S, p, scale, S0=None, lengths=None):
    n = {x: host(y) for x, y in p.items()}
    ref, refS, size = oracle.gated_delta_rule(**n, scale=scale, S0=host(S0), lengths=lengths)
    T, Dk, H = ref.shape[0], n["q"].shape[3], ref.shape[2]
    c = rounding(T, Dk)
    q = np.repeat(np.sqrt(np.square(n["q"]).sum(-1)), H // n["q"].shape[2], axis=2)
    close("o", o, ref, c * abs(scale) * q[..., None] * size[None], p["q"].dtype)
    if S is not None:
        close("S", S, refS, c * size[:, :, None, :], torch.float32)


NAMES = ("dq", "dk", "dv", "dlog_decay", "dbeta", "dS0")


def check_backward(grads, dS0, p, do, scale, S0=None, dS1=None, lengths=None):
    n = {x: host(y) for x, y in p.items()}
    ref, bound = oracle.gated_delta_rule_backward(**n, do=host(do), scale=scale, S0=host(S0), dS1=host(dS1), lengths=lengths)
    c = 3 * rounding(ref[0].shape[0], n["q"].shape[3])
    for i, (name, g) in enumerate(zip(NAMES, (*grads, dS0))):
        if g is not None:
            close(name, g, ref[i], c * bound[i], p["q"].dtype if i < 3 else torch.float32)


# (T, B, H, Hk, Dk, Dv): one token; lengths around and across chunks of 32; heads
# that fill, do not fill and exceed a tile; shared heads; odd sizes.
SHAPES = [(1, 1, 1, 1, 1, 1), (1, 3, 4, 2, 64, 64), (5, 2, 2, 1, 8, 16), (31, 1, 2, 2, 32, 32), (32, 2, 4, 2, 64, 64),
          (33, 1, 3, 3, 128, 128), (65, 1, 3, 1, 128, 128), (130, 2, 3, 1, 96, 80), (200, 1, 2, 2, 128, 64),
          (97, 1, 1, 1, 37, 53), (70, 1, 1, 1, 256, 256), (129, 1, 2, 2, 64, 200), (150, 1, 1, 1, 255, 9)]


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(handle, type, shape):
    p, x = problem(sum(shape), type, *shape)
    S = torch.full_like(x["S0"], float("nan"))
    o = handle.gated_delta_rule(**p, scale=0.3, initial_state=x["S0"], final_state=S)
    check_forward(o, S, p, 0.3, x["S0"])
    o = handle.gated_delta_rule(**p)
    check_forward(o, None, p, shape[4] ** -0.5)


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(handle, type, shape):
    p, x = problem(1 + sum(shape), type, *shape)
    dS0 = torch.full_like(x["S0"], float("nan"))
    grads = handle.gated_delta_rule_backward(**p, grad_out=x["do"], scale=0.3, initial_state=x["S0"],
                                             grad_final_state=x["dS1"], grad_initial_state=dS0)
    check_backward(grads, dS0, p, x["do"], 0.3, x["S0"], x["dS1"])
    grads = handle.gated_delta_rule_backward(**p, grad_out=x["do"])
    check_backward(grads, None, p, x["do"], shape[4] ** -0.5)


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("T", [700, 2500])
def test_long_sequence_of_one_head(handle, type, T):
    p, x = problem(T, type, T, 1, 1, 1, 64, 48, decay=-0.003)
    S, dS0 = torch.empty_like(x["S0"]), torch.empty_like(x["S0"])
    o = handle.gated_delta_rule(**p, scale=0.1, initial_state=x["S0"], final_state=S)
    check_forward(o, S, p, 0.1, x["S0"])
    grads = handle.gated_delta_rule_backward(**p, grad_out=x["do"], scale=0.1, initial_state=x["S0"],
                                             grad_final_state=x["dS1"], grad_initial_state=dS0)
    check_backward(grads, dS0, p, x["do"], 0.1, x["S0"], x["dS1"])


@pytest.mark.parametrize("type", sorted(TYPES))
def test_decays_and_shares(handle, type):
    """No decay, total decay (minus infinity) at every and at one token, fast and
    slow ones; beta 0, 1 and 2."""
    decay = [0.0, -float("inf"), -40.0, -1e-6, -2.0, -0.1]
    for beta in ([0.0, 1.0, 2.0, 0.5, 1.0, 0.0], [1.0, 0.5, 1.0, 2.0, 0.0, 1.5]):
        p, x = problem(5, type, 150, 1, 6, 2, 32, 32, decay=decay, beta=beta)
        p["log_decay"][77, 0, 5] = -float("inf")
        p["log_decay"][40:44, 0, 3] = -300.0
        S, dS0 = torch.empty_like(x["S0"]), torch.empty_like(x["S0"])
        o = handle.gated_delta_rule(**p, scale=0.2, initial_state=x["S0"], final_state=S)
        check_forward(o, S, p, 0.2, x["S0"])
        grads = handle.gated_delta_rule_backward(**p, grad_out=x["do"], scale=0.2, initial_state=x["S0"],
                                                 grad_final_state=x["dS1"], grad_initial_state=dS0)
        check_backward(grads, dS0, p, x["do"], 0.2, x["S0"], x["dS1"])


@pytest.mark.parametrize("type", sorted(TYPES))
def test_without_decay(handle, type):
    p, x = problem(15, type, 70, 2, 2, 1, 64, 64, decay=0.0)
    q = {**p, "log_decay": None}
    S, S2 = torch.empty_like(x["S0"]), torch.empty_like(x["S0"])
    o = handle.gated_delta_rule(**q, initial_state=x["S0"], final_state=S)
    assert torch.equal(o, handle.gated_delta_rule(**p, initial_state=x["S0"], final_state=S2)) and torch.equal(S, S2)
    a, b = (handle.gated_delta_rule_backward(**r, grad_out=x["do"], initial_state=x["S0"]) for r in (p, q))
    assert b[3] is None
    for i in (0, 1, 2, 4):
        assert torch.equal(a[i], b[i])
    one = {m: (t[0] if t is not None else None) for m, t in q.items()}
    s1, s2 = torch.empty_like(S), torch.empty_like(S)
    o1 = handle.gated_delta_rule_step(**one, state=x["S0"], new_state=s1)
    o2 = handle.gated_delta_rule_step(**{**one, "log_decay": p["log_decay"][0]}, state=x["S0"], new_state=s2)
    assert torch.equal(o1, o2) and torch.equal(s1, s2)


@pytest.mark.parametrize("type", sorted(TYPES))
def test_one_key_again_and_again(handle, type):
    """Keys that are all the same, fully corrected: every value replaces the one
    before, and T' has entries of the size of 1 in every place of its band."""
    p, x = problem(16, type, 100, 1, 2, 1, 64, 64, decay=0.0, beta=[1.0, 2.0])
    p["k"] = p["k"][:1].expand(100, 1, 1, 64).contiguous()
    S = torch.empty_like(x["S0"])
    o = handle.gated_delta_rule(**p, scale=0.2, initial_state=x["S0"], final_state=S)
    check_forward(o, S, p, 0.2, x["S0"])


@pytest.mark.parametrize("type", sorted(TYPES))
def test_lengths(handle, type):
    """A padded batch with an empty sequence, one token, a full one, lengths out
    of range; what the padding holds (NaN here) reaches nothing."""
    lengths = [0, 1, 90, 64, 200, -3]
    used = [0, 1, 90, 64, 90, 0]
    p, x = problem(6, type, 90, 6, 2, 1, 64, 32)
    clean = {m: t.clone() for m, t in p.items()}
    clean_do = x["do"].clone()
    for b, n in enumerate(used):
        for t in (*p.values(), x["do"]):
            t[n:, b] = float("nan")
    S, dS0 = torch.empty_like(x["S0"]), torch.empty_like(x["S0"])
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o = handle.gated_delta_rule(**p, scale=0.2, initial_state=x["S0"], final_state=S, lengths=n)
    grads = handle.gated_delta_rule_backward(**p, grad_out=x["do"], scale=0.2, initial_state=x["S0"],
                                             grad_final_state=x["dS1"], grad_initial_state=dS0, lengths=n)
    check_forward(o, S, clean, 0.2, x["S0"], used)
    check_backward(grads, dS0, clean, clean_do, 0.2, x["S0"], x["dS1"], used)
    for b, m in enumerate(used):
        for t in (o, *grads):
            assert not t[m:, b].any()


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("max_len", [None, 100])
def test_packed(handle, type, max_len):
    """Packed sequences, empty ones among them; rows that belong to none keep
    what the outputs held."""
    offsets = [2, 2, 3, 103, 103, 140, 141]
    rows = 143
    B, H, Hk = 6, 4, 2
    p, x = problem(7, type, rows, 1, H, Hk, 48, 64)
    S0 = torch.randn((B, H, 48, 64), device="cuda")
    packed = {m: t[:, 0].contiguous() for m, t in p.items()}
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    S, dS0 = torch.empty_like(S0), torch.empty_like(S0)
    out = torch.full((rows, H, 64), 7.0, dtype=TYPES[type], device="cuda")
    seq = {"scale": 0.2, "offsets": off, "max_len": max_len, "initial_state": S0}
    handle.gated_delta_rule(**packed, final_state=S, out=out, **seq)
    given = {"grad_q": torch.full_like(packed["q"], 7.0), "grad_k": torch.full_like(packed["k"], 7.0),
             "grad_v": torch.full_like(packed["v"], 7.0), "grad_log_decay": torch.full_like(packed["beta"], 7.0),
             "grad_beta": torch.full_like(packed["beta"], 7.0)}
    grads = handle.gated_delta_rule_backward(**packed, grad_out=x["do"][:, 0].contiguous(), grad_final_state=S0 + 1,
                                             grad_initial_state=dS0, **given, **seq)
    for b, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        one = {m: t[lo:hi] for m, t in p.items()}
        check_forward(out[lo:hi, None], S[b:b + 1], one, 0.2, S0[b:b + 1])
        check_backward([g[lo:hi, None] for g in grads], dS0[b:b + 1], one, x["do"][lo:hi], 0.2, S0[b:b + 1],
                       S0[b:b + 1] + 1)
    for t in (out, *grads):
        assert (t[:2] == 7).all() and (t[141:] == 7).all()


def test_offsets_out_of_range_stay_inside(handle):
    """Offsets are clamped to the rows there are, and to max_len."""
    p, _ = problem(8, "f32", 40, 1, 1, 1, 16, 16)
    packed = {m: t[:, 0].contiguous() for m, t in p.items()}
    off = torch.tensor([-5, 10, 10, 1000, 1000], dtype=torch.int32, device="cuda")
    S = torch.empty((4, 1, 16, 16), device="cuda")
    out = torch.zeros((40, 1, 16), device="cuda")
    handle.gated_delta_rule(**packed, scale=1.0, offsets=off, max_len=24, final_state=S, out=out)
    for b, (lo, hi) in enumerate(((0, 10), (10, 10), (10, 34), (40, 40))):
        one = {m: t[lo:hi] for m, t in p.items()}
        check_forward(out[lo:hi, None], S[b:b + 1], one, 1.0)
    assert not out[34:].any()


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("layout", ["batch first", "fused", "unaligned", "repeated"])
def test_strides(handle, type, layout):
    T, B, H, Hk, D = 70, 2, 4, 2, 64
    p, x = problem(9, type, T, B, H, Hk, D, D)
    out = None
    grads = {}
    if layout == "batch first":
        move = lambda t: t.movedim(0, 2).contiguous().movedim(2, 0)
        p = {m: move(t) for m, t in p.items()}
        x["do"] = move(x["do"])
        out = torch.empty((B, H, T, D), dtype=TYPES[type], device="cuda").permute(2, 0, 1, 3)
        grads = {"grad_beta": torch.empty((B, H, T), device="cuda").permute(2, 0, 1)}
    elif layout == "fused":
        fused = torch.cat([p["q"].flatten(2), p["k"].flatten(2), p["v"].flatten(2)], dim=2)
        cut = lambda t: [y.unflatten(2, (n, D)) for y, n in zip(t.split([Hk * D, Hk * D, H * D], dim=2), (Hk, Hk, H))]
        p.update(zip(("q", "k", "v"), cut(fused)))
        both = torch.stack([p["log_decay"], p["beta"]], dim=3)
        p.update(log_decay=both[..., 0], beta=both[..., 1])
        grads = dict(zip(("grad_q", "grad_k", "grad_v"), cut(torch.empty_like(fused))))
        pair = torch.empty_like(both)
        grads.update(grad_log_decay=pair[..., 0], grad_beta=pair[..., 1])
    elif layout == "unaligned":
        def shift(t):
            buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
            buf[1:].view(t.shape).copy_(t)
            return buf[1:].view(t.shape)
        p = {m: shift(t) for m, t in p.items()}
        x["do"] = shift(x["do"])
        out = shift(torch.zeros((T, B, H, D), dtype=TYPES[type], device="cuda"))
        grads = {"grad_q": shift(p["q"]), "grad_v": shift(p["v"])}
    else:
        p["k"] = p["k"][:, :1, :1].expand(T, B, Hk, D)
        p["q"] = p["q"][:1].expand(T, B, Hk, D)
        p["beta"] = p["beta"][:1, :1].expand(T, B, H)
    S = torch.empty_like(x["S0"])
    o = handle.gated_delta_rule(**p, scale=0.2, initial_state=x["S0"], final_state=S, out=out)
    check_forward(o, S, p, 0.2, x["S0"])
    got = handle.gated_delta_rule_backward(**p, grad_out=x["do"], scale=0.2, **grads)
    check_backward(got, None, p, x["do"], 0.2)


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("where", ["q", "k", "v", "log_decay", "beta"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_later_tokens_reach_no_earlier_row(handle, type, where, value):
    """A NaN or infinity at one token: the rows before it are as if it were not
    there, other heads and sequences too; where the recurrence is not finite, so
    is the result."""
    T, t = 150, 75
    p, x = problem(10, type, T, 2, 2, 2, 64, 64, decay=[-0.01, -0.5])
    if where in ("log_decay", "beta"):
        p[where][t, 0, 0] = value
    else:
        p[where][t, 0, 0, 5] = value
    S = torch.empty_like(x["S0"])
    o = handle.gated_delta_rule(**p, scale=0.2, initial_state=x["S0"], final_state=S)
    before = {m: y[:t] for m, y in p.items()}
    check_forward(o[:t], None, before, 0.2, x["S0"])
    others = {m: y[:, :, 1:] for m, y in p.items()}
    check_forward(o[:, :, 1:], S[:, 1:], others, 0.2, x["S0"][:, 1:])
    check_forward(o[:, 1:], S[1:], {m: y[:, 1:] for m, y in p.items()}, 0.2, x["S0"][1:])
    with np.errstate(all="ignore"):
        ref, refS, _ = oracle.gated_delta_rule(**{m: host(y) for m, y in p.items()}, scale=0.2, S0=host(x["S0"]))
    for got, want in ((host(o), ref), (host(S), refS)):
        assert np.array_equal(np.isfinite(got), np.isfinite(want))
    grads = handle.gated_delta_rule_backward(**p, grad_out=x["do"], scale=0.2, initial_state=x["S0"])
    for name, got, want in zip(NAMES, grads, oracle.gated_delta_rule_backward(
            **{m: host(y[:, 1:]) for m, y in p.items()}, do=host(x["do"][:, 1:]), scale=0.2, S0=host(x["S0"][1:]))[0]):
        assert np.isfinite(host(got[:, 1:])).all(), name
        assert np.linalg.norm(host(got[:, 1:]) - want) <= 1e-2 * np.linalg.norm(want), name


def test_large_values_of_fp16(handle):
    """Scores and states beyond fp16's range, outputs inside it."""
    p, x = problem(11, "f16", 100, 1, 1, 1, 64, 64)
    p["q"], p["v"] = p["q"] * 1000, p["v"] * 10000
    S = torch.empty_like(x["S0"])
    o = handle.gated_delta_rule(**p, scale=1e-4, final_state=S)
    check_forward(o, S, p, 1e-4)
    grads = handle.gated_delta_rule_backward(**p, grad_out=x["do"], scale=1e-4)
    check_backward(grads, None, p, x["do"], 1e-4)


def test_row_offsets_past_32_bits(handle):
    T, D, stride = 300, 64, 1 << 23
    buf = torch.empty(T * stride, dtype=torch.float16, device="cuda")  # 5 GB
    p, x = problem(13, "f16", T, 1, 1, 1, D, D)
    views = {}
    for i, m in enumerate(("q", "k", "v", "o", "do", "dq", "dk", "dv")):
        views[m] = buf.as_strided((T, 1, 1, D), (stride, D, D, 1), 100 * i * 64)
        if m in p:
            views[m].copy_(p[m])
    views["do"].copy_(x["do"])
    q = {**p, "q": views["q"], "k": views["k"], "v": views["v"]}
    o = handle.gated_delta_rule(**q, scale=0.2, out=views["o"])
    check_forward(o.contiguous(), None, p, 0.2)
    grads = handle.gated_delta_rule_backward(**q, grad_out=views["do"], scale=0.2, grad_q=views["dq"], grad_k=views["dk"],
                                             grad_v=views["dv"])
    check_backward(grads, None, p, x["do"], 0.2)


def test_gradients_match_differences(handle):
    """Along a direction, central differences of step e: the third derivative's
    e^2 (about 1e-5 of the terms at e = 3e-3) and the rounding of the two
    losses over 2 e (2^-24 of the terms' sum of 5000, as independent ones, over
    6e-3), together below 1e-3 of the terms' 2-norm."""
    p, x = problem(14, "f32", 100, 2, 4, 2, 32, 48)
    do, dS1 = x["do"], x["dS1"]
    dS0 = torch.empty_like(x["S0"])
    grads = handle.gated_delta_rule_backward(**p, grad_out=do, scale=0.3, initial_state=x["S0"], grad_final_state=dS1,
                                             grad_initial_state=dS0)

    def loss(p, S0):
        S = torch.empty_like(S0)
        o = handle.gated_delta_rule(**p, scale=0.3, initial_state=S0, final_state=S)
        return (o.double() * do.double()).sum() + (S.double() * dS1.double()).sum()

    g = torch.Generator().manual_seed(0)
    e = 3e-3
    for name, grad in zip(("q", "k", "v", "log_decay", "beta", "S0"), (*grads, dS0)):
        at = x["S0"] if name == "S0" else p[name]
        d = torch.randn(at.shape, generator=g).cuda()
        d = d / d.square().sum(-1, keepdim=True).sqrt() if name in ("q", "k") else d * 0.3
        hi, lo = (loss(p, at + s * d) if name == "S0" else loss({**p, name: at + s * d}, x["S0"]) for s in (e, -e))
        terms = grad.double() * d.double()
        assert abs((hi - lo) / (2 * e) - terms.sum()) <= 1e-3 * (terms.square().sum().sqrt() + 1), name


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1), (1, 14, 14, 128, 128), (5, 4, 2, 64, 80), (3, 6, 3, 37, 53), (2, 2, 1, 33, 3),
                                   (2, 2, 1, 256, 255)], ids=str)
def test_step(handle, type, shape):
    B, H, Hk, Dk, Dv = shape
    p, x = problem(17, type, 1, B, H, Hk, Dk, Dv)
    one = {m: t[0] for m, t in p.items()}
    S = x["S0"].clone()
    new = torch.full_like(S, float("nan"))
    o = handle.gated_delta_rule_step(**one, state=S, scale=0.3, new_state=new)
    assert torch.equal(S, x["S0"])
    check_forward(o[None], new, p, 0.3, x["S0"])
    o2 = handle.gated_delta_rule_step(**one, state=S, scale=0.3)  # in place
    assert torch.equal(o, o2) and torch.equal(S, new)


@pytest.mark.parametrize("type", sorted(TYPES))
def test_steps_continue_a_prompt(handle, type):
    T, n = 80, 7
    p, x = problem(18, type, T, 2, 4, 2, 64, 96)
    S = x["S0"].clone()
    head = {m: t[:T - n] for m, t in p.items()}
    o = [handle.gated_delta_rule(**head, initial_state=S, final_state=S)]
    for t in range(T - n, T):
        o.append(handle.gated_delta_rule_step(**{m: y[t] for m, y in p.items()}, state=S)[None])
    check_forward(torch.cat(o), S, p, 64 ** -0.5, x["S0"])


def test_states_in_place(handle):
    p, x = problem(19, "bf16", 100, 2, 4, 2, 64, 64)
    S = torch.empty_like(x["S0"])
    o = handle.gated_delta_rule(**p, initial_state=x["S0"], final_state=S)
    S0 = x["S0"].clone()
    assert torch.equal(o, handle.gated_delta_rule(**p, initial_state=S0, final_state=S0)) and torch.equal(S, S0)
    dS0 = torch.empty_like(S)
    a = handle.gated_delta_rule_backward(**p, grad_out=x["do"], initial_state=x["S0"], grad_final_state=x["dS1"],
                                         grad_initial_state=dS0)
    dS = x["dS1"].clone()
    b = handle.gated_delta_rule_backward(**p, grad_out=x["do"], initial_state=x["S0"], grad_final_state=dS,
                                         grad_initial_state=dS)
    assert torch.equal(dS, dS0) and all(torch.equal(y, z) for y, z in zip(a, b))


def test_no_tokens_and_no_sequences(handle):
    p, x = problem(20, "f32", 4, 2, 2, 1, 32, 32)
    none = {m: t[:0] for m, t in p.items()}
    S = torch.full_like(x["S0"], 5.0)
    assert handle.gated_delta_rule(**none, initial_state=x["S0"], final_state=S).shape == (0, 2, 2, 32)
    assert torch.equal(S, x["S0"])
    handle.gated_delta_rule(**none, final_state=S)
    assert not S.any()
    dS0 = torch.empty_like(S)
    handle.gated_delta_rule_backward(**none, grad_out=x["do"][:0], grad_final_state=x["dS1"], grad_initial_state=dS0)
    assert torch.equal(dS0, x["dS1"])
    empty = {m: t[:, :0] for m, t in p.items()}
    assert handle.gated_delta_rule(**empty).shape == (4, 0, 2, 32)


@pytest.mark.parametrize("type", sorted(TYPES))
def test_states_keep_fp32_s_bits(handle, type):
    """States and the scalars' gradients are fp32 whatever the operands: as many
    independent roundings of 2^-24 as a column meets, four times over, which
    16-bit intermediate values (2^-16 each) would exceed."""
    T, D = 256, 128
    p, x = problem(21, type, T, 1, 4, 2, D, D)
    S = torch.empty_like(x["S0"])
    dS0 = torch.empty_like(S)
    handle.gated_delta_rule(**p, initial_state=x["S0"], final_state=S)
    grads = handle.gated_delta_rule_backward(**p, grad_out=x["do"], initial_state=x["S0"], grad_final_state=x["dS1"],
                                             grad_initial_state=dS0)
    n = {m: host(t) for m, t in p.items()}
    _, ref, _ = oracle.gated_delta_rule(**n, S0=host(x["S0"]))
    want = oracle.gated_delta_rule_backward(**n, do=host(x["do"]), S0=host(x["S0"]), dS1=host(x["dS1"]))[0]
    for name, got, r in (("S", S, ref), ("dS0", dS0, want[5]), ("dlog_decay", grads[3], want[3]), ("dbeta", grads[4], want[4])):
        off = np.linalg.norm(host(got) - r) / np.linalg.norm(r)
        print(type, name, off)
        assert off <= 4 * U * np.sqrt(T + D + 64), (name, off)


def test_calls_repeat_bit_for_bit(handle):
    p, x = problem(22, "bf16", 500, 2, 4, 2, 64, 64)
    runs = []
    for _ in range(3):
        S = torch.empty_like(x["S0"])
        runs.append((handle.gated_delta_rule(**p, initial_state=x["S0"], final_state=S), S,
                     *handle.gated_delta_rule_backward(**p, grad_out=x["do"], initial_state=x["S0"])))
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_graphs_replay_with_eager_calls_between(gpu):
    """A prompt, its gradients and a step captured; the inputs change between the
    replays, and eager calls on the same handle and memory run there too."""
    with Handle() as h:
        p, x = problem(23, "bf16", 300, 2, 4, 2, 64, 64)
        big, bx = problem(24, "bf16", 400, 2, 4, 2, 64, 64)
        S1, dS0, Sn = (torch.empty_like(x["S0"]) for _ in range(3))

        def work():
            o = h.gated_delta_rule(**p, initial_state=x["S0"], final_state=S1)
            g = h.gated_delta_rule_backward(**p, grad_out=x["do"], initial_state=x["S0"], grad_initial_state=dS0)
            o1 = h.gated_delta_rule_step(**{m: t[0] for m, t in p.items()}, state=x["S0"], new_state=Sn)
            return (o, S1, *g, dS0, o1, Sn)

        work()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                outs = work()
        torch.cuda.synchronize()
        for i in range(3):
            p["v"].copy_(torch.randn_like(p["v"]))
            x["S0"].normal_()
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in outs]
            h.gated_delta_rule_backward(**big, grad_out=bx["do"])  # a larger workspace than the captured one
            want = work()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_workspace_does_not_grow_while_capturing(gpu):
    with Handle() as h:
        p, _ = problem(25, "f32", 64, 1, 1, 1, 32, 32)
        out = torch.empty((64, 1, 1, 32), device="cuda")
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                with pytest.raises(PrnnError) as e:
                    h.gated_delta_rule(**p, out=out)
                out.zero_()
        assert e.value.status == binding.NOT_SUPPORTED


def test_runs_on_the_stream_given(handle):
    p, x = problem(26, "f32", 200, 1, 2, 2, 64, 64)
    want = handle.gated_delta_rule(**p)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        v = p["v"] * 2
    o = handle.gated_delta_rule(**{**p, "v": v}, stream=side)
    side.synchronize()
    assert torch.equal(o, want * 2)


def test_refusals(handle):
    p, x = problem(27, "f32", 8, 1, 2, 1, 16, 16)
    for change, error in (({"q": p["q"][..., :8]}, None), ({"k": p["k"].half()}, TypeError), ({"beta": p["beta"].double()}, TypeError),
                          ({"beta": p["beta"][:4]}, ValueError), ({"beta": None}, TypeError), ({"v": p["v"].cpu()}, ValueError),
                          ({"q": p["q"].expand(8, 1, 3, 16), "k": p["k"].expand(8, 1, 3, 16)}, PrnnError)):
        with pytest.raises(error or (ValueError, TypeError)):
            handle.gated_delta_rule(**{**p, **change})
    with pytest.raises(PrnnError):
        handle.gated_delta_rule(**p, out=p["v"])
    with pytest.raises(PrnnError):
        handle.gated_delta_rule_backward(**p, grad_out=x["do"], grad_beta=p["beta"])
    with pytest.raises(ValueError):
        handle.gated_delta_rule(**p, initial_state=x["S0"][:, :, :, :8])
    handle.synchronize()


# -- sequences long enough to be split into segments, and groups of chunks ----------

SPLIT = [(530, 2, 3, 1, 96, 80), (600, 1, 2, 2, 128, 128), (420, 1, 1, 1, 256, 40), (401, 3, 2, 1, 33, 5), (777, 1, 1, 1, 100, 256),
         (384, 1, 4, 2, 64, 64)]


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("shape", SPLIT, ids=str)
def test_split_sequences(handle, type, shape):
    """The states are in place: other workgroups may end before the first segment starts."""
    p, x = problem(31 + sum(shape), type, *shape)
    S = x["S0"].clone()
    o = handle.gated_delta_rule(**p, scale=0.3, initial_state=S, final_state=S)
    check_forward(o, S, p, 0.3, x["S0"])
    o = handle.gated_delta_rule(**p, scale=0.3)
    check_forward(o, None, p, 0.3)
    dS = x["dS1"].clone()
    grads = handle.gated_delta_rule_backward(**p, grad_out=x["do"], scale=0.3, initial_state=x["S0"],
                                             grad_final_state=dS, grad_initial_state=dS)
    check_backward(grads, dS, p, x["do"], 0.3, x["S0"], x["dS1"])
    grads = handle.gated_delta_rule_backward(**p, grad_out=x["do"], scale=0.3)
    check_backward(grads, None, p, x["do"], 0.3)


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("Dk", [48, 112])
def test_split_lengths(handle, type, Dk):
    """A padded batch of sequences in none, one and several segments."""
    used = [0, 1, 530, 400, 129, 31, 256]
    p, x = problem(41, type, 530, len(used), 1, 1, Dk, 72)
    clean, clean_do = {m: t.clone() for m, t in p.items()}, x["do"].clone()
    for b, n in enumerate(used):
        for t in (*p.values(), x["do"]):
            t[n:, b] = float("nan")
    S, dS0 = torch.empty_like(x["S0"]), torch.empty_like(x["S0"])
    n = torch.tensor(used, dtype=torch.int32, device="cuda")
    o = handle.gated_delta_rule(**p, scale=0.2, initial_state=x["S0"], final_state=S, lengths=n)
    grads = handle.gated_delta_rule_backward(**p, grad_out=x["do"], scale=0.2, initial_state=x["S0"],
                                             grad_final_state=x["dS1"], grad_initial_state=dS0, lengths=n)
    check_forward(o, S, clean, 0.2, x["S0"], used)
    check_backward(grads, dS0, clean, clean_do, 0.2, x["S0"], x["dS1"], used)
    for b, m in enumerate(used):
        for t in (o, *grads):
            assert not t[m:, b].any()


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("max_len", [None, 450])
@pytest.mark.parametrize("Dk", [64, 100])
def test_split_packed(handle, type, max_len, Dk):
    """Long packed sequences between more short and empty ones than a wave looks at
    at once; segments of one begin inside what would be another's."""
    lens = [3, 450, 0, 0, 131, 1, 389] + [i % 4 for i in range(70)] + [300, 0]
    offsets = np.cumsum([1] + lens)
    rows = int(offsets[-1]) + 5
    B, H, Hk = len(lens), 2, 1
    p, x = problem(43, type, rows, 1, H, Hk, Dk, 24)
    S0 = torch.randn((B, H, Dk, 24), device="cuda")
    packed = {m: t[:, 0].contiguous() for m, t in p.items()}
    S, dS0 = torch.empty_like(S0), torch.empty_like(S0)
    out = torch.full((rows, H, 24), 7.0, dtype=TYPES[type], device="cuda")
    seq = {"scale": 0.2, "offsets": torch.tensor(offsets, dtype=torch.int32, device="cuda"), "max_len": max_len, "initial_state": S0}
    handle.gated_delta_rule(**packed, final_state=S, out=out, **seq)
    given = {f"grad_{m}": torch.full_like(t, 7.0) for m, t in packed.items()}
    grads = handle.gated_delta_rule_backward(**packed, grad_out=x["do"][:, 0].contiguous(), grad_final_state=S0 + 1,
                                             grad_initial_state=dS0, **given, **seq)
    for b in [0, 1, 2, 4, 5, 6, 8, 10, 40, 75, 76, 77, 78]:
        lo, hi = offsets[b:b + 2]
        one = {m: t[lo:hi] for m, t in p.items()}
        check_forward(out[lo:hi, None], S[b:b + 1], one, 0.2, S0[b:b + 1])
        check_backward([g[lo:hi, None] for g in grads], dS0[b:b + 1], one, x["do"][lo:hi], 0.2, S0[b:b + 1], S0[b:b + 1] + 1)
    for t in (out, *grads):
        assert (t[:1] == 7).all() and (t[-5:] == 7).all()


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("T", [32, 63, 64, 65, 96, 97, 128, 129])
def test_groups_of_chunks(handle, type, T):
    """Gradients where the last group of chunks is whole, of one chunk, of one token."""
    p, x = problem(50 + T, type, T, 2, 2, 1, 112, 72)
    dS0 = torch.empty_like(x["S0"])
    grads = handle.gated_delta_rule_backward(**p, grad_out=x["do"], scale=0.3, initial_state=x["S0"],
                                             grad_final_state=x["dS1"], grad_initial_state=dS0)
    check_backward(grads, dS0, p, x["do"], 0.3, x["S0"], x["dS1"])


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("where", ["q", "k", "v", "log_decay", "beta"])
def test_later_tokens_of_a_split_sequence(handle, type, where):
    """As test_later_tokens_reach_no_earlier_row, from a token in a middle segment on."""
    T, t = 520, 300
    p, x = problem(60, type, T, 2, 2, 2, 64, 64, decay=[-0.01, -0.5])
    if where in ("log_decay", "beta"):
        p[where][t, 0, 0] = float("nan")
    else:
        p[where][t, 0, 0, 5] = float("nan")
    S = torch.empty_like(x["S0"])
    o = handle.gated_delta_rule(**p, scale=0.2, initial_state=x["S0"], final_state=S)
    check_forward(o[:t], None, {m: y[:t] for m, y in p.items()}, 0.2, x["S0"])
    check_forward(o[:, 1:], S[1:], {m: y[:, 1:] for m, y in p.items()}, 0.2, x["S0"][1:])
    with np.errstate(all="ignore"):
        ref, refS, _ = oracle.gated_delta_rule(**{m: host(y) for m, y in p.items()}, scale=0.2, S0=host(x["S0"]))
    for got, want in ((host(o), ref), (host(S), refS)):
        assert np.array_equal(np.isfinite(got), np.isfinite(want))


@pytest.mark.parametrize("type", sorted(TYPES))
def test_decays_to_nothing_in_a_split_sequence(handle, type):
    """log_decay of minus infinity forgets what was before, in the middle of a segment and
    at its first token; beta of 0 and keys of zeros change nothing."""
    p, x = problem(61, type, 500, 1, 2, 1, 64, 64)
    p["log_decay"][[200, 256, 384, 385], :, 0] = float("-inf")
    p["beta"][300:340] = 0
    p["k"][400:420] = 0
    S = torch.empty_like(x["S0"])
    o = handle.gated_delta_rule(**p, scale=0.2, initial_state=x["S0"], final_state=S)
    check_forward(o, S, p, 0.2, x["S0"])
    q = {m: y.clone() for m, y in p.items()}
    q["log_decay"].clamp_(min=-200.0)  # exp is 0 all the same, and the oracle's sums of it are finite
    grads = handle.gated_delta_rule_backward(**p, grad_out=x["do"], scale=0.2, initial_state=x["S0"])
    check_backward(grads, None, q, x["do"], 0.2, x["S0"])


def test_two_graphs_share_the_workspace(gpu):
    """Graphs of two calls of one handle, one split, replayed in turn on one stream."""
    with Handle() as h:
        a, ax = problem(62, "bf16", 700, 1, 2, 1, 64, 64)
        b, bx = problem(63, "f16", 200, 3, 4, 4, 96, 40)
        calls = [lambda: h.gated_delta_rule_backward(**a, grad_out=ax["do"], initial_state=ax["S0"]),
                 lambda: (h.gated_delta_rule(**b), h.gated_delta_rule_backward(**b, grad_out=bx["do"])[4])]
        want = [[t.clone() for t in call()] for call in calls]
        for call in calls:
            call()
        torch.cuda.synchronize()
        side, graphs, outs = torch.cuda.Stream(), [], []
        with torch.cuda.stream(side):
            for call in calls:
                graphs.append(torch.cuda.CUDAGraph())
                with torch.cuda.graph(graphs[-1], stream=side):
                    outs.append(call())
        torch.cuda.synchronize()
        for i in (0, 1, 1, 0, 0, 1):
            for t in outs[i]:
                t.zero_()
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                graphs[i].replay()
                graphs[1 - i].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for got, ref in zip(outs, want) for x, y in zip(got, ref)), i


def test_two_handles_on_two_streams(gpu):
    """Each handle has its own workspace: calls that run at once leave each other's results alone."""
    problems = [problem(64, "bf16", 900, 1, 2, 1, 64, 64), problem(65, "f32", 300, 2, 4, 4, 96, 40)]
    with Handle() as a, Handle() as b:
        def call(h, p, x, stream=None):
            S = torch.empty_like(x["S0"])
            return (h.gated_delta_rule(**p, initial_state=x["S0"], final_state=S, stream=stream), S,
                    *h.gated_delta_rule_backward(**p, grad_out=x["do"], initial_state=x["S0"], stream=stream))

        want = [call(h, *p) for h, p in zip((a, b), problems)]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = [[], []]
        for _ in range(5):
            for i, h in enumerate((a, b)):
                with torch.cuda.stream(streams[i]):
                    got[i].append(call(h, *problems[i]))
        torch.cuda.synchronize()
        for i in range(2):
            for run in got[i]:
                assert all(torch.equal(x, y) for x, y in zip(run, want[i])), i
