"""GPU tests of linear attention and layer norm at the edges of what they take:
lengths, strides, buffers that are one, sizes past the usual shapes.

Tolerances are those of test_gpu_sequence.py, whose derivation they share.
"""
import numpy as np
import pytest
import torch

import oracle
from persistent_rnn_fwd_amd import Handle
from test_gpu_sequence import TYPES, attention_problem, check_backward, check_forward, check_norm, check_norm_backward, \
    handle, host, norm_problem  # noqa: F401

pytestmark = pytest.mark.gpu


def packed_problem(seed, type, lengths, H, Hkv, Dk, Dv):
    """A problem of packed sequences: as one row of tokens (T = all, B = 1), and as the call takes it."""
    offsets = [0]
    for n in lengths:
        offsets.append(offsets[-1] + n)
    p, x = attention_problem(seed, type, offsets[-1], 1, H, Hkv, Dk, Dv)
    _, s = attention_problem(seed + 1, type, 1, len(lengths), H, Hkv, Dk, Dv)
    x.update(S0=s["S0"], dS1=s["dS1"])
    packed = {n: (t[:, 0].contiguous() if n != "log_decay" else t) for n, t in p.items()}
    return p, x, packed, torch.tensor(offsets, dtype=torch.int32, device="cuda"), offsets


# -- lengths ---------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("max_len", [2**31 - 1, 2**31 - 64, 2**40])
def test_a_length_past_the_rows_is_the_rows(handle, max_len):  # noqa: F811
    """Packed calls whose longest sequence is not known."""
    lengths, H = [700, 0, 1500, 65], 96
    p, x, packed, off, offsets = packed_problem(1, "bf16", lengths, H, H, 32, 128)
    S, S2 = torch.full_like(x["S0"], float("nan")), torch.full_like(x["S0"], float("nan"))
    o = handle.linear_attention(**packed, scale=0.3, offsets=off, initial_state=x["S0"], final_state=S, max_len=max_len)
    o2 = handle.linear_attention(**packed, scale=0.3, offsets=off, initial_state=x["S0"], final_state=S2)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    one = {n: (t[700:2200, :, :1] if n != "log_decay" else t[:1]) for n, t in p.items()}
    check_forward(o[700:2200, None, :1], S[2:3, :1], one, 0.3, x["S0"][2:3, :1])
    do = x["do"][:, 0].contiguous()
    dS0, dS02 = torch.full_like(S, float("nan")), torch.full_like(S, float("nan"))
    grads = handle.linear_attention_backward(**packed, grad_out=do, scale=0.3, offsets=off, initial_state=x["S0"],
                                             grad_initial_state=dS0, max_len=max_len)
    grads2 = handle.linear_attention_backward(**packed, grad_out=do, scale=0.3, offsets=off, initial_state=x["S0"],
                                              grad_initial_state=dS02)
    assert all(torch.equal(m, n) for m, n in zip((*grads, dS0), (*grads2, dS02)))
    check_backward([g[700:2200, None, :1] for g in grads], dS0[2:3, :1], one, x["do"][700:2200, :, :1], 0.3, x["S0"][2:3, :1])


# -- buffers that are one ----------------------------------------------------------------------------------------

def same(got, want):
    return got.shape == want.shape and bool(((got == want) | (torch.isnan(got) & torch.isnan(want))).all())


@pytest.mark.parametrize("value", [None, float("inf"), float("nan")])
@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("shape", [(90, 3, 4, 2, 64, 80), (200, 16, 9, 9, 64, 64), (130, 40, 8, 4, 128, 128), (2500, 1, 2, 2, 64, 48)],
                         ids=str)
def test_state_gradients_in_place(handle, type, shape, value):  # noqa: F811
    """dS0 over dS1 gives what dS0 elsewhere does: whole and split sequences, of
    equal and of very unequal lengths, also where a value that is not finite has a
    sequence done again."""
    T, B, H, Hkv, Dk, Dv = shape
    p, x = attention_problem(2, type, *shape)
    if value is not None:
        p["v"][T // 3, 0, 0, 3] = value
        x["do"][T // 2, B - 1, H - 1, 5] = value
    short = torch.randint(0, 4, (B,), generator=torch.Generator().manual_seed(3)).int()
    short[:: 7] = T
    for lengths in (None, short.cuda()):
        kw = {"grad_out": x["do"], "scale": 0.3, "initial_state": x["S0"], "lengths": lengths}
        apart = torch.full_like(x["S0"], 7.0)
        want = handle.linear_attention_backward(**p, grad_final_state=x["dS1"], grad_initial_state=apart, **kw)
        state = x["dS1"].clone()
        got = handle.linear_attention_backward(**p, grad_final_state=state, grad_initial_state=state, **kw)
        assert all(same(m, n) for m, n in zip((*got, state), (*want, apart)))
    if value is None:
        check_backward(got, state, p, x["do"], 0.3, x["S0"], x["dS1"], short.tolist())


@pytest.mark.parametrize("type", sorted(TYPES))
def test_state_gradients_in_place_of_packed_sequences(handle, type):  # noqa: F811
    lengths = [0, 1, 1300, 64, 2, 130, 0]
    p, x, packed, off, offsets = packed_problem(4, type, lengths, 4, 2, 64, 64)
    kw = {"grad_out": x["do"][:, 0].contiguous(), "scale": 0.3, "offsets": off, "initial_state": x["S0"]}
    for max_len in (1300, None):
        apart = torch.full_like(x["S0"], 7.0)
        want = handle.linear_attention_backward(**packed, grad_final_state=x["dS1"], grad_initial_state=apart,
                                                max_len=max_len, **kw)
        state = x["dS1"].clone()
        got = handle.linear_attention_backward(**packed, grad_final_state=state, grad_initial_state=state,
                                               max_len=max_len, **kw)
        assert all(same(m, n) for m, n in zip((*got, state), (*want, apart)))
        for b, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
            one = {n: (t[lo:hi] if n != "log_decay" else t) for n, t in p.items()}
            check_backward([g[lo:hi, None] for g in got], state[b:b + 1], one, x["do"][lo:hi], 0.3, x["S0"][b:b + 1],
                           x["dS1"][b:b + 1])


def test_state_gradients_in_place_in_a_graph(gpu):
    p, x = attention_problem(5, "bf16", 300, 2, 4, 2, 64, 64)
    state, given = x["dS1"].clone(), x["dS1"].clone()
    grads = [torch.empty_like(p[n]) for n in ("q", "k", "v")]

    def call(h, s):
        return h.linear_attention_backward(**p, grad_out=x["do"], grad_final_state=s, grad_initial_state=s,
                                           grad_q=grads[0], grad_k=grads[1], grad_v=grads[2])

    with Handle() as h:
        call(h, state.clone())  # the workspace grows here
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(h, state)
        for seed in range(3):
            given.copy_(torch.randn(given.shape, generator=torch.Generator().manual_seed(seed)))
            eager = given.clone()
            want = [g.clone() for g in call(h, eager)]
            state.copy_(given)
            for g in grads:
                g.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(state, eager) and all(torch.equal(m, n) for m, n in zip(grads, want))
        del graph


# -- many heads and sequences ------------------------------------------------------------------------------------

@pytest.mark.parametrize("shape", [(40, 2048, 64, 32, 96, 128), (64, 4096, 32, 16, 128, 32)], ids=str)
def test_gradients_of_shared_heads_at_many_heads_and_sequences(gpu, shape):
    """Batch first: rows of all heads of all sequences together pass 2^31 bytes a
    chunk.  Every sequence is the same, so that all of them can be compared."""
    T, B, H, Hkv, Dk, Dv = shape
    p, x = attention_problem(6, "bf16", T, 1, H, Hkv, Dk, Dv)
    every = lambda t: t.transpose(0, 1).expand(B, T, *t.shape[2:]).contiguous().transpose(0, 1)
    many = {n: (every(t) if n != "log_decay" else t) for n, t in p.items()}
    with Handle() as h:
        into = {"grad_" + n: torch.empty_like(many[n]) for n in ("q", "k", "v")}  # (their strides too)
        grads = h.linear_attention_backward(**many, grad_out=every(x["do"]), scale=0.3, **into)
        for g in grads:
            assert (g == g[:, :1]).all()
        check_backward([g[:, :1, :1] if i else g[:, :1, :2] for i, g in enumerate(grads)], None,
                       {"q": p["q"][:, :, :2], "k": p["k"][:, :, :1], "v": p["v"][:, :, :1], "log_decay": p["log_decay"][:2]},
                       x["do"][:, :, :2], 0.3)
        check_backward([g[:, -1:, -1:] if i else g[:, -1:, -2:] for i, g in enumerate(grads)], None,
                       {"q": p["q"][:, :, -2:], "k": p["k"][:, :, -1:], "v": p["v"][:, :, -1:], "log_decay": p["log_decay"][-2:]},
                       x["do"][:, :, -2:], 0.3)


# -- packed sequences of very unequal lengths --------------------------------------------------------------------

def check_sequences(p, x, offsets, which, o, S, grads, dS0):
    for b in which:
        lo, hi = offsets[b], offsets[b + 1]
        one = {n: (t[lo:hi] if n != "log_decay" else t) for n, t in p.items()}
        check_forward(o[lo:hi, None], S[b:b + 1], one, 0.3, x["S0"][b:b + 1])
        check_backward([g[lo:hi, None] for g in grads], dS0[b:b + 1], one, x["do"][lo:hi], 0.3, x["S0"][b:b + 1],
                       x["dS1"][b:b + 1])


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("lengths", [[n % 41 for n in range(7, 700, 7)] + [1700] + [n % 5 for n in range(60)],
                                     [1700] + [0] * 30 + [129, 64, 65, 1], [0, 0, 64, 128, 640, 0, 900, 1, 63]],
                         ids=["many", "first", "some"])
def test_long_sequences_among_short_ones(handle, type, lengths):  # noqa: F811
    p, x, packed, off, offsets = packed_problem(8, type, lengths, 4, 2, 64, 48)
    by_length = sorted(range(len(lengths)), key=lambda b: lengths[b])
    which = sorted({*by_length[:2], *by_length[-4:], len(lengths) // 2})
    do = x["do"][:, 0].contiguous()
    for max_len in (None, max(lengths)):
        kw = {"scale": 0.3, "offsets": off, "max_len": max_len}
        S, dS0 = torch.full_like(x["S0"], float("nan")), torch.full_like(x["S0"], float("nan"))
        o = handle.linear_attention(**packed, initial_state=x["S0"], final_state=S, **kw)
        grads = handle.linear_attention_backward(**packed, grad_out=do, initial_state=x["S0"], grad_final_state=x["dS1"],
                                                 grad_initial_state=dS0, **kw)
        assert not torch.isnan(S).any() and not torch.isnan(dS0).any()
        check_sequences(p, x, offsets, which, o, S, grads, dS0)
        state = x["S0"].clone()
        again = handle.linear_attention(**packed, initial_state=state, final_state=state, **kw)
        assert torch.equal(again, o) and torch.equal(state, S)
        plain = handle.linear_attention(**packed, **kw)
        lo = offsets[which[-1]]
        one = {n: (t[lo:offsets[which[-1] + 1]] if n != "log_decay" else t) for n, t in p.items()}
        check_forward(plain[lo:offsets[which[-1] + 1], None], None, one, 0.3)


def test_many_sequences_without_a_longest_take_little_memory(gpu):
    """4096 sequences of one token each, of which any could be 4096 long."""
    n, H, D = 4096, 16, 128
    p, x = attention_problem(9, "bf16", n, 1, H, H, D, D)
    packed = {m: (t[:, 0].contiguous() if m != "log_decay" else t) for m, t in p.items()}
    off = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(packed["v"])
    with Handle() as h:
        h.linear_attention(*(packed[m][:1] for m in ("q", "k", "v")), packed["log_decay"], offsets=off[:2])
        torch.cuda.synchronize()
        before = torch.cuda.mem_get_info()[0]
        h.linear_attention(**packed, scale=1.0, offsets=off, out=out)
        torch.cuda.synchronize()
        used = before - torch.cuda.mem_get_info()[0]
    # operands of 67 MB, of which a state of every 128 rows is 33 MB
    assert used < 256 << 20
    for t in (0, 1, 2000, n - 1):
        check_forward(out[t:t + 1, None], None, {m: (y[t:t + 1] if m != "log_decay" else y) for m, y in p.items()}, 1.0)


# -- values that are not finite ----------------------------------------------------------------------------------

def check_kinds(got, want):
    """The same NaN, and the same infinities."""
    got = host(got)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    assert np.isfinite(got[np.isfinite(want)]).all()


DECAYS = [-0.01, -0.5, -0.9, -2.0, -30.0, 0.0, 1e-3, -float("inf")]


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("T", [40, 150, 192, 400, 500, 700, 2500])
@pytest.mark.parametrize("where", ["k", "v", "S0"])
def test_infinities_follow_the_recurrence(handle, type, T, where):  # noqa: F811
    """An infinity in the first tokens (or in the state before them) of sequences of
    one, 2, 3, 6, 7 and more segments, at decays whose power over a segment is 0."""
    H = len(DECAYS)
    p, x = attention_problem(10, type, T, 1, H, H, 16, 16, decay=DECAYS)
    if where == "S0":
        x["S0"][0, :, 3, 4], x["S0"][0, :, 5, 6] = float("inf"), float("nan")
    else:
        p[where][5, 0, :, 3] = float("inf")
    S = torch.empty_like(x["S0"])
    o = handle.linear_attention(**p, scale=0.2, initial_state=x["S0"], final_state=S)
    with np.errstate(invalid="ignore"):
        ref, refS = oracle.linear_attention(**{m: host(y) for m, y in p.items()}, scale=0.2, S0=host(x["S0"]))
    check_kinds(o, ref)
    check_kinds(S, refS)


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("T", [40, 192, 500, 700, 2500])
@pytest.mark.parametrize("where", ["q", "k", "v", "do", "S0", "dS1"])
def test_gradients_of_infinities_follow_the_recurrence(handle, type, T, where):  # noqa: F811
    H = len(DECAYS)
    p, x = attention_problem(11, type, T, 1, H, H, 16, 16, decay=DECAYS)
    if where in ("S0", "dS1"):
        x[where][0, :, 3, 4] = float("inf")
    else:
        (p if where in p else x)[where][T - 5 if where in ("q", "do") else 5, 0, :, 3] = float("inf")
    dS0 = torch.empty_like(x["S0"])
    grads = handle.linear_attention_backward(**p, grad_out=x["do"], scale=0.2, initial_state=x["S0"],
                                             grad_final_state=x["dS1"], grad_initial_state=dS0)
    with np.errstate(invalid="ignore"):
        ref = oracle.linear_attention_backward(**{m: host(y) for m, y in p.items()}, do=host(x["do"]), scale=0.2,
                                               S0=host(x["S0"]), dS1=host(x["dS1"]))
    for got, want in zip((*grads, dS0), ref):
        check_kinds(got, want)


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("T", [192, 700])
def test_growth_leaves_zeros_alone(handle, type, T):  # noqa: F811
    """Decays above 1 whose power over a segment is infinite: rows of the state
    that are zero stay zero."""
    p, _ = attention_problem(12, type, T, 1, 2, 2, 16, 16, decay=[1.5, 2.0])
    p["k"][..., 4:] = 0
    S = torch.full((1, 2, 16, 16), float("nan"), device="cuda")
    handle.linear_attention(**p, scale=0.2, final_state=S)
    assert not S[:, :, 4:].any() and torch.isinf(S[:, :, :4]).any()


# -- layer norm of many rows and of wide ones --------------------------------------------------------------------

@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("M, N", [((1 << 22) + 5, 3), (1, (1 << 27) + 5)], ids=["rows", "columns"])
def test_norm_past_what_one_launch_counts(handle, type, M, N):  # noqa: F811
    """Rows that no vector covers take a workgroup each, the sums of the parameters'
    gradients one for 32 columns."""
    g = torch.Generator(device="cuda").manual_seed(1)
    dt = TYPES[type]
    x, dy = (torch.randn((M, N), generator=g, device="cuda").to(dt) for _ in range(2))
    w = torch.randn(N, generator=g, device="cuda").to(dt)
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    y = handle.layer_norm(x, w, mean=mean, rstd=rstd)
    dx, dw, db = handle.layer_norm_backward(dy, x, mean, rstd, w)
    if M > 1:
        some = torch.cat([torch.arange(5), torch.tensor([1 << 20, (1 << 22) - 1, 1 << 22, M - 1])]).cuda()
        check_norm(y[some], mean[some], rstd[some], x[some], w, None)
        check_norm_backward(dx[some], None, None, dy[some], x[some], w, mean[some], rstd[some])
        n = (x.double() - mean[:, None]) * rstd[:, None]
        want = (dy.double() * n).sum(0), dy.double().sum(0), (dy.double() * n).abs().sum(0)
        for got, ref in ((dw, want[0]), (db, want[1])):  # 2^16 rows in turn at most, of 2^-24 each, and a rounding
            assert ((got.double() - ref).abs() <= 2.0 ** -8 * want[2] + torch.finfo(dt).eps / 2 * ref.abs()).all()
    else:
        # every column of the one row: statistics to the roundings of 2^17 columns a thread
        n = (x.double() - x.double().mean()) * (x.double().var(correction=0) + 1e-5).rsqrt()
        part = slice(N - 4096, None)
        for got, ref in ((y, n * w.double()), (dw, dy.double() * n), (db, dy.double())):
            got, ref = got.view(-1), ref.view(-1)
            for s in (slice(0, 4096), part):
                assert ((got[s].double() - ref[s]).abs() <= (2.0 ** -7 + torch.finfo(dt).eps) * (ref[s].abs() + 1)).all()
        assert torch.isfinite(dx).all() and dx.view(-1)[part].any()
