"""GPU parity of linear attention where the heads fill the chip (the kernels of
32 columns a wave, split and whole), checked on a few heads, and of layer norm on
rows that no vector divides, over several rows a workgroup.

Tolerances are those of test_gpu_sequence.py, whose derivation they share.
"""
import pytest
import torch

from test_gpu_sequence import TYPES, attention_problem, check_backward, check_forward, check_norm, check_norm_backward, \
    handle, norm_problem  # noqa: F401

pytestmark = pytest.mark.gpu

# (T, B, H, Hkv, Dk, Dv): at least 512 pieces of 64 tokens, with Dv > 64.  64 and
# 128 rows of the state; whole, split in 4 and 8, and in 16 (scanned) segments;
# shared heads; sizes and lengths that end inside a tile.
SHAPES = [(130, 8, 32, 32, 64, 128), (70, 8, 64, 16, 128, 128), (300, 4, 32, 32, 100, 75), (600, 2, 33, 11, 128, 80),
          (1100, 2, 16, 16, 37, 128), (2100, 1, 32, 8, 128, 128)]


def some_heads(Hkv):
    return sorted({0, Hkv // 2, Hkv - 1})


def heads_of(p, x, kv, b, group):
    """The problem of key-value head kv of sequence b alone, with its query heads."""
    h = slice(kv * group, (kv + 1) * group)
    part = {"q": p["q"][:, b:b + 1, h], "k": p["k"][:, b:b + 1, kv:kv + 1], "v": p["v"][:, b:b + 1, kv:kv + 1],
            "log_decay": p["log_decay"][h]}
    return part, {"S0": x["S0"][b:b + 1, h], "do": x["do"][:, b:b + 1, h], "dS1": x["dS1"][b:b + 1, h]}, h


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_attention_of_many_heads(handle, type, shape):  # noqa: F811
    T, B, H, Hkv, Dk, Dv = shape
    p, x = attention_problem(sum(shape), type, *shape)
    S = torch.full_like(x["S0"], float("nan"))
    o = handle.linear_attention(**p, scale=0.3, initial_state=x["S0"], final_state=S)
    plain = handle.linear_attention(**p, scale=0.3)
    assert not torch.isnan(S).any()
    for b, kv in zip((0, B // 2, B - 1), some_heads(Hkv) * 3):
        part, y, h = heads_of(p, x, kv, b, H // Hkv)
        check_forward(o[:, b:b + 1, h], S[b:b + 1, h], part, 0.3, y["S0"])
        check_forward(plain[:, b:b + 1, h], None, part, 0.3)


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("shape", SHAPES[1:4], ids=str)
def test_attention_gradients_of_many_heads(handle, type, shape):  # noqa: F811
    T, B, H, Hkv, Dk, Dv = shape
    p, x = attention_problem(1 + sum(shape), type, *shape)
    dS0 = torch.full_like(x["S0"], float("nan"))
    grads = handle.linear_attention_backward(**p, grad_out=x["do"], scale=0.3, initial_state=x["S0"],
                                             grad_final_state=x["dS1"], grad_initial_state=dS0)
    plain = handle.linear_attention_backward(**p, grad_out=x["do"], scale=0.3)
    for b, kv in zip((0, B - 1), some_heads(Hkv)[1:]):
        part, y, h = heads_of(p, x, kv, b, H // Hkv)
        own = [grads[0][:, b:b + 1, h], *(g[:, b:b + 1, kv:kv + 1] for g in grads[1:])]
        check_backward(own, dS0[b:b + 1, h], part, y["do"], 0.3, y["S0"], y["dS1"])
        own = [plain[0][:, b:b + 1, h], *(g[:, b:b + 1, kv:kv + 1] for g in plain[1:])]
        check_backward(own, None, part, y["do"], 0.3)


@pytest.mark.parametrize("type", sorted(TYPES))
def test_attention_of_many_heads_keeps_later_values_out(handle, type):  # noqa: F811
    """A NaN in one token reaches no earlier row and no other head, and every
    later row, across segments."""
    p, _ = attention_problem(5, type, 600, 2, 32, 32, 64, 128)
    before = handle.linear_attention(**p)
    p["k"][333, 1, 7, 5] = float("nan")
    o = handle.linear_attention(**p)
    assert torch.equal(o[:, 0], before[:, 0]) and torch.equal(o[:, 1, 8:], before[:, 1, 8:])
    assert not torch.isnan(o[:333]).any() and torch.isnan(o[333:, 1, 7]).all()
    # the redone rows are the same values from another order of sums: a step of
    # the type, and the rounding of 600 tokens' sums
    tol = 2 * torch.finfo(TYPES[type]).eps
    d = (o[:333, 1, 7].float() - before[:333, 1, 7].float()).abs()
    assert (d <= tol * before[:333, 1, 7].float().abs() + 2.0 ** -11 * before[:333, 1, 7].float().abs().max()).all()


@pytest.mark.parametrize("type", sorted(TYPES))
def test_packed_sequences_that_end_in_early_segments(handle, type):  # noqa: F811
    """Sequences that reach no, one, some and all of the segments."""
    lengths = [0, 1, 63, 64, 65, 700, 129, 1500, 0, 300]
    offsets = [0]
    for n in lengths:
        offsets.append(offsets[-1] + n)
    p, _ = attention_problem(6, type, offsets[-1], 1, 4, 2, 64, 64)
    _, x = attention_problem(7, type, 1, len(lengths), 4, 2, 64, 64)
    packed = {n: (t[:, 0].contiguous() if n != "log_decay" else t) for n, t in p.items()}
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    S = torch.full_like(x["S0"], float("nan"))
    o = handle.linear_attention(**packed, scale=0.3, offsets=off, max_len=1500, initial_state=x["S0"], final_state=S)
    none = torch.full_like(x["S0"], float("nan"))
    handle.linear_attention(**packed, scale=0.3, offsets=off, max_len=1500, final_state=none)
    for b, n in enumerate(lengths):
        lo, hi = offsets[b], offsets[b + 1]
        part = {m: (t[lo:hi] if m != "log_decay" else t) for m, t in p.items()}
        if n == 0:
            assert torch.equal(S[b], x["S0"][b]) and not none[b].any()
        else:
            check_forward(o[lo:hi, None], S[b:b + 1], part, 0.3, x["S0"][b:b + 1])


# the last vector of a row moved back by every number of elements; rows of one
# vector, of every number of threads, and narrower than a vector
@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("N", [2, 4, 5, 8, 9, 10, 11, 12, 13, 14, 15, 259, 500, 517, 1030, 1543, 2051, 4099, 6147, 8197, 12285])
def test_norm_of_rows_no_vector_divides(handle, type, N):  # noqa: F811
    M = 2100 if N < 1100 else 37
    x, w, b, dy = norm_problem(N, type, M, N + 3, "f32")
    x, dy = x[:, 1:N + 1], dy[:, 3:]  # rows that start anywhere
    w, b = w[1:N + 1], b[2:N + 2]
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    y = handle.layer_norm(x, w, b, mean=mean, rstd=rstd)
    check_norm(y, mean, rstd, x, w, b)
    dx, dw, db = handle.layer_norm_backward(dy, x, mean, rstd, w)
    check_norm_backward(dx, dw, db, dy, x, w, mean, rstd)
    # in place, with what lies between the rows left alone
    wide = torch.full((M, N + 3), 7.0, dtype=x.dtype, device="cuda")
    over = wide[:, 1:N + 1]
    over.copy_(x)
    assert torch.equal(handle.layer_norm(over, w, b, out=over), y)
    over.copy_(dy)
    assert torch.equal(handle.layer_norm_backward(over, x, mean, rstd, w, grad_x=over)[0], dx)
    assert (wide[:, 0] == 7).all() and (wide[:, N + 1:] == 7).all()


def test_norm_rows_do_not_mix(handle):  # noqa: F811
    """A row that is not finite leaves every other one as it is."""
    for type, M, N in (("f32", 3000, 321), ("bf16", 2500, 1000), ("f16", 1500, 5001)):
        x, w, b, dy = norm_problem(8, type, M, N, "f32")
        mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        y = handle.layer_norm(x, w, b, mean=mean, rstd=rstd)
        dx, _, _ = handle.layer_norm_backward(dy, x, mean, rstd, w)
        x[M // 2, N - 1] = float("inf")
        m, r = mean.clone(), rstd.clone()
        y2 = handle.layer_norm(x, w, b, mean=m, rstd=r)
        dx2, _, _ = handle.layer_norm_backward(dy, x, m, r, w)
        keep = torch.arange(M, device="cuda") != M // 2
        assert torch.equal(y2[keep], y[keep]) and torch.equal(dx2[keep], dx[keep])
        assert torch.isnan(y2[M // 2]).any() and torch.isnan(dx2[M // 2]).all()


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("Dv", [1, 2, 3, 4, 5, 6, 7, 31, 33, 34, 35, 63, 97, 130, 255])
def test_step_of_rows_no_vector_divides(handle, type, Dv):  # noqa: F811
    """The columns that the last vector of a row shares with the one before it,
    in place (where they may be written before they are read) and out of place,
    states at addresses that only fp32 divides."""
    for B, H, Hkv, Dk, offset in ((3, 4, 2, 37, 0), (9, 6, 6, 128, 1)):
        p, x = attention_problem(Dv + B, type, 1, B, H, Hkv, Dk, Dv)
        one = {n: (t[0] if n != "log_decay" else t) for n, t in p.items()}
        room = torch.full((2, x["S0"].numel() + 8), 7.0, device="cuda")
        states = [r[offset:offset + x["S0"].numel()].view(x["S0"].shape) for r in room]
        for s in states:
            s.copy_(x["S0"])
        o = handle.linear_attention_step(**one, state=states[0], scale=0.3)
        check_forward(o[None], states[0], p, 0.3, x["S0"])
        new = torch.empty_like(x["S0"])
        again = handle.linear_attention_step(**one, state=states[1], scale=0.3, new_state=new)
        assert torch.equal(o, again) and torch.equal(new, states[0]) and torch.equal(states[1], x["S0"])
        assert (room[:, :offset] == 7).all() and (room[:, offset + x["S0"].numel():] == 7).all()
