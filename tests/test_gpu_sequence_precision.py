"""GPU precision of linear attention between its products: what is fp32 there
(decayed scores, states, the decayed values that enter a state) keeps fp32's
bits for 16-bit types too.  Results in which large terms cancel show it, since
the rounding of the output itself is then small.

Tolerances: half a step of the output's type, and a count of fp32 roundings of
2^-24 each relative to A, the result from absolute values.
"""
import pytest
import torch

import oracle
from test_gpu_sequence import U, TYPES, absolute, attention_problem, close, handle, host  # noqa: F401

pytestmark = pytest.mark.gpu


def check(handle, p, S0, roundings, **call):  # noqa: F811
    o = handle.linear_attention(**p, scale=1.0, initial_state=S0, **call)
    n = {x: host(y) for x, y in p.items()}
    s0 = host(S0) if S0 is not None else None
    ref, _ = oracle.linear_attention(**n, scale=1.0, S0=s0)
    A, _ = oracle.linear_attention(**absolute(n), scale=1.0, S0=abs(s0) if s0 is not None else None)
    close("o", o, ref, A, o.dtype, roundings * U)


@pytest.mark.parametrize("type", sorted(TYPES))
def test_decayed_scores_keep_their_bits(handle, type):  # noqa: F811
    """o[1] = d - hi - lo, where hi + lo is d to at least 16 bits.  Roundings: d
    (4), its product with the score (2), the sums (4); 16 allowed."""
    dt, H = TYPES[type], 64
    g = torch.Generator().manual_seed(1)
    a = -torch.rand(H, generator=g)
    d = torch.exp(a)
    hi = d.to(dt)
    lo = (d - hi.float()).to(dt)
    k = torch.zeros((2, 1, H, 2), dtype=dt)
    k[0, 0, :, 0] = 1
    k[1, 0, :, 0], k[1, 0, :, 1] = -hi, -lo
    p = {"q": torch.ones((2, 1, H, 2), dtype=dt).cuda(), "k": k.cuda(),
         "v": torch.ones((2, 1, H, 1), dtype=dt).cuda(), "log_decay": a.cuda()}
    check(handle, p, None, 16)


@pytest.mark.parametrize("type", sorted(TYPES))
def test_states_keep_their_bits(handle, type):  # noqa: F811
    """o = s - s (1 - 2^-12), read from a state of two rows.  Roundings: one sum,
    the state's last parts and the scale; 8 allowed."""
    dt, H = TYPES[type], 64
    s = 1 + torch.rand((1, H, 1), generator=torch.Generator().manual_seed(2))
    S0 = torch.stack([s, -s * (1 - 2.0 ** -12)], dim=2).cuda()
    p = {"q": torch.ones((1, 1, H, 2), dtype=dt).cuda(), "k": torch.zeros((1, 1, H, 2), dtype=dt).cuda(),
         "v": torch.zeros((1, 1, H, 1), dtype=dt).cuda(), "log_decay": torch.zeros(H).cuda()}
    check(handle, p, S0, 8)


@pytest.mark.parametrize("type", ["f16", "bf16"])
def test_scores_see_their_operands_whole(handle, type):  # noqa: F811
    """o = x x - round(x x): the products of the operands' lowest bits show.
    Roundings: the sum of two products, 8 allowed."""
    dt, H = TYPES[type], 64
    x = (1 + 0.4 * torch.rand(H, generator=torch.Generator().manual_seed(3))).to(dt)
    x[0] = 1 + 2.0 ** -7 - 2.0 ** -10  # (fp16: all the bits below the upper eight)
    q, k = torch.ones((1, 1, H, 2), dtype=dt), torch.empty((1, 1, H, 2), dtype=dt)
    q[0, 0, :, 0] = k[0, 0, :, 0] = x
    k[0, 0, :, 1] = -(x.float() * x.float()).to(dt)
    p = {"q": q.cuda(), "k": k.cuda(), "v": torch.ones((1, 1, H, 1), dtype=dt).cuda(), "log_decay": torch.zeros(H).cuda()}
    check(handle, p, None, 8)


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("shape", [(200, 2, 4, 2, 64, 64), (300, 1, 2, 1, 128, 80), (1100, 1, 16, 16, 64, 128)], ids=str)
def test_outputs_do_not_depend_on_the_states_asked_for(handle, type, shape):  # noqa: F811
    p, x = attention_problem(4, type, *shape)
    S = torch.empty_like(x["S0"])
    one = handle.linear_attention(**p, initial_state=x["S0"])
    two = handle.linear_attention(**p, initial_state=x["S0"], final_state=S)
    assert torch.equal(one, two)
    one = handle.linear_attention_backward(**p, grad_out=x["do"], grad_final_state=x["dS1"])
    two = handle.linear_attention_backward(**p, grad_out=x["do"], grad_final_state=x["dS1"], grad_initial_state=S)
    assert all(torch.equal(m, n) for m, n in zip(one, two))
