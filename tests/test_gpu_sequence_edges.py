"""GPU tests of linear attention and layer norm at the edges of what they take:
lengths, strides, buffers that are one, sizes past the usual shapes.

Tolerances are those of test_gpu_sequence.py, whose derivation they share.
"""
import pytest
import torch

from test_gpu_sequence import TYPES, attention_problem, check_backward, check_forward, handle  # noqa: F401

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
