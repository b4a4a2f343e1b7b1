"""Calls with more than 1024 chunks and heads: the first launch then has four
waves a workgroup, each with a chunk and head, and a last workgroup that some of
them leave.  Against the oracle and, bit for bit, against the sequences one by
one (whose chunks have a workgroup each)."""
import numpy as np
import pytest
import torch

from persistent_rnn_fwd_amd import Handle
from test_gpu_delta import TYPES, check_backward, check_forward, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle(gpu):
    h = Handle()
    yield h
    h.close()


def call(handle, p, do, S0, dS1, **seq):
    S, dS0 = torch.full_like(S0, float("nan")), torch.full_like(S0, float("nan"))
    o = handle.gated_delta_rule(**p, scale=0.3, initial_state=S0, final_state=S, **seq)
    grads = handle.gated_delta_rule_backward(**p, grad_out=do, scale=0.3, initial_state=S0, grad_final_state=dS1,
                                             grad_initial_state=dS0, **seq)
    return o, S, grads, dS0


# 3 chunks of 23 sequences and 15 heads: 1035, three more than a multiple of 4; rows at 16 bytes and not.
@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("Dk,Dv", [(16, 8), (112, 40), (33, 5)])
def test_many_chunks(handle, type, Dk, Dv):
    T, B, H = 65, 23, 15
    p, x = problem(80 + Dk, type, T, B, H, 5, Dk, Dv)
    o, S, grads, dS0 = call(handle, p, x["do"], x["S0"], x["dS1"])
    check_forward(o, S, p, 0.3, x["S0"])
    check_backward(grads, dS0, p, x["do"], 0.3, x["S0"], x["dS1"])
    for b in range(B):
        cut = slice(b, b + 1)
        o1, S1, grads1, dS01 = call(handle, {m: t[:, cut] for m, t in p.items()}, x["do"][:, cut], x["S0"][cut], x["dS1"][cut])
        assert torch.equal(o[:, cut], o1) and torch.equal(S[cut], S1) and torch.equal(dS0[cut], dS01)
        assert all(torch.equal(g[:, cut], g1) for g, g1 in zip(grads, grads1))


# 79 chunks' places (1555 rows and 31 sequences) and 15 heads: 1185, one more than a multiple of 4, some
# places without a chunk.
@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("Dk,Dv", [(16, 8), (112, 40), (33, 5)])
def test_many_chunks_packed(handle, type, Dk, Dv):
    lens = [i * 37 % 100 for i in range(30)] + [60]
    offsets = np.cumsum([0] + lens)
    rows, B, H = int(offsets[-1]), len(lens), 15
    assert (rows // 32 + B) * H > 1024 and (rows // 32 + B) * H % 4 != 0
    p, x = problem(90 + Dk, type, rows, 1, H, 5, Dk, Dv)
    packed = {m: t[:, 0].contiguous() for m, t in p.items()}
    do = x["do"][:, 0].contiguous()
    g = torch.Generator().manual_seed(Dk)
    S0, dS1 = (torch.randn((B, H, Dk, Dv), generator=g).cuda() for _ in range(2))
    o, S, grads, dS0 = call(handle, packed, do, S0, dS1, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"), max_len=99)
    for b, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        one, cut = {m: t[lo:hi] for m, t in p.items()}, slice(b, b + 1)
        check_forward(o[lo:hi, None], S[cut], one, 0.3, S0[cut])
        check_backward([y[lo:hi, None] for y in grads], dS0[cut], one, x["do"][lo:hi], 0.3, S0[cut], dS1[cut])
        if hi == lo:
            continue
        o1, S1, grads1, dS01 = call(handle, one, x["do"][lo:hi], S0[cut], dS1[cut])
        assert torch.equal(o[lo:hi, None], o1) and torch.equal(S[cut], S1) and torch.equal(dS0[cut], dS01)
        assert all(torch.equal(y[lo:hi, None], y1) for y, y1 in zip(grads, grads1))
