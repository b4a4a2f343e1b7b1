"""The gradient of a log decay whose exp is 0: the decayed state is 0 whatever the
log decay is, so it is 0 and not the rounding of the sums it is taken from."""
import pytest
import torch

from persistent_rnn_fwd_amd import Handle
from test_gpu_delta import TYPES, check_backward, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle(gpu):
    h = Handle()
    yield h
    h.close()


# Tokens at the start of a sequence, of a chunk of 32 and of a group of 64, inside them, next to each other.
FORGET = [0, 7, 8, 31, 32, 64, 77, 96, 128, 129, 190]


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("shape", [(200, 2, 2, 1, 64, 64), (200, 1, 2, 2, 112, 40), (200, 1, 1, 1, 200, 33), (500, 1, 2, 1, 96, 48)],
                         ids=str)
@pytest.mark.parametrize("value", [float("-inf"), -3e38, -105.0])
def test_gradients_of_decays_to_nothing_are_zero(handle, type, shape, value):
    p, x = problem(70 + sum(shape), type, *shape)
    p["log_decay"][FORGET] = value
    grads = handle.gated_delta_rule_backward(**p, grad_out=x["do"], scale=0.3, initial_state=x["S0"], grad_final_state=x["dS1"])
    assert not grads[3][FORGET].any()
    others = [t for t in range(shape[0]) if t not in FORGET]
    assert (grads[3][others] != 0).all()
    q = {**p, "log_decay": p["log_decay"].clamp(min=-200.0)}  # (exp is 0 all the same, and the oracle's sums are finite)
    check_backward(grads, None, q, x["do"], 0.3, x["S0"], x["dS1"])


@pytest.mark.parametrize("type", sorted(TYPES))
def test_packed_gradients_of_decays_to_nothing_are_zero(handle, type):
    offsets = [0, 1, 1, 40, 41, 171]
    p, x = problem(71, type, 171, 1, 2, 1, 80, 24)
    at = [0, 1, 33, 40, 41, 104, 105, 170]
    p["log_decay"][at] = float("-inf")
    packed = {m: t[:, 0].contiguous() for m, t in p.items()}
    S0 = torch.randn((5, 2, 80, 24), device="cuda")
    grads = handle.gated_delta_rule_backward(**packed, grad_out=x["do"][:, 0].contiguous(), initial_state=S0,
                                             offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    assert not grads[3][at].any()
    assert (grads[3][[t for t in range(171) if t not in at]] != 0).all()
