"""Rms norm of more rows than its grid takes at once (64 workgroups a compute
unit, each with the rows its threads hold): a workgroup then walks on to further
rows, the next ones' loads ahead of the sums, the last of them past the end.
Bit for bit as the same rows in calls that need no second walk, which other
tests compare with the oracle; rows at the start of the second walk, and the
last ones, against the oracle too."""
import pytest
import torch

from persistent_rnn_fwd_amd import Handle
from test_gpu_rms import TYPES, check, check_e4m3, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle(gpu):
    h = Handle()
    yield h
    h.close()


def equal(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8)) if a.dtype == torch.float8_e4m3fn else torch.equal(a, b)


# Widths whose rows lie in 16, 64 (fp32: up to 128) and 256 (fp32: 512) threads, of which a workgroup holds
# 16, 4 and 1 rows at most; some not a multiple of a vector.
@pytest.mark.parametrize("type,params", [("f32", "f32"), ("f16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("N,sets,more", [(96, 16, 5), (67, 16, 11), (1152, 4, 3), (1153, 4, 6), (5760, 1, 1), (4099, 1, 3)])
def test_second_walk(handle, type, params, N, sets, more):
    units = torch.cuda.get_device_properties(0).multi_processor_count
    whole = 64 * units * sets
    M = whole + more
    x, res, w, _, _ = rows(N, type, params, 2048, N)
    # (row m: one of 2048 times a power of two, so that neighbours in a workgroup's walk differ)
    m = torch.arange(M, device="cuda")
    x, res = x[(m * 7 + m // 2048) % 2048], res[(m * 5 + m // 2048 * 3) % 2048]
    x = x * torch.exp2((m % 5 - 2).float())[:, None].to(x.dtype)
    parts = [slice(lo, min(M, lo + 32 * units)) for lo in range(0, M, 32 * units)]
    some = torch.cat([m[whole - 8:], m[64 * units - 4:64 * units + 8], m[:4]]).cpu()

    def call(cut, residual, out):
        r = res[cut] if residual else None
        total = torch.full_like(x[cut], float("nan")) if residual else None
        rstd = torch.full((x[cut].shape[0],), float("nan"), device="cuda")
        y = ((handle.rms_norm(x[cut], w, residual=r, sum_out=total, rstd=rstd),) if out == "same" else
             handle.rms_norm_e4m3(x[cut], w, residual=r, sum_out=total, rstd=rstd, group=128 if out == "group" else None))
        return [*y, rstd] + ([total] if residual else [])

    for out in ("same", "row", "group"):
        for residual in (False, True):
            got = call(slice(0, M), residual, out)
            for cut in parts:
                assert all(equal(a[cut], b) for a, b in zip(got, call(cut, residual, out))), (out, residual, cut)
            r = res[some] if residual else None
            if out == "same":
                check(got[0][some], x[some], w, 1e-6, r, got[2][some] if residual else None, got[1][some])
            else:
                check_e4m3(got[0].view(torch.uint8)[some].view(torch.float8_e4m3fn), got[1][some], x[some], w, 1e-6,
                           128 if out == "group" else None, r)
            if residual and out == "same":  # in place
                a, b = x.clone(), res.clone()
                handle.rms_norm(a, w, residual=b, sum_out=b, out=a)
                assert torch.equal(a, got[0]) and torch.equal(b, got[2])
