"""GPU parity of rms norm (through the C ABI) against the fp64 oracle.

Tolerances come from the arithmetic.  Sums are of at most 96 sequential roundings
(registers, lanes, waves) of 2^-24 each, so statistics and outputs are right to 128
* 2^-24 of their absolute terms, plus half a step of the output's type.  e4m3: a
value lies within half a step of e4m3 (2^-4 of it, or 2^-10 below 2^-6) of y / scale,
and whatever the library's y / scale differs by from the exact one (128 * 2^-24).
"""
import numpy as np
import pytest
import torch

import oracle
from persistent_rnn_fwd_amd import Handle, PrnnError

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
C = 128 * 2.0 ** -24


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


def rows(seed, type, params, M, N):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[type]
    x = (torch.randn((M, N), generator=g) * (0.5 + 2 * torch.rand((M, 1), generator=g))).to(dt).cuda()
    res = torch.randn((M, N), generator=g).to(dt).cuda()
    w = (1 + 0.1 * torch.randn(N, generator=g)).to(TYPES[params]).cuda() if params else None
    dy, ds = (torch.randn((M, N), generator=g).to(dt).cuda() for _ in range(2))
    return x, res, w, dy, ds


def close(name, got, ref, bound):
    got = host(got)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (name, int(bad.sum()), float(np.nanmax(np.abs(got - ref) / np.maximum(bound, 1e-300))))


def check(y, x, w, eps, res=None, total=None, rstd=None):
    ref, r, s = oracle.rms_norm(host(x), host(w), eps, host(res))
    # (the sum's own rounding is 2^-24 of its terms, which may cancel in it)
    terms = np.abs(host(x)) + (np.abs(host(res)) if res is not None else 0)
    scaled = terms * r[:, None] * (np.abs(host(w)) if w is not None else 1)
    close("y", y, ref, half_step(x.dtype, ref) + C * scaled)
    if rstd is not None:
        close("rstd", rstd, r, C * r)
    if total is not None:
        close("sum", total, s, half_step(x.dtype, s) + 2.0 ** -24 * terms)


def check_e4m3(q, scales, x, w, eps, group, res=None):
    ref, r, _ = oracle.rms_norm(host(x), host(w), eps, host(res))
    M, N = ref.shape
    width = N if group is None else group
    terms = (np.abs(host(x)) + (np.abs(host(res)) if res is not None else 0)) * r[:, None] * (np.abs(host(w)) if w is not None else 1)
    values = oracle.e4m3_values()
    s = host(scales).reshape(M, -1)
    assert s.shape[1] == -(-N // width)
    got = q.float().double().cpu().numpy()
    for j in range(s.shape[1]):
        cols = slice(j * width, min(N, (j + 1) * width))
        most = np.abs(ref[:, cols]).max(1)
        want = np.maximum(most / 448, 2.0 ** -126)
        close("scale", scales.reshape(M, -1)[:, j], want, 2.0 ** -23 * want + C * terms[:, cols].max(1) / 448)
        at = ref[:, cols] / s[:, j:j + 1]
        off = np.abs(got[:, cols] - at)
        above = values[np.clip(np.searchsorted(values, np.abs(at)), 0, 126)]
        step = np.where(above <= 2.0 ** -6, 2.0 ** -9, 2.0 ** (np.floor(np.log2(np.maximum(above, 2.0 ** -6))) - 3))
        assert (off <= step / 2 + C * terms[:, cols] / s[:, j:j + 1] + 2.0 ** -22 * np.abs(at)).all(), float((off / step).max())


# rows that one wave, several and a workgroup hold, and wider ones; odd widths; fewer columns than a vector
SIZES = [(1, 1), (3, 5), (1, 16), (7, 96), (5, 128), (4, 129), (2, 500), (9, 1153), (4, 1792), (3, 4099), (2, 5760),
         (2, 16384), (2, 20001)]
KINDS = [("f32", "f32"), ("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("bf16", None)]


@pytest.mark.parametrize("type,params", KINDS)
@pytest.mark.parametrize("M,N", SIZES)
def test_forward(handle, type, params, M, N):
    x, res, w, _, _ = rows(M + N, type, params, M, N)
    rstd = torch.full((M,), float("nan"), device="cuda")
    y = handle.rms_norm(x, w, 1e-5, rstd=rstd)
    check(y, x, w, 1e-5, rstd=rstd)
    total = torch.full_like(x, float("nan"))
    y = handle.rms_norm(x, w, 1e-6, residual=res, sum_out=total, rstd=rstd)
    check(y, x, w, 1e-6, res, total, rstd)
    assert torch.equal(y, handle.rms_norm(x, w, 1e-6, residual=res))


@pytest.mark.parametrize("type,params", KINDS)
@pytest.mark.parametrize("group", [None, 128])
@pytest.mark.parametrize("M,N", SIZES)
def test_e4m3(handle, type, params, group, M, N):
    x, res, w, _, _ = rows(M + N + 1, type, params, M, N)
    q, s = handle.rms_norm_e4m3(x, w, group=group)
    assert q.dtype == torch.float8_e4m3fn and s.shape == ((M,) if group is None else (M, -(-N // 128)))
    check_e4m3(q, s, x, w, 1e-6, group)
    total, rstd = torch.empty_like(x), torch.empty(M, device="cuda")
    q, s = handle.rms_norm_e4m3(x, w, residual=res, sum_out=total, rstd=rstd, group=group)
    check_e4m3(q, s, x, w, 1e-6, group, res)
    plain = torch.empty_like(x)
    handle.rms_norm(x, w, residual=res, sum_out=plain)
    assert torch.equal(total, plain)


@pytest.mark.parametrize("type,params", KINDS)
@pytest.mark.parametrize("M,N", SIZES + [(700, 24), (2000, 64), (300, 1153)])
def test_backward(handle, type, params, M, N):
    x, _, w, dy, ds = rows(M + N + 2, type, params, M, N)
    _, r, _ = oracle.rms_norm(host(x))
    rstd = torch.from_numpy(r).float().cuda()
    for dsum in (None, ds):
        given = torch.full((N,), float("nan"), device="cuda") if params is None else None
        dx, dw = handle.rms_norm_backward(dy, x, rstd, w, grad_sum=dsum, grad_weight=given)
        want, wantw = oracle.rms_norm_backward(host(dy), host(x), host(rstd), host(w), host(dsum))
        n, g = np.abs(host(x)) * r[:, None], np.abs(host(dy)) * (np.abs(host(w)) if w is not None else 1)
        terms = r[:, None] * (g + n * (g * n).mean(1, keepdims=True)) + (np.abs(host(dsum)) if dsum is not None else 0)
        close("dx", dx, want, half_step(x.dtype, want) + C * terms)
        sums = (np.abs(host(dy)) * n).sum(0)
        # (a column's sum: rows of one set in order, then the sets' and the workgroups' partial sums)
        close("dw", dw, wantw, half_step(dw.dtype, wantw) + (C + 2.0 ** -24 * min(M, 200)) * sums)
    assert handle.rms_norm_backward(dy, x, rstd)[1] is None


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("N", [96, 500, 1153, 20001])
def test_in_place(handle, type, N):
    x, res, w, dy, ds = rows(N, type, type, 37, N)
    total = torch.empty_like(x)
    y = handle.rms_norm(x, w, residual=res, sum_out=total)
    a, b = x.clone(), res.clone()
    handle.rms_norm(a, w, residual=b, sum_out=b, out=a)
    assert torch.equal(a, y) and torch.equal(b, total)
    a, b = x.clone(), res.clone()
    handle.rms_norm(a, w, residual=b, sum_out=a, out=b)
    assert torch.equal(a, total) and torch.equal(b, y)
    b = res.clone()
    q, s = handle.rms_norm_e4m3(x, w, residual=res)
    q2, s2 = handle.rms_norm_e4m3(x, w, residual=b, sum_out=b)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2) and torch.equal(b, total)
    rstd = torch.rand(37, device="cuda") + 0.5
    dx, dw = handle.rms_norm_backward(dy, total, rstd, w, grad_sum=ds)
    for i in range(3):
        t = [dy.clone(), total.clone(), ds.clone()]
        dx2, dw2 = handle.rms_norm_backward(t[0], t[1], rstd, w, grad_sum=t[2], grad_x=t[i])
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2), i


@pytest.mark.parametrize("type", sorted(TYPES))
@pytest.mark.parametrize("N", [96, 501, 1152])
def test_strides(handle, type, N):
    """Rows apart, in buffers whose other elements stay as they were; more rows
    than the grid has row sets; more axes than two."""
    M = 3000
    x, res, w, dy, ds = rows(N, type, "f32", M, N)

    def apart(t, gap):
        buf = torch.full((M, N + gap), 7.0, device="cuda").to(t.dtype)
        buf[:, 1:N + 1].copy_(t) if t.dtype != torch.float8_e4m3fn else None
        return buf, buf[:, 1:N + 1]

    total, y = torch.empty_like(x), None
    y = handle.rms_norm(x, w, residual=res, sum_out=total)
    (_, a), (_, b), (bt, t), (by, o) = apart(x, 3), apart(res, 9), apart(torch.zeros_like(x), 5), apart(torch.zeros_like(x), 8)
    handle.rms_norm(a, w, residual=b, sum_out=t, out=o)
    assert torch.equal(o, y) and torch.equal(t, total)
    for buf in (bt, by):
        assert (buf[:, 0] == 7).all() and (buf[:, N + 1:] == 7).all()
    for group in (None, 128):
        q, s = handle.rms_norm_e4m3(x, w, residual=res, group=group)
        bq = torch.full((M, N + 5), 7, dtype=torch.uint8, device="cuda")
        q2, s2 = handle.rms_norm_e4m3(a, w, residual=b, group=group, out=bq.view(torch.float8_e4m3fn)[:, 1:N + 1])
        assert torch.equal(q.view(torch.uint8), bq[:, 1:N + 1]) and torch.equal(s, s2)
        assert (bq[:, 0] == 7).all() and (bq[:, N + 1:] == 7).all()
    rstd = torch.rand(M, device="cuda") + 0.5
    dx, dw = handle.rms_norm_backward(dy, x, rstd, w, grad_sum=ds)
    (_, c), (_, d), (be, e) = apart(dy, 4), apart(ds, 6), apart(torch.zeros_like(x), 8)
    dx2, dw2 = handle.rms_norm_backward(c, a, rstd, w, grad_sum=d, grad_x=e)
    close("dw", dw2, host(dw), C * host(dw.abs()) + C * M)
    assert torch.equal(dx, dx2)
    assert (be[:, 0] == 7).all() and (be[:, N + 1:] == 7).all()
    assert torch.equal(handle.rms_norm(x.view(30, 100, N), w, residual=res.view(30, 100, N)), y.view(30, 100, N))


def test_zeros_and_values_that_are_not_finite(handle):
    x = torch.randn((6, 300), device="cuda")
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 5] = float("inf")
    x[4] *= 1e-30
    clean = x[[0, 5]]
    y = handle.rms_norm(x)
    assert torch.equal(y[[0, 5]], handle.rms_norm(clean)) and not y[1].any() and y[2].isnan().all() and not y[3].isfinite().all()
    for group in (None, 128):
        q, s = handle.rms_norm_e4m3(x, group=group)
        q2, s2 = handle.rms_norm_e4m3(clean.contiguous(), group=group)
        assert torch.equal(q.view(torch.uint8)[[0, 5]], q2.view(torch.uint8)) and torch.equal(s[[0, 5]], s2)
        assert (s[1] == 2.0 ** -126).all() and not q[1].float().any()
        assert q[2].float().isnan().all()
    q, s = handle.rms_norm_e4m3(x, eps=0.0)
    assert not (q[1].float() == 0).any()  # 0 / 0


def test_no_rows(handle):
    x = torch.empty((0, 64), device="cuda")
    assert handle.rms_norm(x).shape == (0, 64)
    w = torch.ones(64, device="cuda")
    _, dw = handle.rms_norm_backward(x, x, torch.empty(0, device="cuda"), w)
    assert not dw.any()


def test_graph_replays(gpu):
    with Handle() as h:
        x, res, w, dy, ds = rows(3, "bf16", "f32", 500, 1792)
        rstd, total = torch.empty(500, device="cuda"), torch.empty_like(x)

        def work():
            y = h.rms_norm_e4m3(x, w, residual=res, sum_out=total, rstd=rstd)
            return (*y, total, rstd, *h.rms_norm_backward(dy, total, rstd, w, grad_sum=ds))

        work()
        side = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                outs = work()
        torch.cuda.synchronize()
        for i in range(3):
            x.copy_(torch.randn_like(x))
            graph.replay()
            torch.cuda.synchronize()
            got = [t.float().clone() for t in outs]
            want = work()
            assert all(torch.equal(a, b.float()) for a, b in zip(got, want)), i


def test_refusals(handle):
    x = torch.zeros((4, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    other = torch.zeros((4, 64), device="cuda", dtype=torch.float16)
    for call in (lambda: handle.rms_norm(x.cpu()), lambda: handle.rms_norm(x, w[:32]), lambda: handle.rms_norm(x, w.half()),
                 lambda: handle.rms_norm(x, residual=other), lambda: handle.rms_norm(x.double()),
                 lambda: handle.rms_norm_e4m3(x, group=64), lambda: handle.rms_norm_e4m3(x, out=torch.empty_like(x)),
                 lambda: handle.rms_norm_e4m3(x, scales=torch.empty(3, device="cuda")),
                 lambda: handle.rms_norm_backward(x, x, w[:4], w, grad_sum=other)):
        with pytest.raises((TypeError, ValueError)):
            call()
    for call in (lambda: handle.rms_norm(x, eps=-1.0), lambda: handle.rms_norm(x, eps=float("nan")),
                 lambda: handle.rms_norm(x, residual=x.clone(), sum_out=x, out=x),
                 lambda: handle.rms_norm(x[:2], out=x.view(-1)[32:160].view(2, 64)),
                 lambda: handle.rms_norm(x, w, rstd=x[0, :4]),
                 lambda: handle.rms_norm_backward(x, x.clone(), w[:4].clone(), w, grad_weight=w)):
        with pytest.raises(PrnnError):
            call()
    handle.synchronize()
