"""GPU: the layer norm over groups against float64, forward and backward.

Bounds: a value in bf16 is off by half a step, 2^-8 of itself; float32 sums of D (rows' statistics) and M (the
weight's gradient) terms by at most that many steps of 2^-24 of the sum of their magnitudes, and a handful
of operations per element."""

import pytest
import torch

import linattn_ref as ref
import rwkv_delta_rule_b200 as lib7
from helpers import need_cuda

pytestmark = pytest.mark.gpu
EPS32 = 2.0 ** -24

SHAPES = [
    (1, 1, 1), (3, 1, 2), (5, 1, 3), (4, 1, 64), (37, 1, 1001), (9, 1, 1000), (7, 1, 1002), (64, 1, 768), (1, 1, 4096), (300, 1, 4096),
    (33, 1, 2048), (5, 1, 8192), (3, 1, 8191), (2, 1, 8194), (3, 1, 16384), (2, 1, 16383), (2, 1, 40000), (2, 1, 70001),
    (100, 12, 64), (1, 64, 64), (257, 64, 64), (50, 40, 64), (11, 3, 300), (6, 5, 7), (13, 16, 8), (4, 300, 64), (3, 2, 5000), (2, 2, 9000),
    (2000, 1, 130), (70, 7, 96), (5000, 1, 64),
]


def inputs(M, G, D, dtype, seed, params=True):
    need_cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(M, G, D, generator=g, device="cuda") * 1.5 + 0.25).to(dtype)
    dy = (torch.randn(M, G, D, generator=g, device="cuda") * 0.5).to(dtype)
    w = torch.randn(G, D, generator=g, device="cuda") * 0.2 + 1 if params else None
    b = torch.randn(G, D, generator=g, device="cuda") * 0.2 if params else None
    return x, dy, w, b


def half_step(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else EPS32


def near(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), (what, bad.nonzero()[:4].tolist(), float((got.double() - want).abs().max()))


def check(x, dy, w, b, eps, y, mean, rstd, dx, dw, db):
    M, G, D = x.shape
    ry, rmean, rrstd = ref.norm(x, w, b, eps)
    n = (D + 32) * EPS32
    absx = x.double().abs().mean(-1)
    near(mean, rmean, n * absx + 1e-37, "mean")
    # the variance's relative error, and the mean's twice through (x - mean)^2; rstd's is half of it
    dm = n * absx
    near(rstd, rrstd, rrstd * (n + 2 * dm * rrstd + (dm * rrstd) ** 2 + 8 * EPS32), "rstd")
    wd = 1.0 if w is None else w.double()
    xh = (x.double() - rmean[..., None]) * rrstd[..., None]
    slack = (n + 2 * dm * rrstd + (dm * rrstd) ** 2 + 16 * EPS32)[..., None]
    tol = (xh.abs() * slack + (dm * rrstd)[..., None]) * (wd.abs() if w is not None else 1.0)
    tol = tol + 4 * EPS32 * ry.abs() + (EPS32 * 4 * b.double().abs() if b is not None else 0.0)
    near(y, ry, tol * 1.01 + half_step(y.dtype) * ry.abs() + 1e-37, "y")

    gx, gw, gb = ref.norm_backward(dy, x, w, mean, rstd)
    m, r = mean.double()[..., None], rstd.double()[..., None]
    xh = ((x.double() - m) * r).abs()
    g = (dy.double() * wd).abs()
    each = g + g.mean(-1, keepdim=True) + xh * (g * xh).mean(-1, keepdim=True)
    near(dx, gx, (n + 16 * EPS32) * r * each + half_step(dx.dtype) * gx.abs() + 1e-37, "dx")
    if dw is not None:
        k = (M + 32) * EPS32
        near(dw, gw, (k + 8 * EPS32) * (dy.double().abs() * xh).sum(0) + 1e-37, "dweight")
        near(db, gb, k * dy.double().abs().sum(0) + 1e-37, "dbias")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,G,D", SHAPES)
def test_norm(M, G, D, dtype):
    x, dy, w, b = inputs(M, G, D, dtype, M + G + D)
    y, mean, rstd = lib7.layer_norm(x, w, b, 64e-5)
    dx, dw, db = lib7.layer_norm_backward(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    check(x, dy, w, b, 64e-5, y, mean, rstd, dx, dw, db)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,G,D", [(40, 12, 64), (9, 1, 1001), (6, 1, 4096), (2, 1, 40000)])
def test_without_parameters(M, G, D, dtype):
    x, dy, _, _ = inputs(M, G, D, dtype, 1, params=False)
    y, mean, rstd = lib7.layer_norm(x, grouped=True)
    dx, dw, db = lib7.layer_norm_backward(dy, x, None, mean, rstd, grouped=True)
    frozen = torch.empty_like(dx)
    f = lib7.rwkv7_layer_norm_backward if dtype == torch.float32 else lib7.rwkv7_layer_norm_backward_bf16
    f(dy, x, None, mean, rstd, frozen)
    torch.cuda.synchronize()
    check(x, dy, None, None, 1e-5, y, mean, rstd, dx, dw, db)
    assert torch.equal(frozen, dx)


def test_no_rows_and_outputs_left_out():
    x, dy, w, b = inputs(0, 2, 64, torch.bfloat16, 2)
    y, mean, rstd = lib7.layer_norm(x, w, b)
    dx, dw, db = lib7.layer_norm_backward(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    assert y.shape == x.shape and dx.shape == x.shape and not bool(dw.any()) and not bool(db.any())
    x, _, w, b = inputs(5, 2, 64, torch.bfloat16, 3)
    y = torch.empty_like(x)
    lib7.rwkv7_layer_norm_bf16(x, w, b, 1e-5, y)
    torch.cuda.synchronize()
    assert torch.equal(y, lib7.layer_norm(x, w, b)[0])


def test_shapes_of_the_convenience():
    x, dy, w, b = inputs(6, 4, 64, torch.bfloat16, 4)
    y, mean, rstd = lib7.layer_norm(x.view(2, 3, 4, 64), w, b)
    assert y.shape == (2, 3, 4, 64) and mean.shape == rstd.shape == (2, 3, 4)
    flat = lib7.layer_norm(x.view(2, 3, 256), w.view(256), b.view(256))
    assert flat[1].shape == (2, 3)
    g = lib7.layer_norm_backward(dy.view(2, 3, 256), x.view(2, 3, 256), w.view(256), flat[1], flat[2])
    torch.cuda.synchronize()
    assert g[0].shape == (2, 3, 256) and g[1].shape == g[2].shape == (256,)
    check(x.view(6, 1, 256), dy.view(6, 1, 256), w.view(1, 256), b.view(1, 256), 1e-5, flat[0].view(6, 1, 256),
          flat[1].view(6, 1), flat[2].view(6, 1), g[0].view(6, 1, 256), g[1].view(1, 256), g[2].view(1, 256))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 1001, 4096, 40000])
def test_special_values(dtype, D):
    """A NaN or an infinity spoils its own vector only; a constant vector gives the bias."""
    x, _, w, b = inputs(6, 1, D, dtype, 5)
    clean = lib7.layer_norm(x, w, b)
    x2 = x.clone()
    x2[1, 0, D // 2] = float("nan")
    x2[3, 0, 0] = float("inf")
    x2[4] = 3.0
    y, mean, rstd = lib7.layer_norm(x2, w, b)
    torch.cuda.synchronize()
    for m in (0, 2, 5):
        assert torch.equal(y[m], clean[0][m])
    assert bool(y[1].isnan().all()) and bool(y[3].isnan().all())
    # mean 3 is off by D float32 steps at most, and rstd is 1 / sqrt(eps)
    assert bool(((y[4].float() - b).abs() <= (3 * (D + 32) * EPS32 * 320 * w.abs()) + half_step(dtype) * 1.1 * b.abs() + 1e-6).all())


def test_repeats_bit_for_bit_on_other_streams_and_in_graphs():
    x, dy, w, b = inputs(3000, 1, 768, torch.bfloat16, 6)
    y, mean, rstd = lib7.layer_norm(x, w, b)
    want = lib7.layer_norm_backward(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = lib7.layer_norm_backward(dy, x, w, mean, rstd, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, m2, r2 = lib7.layer_norm(x, w, b)
        got = lib7.layer_norm_backward(dy, x, w, m2, r2)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and all(torch.equal(a, c) for a, c in zip(got, want))


def test_guard_bands():
    for M, G, D in ((37, 1, 1001), (21, 12, 64), (3, 1, 8192)):
        x, dy, w, b = inputs(M, G, D, torch.bfloat16, 7)
        pad = 512

        def banded(like, dtype):
            buf = torch.full((like.numel() + 2 * pad,), 3.0, dtype=dtype, device="cuda")
            return buf, buf[pad:pad + like.numel()].view(like.shape)
        stat = torch.empty(M, G)
        bufs = [banded(x, x.dtype), banded(stat, torch.float32), banded(stat, torch.float32), banded(x, x.dtype),
                banded(w, torch.float32), banded(w, torch.float32)]
        y, mean, rstd, dx, dw, db = (t for _, t in bufs)
        n = lib7.rwkv7_layer_norm_workspace(True, M, G, D) // 4
        wbuf = torch.full((n + 2 * pad,), 3.0, device="cuda")
        lib7.rwkv7_layer_norm_bf16(x, w, b, 1e-5, y, mean, rstd)
        lib7.rwkv7_layer_norm_backward_bf16(dy, x, w, mean, rstd, dx, dw, db, wbuf[pad:pad + n])
        torch.cuda.synchronize()
        for buf in [t for t, _ in bufs] + [wbuf]:
            assert bool((buf[:pad] == 3.0).all()) and bool((buf[-pad:] == 3.0).all())
        check(x, dy, w, b, 1e-5, y, mean, rstd, dx, dw, db)


def test_most_columns():
    """G * D of 2^24, the most there may be: 65536 tiles of columns."""
    x, dy, w, b = inputs(2, 256, 65536, torch.bfloat16, 9)
    y, mean, rstd = lib7.layer_norm(x, w, b)
    dx, dw, db = lib7.layer_norm_backward(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    check(x, dy, w, b, 1e-5, y, mean, rstd, dx, dw, db)


def test_rows_past_32_bits():
    """More than 2^31 elements: the last rows are right."""
    M, D = (1 << 31) // 4096 + 9, 4096
    need_cuda()
    x = torch.empty(M, D, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(8))
    w = torch.ones(D, device="cuda")
    y, mean, rstd = lib7.layer_norm(x, w)
    dx, dw, db = lib7.layer_norm_backward(x, x, w, mean, rstd)
    torch.cuda.synchronize()
    t = slice(M - 12, M)
    ry, rm, rr = ref.norm(x[t], None, None, 1e-5)
    assert float((y[t].double() - ry).abs().max()) <= 2.0 ** -8 * float(ry.abs().max()) + 1e-5
    gx, _, _ = ref.norm_backward(x[t], x[t], None, mean[t], rstd[t])
    # dx = rstd x (1 - rstd^2 var) is all cancellation here: a few float32 steps of the terms
    assert float((dx[t].double() - gx).abs().max()) <= 4200 * EPS32 * 40 + 2.0 ** -8 * float(gx.abs().max())
