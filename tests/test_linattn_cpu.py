"""The head-decay linear attention and the layer norm without a GPU: the entry points' refusals (no call
here reaches a launch), and the gradients' formulas against differences and automatic differentiation."""

import pytest
import torch

import linattn_ref as ref
import rwkv_delta_rule_b200 as lib7

FAKE = 0x10000  # 16-byte aligned, never dereferenced
MIS = 0x10008


@pytest.fixture(scope="module")
def cdll():
    from rwkv_delta_rule_b200 import build

    build.build()
    return lib7.load_library()


def prefill(cdll, name="rwkv7_linattn_prefill_bf16", B=1, T=4, H=1, N=64, op=FAKE, w=FAKE, s_in=None, s_out=FAKE,
            ws=None, nb=0):
    return getattr(cdll, name)(B, T, H, N, op, op, op, w, s_in, op, s_out, ws, nb, None)


@pytest.mark.parametrize("name", ["rwkv7_linattn_prefill_bf16", "rwkv7_linattn_prefill"])
def test_prefill_rejects(cdll, name):
    assert prefill(cdll, name, N=32) == 5
    assert prefill(cdll, name, B=0) == 1
    assert prefill(cdll, name, B=65536) == 1
    assert prefill(cdll, name, H=-1) == 1
    assert prefill(cdll, name, H=65536) == 1
    assert prefill(cdll, name, T=-1) == 1
    assert prefill(cdll, name, B=65535, T=65535) == 1  # more tokens than an int counts
    assert prefill(cdll, name, op=None) == 1
    assert prefill(cdll, name, w=None) == 1
    assert prefill(cdll, name, s_out=None) == 1
    assert prefill(cdll, name, nb=16) == 1  # bytes without a workspace
    assert prefill(cdll, name, ws=FAKE, nb=-1) == 1
    assert prefill(cdll, name, op=MIS) == 2
    assert prefill(cdll, name, w=MIS) == 2
    assert prefill(cdll, name, s_in=MIS) == 2
    assert prefill(cdll, name, ws=MIS, nb=1 << 20) == 2


def test_varlen_rejects(cdll):
    def call(cu=FAKE, max_T=8, N=64, op=FAKE, total=10):
        return cdll.rwkv7_linattn_prefill_varlen_bf16(2, total, max_T, 1, N, cu, op, op, op, FAKE, None, op, FAKE, None,
                                                      0, None)
    assert call(cu=None) == 1
    assert call(cu=MIS) == 2
    assert call(max_T=-1) == 1
    assert call(total=-1) == 1
    assert call(N=48) == 5
    assert call(op=None) == 1
    assert call(op=MIS) == 2


@pytest.mark.parametrize("name", ["rwkv7_linattn_decode", "rwkv7_linattn_decode_bf16"])
def test_decode_rejects(cdll, name):
    def call(B=1, H=1, N=64, op=FAKE, w=FAKE, s=FAKE):
        return getattr(cdll, name)(B, H, N, op, op, op, w, s, op, None)
    assert call(B=0) == 1
    assert call(H=0) == 1
    assert call(N=128) == 5
    assert call(op=None) == 1
    assert call(w=None) == 1
    assert call(s=None) == 1
    assert call(op=MIS) == 2
    assert call(s=MIS) == 2


def test_backward_rejects(cdll):
    def call(B=1, T=4, H=1, N=64, op=FAKE, dy=FAKE, dr=FAKE, dk=FAKE, w=FAKE, ds=None, ds_in=None, ws=None, nb=0):
        return cdll.rwkv7_linattn_backward_bf16(B, T, H, N, op, op, op, w, None, dy, ds, dr, dk, FAKE, ds_in, ws, nb, None)
    assert call(N=16) == 5
    assert call(B=0) == 1
    assert call(T=-1) == 1
    for gone in ("op", "dy", "dr", "dk", "w"):
        assert call(**{gone: None}) == 1, gone
    for off in ("op", "dy", "dr", "dk", "w", "ds", "ds_in"):
        assert call(**{off: MIS}) == 2, off
    assert call(nb=8) == 1
    assert call(T=0, op=None, dy=None, dr=None, dk=None) == 0  # nothing to do, no ds_in wanted


@pytest.mark.parametrize("suffix", ["", "_bf16"])
def test_layer_norm_rejects(cdll, suffix):
    fwd, bwd = getattr(cdll, "rwkv7_layer_norm" + suffix), getattr(cdll, "rwkv7_layer_norm_backward" + suffix)

    def f(M=2, G=1, D=64, eps=1e-5, x=FAKE, w=FAKE, y=FAKE, mean=None):
        return fwd(M, G, D, eps, x, w, None, y, mean, None, None)
    assert f(M=-1) == 1
    assert f(G=0) == 1
    assert f(D=0) == 1
    assert f(G=1 << 12, D=(1 << 12) + 1) == 1  # more than 2^24 channels
    assert f(M=1 << 30, G=2) == 1
    assert f(eps=-1.0) == 1
    assert f(eps=float("nan")) == 1
    assert f(x=None) == 1
    assert f(y=None) == 1
    assert f(x=MIS) == 2
    assert f(w=MIS) == 2
    assert f(mean=MIS) == 2
    assert f(M=0, x=None, y=None) == 0

    need = lib7.rwkv7_layer_norm_workspace(suffix == "_bf16", 2, 1, 64)
    assert need > 0

    def g(M=2, dy=FAKE, mean=FAKE, dx=FAKE, dw=FAKE, db=FAKE, ws=FAKE, nb=need):
        return bwd(M, 1, 64, dy, FAKE, None, mean, FAKE, dx, dw, db, ws, nb, None)
    assert g(M=-1) == 1
    assert g(dy=None) == 1
    assert g(mean=None) == 1
    assert g(dx=None) == 1
    assert g(dw=None) == 1  # both or neither
    assert g(db=None) == 1
    assert g(ws=None, nb=0) == 1
    assert g(nb=need - 1) == 1
    assert g(dy=MIS) == 2
    assert g(dw=MIS) == 2
    assert g(ws=MIS) == 2
    assert g(M=0, dw=None, db=None, ws=None, nb=0) == 0


def test_workspace_sizes():
    assert lib7.rwkv7_linattn_workspace(0, 10, 1) == 0
    assert lib7.rwkv7_linattn_workspace(1, 0, 1) == 0
    assert lib7.rwkv7_linattn_workspace(1, 1, 1) == 0  # one token is not split
    assert lib7.rwkv7_linattn_workspace(64, 4096, 64) == 0  # enough chains as they are
    n = lib7.rwkv7_linattn_workspace(1, 4096, 12)
    assert n > 0 and n % (12 * 64 * 64 * 4) == 0
    n = lib7.rwkv7_linattn_backward_workspace(1, 4096, 12)
    assert n > 0 and n % (3 * 12 * 64 * 64 * 4) == 0
    assert lib7.rwkv7_layer_norm_workspace(True, 0, 1, 64) == 0
    assert lib7.rwkv7_layer_norm_workspace(True, 5, 0, 64) == 0


def test_bindings_reject_wrong_tensors():
    x = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    w, s = torch.ones(1), torch.zeros(1, 1, 64, 64)
    with pytest.raises(ValueError):
        lib7.rwkv7_linattn_prefill_bf16(x, x, x, w, None, x, s)
    with pytest.raises(ValueError):
        lib7.rwkv7_linattn_decode_bf16(x[0], x[0], x[0], w, s, x[0])
    with pytest.raises(ValueError):
        lib7.rwkv7_layer_norm(torch.zeros(2, 1, 64), None, None, 1e-5, torch.zeros(2, 1, 64))
    with pytest.raises(ValueError):
        lib7.layer_norm(torch.zeros(2, 64))


def _inputs(B, T, H, seed):
    g = torch.Generator().manual_seed(seed)
    r, k, v, dy = (torch.randn(B, T, H, 64, generator=g, dtype=torch.float64) for _ in range(4))
    s0, ds = (torch.randn(B, H, 64, 64, generator=g, dtype=torch.float64) for _ in range(2))
    return r, k / 8, v, dy, s0, ds


def _by_formula(r, k, v, w, dy, s0, ds):
    """The three passes of the backward: (dr, dk, dv, ds_in)."""
    t = lambda x: x.transpose(-1, -2)  # noqa: E731
    dr, _ = ref.mix(dy, v, k, w, t(s0))
    dk, _ = ref.mix(v, dy, r, w, t(ds), reverse=True)
    dv, g = ref.mix(k, r, dy, w, ds, reverse=True)
    return dr, dk, dv, g


def test_gradient_formula_against_autograd():
    r, k, v, dy, s0, ds = _inputs(2, 9, 3, 1)
    w = torch.tensor([0.0, 0.9, 1.0], dtype=torch.float64)
    leaves = [x.clone().requires_grad_() for x in (r, k, v, s0)]
    S, ys = leaves[3], []
    for t in range(9):
        S = w.view(1, 3, 1, 1) * S + leaves[2][:, t, :, :, None] * leaves[1][:, t, :, None, :]
        ys.append((S @ leaves[0][:, t, :, :, None])[..., 0])
    loss = (torch.stack(ys, 1) * dy).sum() + (S * ds).sum()
    want = torch.autograd.grad(loss, leaves)
    for got, w_ in zip(_by_formula(r, k, v, w, dy, s0, ds), want):
        torch.testing.assert_close(got, w_, rtol=1e-12, atol=1e-12)


def test_gradient_formula_against_differences():
    # the loss is linear in each of r, v, s_in and k alone, so a central difference is exact up to rounding
    r, k, v, dy, s0, ds = _inputs(1, 6, 2, 2)
    w = torch.tensor([0.5, 0.97], dtype=torch.float64)

    def loss(r, k, v, s0):
        y, s = ref.mix(r, k, v, w, s0)
        return float((y * dy).sum() + (s * ds).sum())
    grads = _by_formula(r, k, v, w, dy, s0, ds)
    g = torch.Generator().manual_seed(3)
    args = [r, k, v, s0]
    for n in range(4):
        d = torch.randn(args[n].shape, generator=g, dtype=torch.float64)
        up, down = list(args), list(args)
        up[n], down[n] = args[n] + 0.5 * d, args[n] - 0.5 * d
        diff = loss(*up) - loss(*down)
        assert abs(diff - float((grads[n] * d).sum())) <= 1e-10 * (1 + abs(diff)), n


def test_norm_gradient_formula_against_autograd():
    g = torch.Generator().manual_seed(4)
    x, dy = (torch.randn(5, 3, 7, generator=g, dtype=torch.float64) for _ in range(2))
    w, b = (torch.randn(3, 7, generator=g, dtype=torch.float64).requires_grad_() for _ in range(2))
    x.requires_grad_()
    y, mean, rstd = ref.norm(x, None, None, 1e-5)
    want = torch.autograd.grad(((y * w + b) * dy).sum(), (x, w, b))
    got = ref.norm_backward(dy, x.detach(), w.detach(), mean.detach(), rstd.detach())
    for a, c in zip(got, want):
        torch.testing.assert_close(a, c, rtol=1e-11, atol=1e-11)
