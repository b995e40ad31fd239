"""GPU: the norms and the head-decay linear attention together, as a token-mixing layer runs them: input
norm, projections, mixing, per-head norm, and the way back through all of it; then the same layer serving:
ragged prompts and tokens one by one.  Every stage is checked against float64 on what the stage before
it handed over, with the bounds of the single operators."""

import pytest
import torch

import linattn_ref as ref
import rwkv_delta_rule_b200 as lib7
from helpers import need_cuda
from test_parity_gpu_layer_norm import check as check_norm

pytestmark = pytest.mark.gpu

H, D = 4, 256


def layer(seed):
    need_cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s, scale=1.0: torch.randn(s, generator=g, device="cuda") * scale  # noqa: E731
    p = {n: rn(D, D, scale=D ** -0.5).bfloat16() for n in ("r", "k", "v")}
    p.update(w=torch.tensor([0.5, 0.9, 0.99, 1.0], device="cuda"), ln_w=1 + rn(D, scale=0.2), ln_b=rn(D, scale=0.2),
             lnx_w=1 + rn(H, 64, scale=0.2), lnx_b=rn(H, 64, scale=0.2))
    return p, rn


@pytest.mark.parametrize("B,T", [(2, 150), (1, 300)])
def test_training_step(B, T):
    p, rn = layer(1)
    x, dz = rn(B, T, D).bfloat16(), rn(B, T, H, 64).bfloat16()
    h, m1, s1 = lib7.layer_norm(x, p["ln_w"], p["ln_b"])
    r, k, v = ((h @ p[n]).view(B, T, H, 64) for n in ("r", "k", "v"))
    y, s = lib7.linattn_prefill(r, k, v, p["w"])
    z, m2, s2 = lib7.layer_norm(y, p["lnx_w"], p["lnx_b"], 64e-5)
    dy, dlnx_w, dlnx_b = lib7.layer_norm_backward(dz, y, p["lnx_w"], m2, s2)
    dr, dk, dv, _ = lib7.linattn_backward(r, k, v, p["w"], dy)
    dh = sum(d.reshape(B, T, D).float() @ p[n].float().t() for n, d in (("r", dr), ("k", dk), ("v", dv))).bfloat16()
    dx, dln_w, dln_b = lib7.layer_norm_backward(dh, x, p["ln_w"], m1, s1)
    torch.cuda.synchronize()
    assert lib7.rwkv7_get_last_error() == 0

    def flat(G, *ts):
        return [t.reshape(-1, G, t.shape[-1]) for t in ts]
    check_norm(*flat(1, x, dh), p["ln_w"].view(1, D), p["ln_b"].view(1, D), 1e-5, *flat(1, h), m1.view(-1, 1), s1.view(-1, 1),
               *flat(1, dx), dln_w.view(1, D), dln_b.view(1, D))
    ref.check_mix(y, s, r, k, v, p["w"])
    check_norm(*flat(H, y, dz), p["lnx_w"], p["lnx_b"], 64e-5, *flat(H, z), m2.view(-1, H), s2.view(-1, H), *flat(H, dy),
               dlnx_w, dlnx_b)
    ref.check_mix(dr, None, dy, v, k, p["w"], what="dr")
    ref.check_mix(dk, None, v, dy, r, p["w"], reverse=True, what="dk")
    ref.check_mix(dv, None, k, r, dy, p["w"], reverse=True, what="dv")


def test_serving():
    """Three prompts of unequal lengths, then five tokens each, in a captured graph."""
    p, rn = layer(2)
    lens, steps = [70, 1, 200], 5
    x = rn(sum(lens), D).bfloat16()
    nxt = rn(steps, len(lens), D).bfloat16()
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()

    def qkv(t):
        h, _, _ = lib7.layer_norm(t, p["ln_w"], p["ln_b"])
        return [(h @ p[n]).view(*t.shape[:-1], H, 64) for n in ("r", "k", "v")]
    r, k, v = qkv(x)
    y, s = lib7.linattn_prefill_varlen(cu, max(lens), r, k, v, p["w"])
    state = s.clone()
    step = torch.empty_like(nxt[0])
    ops = qkv(nxt[0])  # warm-up of the library products
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops = qkv(step)
        out = lib7.linattn_decode_(*ops, p["w"], state)
        z, _, _ = lib7.layer_norm(out, p["lnx_w"], p["lnx_b"], 64e-5)
    got = []
    for t in range(steps):
        step.copy_(nxt[t])
        graph.replay()
        got.append([a.clone() for a in ops] + [out.clone(), z.clone()])
    torch.cuda.synchronize()
    assert lib7.rwkv7_get_last_error() == 0
    at = cu.tolist()
    for b in range(len(lens)):
        row = [a[None, at[b]:at[b + 1]] for a in (r, k, v)]
        ref.check_mix(y[None, at[b]:at[b + 1]], s[b:b + 1], *row, p["w"], what=b)
    rs, ks, vs, ys, zs = (torch.stack([g[i] for g in got], 1) for i in range(5))
    ref.check_mix(ys, state, rs, ks, vs, p["w"], s, what="steps")
    want, _, _ = ref.norm(ys.view(-1, H, 64), p["lnx_w"], p["lnx_b"], 64e-5)
    # bf16's half step, and float32 sums of 64 values around a mean
    assert bool(((zs.view(-1, H, 64).double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4).all())
