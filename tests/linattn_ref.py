"""Plain float64 forms of the head-decay linear attention and the layer norm, and bounds on what
rounding may do to the kernels' results.

A bound is formed per element from the magnitudes of what is summed: a rounding of a term to bf16 moves
it by at most 2^-8 of itself, one float32 operation by 2^-24, and a sum of n terms in float32 by n 2^-24 of
the sum of their magnitudes.
"""

import torch

BF16_HALF_STEP = 2.0 ** -8
F32_HALF_STEP = 2.0 ** -24


def mix(q, k, v, w, s0=None, reverse=False):
    """Token by token: (out [B,T,H,64], end state) of S <- w S + v k^T, out = S q, or reversed
    S <- S + v k^T, out = S q, S <- w S from the last token.  float64; states [B,H,64,64]."""
    q, k, v, w = (x.double() for x in (q, k, v, w))
    B, T, H, N = q.shape
    S = torch.zeros(B, H, N, N, dtype=torch.float64, device=q.device) if s0 is None else s0.double().clone()
    wb = w.view(1, H, 1, 1)
    out = torch.empty(B, T, H, N, dtype=torch.float64, device=q.device)
    for t in (range(T - 1, -1, -1) if reverse else range(T)):
        vk = v[:, t, :, :, None] * k[:, t, :, None, :]
        S = S + vk if reverse else wb * S + vk
        out[:, t] = (S @ q[:, t, :, :, None])[..., 0]
        if reverse:
            S = wb * S
    return out, S


def products(q, k, v, w, reverse=False):
    """sum_s w^|t-s| |q_t . k_s| |v_s|, what a rounding of the products q_t . k_s is multiplied by."""
    q, k, v = (x.double().transpose(1, 2) for x in (q, k, v))
    w = w.double()
    T = q.shape[2]
    i = torch.arange(T, device=q.device)
    d = (i[None, :] - i[:, None]) if reverse else (i[:, None] - i[None, :])
    D = torch.pow(w.view(-1, 1, 1), d.clamp(min=0).double()) * (d >= 0)
    return (((q @ k.transpose(-1, -2)) * D).abs() @ v.abs()).transpose(1, 2)


def state_products(q, k, v, w, s0=None, reverse=False, C=128):
    """What a rounding of the state that a chunk of C tokens begins with (reversed: of the one behind it) is
    multiplied by: w^(tokens between) |S| |q_t|, summed over the 64 key channels."""
    q, k, v, w = (x.double() for x in (q, k, v, w))
    B, T, H, N = q.shape
    out, S = torch.zeros_like(q), s0
    starts = list(range(0, T, C))
    for t0 in (reversed(starts) if reverse else starts):
        n = min(C, T - t0)
        part = [x[:, t0:t0 + n] for x in (q, k, v)]
        if S is not None:
            i = torch.arange(n, device=q.device, dtype=torch.float64)
            f = torch.pow(w.view(1, 1, H, 1), ((n - 1 - i) if reverse else (i + 1)).view(1, n, 1, 1))
            out[:, t0:t0 + n] = torch.einsum("bhij,bthj->bthi", S.double().abs(), part[0].abs()) * f
        _, S = mix(*part, w, S, reverse)
    return out


def check_mix(out, s_end, q, k, v, w, s0=None, reverse=False, what=""):
    """out (its dtype says how it was rounded) and the end state (or None) of a pass against float64."""
    T = q.shape[1]
    ref, ref_s = mix(q, k, v, w, s0, reverse)
    mag, mag_s = mix(q.abs(), k.abs(), v.abs(), w, None if s0 is None else s0.abs(), reverse)
    # float32 sums: T tokens, 64 channels, and a handful of operations per chunk on the way
    n = (2 * T + 256) * F32_HALF_STEP
    if out is not None and T > 0:
        tol = n * mag
        if out.dtype == torch.bfloat16:
            # the result's own rounding, the products' q_t . k_s one, and the one of the state that a chunk
            # begins with: each moves its term by at most half a step, and nothing else is in bf16
            tol = tol + BF16_HALF_STEP * (ref.abs() + products(q, k, v, w, reverse)
                                          + state_products(q, k, v, w, s0, reverse)) * (1 + 2.0 ** -6)
            if s_end is None:
                # no state leaves the pass, which may then form its products v k^T from two bf16 terms of v: the
                # first, cut to 8 bits, leaves less than 2^-7 of v, and rounding that to 8 bits leaves 2^-9 of it
                tol = tol + 2.0 ** -16 * mag
        bad = ~((out.double() - ref).abs() <= tol + 1e-37)
        assert not bool(bad.any()), (what, "out", bad.nonzero()[:4].tolist(), float((out.double() - ref).abs().max()))
    if s_end is not None:
        bad = ~((s_end.double() - ref_s).abs() <= n * mag_s + 1e-37)
        assert not bool(bad.any()), (what, "state", bad.nonzero()[:4].tolist(), float((s_end.double() - ref_s).abs().max()))


def norm(x, weight, bias, eps):
    """[M,G,D]: (y, mean, rstd) in float64."""
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    y = (x - mean) * rstd
    y = y * (1.0 if weight is None else weight.double()) + (0.0 if bias is None else bias.double())
    return y, mean[..., 0], rstd[..., 0]


def norm_backward(dy, x, weight, mean, rstd):
    """[M,G,D]: (dx, dweight, dbias) in float64, from the mean and rstd given."""
    dy, x, rs = dy.double(), x.double(), rstd.double()[..., None]
    xh = (x - mean.double()[..., None]) * rs
    g = dy * (1.0 if weight is None else weight.double())
    dx = rs * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)
