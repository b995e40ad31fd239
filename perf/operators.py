"""Cases of the head-decay linear attention and of the layer norm, with their plain forms.

Linear attention with one decay per head (per batch row b and head h, 64 x 64 float32 state S,
row = value channel, column = key channel, as for the wkv recurrence):

    S_t = w_h S_{t-1} + v_t k_t^T,    y_t = S_t r_t

as prefill (dense and ragged batches), one decode step, and the gradients of r, k, v and the
initial state.  Layer norm over groups of D channels, x [M, G, D] with weight and bias [G, D]
(G = 1: the ln1 / ln2 of a block, weight [D]; G = heads, D = 64: the ln_x of the time mix), forward and backward.

``run`` computes the operators in elementary float32 torch operations, or, with ``own`` set, calls
the framework.  ``exact`` follows the definitions in float64, token by token.
"""

import math

import torch

own = False
N = 64
DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ---- cases ------------------------------------------------------------------------------------------

def listed():
    return [
        # one user's next token, width 768: latency
        {"name": "decode_b1_h12_f32", "op": "decode", "dtype": "f32", "B": 1, "H": 12},
        # a serving batch's next token, width 1024
        {"name": "decode_b256_h16", "op": "decode", "dtype": "bf16", "B": 256, "H": 16},
        # one prompt of odd length in float32: few heads, so the length has to be split
        {"name": "prefill_f32_b1_t1000_h12", "op": "prefill", "dtype": "f32", "B": 1, "T": 1000, "H": 12, "s0": False},
        # a batch of prompts at width 768, continuing from states
        {"name": "prefill_d768_b8_t4096", "op": "prefill", "dtype": "bf16", "B": 8, "T": 4096, "H": 12, "s0": True},
        # prompts of unequal lengths packed together, width 2048
        {"name": "prefill_ragged_d2048_b16", "op": "varlen", "dtype": "bf16", "B": 16, "T": 2500, "H": 32, "s0": True},
        # long contexts at width 4096: the largest
        {"name": "prefill_d4096_b4_t16384", "op": "prefill", "dtype": "bf16", "B": 4, "T": 16384, "H": 64, "s0": False},
        # a training step's gradients at width 768
        {"name": "backward_d768_b8_t1024", "op": "backward", "dtype": "bf16", "B": 8, "T": 1024, "H": 12, "s0": False},
        # gradients of long sequences at width 4096, odd length, with state gradients
        {"name": "backward_d4096_b2_t4001", "op": "backward", "dtype": "bf16", "B": 2, "T": 4001, "H": 64, "s0": True},
        # a block's input norm over a prefill's tokens, width 4096
        {"name": "norm_m65536_d4096", "op": "norm", "dtype": "bf16", "M": 65536, "G": 1, "D": 4096, "eps": 1e-5},
        # the same norm on one float32 token batch of odd width: latency and unaligned rows
        {"name": "norm_f32_m37_d1001", "op": "norm", "dtype": "f32", "M": 37, "G": 1, "D": 1001, "eps": 1e-5},
        # its gradients in a training step, width 768
        {"name": "norm_grad_m32768_d768", "op": "norm_grad", "dtype": "bf16", "M": 32768, "G": 1, "D": 768, "eps": 1e-5},
        # gradients of the per-head norm after the token mixing, width 4096
        {"name": "norm_grad_m16384_g64_d64", "op": "norm_grad", "dtype": "bf16", "M": 16384, "G": 64, "D": 64, "eps": 64e-5},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "prefill", "prefill", "varlen", "backward", "norm", "norm_grad"])
    dtype = "bf16" if op in ("varlen", "backward") else rng.choice(["bf16", "bf16", "f32"])
    if op == "decode":
        return {"op": op, "dtype": dtype, "B": _spread(rng, 1, 256), "H": rng.choice([1, 12, 16, 32, 40, 64])}
    if op in ("prefill", "varlen", "backward"):
        B, H, T = _spread(rng, 1, 16), rng.choice([1, 2, 12, 16, 32, 64]), _spread(rng, 1, 16384)
        most = 1 << (22 if op == "prefill" and dtype == "bf16" else 19)
        T = max(1, min(T, most // (B * H)))
        return {"op": op, "dtype": dtype, "B": B, "T": T, "H": H, "s0": rng.random() < 0.5}
    # from 8 channels on: the gradient of a norm over two or three is all cancellation
    G, D = rng.choice([(1, _spread(rng, 8, 16384)), (1, 64 * rng.randint(1, 128)), (rng.choice([1, 12, 32, 64]), 64),
                       (rng.randint(2, 16), rng.randint(8, 300))])
    M = max(1, min(_spread(rng, 1, 65536), (1 << 27) // (G * D)))
    return {"op": op, "dtype": dtype, "M": M, "G": G, "D": D, "eps": 64e-5 if G > 1 else 1e-5}


def _lengths(B, T):
    """Row lengths of a ragged batch: between nothing and T tokens, the first row T."""
    g = torch.Generator().manual_seed(B * 100003 + T)
    n = (torch.rand(B, generator=g) * (T + 1)).long().clamp_(max=T)
    n[0] = T
    return n


def _type(case):
    return BF16 if case["dtype"] == "bf16" else F32


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    ty, op = _type(case), case["op"]

    def randn(*shape, scale=1.0, shift=0.0, dtype=None):
        return torch.randn(shape, generator=g, device=DEV).mul_(scale).add_(shift).to(dtype or ty)

    s = {"case": dict(case)}
    if op in ("norm", "norm_grad"):
        M, G, D = case["M"], case["G"], case["D"]
        shape = (M, D) if G == 1 else (M, G, D)
        s["x"] = randn(*shape, scale=1.5, shift=0.25)
        s["weight"] = randn(*shape[1:], scale=0.2, shift=1.0, dtype=F32)
        s["bias"] = randn(*shape[1:], scale=0.2, dtype=F32)
        if op == "norm_grad":
            s["dy"] = randn(*shape, scale=0.5)
            # what the forward pass left behind
            x = s["x"].to(F64)
            mean = x.mean(-1)
            s["mean"] = mean.to(F32)
            s["rstd"] = ((x - mean[..., None]).square().mean(-1) + case["eps"]).rsqrt().to(F32)
        return s
    H = case["H"]
    # one decay per head, from a memory of 32 tokens to one of 4096
    s["w"] = (1.0 - torch.exp2(-5.0 - 7.0 * torch.arange(H, device=DEV, dtype=F64) / max(1, H - 1))).to(F32)
    if op == "varlen":
        n = _lengths(case["B"], case["T"])
        s["lens"] = n.to(DEV)
        s["cu"] = torch.cat([torch.zeros(1, dtype=torch.long), n.cumsum(0)]).to(torch.int32).to(DEV)
        shape = (int(n.sum()), H, N)
    else:
        shape = (case["B"], H, N) if op == "decode" else (case["B"], case["T"], H, N)
    s["r"], s["k"], s["v"] = randn(*shape), randn(*shape, scale=0.125), randn(*shape)
    st = (case["B"], H, N, N)
    if op == "decode" or case["s0"]:
        s["s0"] = randn(*st, scale=0.3, dtype=F32)
    if op == "backward":
        s["dy"] = randn(*shape)
        if case["s0"]:
            s["ds"] = randn(*st, scale=0.3, dtype=F32)
    return s


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op in ("norm", "norm_grad"):
        n, w = case["M"] * case["G"] * case["D"], case["G"] * case["D"]
        stats = 8 * case["M"] * case["G"]
        if op == "norm":
            return {"bytes": 2 * n * e + 8 * w + stats, "flops": 8 * n}
        return {"bytes": 3 * n * e + 12 * w + stats, "flops": 14 * n}
    B, H = case["B"], case["H"]
    tok = int(_lengths(B, case["T"]).sum()) if op == "varlen" else B * case.get("T", 1)
    st = B * H * N * N * 4
    if op == "backward":
        return {"bytes": 7 * tok * H * N * e + (3 * st if case["s0"] else st), "flops": 14 * tok * H * N * N}
    return {"bytes": 4 * tok * H * N * e + (2 * st if op == "decode" or case["s0"] else st), "flops": 4 * tok * H * N * N}


# ---- plain forms ----------------------------------------------------------------------------------------

def _powers(w, e):
    """w[h] ** e for exponents >= 0, formed in float64."""
    return torch.pow(w.to(F64).view(-1, *([1] * e.dim())), e.to(F64)).to(F32)


def _mix(q, k, v, w, C=64):
    """[B,T,H,N] float32 from a zero state: (out, final state), chunk by chunk all at once.
    T is filled up in front with empty tokens, which leave a zero state as it is."""
    B, T, H, _ = q.shape
    nc = -(-T // C)
    q, k, v = (torch.cat([x.new_zeros(B, nc * C - T, H, N), x], 1).view(B, nc, C, H, N).permute(3, 0, 1, 2, 4)
               for x in (q, k, v))  # [H,B,nc,C,N]
    i = torch.arange(C, device=DEV)
    d = i[:, None] - i[None, :]
    D = _powers(w, d.clamp(min=0)) * (d >= 0)
    out = ((q @ k.transpose(-1, -2)) * D[:, None, None]) @ v
    U = (v * _powers(w, C - 1 - i)[:, None, None, :, None]).transpose(-1, -2) @ k  # [H,B,nc,N,N] what a chunk adds
    c = torch.arange(nc + 1, device=DEV)
    d = c[:, None] - 1 - c[None, :nc]
    M = _powers(w, C * d.clamp(min=0)) * (d >= 0)  # a chunk's start from the chunks before it
    S = (M[:, None] @ U.reshape(H, B, nc, N * N)).view(H, B, nc + 1, N, N)
    out = out + (q @ S[:, :, :nc].transpose(-1, -2)) * _powers(w, i + 1)[:, None, None, :, None]
    return out.permute(1, 2, 3, 0, 4).reshape(B, nc * C, H, N)[:, nc * C - T:], S[:, :, nc].transpose(0, 1)


def _plain_prefill(r, k, v, w, s0):
    r, k, v = r.float(), k.float(), v.float()
    y, s = _mix(r, k, v, w)
    if s0 is not None:
        T = r.shape[1]
        p = _powers(w, torch.arange(T + 1, device=DEV))  # [H,T+1]
        y = y + (r.transpose(1, 2) @ s0.transpose(-1, -2)).transpose(1, 2) * p[:, 1:].t()[None, :, :, None]
        s = s + s0 * p[:, T].view(-1, 1, 1)
    return y, s


def _plain_varlen(r, k, v, w, s0, cu, lens, T):
    # rows end together at T; what is in front of a row is empty
    B = lens.numel()
    pos = torch.arange(T, device=DEV)[None] - (T - lens)[:, None]  # token of the row, negative in front
    at = (cu[:-1, None] + pos).clamp(min=0)
    there = (pos >= 0)[:, :, None, None]
    r, k, v = (x.float()[at] * there for x in (r, k, v))
    y, s = _mix(r, k, v, w)
    if s0 is not None:
        y = y + (r.transpose(1, 2) @ s0.transpose(-1, -2)).transpose(1, 2) * _powers(w, (pos + 1).clamp(min=0)).permute(1, 2, 0)[..., None]
        s = s + s0 * _powers(w, lens).t()[:, :, None, None]
    return y[pos >= 0], s


def _plain_backward(r, k, v, w, dy, s0, ds):
    r, k, v, dy = r.float(), k.float(), v.float(), dy.float()
    T = r.shape[1]
    p = _powers(w, torch.arange(T + 1, device=DEV))
    dr, _ = _mix(dy, v, k, w)
    rk, rv, rr, rdy = (x.flip(1) for x in (k, v, r, dy))
    dk, _ = _mix(rv, rdy, rr, w)
    dv, g = _mix(rk, rr, rdy, w)
    dk, dv = dk.flip(1), dv.flip(1)
    g = g * w.view(-1, 1, 1)
    if s0 is not None:
        dr = dr + (dy.transpose(1, 2) @ s0).transpose(1, 2) * p[:, 1:].t()[None, :, :, None]
    if ds is not None:
        f = p[:, :T].flip(1).t()[None, :, :, None]
        dk = dk + (v.transpose(1, 2) @ ds).transpose(1, 2) * f
        dv = dv + (k.transpose(1, 2) @ ds.transpose(-1, -2)).transpose(1, 2) * f
        g = g + ds * p[:, T].view(-1, 1, 1)
    return dr, dk, dv, g


def run(s):
    case = s["case"]
    op, ty = case["op"], _type(case)
    if own:
        return _own(s, op, case)
    if op == "norm":
        x = s["x"].float()
        mean = x.sum(-1, keepdim=True) / x.shape[-1]
        c = x - mean
        rstd = 1.0 / torch.sqrt((c * c).sum(-1, keepdim=True) / x.shape[-1] + case["eps"])
        return {"y": (c * rstd * s["weight"] + s["bias"]).to(ty), "mean": mean[..., 0], "rstd": rstd[..., 0]}
    if op == "norm_grad":
        x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][..., None]
        xh = (x - s["mean"][..., None]) * rstd
        g = dy * s["weight"]
        D = x.shape[-1]
        dx = rstd * (g - g.sum(-1, keepdim=True) / D - xh * ((g * xh).sum(-1, keepdim=True) / D))
        return {"dx": dx.to(ty), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}
    r, k, v, w, s0 = s["r"], s["k"], s["v"], s["w"], s.get("s0")
    if op == "decode":
        kf, vf, rf = k.float(), v.float(), r.float()
        s0.mul_(w.view(-1, 1, 1)).add_(vf[..., :, None] * kf[..., None, :])
        return {"y": (s0 * rf[..., None, :]).sum(-1).to(ty), "s": s0}
    if op == "backward":
        dr, dk, dv, dsi = _plain_backward(r, k, v, w, s["dy"], s0, s.get("ds"))
        return {"dr": dr.to(ty), "dk": dk.to(ty), "dv": dv.to(ty), "ds_in": dsi}
    y, so = _plain_varlen(r, k, v, w, s0, s["cu"], s["lens"], case["T"]) if op == "varlen" else _plain_prefill(r, k, v, w, s0)
    return {"y": y.to(ty), "s": so}


def _own(s, op, case):
    import rwkv_delta_rule_b200 as rk

    if op == "norm":
        y, mean, rstd = rk.layer_norm(s["x"], s["weight"], s["bias"], case["eps"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        dx, dw, db = rk.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])
        return {"dx": dx, "dweight": dw, "dbias": db}
    r, k, v, w, s0 = s["r"], s["k"], s["v"], s["w"], s.get("s0")
    if op == "decode":
        return {"y": rk.linattn_decode_(r, k, v, w, s0), "s": s0}
    if op == "backward":
        dr, dk, dv, dsi = rk.linattn_backward(r, k, v, w, s["dy"], s0, s.get("ds"))
        return {"dr": dr, "dk": dk, "dv": dv, "ds_in": dsi}
    if op == "varlen":
        y, so = rk.linattn_prefill_varlen(s["cu"], case["T"], r, k, v, w, s0)
    else:
        y, so = rk.linattn_prefill(r, k, v, w, s0)
    return {"y": y, "s": so}


# ---- the definitions in float64 ------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        return _exact_norm(s, op, case)
    H, B = case["H"], case["B"]
    w = s["w"].to(F64)[None, :, None, None]
    S = s["s0"].to(F64) if "s0" in s else torch.zeros(B, H, N, N, dtype=F64, device=DEV)
    if op == "decode":
        S = w * S + torch.einsum("bhi,bhj->bhij", s["v"].to(F64), s["k"].to(F64))
        return {"y": torch.einsum("bhij,bhj->bhi", S, s["r"].to(F64)), "s": S}
    if op == "varlen":
        y, at, out = torch.empty(s["r"].shape, dtype=F64, device=DEV), s["cu"].tolist(), S.clone()
        # rows in order of length: at token t the first `live` rows still run
        n = [at[b + 1] - at[b] for b in range(B)]
        order = sorted(range(B), key=lambda b: -n[b])
        first = torch.tensor([at[b] for b in order], device=DEV)
        S = S[order].contiguous()
        live = B
        for t in range(max(n)):
            while n[order[live - 1]] <= t:
                live -= 1
            rows = first[:live] + t
            v, k, r = (s[x][rows].to(F64) for x in ("v", "k", "r"))
            A = S[:live]
            A.mul_(w)
            A.add_(v[..., :, None] * k[..., None, :])
            y[rows] = (A @ r[..., None])[..., 0]
        out[order] = S
        return {"y": y, "s": out}
    T = case["T"]
    if op == "prefill":
        y = torch.empty(s["r"].shape, dtype=F64, device=DEV)
        for t in range(T):
            v, k, r = (s[x][:, t].to(F64) for x in ("v", "k", "r"))
            S.mul_(w)
            S.add_(v[..., :, None] * k[..., None, :])
            y[:, t] = (S @ r[..., None])[..., 0]
        return {"y": y, "s": S}
    dr, dk, dv = (torch.empty(s["r"].shape, dtype=F64, device=DEV) for _ in range(3))
    for t in range(T):
        S = w * S + s["v"][:, t].to(F64)[..., :, None] * s["k"][:, t].to(F64)[..., None, :]
        dr[:, t] = torch.einsum("bhij,bhi->bhj", S, s["dy"][:, t].to(F64))
    Gm = s["ds"].to(F64) if "ds" in s else torch.zeros_like(S)
    for t in range(T - 1, -1, -1):
        Gm = Gm + s["dy"][:, t].to(F64)[..., :, None] * s["r"][:, t].to(F64)[..., None, :]
        dk[:, t] = torch.einsum("bhij,bhi->bhj", Gm, s["v"][:, t].to(F64))
        dv[:, t] = torch.einsum("bhij,bhj->bhi", Gm, s["k"][:, t].to(F64))
        Gm = w * Gm
    return {"dr": dr, "dk": dk, "dv": dv, "ds_in": Gm}


def _exact_norm(s, op, case):
    M = case["M"]
    step = max(1, (1 << 26) // (case["G"] * case["D"]))
    parts, dw, db = [], 0.0, 0.0
    for a in range(0, M, step):
        x = s["x"][a:a + step].to(F64)
        if op == "norm":
            mean = x.mean(-1)
            var = x.square().mean(-1) - mean.square()  # the other formula of the variance, safe in 64 bits here
            rstd = (var.clamp(min=0) + case["eps"]).rsqrt()
            y = ((x - mean[..., None]) * rstd[..., None]) * s["weight"].to(F64) + s["bias"].to(F64)
            parts.append((y.to(F32) if M * case["G"] * case["D"] > 1 << 27 else y, mean, rstd))
            continue
        dy, rstd = s["dy"][a:a + step].to(F64), s["rstd"][a:a + step].to(F64)
        xh = torch.einsum("...d,...->...d", x - s["mean"][a:a + step].to(F64)[..., None], rstd)
        g = dy * s["weight"].to(F64)
        dot = torch.einsum("...d,...d->...", g, xh)[..., None]
        dx = rstd[..., None] * (g - (g.sum(-1, keepdim=True) + xh * dot) / case["D"])
        parts.append((dx,))
        dw, db = dw + torch.einsum("m...,m...->...", dy, xh), db + dy.sum(0)
    out = [torch.cat(p) for p in zip(*parts)]
    if op == "norm":
        return {"y": out[0], "mean": out[1], "rstd": out[2]}
    return {"dx": out[0], "dweight": dw, "dbias": db}
