"""GPU: NaN and infinity among the operands of the head-decay linear attention.  The recurrence in float64 says which
results they reach (a token's own, later ones, and in the gradients of k and v earlier ones): those are
not finite, and all others have the bits that they have without the bad values.  Float32 and T = 20 go
token by token, bf16 from 32 tokens on in chunks of 128."""

import pytest
import torch

import linattn_ref as ref
import rwkv_delta_rule_b200 as lib7
from test_parity_gpu_linattn import done, inputs

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
F32, BF16 = torch.float32, torch.bfloat16


def meets(got, clean, want, what):
    """got is finite where want (float64) is, with clean's bits, and not finite elsewhere."""
    fine = torch.isfinite(want)
    wrong = fine != torch.isfinite(got)
    n = int(wrong.sum())
    assert n == 0, (what, "not finite, or finite, at", wrong.nonzero()[:4].tolist(), n)
    changed = int((got[fine] != clean[fine]).sum())
    assert changed == 0, (what, "changed", changed)


def spoil(ops, name, at, bad):
    """ops with values of operand `name` replaced: at = [(token, channel), ...], of row 1 and of every head"""
    ops = dict(ops, **{name: ops[name].clone()})
    for t, c in at:
        ops[name][1, t, :, c] = bad
    return ops


PLACES = [[(0, 5)], [(127, 0), (126, 63)], [(128, 63)], [(299, 31)], [(200, 7), (210, 7), (190, 40), (297, 40), (201, 8)]]


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("name", ["r", "k", "v"])
@pytest.mark.parametrize("dtype,T", [(BF16, 300), (BF16, 20), (F32, 300)])
def test_prefill(dtype, T, name, bad):
    r, k, v, w, _, st, _ = inputs(2, T, 7, 30, dtype)
    ops = dict(r=r, k=k, v=v)
    clean = lib7.linattn_prefill(**ops, w=w, s_in=st)
    for at in PLACES:
        at = [(t % T, c) for t, c in at]
        x = spoil(ops, name, at, bad)
        got = lib7.linattn_prefill(**x, w=w, s_in=st)
        done()
        for g, c, r_, n in zip(got, clean, ref.mix(x["r"], x["k"], x["v"], w, st), ("y", "s_out")):
            meets(g, c, r_, (n, at))


@pytest.mark.parametrize("bad", [NAN, -INF])
def test_prefill_in_segments(bad):
    """1100 tokens in segments that run side by side; the state that arrives is bad, too."""
    r, k, v, w, _, st, _ = inputs(2, 1100, 3, 31, BF16)
    ops = dict(r=r, k=k, v=v)
    assert lib7.rwkv7_linattn_workspace(2, 1100, 3) > 0
    clean = lib7.linattn_prefill(**ops, w=w, s_in=st)
    for name, at in (("v", [(700, 3), (760, 3), (701, 4)]), ("k", [(1023, 3)]), ("r", [(1024, 3)])):
        x = spoil(ops, name, at, bad)
        got = lib7.linattn_prefill(**x, w=w, s_in=st)
        done()
        for g, c, r_ in zip(got, clean, ref.mix(x["r"], x["k"], x["v"], w, st)):
            meets(g, c, r_, (name, at))
    s2 = st.clone()
    s2[0, 1, 9, 40] = bad
    got = lib7.linattn_prefill(**ops, w=w, s_in=s2)
    done()
    for g, c, r_ in zip(got, clean, ref.mix(r, k, v, w, s2)):
        meets(g, c, r_, "s_in")


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("name", ["r", "k", "v", "dy"])
@pytest.mark.parametrize("T", [20, 300])
def test_backward(T, name, bad):
    r, k, v, w, dy, st, ds = inputs(2, T, 7, 32, BF16)
    ops = dict(r=r, k=k, v=v, dy=dy)
    clean = lib7.linattn_backward(**ops, w=w, s_in=st, ds_out=ds)
    t = lambda x: x.transpose(-1, -2)  # noqa: E731
    for at in PLACES:
        at = [(u % T, c) for u, c in at]
        x = spoil(ops, name, at, bad)
        got = lib7.linattn_backward(**x, w=w, s_in=st, ds_out=ds)
        done()
        want = [ref.mix(x["dy"], x["v"], x["k"], w, t(st))[0], ref.mix(x["v"], x["dy"], x["r"], w, t(ds), reverse=True)[0],
                *ref.mix(x["k"], x["r"], x["dy"], w, ds, reverse=True)]
        for g, c, r_, n in zip(got, clean, want, ("dr", "dk", "dv", "ds_in")):
            meets(g, c, r_, (n, at))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [33, 128, 200, 255])
def test_padded_batch(n, dtype):
    """Rows filled up with anything behind their last token: the tokens that count have the outputs of the row alone."""
    r, k, v, w, _, st, _ = inputs(2, 290, 7, 33, dtype)
    f = lib7.rwkv7_linattn_prefill if dtype == F32 else lib7.rwkv7_linattn_prefill_bf16

    def call(r, k, v):  # whole sequences, so that the sums are the same whatever the length
        y, s = torch.empty_like(r), torch.empty_like(st)
        f(r, k, v, w, st, y, s)
        return y
    alone = call(*(x[:, :n].contiguous() for x in (r, k, v)))
    for x, bad in ((r, INF), (k, NAN), (v, NAN)):
        x[:, n:] = bad
    v[0, n:] = INF
    padded = call(r, k, v)
    done()
    changed = int((padded[:, :n] != alone).sum())  # a NaN differs from anything
    assert changed == 0


def test_bad_values_in_many_chunks():
    """Several CTAs per SM, bad values in most chunks of some heads, in ragged rows with a part of a chunk at their end."""
    H, rows = 32, [1500, 700, 1, 129, 640]
    total = sum(rows)
    r, k, v, w, *_ = (x[0] if x is not None and x.dim() == 4 else x for x in inputs(1, total, H, 36, BF16, False))
    st = inputs(len(rows), 1, H, 37, BF16)[5]
    cu = torch.tensor([0] + rows).cumsum(0).to(torch.int32).cuda()
    clean = lib7.linattn_prefill_varlen(cu, max(rows), r, k, v, w, st)
    g = torch.Generator().manual_seed(38)
    for n in range(60):
        t, h, c = (int(torch.randint(m, (1,), generator=g)) for m in (total, H // 2, 64))
        (k if n % 6 == 0 else v)[t, 2 * h, c] = (NAN, INF, -INF)[n % 3]
    y, s = lib7.linattn_prefill_varlen(cu, max(rows), r, k, v, w, st)
    done()
    at = cu.tolist()
    for b in range(len(rows)):
        want = ref.mix(*(x[None, at[b]:at[b + 1]] for x in (r, k, v)), w, st[b:b + 1])
        meets(y[None, at[b]:at[b + 1]], clean[0][None, at[b]:at[b + 1]], want[0], ("y", b))
        meets(s[b:b + 1], clean[1][b:b + 1], want[1], ("s_out", b))
