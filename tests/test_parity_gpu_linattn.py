"""GPU: the head-decay linear attention against the token-by-token form in float64, with bounds per
element (linattn_ref).  Heads span the decay domain: 0, a denormal-making one, 0.3 .. 0.9999 and 1."""

import pytest
import torch

import linattn_ref as ref
import rwkv_delta_rule_b200 as lib7
from helpers import need_cuda

pytestmark = pytest.mark.gpu

DECAYS = [0.0, 1e-30, 0.3, 0.9, 0.99, 0.9999, 1.0]
LENGTHS = [1, 2, 31, 32, 33, 64, 127, 128, 129, 255, 256, 257, 300, 640]


def inputs(B, T, H, seed, dtype, s0=True):
    need_cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale
    r, k, v, dy = (randn(B, T, H, 64, scale=s).to(dtype) for s in (1, 0.125, 1, 1))
    w = torch.tensor([DECAYS[i % len(DECAYS)] for i in range(H)], device="cuda")
    st = randn(B, H, 64, 64, scale=0.3) if s0 else None
    ds = randn(B, H, 64, 64, scale=0.3) if s0 else None
    return r, k, v, w, dy, st, ds


def done():
    torch.cuda.synchronize()
    assert lib7.rwkv7_get_last_error() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", LENGTHS)
def test_prefill(T, dtype):
    r, k, v, w, _, st, _ = inputs(2, T, 7, T, dtype, s0=T % 2 == 1)
    y, s = lib7.linattn_prefill(r, k, v, w, st)
    done()
    ref.check_mix(y, s, r, k, v, w, st, what=T)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("states", [0, 1, 2, 3, 100])
def test_prefill_with_less_workspace(states, dtype):
    """Every number of segments that a workspace of `states` states per pair allows."""
    B, T, H = 1, 1100, 7
    r, k, v, w, _, st, _ = inputs(B, T, H, 5, dtype)
    y, s = torch.full_like(r, float("nan")), torch.full_like(st, float("nan"))
    ws = torch.full((states * B * H * 4096,), float("nan"), device="cuda") if states else None
    f = lib7.rwkv7_linattn_prefill if dtype == torch.float32 else lib7.rwkv7_linattn_prefill_bf16
    f(r, k, v, w, st, y, s, ws)
    done()
    ref.check_mix(y, s, r, k, v, w, st, what=states)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prefill_state_in_place_and_chained(dtype):
    """s_out = s_in, with segments that run side by side, and a sequence in two calls."""
    r, k, v, w, _, st, _ = inputs(1, 900, 7, 6, dtype)
    s = st.clone()
    y = torch.empty_like(r)
    f = lib7.rwkv7_linattn_prefill if dtype == torch.float32 else lib7.rwkv7_linattn_prefill_bf16
    ws = torch.empty(lib7.rwkv7_linattn_workspace(1, 900, 7), dtype=torch.uint8, device="cuda")
    f(r, k, v, w, s, y, s, ws)
    done()
    ref.check_mix(y, s, r, k, v, w, st)
    cut = 391
    part = [(r[:, a:b].contiguous(), k[:, a:b].contiguous(), v[:, a:b].contiguous()) for a, b in ((0, cut), (cut, 900))]
    y1, s1 = lib7.linattn_prefill(*part[0], w, st)
    y2, s2 = lib7.linattn_prefill(*part[1], w, s1)
    done()
    ref.check_mix(y1, s1, *part[0], w, st)
    ref.check_mix(y2, s2, *part[1], w, s1)
    ref.check_mix(None, s2, r, k, v, w, st)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 7), (37, 14)])
def test_decode(B, H, dtype):
    r, k, v, w, _, st, _ = inputs(B, 3, H, 7, dtype)
    s = st.clone()
    ys = [lib7.linattn_decode_(*[x[:, t].contiguous() for x in (r, k, v)], w, s) for t in range(3)]
    done()
    ref.check_mix(torch.stack(ys, 1), s, r, k, v, w, st)


def test_prefill_equals_decode_steps():
    r, k, v, w, _, st, _ = inputs(2, 140, 7, 8, torch.bfloat16)
    _, s = lib7.linattn_prefill(r, k, v, w, st)
    d = st.clone()
    for t in range(140):
        lib7.linattn_decode_(*[x[:, t].contiguous() for x in (r, k, v)], w, d)
    done()
    ref.check_mix(None, d, r, k, v, w, st)
    _, mag = ref.mix(r.abs(), k.abs(), v.abs(), w, st.abs())
    assert bool(((s - d).abs() <= 2 * (2 * 140 + 256) * 2.0 ** -24 * mag + 1e-37).all())


def test_no_tokens():
    r, k, v, w, _, st, ds = inputs(2, 0, 7, 9, torch.bfloat16)
    y, s = lib7.linattn_prefill(r, k, v, w, st)
    _, z = lib7.linattn_prefill(r, k, v, w)
    dr, dk, dv, ds_in = lib7.linattn_backward(r, k, v, w, r, st, ds)
    *_, zero = lib7.linattn_backward(r, k, v, w, r)
    done()
    assert y.shape == r.shape and torch.equal(s, st) and not bool(z.any())
    assert torch.equal(ds_in, ds) and not bool(zero.any())


# rows of a ragged batch: none, one, around a chunk, several; max_T below the longest, at it, above it
ROWS = [129, 0, 1, 300, 128, 0, 127, 31]


@pytest.mark.parametrize("max_T", [1, 40, 300, 5000])
@pytest.mark.parametrize("s0", [True, False])
def test_varlen(max_T, s0):
    H, B = 7, len(ROWS)
    gap = 70  # tokens behind the last row
    total = sum(ROWS) + gap
    r, k, v, w, *_ = (x[0] if x is not None and x.dim() == 4 else x for x in inputs(1, total, H, 10, torch.bfloat16, False))
    st = inputs(B, 1, H, 11, torch.bfloat16)[5] if s0 else None
    cu = torch.tensor([0] + ROWS).cumsum(0).to(torch.int32).cuda()
    # what no row owns may hold anything and must stay out of the results
    r, k, v = (x.clone() for x in (r, k, v))
    for x in (r, k, v):
        x[sum(ROWS):] = float("nan")
    y = torch.full_like(r, 7.0)
    s = torch.full((B, H, 64, 64), 7.0, device="cuda")
    n = lib7.rwkv7_linattn_workspace(B, max_T, H)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    lib7.rwkv7_linattn_prefill_varlen_bf16(cu, max_T, r, k, v, w, st, y, s, ws)
    done()
    assert bool((y[sum(ROWS):] == 7.0).all())
    at = cu.tolist()
    for b in range(B):
        row = [x[None, at[b]:at[b + 1]] for x in (r, k, v)]
        ref.check_mix(y[None, at[b]:at[b + 1]], s[b:b + 1], *row, w, None if st is None else st[b:b + 1], what=(max_T, b))


def test_varlen_neighbours_do_not_mix():
    """A row beside rows full of infinities and NaN gets the results that it gets alone."""
    H, n = 7, [100, 200, 60]
    r, k, v, w, *_ = (x[0] if x is not None and x.dim() == 4 else x for x in inputs(1, sum(n), H, 12, torch.bfloat16, False))
    alone_y, alone_s = lib7.linattn_prefill(*[x[None, 100:300].contiguous() for x in (r, k, v)], w)
    for x, bad in ((r, float("nan")), (k, float("inf")), (v, float("nan"))):
        x[:100] = bad
        x[300:] = bad
    cu = torch.tensor([0, 100, 300, 360], dtype=torch.int32, device="cuda")
    y, s = lib7.linattn_prefill_varlen(cu, 200, r, k, v, w)
    done()
    assert torch.equal(y[100:300], alone_y[0]) and torch.equal(s[1], alone_s[0])


@pytest.mark.parametrize("max_T", [20, 600])
def test_varlen_skips_rows_out_of_range(max_T):
    H = 3
    r, k, v, w, *_ = (x[0] if x is not None and x.dim() == 4 else x for x in inputs(1, 200, H, 13, torch.bfloat16, False))
    cu = torch.tensor([0, 50, 40, 200, 900], dtype=torch.int32, device="cuda")  # row 1 runs back, row 3 past the end
    y = torch.full_like(r, 7.0)
    s = torch.full((4, H, 64, 64), 7.0, device="cuda")
    n = lib7.rwkv7_linattn_workspace(4, max_T, H)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    lib7.rwkv7_linattn_prefill_varlen_bf16(cu, max_T, r, k, v, w, None, y, s, ws)
    done()
    assert bool((s[1] == 7.0).all()) and bool((s[3] == 7.0).all())
    row = [x[None, 40:200] for x in (r, k, v)]
    got = y[None, 40:200].clone()
    got[:, :10] = ref.mix(*row, w)[0][:, :10].to(torch.bfloat16)  # tokens 40 .. 49 are row 0's too
    ref.check_mix(got, s[2:3], *row, w)


@pytest.mark.parametrize("T", LENGTHS)
def test_backward(T):
    r, k, v, w, dy, st, ds = inputs(2, T, 7, 100 + T, torch.bfloat16, s0=T % 2 == 0)
    dr, dk, dv, ds_in = lib7.linattn_backward(r, k, v, w, dy, st, ds)
    done()
    t = lambda x: None if x is None else x.transpose(-1, -2)  # noqa: E731
    ref.check_mix(dr, None, dy, v, k, w, t(st), what="dr")
    ref.check_mix(dk, None, v, dy, r, w, t(ds), reverse=True, what="dk")
    ref.check_mix(dv, ds_in, k, r, dy, w, ds, reverse=True, what="dv")


@pytest.mark.parametrize("states", [0, 2, 3])
def test_backward_with_less_workspace_and_in_place(states):
    B, T, H = 1, 1000, 7
    r, k, v, w, dy, st, ds = inputs(B, T, H, 14, torch.bfloat16)
    dr, dk, dv = (torch.full_like(r, float("nan")) for _ in range(3))
    io = ds.clone()
    ws = torch.full((3 * states * B * H * 4096,), float("nan"), device="cuda") if states else None
    lib7.rwkv7_linattn_backward_bf16(r, k, v, w, st, dy, io, dr, dk, dv, io, ws)
    done()
    t = lambda x: x.transpose(-1, -2)  # noqa: E731
    ref.check_mix(dr, None, dy, v, k, w, t(st), what="dr")
    ref.check_mix(dk, None, v, dy, r, w, t(ds), reverse=True, what="dk")
    ref.check_mix(dv, io, k, r, dy, w, ds, reverse=True, what="dv")


@pytest.mark.parametrize("T", [20, 1000])
@pytest.mark.parametrize("states", [0, 3])
def test_backward_over_the_initial_state(states, T):
    """ds_in may be s_in, which another pass reads."""
    B, H = 40, 7
    r, k, v, w, dy, st, ds = inputs(B, T, H, 16, torch.bfloat16)
    dr, dk, dv = (torch.full_like(r, float("nan")) for _ in range(3))
    io = st.clone()
    ws = torch.full((3 * states * B * H * 4096,), float("nan"), device="cuda") if states else None
    lib7.rwkv7_linattn_backward_bf16(r, k, v, w, io, dy, ds, dr, dk, dv, io, ws)
    done()
    t = lambda x: x.transpose(-1, -2)  # noqa: E731
    ref.check_mix(dr, None, dy, v, k, w, t(st), what="dr")
    ref.check_mix(dk, None, v, dy, r, w, t(ds), reverse=True, what="dk")
    ref.check_mix(dv, io, k, r, dy, w, ds, reverse=True, what="dv")


def test_backward_without_state_gradient():
    r, k, v, w, dy, st, ds = inputs(1, 200, 2, 15, torch.bfloat16)
    want = lib7.linattn_backward(r, k, v, w, dy, st, ds)
    dr, dk, dv = (torch.empty_like(r) for _ in range(3))
    lib7.rwkv7_linattn_backward_bf16(r, k, v, w, st, dy, ds, dr, dk, dv, None)
    done()
    assert torch.equal(dr, want[0]) and torch.equal(dk, want[1]) and torch.equal(dv, want[2])


def test_gradient_against_differences_of_the_prefill():
    """The prefill in float32 is linear in v and in s_in: differences of its loss meet dv and ds_in."""
    r, k, v, w, dy, st, ds = inputs(1, 150, 7, 16, torch.bfloat16)
    _, _, dv, ds_in = lib7.linattn_backward(r, k, v, w, dy, st, ds)

    def loss(vf, s0):
        y, s = lib7.linattn_prefill(r.float(), k.float(), vf, w, s0)
        return float((y.double() * dy.double()).sum() + (s.double() * ds.double()).sum())
    g = torch.Generator(device="cuda").manual_seed(17)
    for n, (base, grad, half) in enumerate(((v.float(), dv, 2.0 ** -8), (st, ds_in, 2.0 ** -22))):
        d = torch.randn(base.shape, generator=g, device="cuda")
        up, down = base + 0.5 * d, base - 0.5 * d
        diff = loss(up, st) - loss(down, st) if n == 0 else loss(v.float(), up) - loss(v.float(), down)
        # each rounding of the gradient is independent; four standard deviations of twice their half step
        # (bf16: the result's and the products' one), and the float32 sums of the two losses
        tol = 8 * half * float((grad.double() * d.double()).norm()) + 1e-4 * (1 + float(dy.float().norm()))
        assert abs(diff - float((grad.double() * d.double()).sum())) <= tol, (n, diff)


def test_other_stream_and_two_calls_at_once():
    r, k, v, w, dy, st, ds = inputs(1, 700, 7, 18, torch.bfloat16)
    want = lib7.linattn_prefill(r, k, v, w, st)
    grads = lib7.linattn_backward(r, k, v, w, dy, st, ds)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):  # the workspaces come from each stream's own pool
        got.append((lib7.linattn_prefill(r, k, v, w, st, stream=a), lib7.linattn_backward(r, k, v, w, dy, st, ds, stream=b.cuda_stream)))
    done()
    for (y, s), g in got:
        assert torch.equal(y, want[0]) and torch.equal(s, want[1])
        assert all(torch.equal(p, q) for p, q in zip(g, grads))


def test_graph_replays():
    """A captured prefill, decode and backward, replayed on new values, give what plain calls give."""
    r, k, v, w, dy, st, ds = inputs(1, 500, 7, 19, torch.bfloat16)
    one = [x[:, 0].contiguous() for x in (r, k, v)]
    s = st.clone()
    lib7.linattn_prefill(r, k, v, w, st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lib7.linattn_prefill(r, k, v, w, st) + lib7.linattn_backward(r, k, v, w, dy, st, ds)
        step = lib7.linattn_decode_(*one, w, s)
    other = inputs(1, 500, 7, 20, torch.bfloat16)
    for x, y in zip((r, k, v, dy, st, ds), (other[0], other[1], other[2], other[4], other[5], other[6])):
        x.copy_(y)
    s.copy_(st)
    graph.replay()
    graph.replay()
    done()
    want = lib7.linattn_prefill(r, k, v, w, st) + lib7.linattn_backward(r, k, v, w, dy, st, ds)
    d = st.clone()
    for _ in range(2):
        y = lib7.linattn_decode_(*one, w, d)
    done()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert torch.equal(step, y) and torch.equal(s, d)


def test_long_sequence_state_keeps_its_precision():
    """64 chunks with no decay at all: the state is a plain sum of 8192 products."""
    r, k, v, _, _, st, _ = inputs(1, 8192, 2, 21, torch.bfloat16)
    w = torch.tensor([1.0, 0.99999], device="cuda")
    _, s = lib7.linattn_prefill(r, k, v, w, st)
    done()
    _, want = ref.mix(r, k, v, w, st)
    assert float((s.double() - want).norm() / want.norm()) <= 2e-6


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_stay_in_their_sequence(bad):
    """One bad value of head 1 of row 1: nothing else changes, and of that sequence only the tokens from its
    chunk on."""
    r, k, v, w, dy, st, ds = inputs(2, 400, 3, 24, torch.bfloat16)
    w = torch.full_like(w, 0.9)
    clean = lib7.linattn_prefill(r, k, v, w, st) + lib7.linattn_backward(r, k, v, w, dy, st, ds)
    v[1, 200, 1, 5] = bad
    got = lib7.linattn_prefill(r, k, v, w, st) + lib7.linattn_backward(r, k, v, w, dy, st, ds)
    done()
    for n, (a, b) in enumerate(zip(got, clean)):
        head = 2 if a.shape == r.shape else 1
        assert torch.equal(a[0], b[0]), n
        others = [h for h in range(3) if h != 1]
        assert torch.equal(a[1].transpose(0, head - 1)[others], b[1].transpose(0, head - 1)[others]), n
    y, s = got[:2]
    assert torch.equal(y[1, :128, 1], clean[0][1, :128, 1])
    assert not bool(torch.isfinite(y[1, 200:, 1, 5]).any()) and not bool(torch.isfinite(s[1, 1, 5]).any())
    dr, dk = got[2:4]
    assert torch.equal(dr[1, :128, 1], clean[2][1, :128, 1])  # dr reads the states before it alone
    assert torch.equal(dk[1, 256:, 1], clean[3][1, 256:, 1])  # dk of a later token does not see an earlier v


def test_guard_bands():
    """Nothing outside the outputs is written: outputs inside larger buffers, odd sizes."""
    B, T, H = 2, 333, 3
    r, k, v, w, dy, st, ds = inputs(B, T, H, 22, torch.bfloat16)
    pad = 1024

    def banded(like):
        buf = torch.full((like.numel() + 2 * pad,), 3.0, dtype=like.dtype, device="cuda")
        return buf, buf[pad:pad + like.numel()].view(like.shape)
    bufs = [banded(x) for x in (r, st, r, r, r, st)]
    y, s, dr, dk, dv, dsi = (v_ for _, v_ in bufs)
    nb = lib7.rwkv7_linattn_backward_workspace(B, T, H)
    wbuf = torch.full((nb // 4 + 2 * pad,), 3.0, device="cuda")
    ws = wbuf[pad:pad + nb // 4] if nb else None
    lib7.rwkv7_linattn_prefill_bf16(r, k, v, w, st, y, s, ws)
    lib7.rwkv7_linattn_backward_bf16(r, k, v, w, st, dy, ds, dr, dk, dv, dsi, ws)
    done()
    for buf in [b for b, _ in bufs] + [wbuf]:
        assert bool((buf[:pad] == 3.0).all()) and bool((buf[-pad:] == 3.0).all())
    ref.check_mix(y, s, r, k, v, w, st)


@pytest.mark.parametrize("T", [1500, 2048])
def test_many_chains_in_segments_of_several_chunks(T):
    """96 chains in 3 segments of 4 to 6 chunks each: several CTAs per SM, forward and backward."""
    r, k, v, w, dy, st, ds = inputs(3, T, 32, 23, torch.bfloat16)
    assert lib7.rwkv7_linattn_workspace(3, T, 32) >= 3 * 96 * 64 * 64 * 4
    y, s = lib7.linattn_prefill(r, k, v, w, st)
    done()
    ref.check_mix(y, s, r, k, v, w, st)
    r, k, v, dy, st, ds = (x[:1].contiguous() for x in (r, k, v, dy, st, ds))  # 3 passes of 32 chains
    grads = torch.full((3 * 3 * 32 * 64 * 64,), float("nan"), device="cuda")
    dr, dk, dv, dsi = (torch.full_like(x, float("nan")) for x in (r, r, r, st))
    lib7.rwkv7_linattn_backward_bf16(r, k, v, w, st, dy, ds, dr, dk, dv, dsi, grads)
    done()
    t = lambda x: x.transpose(-1, -2)  # noqa: E731
    ref.check_mix(dr, None, dy, v, k, w, t(st), what="dr")
    ref.check_mix(dk, None, v, dy, r, w, t(ds), reverse=True, what="dk")
    ref.check_mix(dv, dsi, k, r, dy, w, ds, reverse=True, what="dv")
