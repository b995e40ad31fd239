"""GPU: what the outputs of the head-decay linear attention do not depend on: whether the state's gradient is asked
for, and whether a sequence comes in one call or in several."""

import pytest
import torch

import linattn_ref as ref
import rwkv_delta_rule_b200 as lib7
from test_parity_gpu_linattn import done, inputs

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("T", [100, 1500])
def test_gradients_do_not_depend_on_the_state_gradient_being_asked_for(T):
    """dr, dk, dv bit for bit, with ds_in and without, with the same workspace."""
    B, H = 4, 7
    r, k, v, w, dy, st, ds = inputs(B, T, H, 34, BF16)
    w = torch.linspace(0.9, 1.0, H, device="cuda")
    ws = torch.empty(lib7.rwkv7_linattn_backward_workspace(B, T, H), dtype=torch.uint8, device="cuda")
    outs = []
    for ds_in in (torch.empty_like(st), None):
        dr, dk, dv = (torch.empty_like(r) for _ in range(3))
        lib7.rwkv7_linattn_backward_bf16(r, k, v, w, st, dy, ds, dr, dk, dv, ds_in, ws)
        outs.append((dr, dk, dv))
    done()
    for a, b, n in zip(*outs, ("dr", "dk", "dv")):
        changed = int((a != b).sum())
        assert changed == 0, (n, changed)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cuts", [(128,), (1,), (391,), (40, 168, 512), (899,)])
def test_outputs_of_a_chained_prefill(cuts, dtype):
    """A sequence in several calls, each from the state that the one before left: every output against the whole
    sequence in float64."""
    T = 900
    r, k, v, w, _, st, _ = inputs(1, T, 7, 35, dtype)
    want, want_s = ref.mix(r, k, v, w, st)
    mag, mag_s = ref.mix(r.abs(), k.abs(), v.abs(), w, st.abs())
    # float32 sums of T tokens and 64 channels, a handful of operations per chunk, and per call a join more
    n = (2 * T + 256 + 64 * len(cuts)) * 2.0 ** -24
    s, exact = st, st
    for a, b in zip((0,) + cuts, cuts + (T,)):
        part = [x[:, a:b].contiguous() for x in (r, k, v)]
        y, s = lib7.linattn_prefill(*part, w, s)
        tol = n * mag[:, a:b] + 1e-37
        if dtype == BF16:
            # half a step, 2^-8, of the result, of each product within the call and of the states that its chunks begin with
            tol = tol + 2.0 ** -8 * (want[:, a:b].abs() + ref.products(*part, w) + ref.state_products(*part, w, exact)) * (1 + 2.0 ** -6)
        bad = ~((y.double() - want[:, a:b]).abs() <= tol)
        count = int(bad.sum())
        assert count == 0, (a, b, count)
        _, exact = ref.mix(*part, w, exact)
    done()
    bad = ~((s.double() - want_s).abs() <= n * mag_s + 1e-37)
    assert not bool(bad.any())
