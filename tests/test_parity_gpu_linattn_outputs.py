"""GPU: what the outputs of the head-decay linear attention do not depend on: whether the state's gradient is asked
for."""

import pytest
import torch

import rwkv_delta_rule_b200 as lib7
from test_parity_gpu_linattn import done, inputs

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


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
