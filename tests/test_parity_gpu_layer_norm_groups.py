"""GPU: the layer norm's gradients over every number of groups, the ones among them that leave lanes of a CTA
without a group: the sums over the rows against float64, and the same bits from repeated calls.  Bounds as for the
other shapes (test_parity_gpu_layer_norm.check)."""

import pytest
import torch

import rwkv_delta_rule_b200 as lib7
from test_parity_gpu_layer_norm import check, inputs

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def both_ways(M, G, D, dtype, repeats):
    x, dy, w, b = inputs(M, G, D, dtype, 1000 * G + D + M)
    y, mean, rstd = lib7.layer_norm(x, w, b)
    grads = [lib7.layer_norm_backward(dy, x, w, mean, rstd) for _ in range(1 + repeats)]
    torch.cuda.synchronize()
    check(x, dy, w, b, 1e-5, y, mean, rstd, *grads[0])
    for again in grads[1:]:
        for a, c in zip(again, grads[0]):
            assert torch.equal(a, c), (M, G, D)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M", [1, 2, 3001])
def test_every_number_of_heads(M, dtype):
    for G in range(1, 65):
        both_ways(M, G, 64, dtype, 2)


# D = 16 and 30: many units per CTA, whole pieces and odd ones
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,groups", [(96, range(4, 18)), (128, range(4, 18)), (256, range(3, 18)), (16, (33, 47, 63, 65, 100, 127)),
                                      (30, (9, 15, 17, 23, 31, 33)), (33, (5, 6, 7, 9, 13))])
def test_groups_of_other_widths(D, groups, dtype):
    for G in groups:
        for M in (1, 1777):
            both_ways(M, G, D, dtype, 2)


# float32 D = 64: 16 units, so idle ones share a warp with units that have rows where G is odd; bf16: 32 units
@pytest.mark.parametrize("dtype,G,D", [(F32, 9, 64), (F32, 12, 64), (F32, 15, 64), (BF16, 17, 64), (BF16, 18, 64), (BF16, 25, 64),
                                       (BF16, 31, 64), (F32, 5, 128), (F32, 6, 128), (BF16, 5, 256), (BF16, 6, 256),
                                       (F32, 4, 64), (BF16, 12, 64), (BF16, 2, 72)])
def test_repeats_bit_for_bit(dtype, G, D):
    """Sums in a fixed order, with one unit per group in a CTA and with several."""
    both_ways(5003, G, D, dtype, 30)
