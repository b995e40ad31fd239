"""The layer norm's gradients over vectors too long for registers and many rows: the workspace that the sums over the rows
need stays near the size of what they give, and the sums are right and repeat bit for bit."""

import pytest
import torch

import rwkv_delta_rule_b200 as lib7
from test_parity_gpu_layer_norm import check, inputs

F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("G,D", [(1, 1 << 24), (256, 65536), (1, 1 << 20), (3, 70001), (1, 16384), (1, 9001)])
def test_workspace_of_long_vectors(G, D, bf16):
    """dweight and dbias, 8 bytes a channel, once per row block: as many of those as fill the device eight times (8 CTAs of
    256 columns on each of 148 SMs), and one in any case."""
    tiles = -(-G * D // 256)
    most = 8 * G * D * max(1, -(-148 * 8 * 8 // tiles))
    for M in (1, 7, 300, 100000):
        n = lib7.rwkv7_layer_norm_workspace(bf16, M, G, D)
        assert 8 * G * D <= n <= min(most, 8 * G * D * M), (M, n)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,G,D", [(300, 1, 16384), (700, 1, 9001), (37, 3, 20000), (513, 1, 12288), (9, 1, 400000), (2000, 1, 8448)])
def test_gradients_of_long_vectors(M, G, D, dtype):
    x, dy, w, b = inputs(M, G, D, dtype, M + D)
    y, mean, rstd = lib7.layer_norm(x, w, b)
    grads = [lib7.layer_norm_backward(dy, x, w, mean, rstd) for _ in range(3)]
    torch.cuda.synchronize()
    check(x, dy, w, b, 1e-5, y, mean, rstd, *grads[0])
    for again in grads[1:]:
        assert all(torch.equal(a, c) for a, c in zip(again, grads[0]))
