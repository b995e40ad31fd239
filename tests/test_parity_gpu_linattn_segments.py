"""GPU: the states of a sequence that is split into segments are as near to float64 as those of the whole sequence.

What a head's results may be off by, as a part of their norm: a token rounds each element of the state twice (its product and
the sum), by at most 2^-24 of it and independently, so by 2^-24 / sqrt(3) on average; w^t of a rounding is left t tokens
later, so sqrt(2 M / 3) 2^-24 with M = sum_t w^2t in all, and over the 4096 elements of a state this average hardly
varies: twice as much is allowed.  Reading a state (64 products and their sum), the powers and the joins add what does
not grow with the length: 16 x 2^-24.  A power of w that is off by one rounding and used n times would add n times
that in one direction, which is what this is about."""

import pytest
import torch

import linattn_ref as ref
import rwkv_delta_rule_b200 as lib7
from helpers import need_cuda

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
STEP = 2.0 ** -24


# one decay per memory of 32 to 4096 tokens, and one a good deal longer
def decays(H):
    w = 1 - torch.exp2(-5 - 7 * torch.arange(H, dtype=torch.float64) / max(1, H - 2))
    w[-1] = 1 - 1.1e-5
    return w.float().cuda()


def rel(a, b):
    """Per head, heads in dimension 0."""
    return ((a.double() - b).flatten(1).norm(dim=1) / b.flatten(1).norm(dim=1)).cpu()


# float32: 10, 4, 129 and 518 segments; bf16 on the tensor cores: 3 (joined by the pass itself), 37, 148
@pytest.mark.parametrize("dtype,B,T,H", [(F32, 8, 4096, 12), (F32, 4, 8192, 64), (F32, 1, 5000, 8), (F32, 1, 16384, 2),
                                         (BF16, 8, 4096, 12), (BF16, 1, 8192, 8), (BF16, 1, 20000, 2)])
def test_segments_keep_the_precision(dtype, B, T, H):
    need_cuda()
    g = torch.Generator(device="cuda").manual_seed(T + H)
    r, k, v = ((torch.randn(B, T, H, 64, generator=g, device="cuda") * s).to(dtype) for s in (1, 0.125, 1))
    w = decays(H)
    want_y, want_s = ref.mix(r, k, v, w)
    assert lib7.rwkv7_linattn_workspace(B, T, H) > 0
    y, s = lib7.linattn_prefill(r, k, v, w)
    torch.cuda.synchronize()
    assert lib7.rwkv7_get_last_error() == 0
    w = w.double().cpu()
    M = (1 - w ** (2 * T)) / (1 - w ** 2)
    tol = 2 * STEP * torch.sqrt(2 * M / 3) + 16 * STEP
    off = rel(s.transpose(0, 1), want_s.transpose(0, 1))
    assert bool((off <= tol).all()), ("state", float((off / tol).max()))
    if dtype == F32:
        off = rel(y.transpose(0, 2), want_y.transpose(0, 2))
        assert bool((off <= tol).all()), ("y", float((off / tol).max()))


@pytest.mark.parametrize("max_T", [0, 20, 5000])
def test_ragged_batch_without_tokens(max_T):
    """Rows of no tokens at all leave the states as they are, whatever max_T and the workspace would allow."""
    need_cuda()
    B, H = 3, 2
    e = torch.empty(0, H, 64, dtype=BF16, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    st = torch.randn(B, H, 64, 64, device="cuda")
    w = torch.full((H,), 0.5, device="cuda")
    _, s = lib7.linattn_prefill_varlen(cu, max_T, e, e, e, w, st)
    _, z = lib7.linattn_prefill_varlen(cu, max_T, e, e, e, w)
    torch.cuda.synchronize()
    assert torch.equal(s, st) and not bool(z.any())
