"""A required tensor left out (None) is refused with a ValueError that names it, as by the other entry points."""

import pytest
import torch

import rwkv_delta_rule_b200 as lib7
from helpers import need_cuda


def test_first_tensor():
    x = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    calls = [
        lambda: lib7.rwkv7_linattn_prefill(None, x, x, x, None, x, x),
        lambda: lib7.rwkv7_linattn_prefill_bf16(None, x, x, x, None, x, x),
        lambda: lib7.rwkv7_linattn_prefill_varlen_bf16(cu, 2, None, x, x, x, None, x, x),
        lambda: lib7.rwkv7_linattn_decode(None, x, x, x, x, x),
        lambda: lib7.rwkv7_linattn_decode_bf16(None, x, x, x, x, x),
        lambda: lib7.rwkv7_linattn_backward_bf16(None, x, x, x, None, x, None, x, x, x, None),
        lambda: lib7.linattn_prefill(None, x, x, x),
        lambda: lib7.linattn_prefill_varlen(cu, 2, None, x, x, x),
        lambda: lib7.linattn_decode_(None, x, x, x, x),
        lambda: lib7.linattn_decode_(None, x, x, x, x, x),
        lambda: lib7.linattn_backward(None, x, x, x, x),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="r is required"):
            call()
    for call in (lambda: lib7.rwkv7_layer_norm(None, x, x, 1e-5, x), lambda: lib7.rwkv7_layer_norm_bf16(None, x, x, 1e-5, x),
                 lambda: lib7.rwkv7_layer_norm_backward(x, None, x, x, x, x),
                 lambda: lib7.rwkv7_layer_norm_backward_bf16(x, None, x, x, x, x),
                 lambda: lib7.layer_norm(None), lambda: lib7.layer_norm_backward(x, None, x, x, x)):
        with pytest.raises(ValueError, match="x is required"):
            call()


def test_offsets():
    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="cu_seqlens is required"):
        lib7.linattn_prefill_varlen(None, 2, x, x, x, x)
    with pytest.raises(ValueError, match="cu_seqlens"):
        lib7.linattn_prefill_varlen(torch.zeros(0, dtype=torch.int32), 2, x, x, x, x)
    with pytest.raises(ValueError, match="cu_seqlens"):
        lib7.rwkv7_linattn_prefill_varlen_bf16(torch.zeros(1, 3, dtype=torch.int32), 2, x, x, x, x, None, x, x)


def test_other_tensors():
    # the check itself: the calls reach it with tensors of a CUDA device only
    with pytest.raises(ValueError, match="k is required"):
        lib7._fits(None, "k", torch.bfloat16, (1, 2, 1, 64), torch.device("cuda", 0))
    assert lib7._fits_or_none(None, "s_in", torch.float32, (1, 1, 64, 64), torch.device("cuda", 0)) is None


@pytest.mark.gpu
def test_calls_on_the_device():
    need_cuda()
    x = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    w, s = torch.ones(1, device="cuda"), torch.zeros(1, 1, 64, 64, device="cuda")
    cu = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    m, st = torch.zeros(2, 64, device="cuda"), torch.zeros(2, device="cuda")
    for name, call in (("k", lambda: lib7.linattn_prefill(x, None, x, w)), ("w", lambda: lib7.linattn_prefill(x, x, x, None)),
                       ("s_out", lambda: lib7.rwkv7_linattn_prefill_bf16(x, x, x, w, None, x, None)),
                       ("v", lambda: lib7.linattn_prefill_varlen(cu, 2, x[0], x[0], None, w)),
                       ("cu_seqlens", lambda: lib7.rwkv7_linattn_prefill_varlen_bf16(None, 2, x[0], x[0], x[0], w, None, x[0], s)),
                       ("s_inout", lambda: lib7.linattn_decode_(x[:, 0], x[:, 0], x[:, 0], w, None)),
                       ("dy", lambda: lib7.linattn_backward(x, x, x, w, None)),
                       ("dy", lambda: lib7.layer_norm_backward(None, m, None, st, st)),
                       ("rstd", lambda: lib7.layer_norm_backward(m, m, None, st, None))):
        with pytest.raises(ValueError, match=name + " is required"):
            call()
