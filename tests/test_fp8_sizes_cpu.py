"""Sizes past 32 bits are refused by the binding, not cut to their lowest bits (tensors without memory)."""
import pytest
import torch

import gated_deltanet_03_b200 as g

F8, BF, F32, I32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32
BIG = 2 ** 32 + 16


def t(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device="meta")


def step(B=3, Hk=1, Hv=2, slots=5):
    return dict(q=t(B, Hk, 128), k=t(B, Hk, 128), v=t(B, Hv, 128), a=t(B, Hv), b=t(B, Hv), A_log=t(Hv, dtype=F32), dt_bias=t(Hv, dtype=F32),
                state_pool=t(slots, Hv, 128, 128, dtype=F32), slots=t(B, dtype=I32))


@pytest.mark.parametrize("call", [
    lambda: g.fp8_quantize_act(t(BIG, 16)),
    lambda: g.fp8_quantize_weight(t(16, BIG)),
    lambda: g.fp8_gemm(t(BIG, 16, dtype=F8), t(BIG, 1, dtype=F32), t(16, 16, dtype=F8), t(1, 1, dtype=F32)),
    lambda: g.fp8_gemm(t(1, 16, dtype=F8), t(1, 1, dtype=F32), t(BIG, 16, dtype=F8), t(BIG // 128 + 1, 1, dtype=F32)),
    lambda: g.gdn_gated_rmsnorm_silu_fp8(t(BIG, 1, 128), t(BIG, 1, 128), t(128, dtype=F32)),
    lambda: g.gdn_decode_step_pooled(**step(slots=BIG)),
    lambda: g.gdn_decode_step_pooled(**step(B=BIG)),
    lambda: g.gdn_decode_step_pooled_gated_fp8(**step(slots=BIG), z=t(3, 2, 128), norm_weight=t(128, dtype=F32)),
    lambda: g.gdn_short_conv1d_silu_decode_pooled(t(BIG, 64), t(64, 4, dtype=F32), t(5, 3, 64), t(BIG, dtype=I32)),
    lambda: g.gdn_short_conv1d_silu_decode_pooled(t(3, 64), t(64, 4, dtype=F32), t(BIG, 3, 64), t(3, dtype=I32)),
])
def test_sizes_past_32_bits_are_refused(call):
    with pytest.raises(ValueError, match="more than the library takes"):
        call()
