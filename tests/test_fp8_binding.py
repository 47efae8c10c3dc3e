"""Row operands that the e4m3 calls' Python binding refuses, without a GPU."""
import pytest

import sparse_mixture_experts_rmsnorm_b200 as moe


def test_row_operands_that_are_too_narrow_or_not_of_codes():
    import torch
    codes = torch.zeros(4, 64, dtype=torch.uint8)
    ws = torch.zeros(256, dtype=torch.uint8)
    cfg = moe.Config(4, 128, 1, 1, 16)

    def gemm(a, k):
        moe.moe_gemm_fp8(1, None, 4, 32, k, a, None, None, None, "f32", None, ws, stream=0)

    def ffn(x):
        moe.moe_expert_ffn_fp8(cfg, 1, None, 4, x, None, None, None, None, None, None, None, 16, None, ws, stream=0)

    for call in (lambda: gemm(codes, 128), lambda: gemm(codes[:, :32], 64), lambda: ffn(codes)):
        with pytest.raises(ValueError, match="columns"):
            call()
    for wrong in (codes.bfloat16(), codes.bfloat16()[:, :32]):
        with pytest.raises(ValueError, match="one-byte"):
            gemm(wrong, 32)
