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


def test_norm_refuses_one_place_for_both_outputs():
    """xn and res_out hold different values: the same place is refused; either may be an input's place."""
    lib = moe.library()
    cfg = moe.Config(64, 256, 8, 2, 128).c()

    def norm(x, res, res_out, xn):
        return lib.moe_add_rmsnorm(cfg, x, res, 1 << 16, res_out, xn, None, None, None)

    assert norm(4096, 8192, 256, 256) == moe.MOE_ERR_INVALID_ARG
    assert norm(4096, 8192, 4096, 4096) == moe.MOE_ERR_INVALID_ARG
    assert norm(4096, None, 4096, 4096) == moe.MOE_ERR_INVALID_ARG
