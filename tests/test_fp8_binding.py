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


def test_extents_that_tiles_would_carry_past_an_int_are_refused():
    """Rounded up to whole tiles, rows, columns and weight rows must fit an int; rows lie less than 2^40 bytes apart."""
    lib, big, edge = moe.library(), 1 << 62, 0x7FFFFF00

    def gemm(rows=64, n=256, k=256, g=1, lda=None):
        return lib.moe_gemm_fp8(g, 256, rows, n, k, 256, lda or k, 256, 256, 256, 1, 256, 256, big, None)

    for call in (dict(rows=edge + 1), dict(n=edge + 1), dict(k=edge + 16), dict(n=edge // 2 + 1, g=2), dict(lda=1 << 40)):
        assert gemm(**call) == moe.MOE_ERR_UNSUPPORTED, call
    assert lib.moe_quantize_fp8(1, 1, 1, 1, edge + 1, 256, 256, 256, None) == moe.MOE_ERR_UNSUPPORTED
    assert lib.moe_quantize_fp8(1, 128, 1, 1, edge + 1, 256, 256, 256, None) == moe.MOE_ERR_UNSUPPORTED

    def ffn(cfg, rows, h, g=1, ldx=256):
        return lib.moe_expert_ffn_fp8(cfg.c(), g, 256, rows, 256, ldx, 256, 4096, 256, 8192, 256, 256, 256, h, 256, 256,
                                      big, None)

    many = moe.Config(edge + 64, 256, 1, 1, 16)
    assert ffn(many, edge + 1, 16) == moe.MOE_ERR_UNSUPPORTED
    assert ffn(many, 64, edge + 16) == moe.MOE_ERR_UNSUPPORTED
    assert ffn(many, 64, 16, ldx=1 << 40) == moe.MOE_ERR_UNSUPPORTED
    w = moe.MoeWeightsFp8(*[256 * (i + 1) for i in range(len(moe.MoeWeightsFp8._fields_))])
    for cfg in (many, moe.Config(edge // 3 + 1, 128, 2, 2, 16)):
        assert lib.moe_layer_forward_fp8(cfg.c(), w, 256, None, None, 256, None, None, 256, big,
                                         None) == moe.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("n,k", [(0x7FFFFFFF, 128), (128, 0x7FFFFFFF)])
def test_workspace_sizes_of_the_largest_extents(n, k):
    assert moe.library().moe_workspace_size_gemm_fp8(1, 1, n, k) % 256 == 0
    assert 1024 <= moe.library().moe_workspace_size_gemm_fp8(1, 1, n, k) < 1 << 40


def test_tiling_of_a_product():
    """The documented rule: groups averaging 256 rows are wide; few tiles get smaller or are cut."""
    tiling = moe.moe_gemm_fp8_tiling
    assert tiling(False, 1, False, 8192, 4096, 7168) == (True, 256, 1)
    assert tiling(True, 256, True, 65536, 2048, 7168) == (True, 256, 1)
    assert tiling(True, 256, True, 65535, 2048, 7168) == (False, 256, 1)
    wide, rows, parts = tiling(False, 1, False, 1, 4096, 7168)
    assert not wide and parts > 1
    assert tiling(False, 1, False, 200, 2048, 7168) == (False, 32, 1)
    for bad in ((False, 0, True, 1, 16, 16), (False, 2, False, 1, 16, 16), (False, 1, False, 0, 16, 16),
                (False, 1, False, 1, 0, 16), (False, 1, False, 1, 16, 0), (True, 1025, True, 1, 16, 16)):
        with pytest.raises(moe.MoEError):
            tiling(*bad)
    assert moe.library().moe_gemm_fp8_tiling(0, 1, 0, 1, 16, 16, None) == moe.MOE_ERR_INVALID_ARG
