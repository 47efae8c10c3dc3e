"""The e4m3 entry points without a GPU: workspace sizes, and bad arguments
refused on the host before anything is launched."""
import ctypes

import pytest

import sparse_mixture_experts_rmsnorm_b200 as moe

BAD, UNSUPPORTED, WORKSPACE = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE
BIG = 1 << 40
lib = moe.library()


def _cfg(**kw):
    base = dict(n_tokens=64, d_model=256, n_experts=8, top_k=2, d_ff=128)
    base.update(kw)
    return moe.Config(**base)


def test_workspace_size_holds_the_documented_regions():
    c = _cfg(n_tokens=1000, d_model=512, n_experts=16, top_k=4, d_ff=384, d_ff_shared=256)
    N, d, E, k, H = 1000, 512, 16, 4, 384
    R = N * k
    need = N * d * 2 + N * d + N * 4 * 4 + N * E * 4 + 4 * N * k * 4 + R * d + R * 4 * 4 + R * H + R * 3 * 4 + \
        R * d * 2 + N * d * 2
    size = lib.moe_workspace_size_fp8(c.c())
    assert need <= size <= need + 64 * 1024 and size % 256 == 0
    # a shared expert as wide as the routed ones: N more rows of activations and outputs, no y_shared
    f = _cfg(n_tokens=1000, d_model=512, n_experts=16, top_k=4, d_ff=384, d_ff_shared=384)
    assert lib.moe_workspace_size_fp8(f.c()) > size - N * d * 2
    assert lib.moe_workspace_size_fp8(_cfg(top_k=9).c()) == 0
    assert lib.moe_workspace_size_gemm_fp8(1, 64, 256, 256) >= 256
    for bad in ((0, 64, 256, 256), (1025, 64, 256, 256), (1, -1, 256, 256), (1, 64, 0, 256), (1, 64, 256, 0)):
        assert lib.moe_workspace_size_gemm_fp8(*bad) == 0
    with pytest.raises(moe.MoEError):
        moe.workspace_gemm_fp8(0, 64, 256, 256)
    with pytest.raises(moe.MoEError):
        moe.workspace_fp8(_cfg(top_k=9))


def test_few_tiles_have_room_for_their_parts():
    """Partial sums of products with few tiles; none where the tiles alone fill the GPU."""
    size = lib.moe_workspace_size_gemm_fp8
    assert size(1, 1, 4096, 7168) > 1 << 20
    assert size(1, 8192, 4096, 7168) == 1024 == size(64, 9000, 2048, 7168)
    assert size(1, 1, 4096, 128) == 1024  # a single block along K is not cut


def test_norm_refusals():
    def norm(cfg=None, x=256, res=None, w=256, res_out=256, xn=256, q=None, s=None):
        return lib.moe_add_rmsnorm(ctypes.byref((cfg or _cfg()).c()), x, res, w, res_out, xn, q, s, None)

    assert norm(cfg=_cfg(top_k=9)) == BAD
    assert norm(x=None) == BAD and norm(w=None) == BAD
    assert norm(q=256) == BAD and norm(s=256) == BAD
    assert norm(res_out=None, xn=None) == BAD
    assert norm(cfg=_cfg(d_model=49168)) == UNSUPPORTED
    assert norm(cfg=_cfg(n_tokens=0), x=None, w=None) == moe.MOE_OK


def test_quantize_refusals():
    def quant(dtype=1, br=1, m=1, r=4, c=8, x=256, q=256, s=256):
        return lib.moe_quantize_fp8(dtype, br, m, r, c, x, q, s, None)

    assert quant(dtype=2) == BAD and quant(br=64) == BAD and quant(br=0) == BAD
    assert quant(m=-1) == BAD and quant(r=-1) == BAD and quant(c=0) == BAD
    assert quant(x=None) == BAD and quant(q=None) == BAD and quant(s=None) == BAD
    assert quant(r=0, x=None) == moe.MOE_OK and quant(m=0, x=None) == moe.MOE_OK


def test_gemm_refusals():
    def gemm(g=1, offs=None, rows=64, n=256, k=256, a=256, sa=256, b=256, sb=256, t=1, c=256, ws=256, bytes=BIG, lda=None):
        return lib.moe_gemm_fp8(g, offs, rows, n, k, a, k if lda is None else lda, sa, b, sb, t, c, ws, bytes, None)

    assert gemm(g=2) == BAD and gemm(g=0, offs=256) == BAD and gemm(g=1025, offs=256) == BAD
    assert gemm(rows=-1) == BAD and gemm(n=0) == BAD and gemm(k=0) == BAD and gemm(t=2) == BAD
    for p in ("a", "sa", "b", "sb", "c", "ws"):
        assert gemm(**{p: None}) == BAD, p
    assert gemm(ws=128) == BAD
    assert gemm(k=264) == UNSUPPORTED and gemm(a=264) == UNSUPPORTED and gemm(b=257) == UNSUPPORTED
    assert gemm(lda=240) == BAD and gemm(lda=264) == UNSUPPORTED
    assert gemm(g=1024, offs=256, n=1 << 22) == UNSUPPORTED
    assert gemm(bytes=1023) == WORKSPACE
    assert gemm(rows=0, a=None, sa=None, b=None, sb=None, c=None) == moe.MOE_OK


def test_ffn_refusals():
    PTRS = ("x", "x_scale", "w_gate", "w_gate_scale", "w_up", "w_up_scale", "w_down", "w_down_scale", "y")

    def ffn(cfg=None, ldx=256, g=1, offs=None, rows=64, h=128, ws=256, bytes=BIG, **null):
        p = {n: 256 for n in PTRS}
        p.update(null)
        return lib.moe_expert_ffn_fp8(ctypes.byref((cfg or _cfg()).c()), g, offs, rows, p["x"], ldx, *(p[n] for n in PTRS[1:-1]), h,
                                      p["y"], ws, bytes, None)

    assert ffn(cfg=_cfg(top_k=9)) == BAD and ffn(ws=None) == BAD and ffn(ws=128) == BAD
    assert ffn(g=2) == BAD and ffn(g=0) == BAD and ffn(rows=-1) == BAD and ffn(h=0) == BAD
    for n in PTRS:
        assert ffn(**{n: None}) == BAD, n
    assert ffn(cfg=_cfg(d_model=264)) == UNSUPPORTED and ffn(cfg=_cfg(d_ff=136)) == UNSUPPORTED
    assert ffn(h=24) == UNSUPPORTED and ffn(w_up=264) == UNSUPPORTED
    assert ffn(ldx=240) == BAD and ffn(ldx=264) == UNSUPPORTED
    assert ffn(bytes=256) == WORKSPACE
    assert ffn(rows=100000) == WORKSPACE
    assert ffn(h=16, rows=1024) == WORKSPACE  # the codes fit, their scales do not
    assert ffn(rows=0) == moe.MOE_OK


def test_layer_refusals():
    def layer(cfg=None, weights=None, h=256, out=256, ws=256, bytes=BIG, **null):
        w = moe.MoeWeightsFp8()
        for n, _ in moe.MoeWeightsFp8._fields_:
            setattr(w, n, null.get(n, 256))
        return lib.moe_layer_forward_fp8(ctypes.byref((cfg or _cfg()).c()), weights or ctypes.byref(w), h, None, None,
                                         out, None, None, ws, bytes, None)

    assert layer(cfg=_cfg(top_k=9)) == BAD and layer(h=None) == BAD and layer(out=None) == BAD and layer(ws=None) == BAD
    for n, _ in moe.MoeWeightsFp8._fields_:
        cfg = _cfg(d_ff_shared=64)
        assert layer(cfg=cfg, **{n: None}) == BAD, n
    assert layer(cfg=_cfg(d_model=264)) == UNSUPPORTED and layer(cfg=_cfg(d_ff_shared=72)) == UNSUPPORTED
    assert layer(w_down=264) == UNSUPPORTED and layer(cfg=_cfg(d_ff_shared=64), ws_up=264) == UNSUPPORTED
    assert layer(bytes=1024) == WORKSPACE
    assert lib.moe_layer_forward_fp8(ctypes.byref(_cfg().c()), None, 256, None, None, 256, None, None, 256, BIG,
                                     None) == BAD


def test_gate_and_up_must_be_two_places_within_reach():
    """Gate and up are one view with their distance as a stride of at most 40 bits."""
    def ffn(gate, up):
        return lib.moe_expert_ffn_fp8(ctypes.byref(_cfg().c()), 1, None, 64, 256, 256, 256, gate, 256, up, 256, 256,
                                      256, 128, 256, 256, BIG, None)

    def layer(gate, up, s_gate, s_up):
        w = moe.MoeWeightsFp8()
        for n, _ in moe.MoeWeightsFp8._fields_:
            setattr(w, n, 256)
        w.w_gate, w.w_up, w.ws_gate, w.ws_up = gate, up, s_gate, s_up
        return lib.moe_layer_forward_fp8(ctypes.byref(_cfg(d_ff_shared=64).c()), ctypes.byref(w), 256, None, None, 256,
                                         None, None, 256, BIG, None)

    assert ffn(4096, 4096) == UNSUPPORTED
    assert ffn(4096, 4096 + (1 << 40)) == UNSUPPORTED and ffn(4096 + (1 << 40), 4096) == UNSUPPORTED
    assert layer(4096, 4096, 4096, 8192) == UNSUPPORTED
    assert layer(4096, 8192, 4096, 4096) == UNSUPPORTED
    assert layer(4096, 8192, 4096, 4096 + (1 << 40)) == UNSUPPORTED


def test_python_wrapper_refuses_strided_tensors():
    import torch
    x = torch.zeros(4, 64)[:, ::2]
    with pytest.raises(ValueError):
        moe.moe_quantize_fp8("f32", 1, 1, 4, 32, x, None, None, stream=0)
    with pytest.raises(ValueError):  # columns apart; rows may be
        moe.moe_gemm_fp8(1, None, 4, 32, 32, x, None, None, None, "f32", None, torch.zeros(256), stream=0)
    with pytest.raises(KeyError):
        moe.moe_quantize_fp8("f16", 1, 1, 4, 32, None, None, None, stream=0)
