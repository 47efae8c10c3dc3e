"""The tilings of the e4m3 products that only larger calls take, against plain 64-bit forms.

A call with more tiles than SM pairs takes 256 rows of a group on the MMA's M side (wide) where its groups average
256 rows or more, else chunks of up to 256 rows on the N side (swapped); calls of fewer tiles are covered elsewhere.
Each case asserts the tiling that it is meant for, so that another rule cannot leave a tiling without its cases.

Tolerances are those of the other e4m3 tests.  For the FFN: an fp32 error of about 1e-6 of an activation moves its code
one step with a probability of at most 1e-4 (1e-6 of the value against half a step of 2^-4 of it, on both sides and with
room for sums that cancel), so of rows of h activations a share of h / 10^4 at most has a moved code on average (twice
that is allowed), and for h = 2560 more than five are in one row with a probability below 10^-6: five steps are allowed.
"""
import pytest

import fp8_helpers as f8
from test_gpu_fp8 import (HALF, LAYERS, U32, _close, _ffn_want, _layer_case, _layer_want, _offsets, _operands, _type,
                          env)  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def _ordered(torch, first, second, swap):
    """Copies of two weight stacks in one buffer, the second in front where swap is set."""
    both = torch.empty(2, *first.shape, dtype=torch.uint8, device="cuda").view(f8.E4M3)
    both[int(swap)], both[1 - int(swap)] = first, second
    return both[int(swap)], both[1 - int(swap)]


def _run(torch, moe, sizes, spare, x, xs, gq, gs, uq, us, dq, ds, out, repeats=1):
    """The FFN's results; every repeat has the same bits and leaves the rows behind the last group as they were."""
    g, rows, d, h = len(sizes), sum(sizes), x.shape[1], gq.shape[1]
    cfg = moe.Config(rows + spare, d, g, 1, h, dtype=out)
    ws = moe.workspace_fp8(cfg)
    first = None
    for _ in range(repeats):
        y = torch.full((rows + spare, d), 7.0, dtype=_type(torch, out), device="cuda")
        moe.moe_expert_ffn_fp8(cfg, g, _offsets(torch, sizes), rows + spare, x, xs, gq, gs, uq, us, dq, ds, h, y, ws)
        first = y if first is None else first
        assert torch.equal(y, first)
    assert torch.all(first[rows:] == 7.0)
    assert moe.moe_check_device_error(ws)[0] == 0
    return first[:rows]


def _check_codes(torch, moe, sizes, d, h, swap=False, repeats=1):
    """The activation's codes and scales themselves: each column of the down projection picks one hidden unit, so a
    result is a code times its scale."""
    g, rows, spare = len(sizes), sum(sizes), 5
    x, xs, gq, gs = _operands(torch, sizes + [spare], h, d, g)
    _, _, uq, us = _operands(torch, [1], h, d, g)
    gq, uq = _ordered(torch, gq, uq, swap)
    unit = (torch.arange(d, device="cuda") * h // d + torch.arange(d, device="cuda") % max(1, h // d)) % h
    dq = torch.zeros(g, d, h, device="cuda")
    dq[:, torch.arange(d), unit] = 1.0
    ds = torch.ones(g, f8.blocks(d), f8.blocks(h), device="cuda")
    y = _run(torch, moe, sizes, spare, x, xs, gq, gs, uq, us, dq.to(f8.E4M3), ds, "f32", repeats).double()
    xv = f8.values(x, xs, 1)
    zg, mg = f8.product(xv, f8.values(gq, gs, 128), sizes)
    zu, mu = f8.product(xv, f8.values(uq, us, 128), sizes)
    act = (zg * torch.sigmoid(zg) * zu)[:rows]
    # silu's slope is below 1.1, and each product is off by at most 2^-24 (d + 32) of its absolute sum
    slack = (1.1 * mg * zu.abs() + mu * zg.abs())[:rows] * 2.0 ** -24 * (d + 32) + act.abs() * 2.0 ** -20
    step = f8.spread(f8.block_scales(act, 1), rows, h, 1) * 2.0 ** -10
    half = torch.maximum(act.abs() * 2.0 ** -4, step)
    err = (y - act[:, unit]).abs()
    assert torch.all(err <= ((half + slack) * (1 + 2.0 ** -16))[:, unit])
    scale = f8.block_scales(act, 1)[:, unit // 128]
    # and every value is a code times the scale, which is off by the slack of its block's largest
    code = y / scale
    off = (code - f8.e4m3_round(code)).abs() / code.abs().clamp_min(2.0 ** -6)
    worst = f8.spread(f8.block_scales(slack, 1), rows, h, 1)[:, unit] / scale
    assert torch.all(off <= worst + 2.0 ** -20)


def test_wide_ffn_of_one_block_along_k_with_tiles_whose_last_rows_are_missing(env):
    """d_model 128: every tile is one k-block, and tiles that lack a warp's rows lie between tiles that have them, so
    the rows' largest magnitudes pass between the warps with nothing but their own barrier to order them."""
    torch, moe = env
    _check_codes(torch, moe, [270, 256, 300, 0, 520, 257, 512, 269], 128, 2048, repeats=8)


@pytest.mark.parametrize("rows,n,k", [(1, 512, 8192), (24, 1024, 7168), (5, 2000, 16384)])
def test_parts_of_every_column_meet_in_order(env, rows, n, k):
    """Tiles cut along K, both CTAs of a pair holding columns of each: the operands are small whole numbers whose sums are
    exact, so every result has the sum of all parts and nothing else, call after call on changing operands."""
    torch, moe = env
    assert moe.library().moe_workspace_size_gemm_fp8(1, rows, n, k) > 4096  # parts are held
    ws = moe.workspace_gemm_fp8(1, rows, n, k)
    sa, sb = torch.ones(rows, f8.blocks(k), device="cuda"), torch.ones(1, f8.blocks(n), f8.blocks(k), device="cuda")
    c = torch.empty(rows, n, device="cuda")
    for i in range(50):
        a = torch.randint(-2, 3, (rows, k), device="cuda").float()
        b = torch.randint(-2, 3, (1, n, k), device="cuda").float()
        moe.moe_gemm_fp8(1, None, rows, n, k, a.to(f8.E4M3), sa, b.to(f8.E4M3), sb, "f32", c, ws)
        assert torch.equal(c.double(), a.double() @ b[0].double().T), i  # |sums| <= 4 k < 2^24
    assert moe.moe_check_device_error(ws)[0] == 0


# ---------------------------------------------------------------- more tiles than SM pairs
RAGGED = [300, 0, 520, 257, 400]                # wide: averages above 256 with the spare rows, an empty group
FULL = [256, 512, 257, 255, 256]
BELOW = [200, 255, 130, 180, 250, 193, 224, 1]  # swapped: chunks of 131 to 256 rows
ONE_LARGE = [3, 600, 0, 40, 257, 33]            # swapped, groups of several chunks
SPARE = 9                                       # rows of the buffers behind the last group


def _tiling(moe, swiglu, sizes, n, k, spare=SPARE, offsets=True):
    """(wide, most rows of a tile); these calls cut nothing along K."""
    wide, rows, parts = moe.moe_gemm_fp8_tiling(swiglu, len(sizes), offsets, sum(sizes) + spare, n, k)
    assert parts == 1
    return wide, rows


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,wide", [(RAGGED, True), (FULL, True), (BELOW, False), (ONE_LARGE, False)])
@pytest.mark.parametrize("n,k", [(4097, 144), (4112, 256), (4100, 400), (4097, 16), (4104, 1280)])
def test_grouped_product_of_many_tiles(env, out, sizes, wide, n, k):
    """Results that are whole 16-byte pieces and others, K in whole blocks and not; rows before the buffer, behind the
    last group and behind the buffer stay as they were."""
    torch, moe = env
    assert _tiling(moe, False, sizes, n, k) == (wide, 256)
    g, rows = len(sizes), sum(sizes)
    aq, as_, bq, bs = _operands(torch, sizes + [SPARE], n, k, g)
    want, mag = f8.product(f8.values(aq, as_, 1), f8.values(bq, bs, 128), sizes)
    band = torch.full((rows + SPARE + 2, n), 7.0, dtype=_type(torch, out), device="cuda")
    c = band[1:-1]
    ws = moe.workspace_gemm_fp8(g, rows + SPARE, n, k)
    moe.moe_gemm_fp8(g, _offsets(torch, sizes), rows + SPARE, n, k, aq, as_, bq, bs, out, c, ws)
    _close(c[:rows], want[:rows], mag[:rows] * U32 * (k + 32), out)
    assert torch.all(band[0] == 7.0) and torch.all(c[rows:] == 7.0) and torch.all(band[-1] == 7.0)
    assert moe.moe_check_device_error(ws)[0] == 0
    again = torch.full_like(c, 7.0)
    moe.moe_gemm_fp8(g, _offsets(torch, sizes), rows + SPARE, n, k, aq, as_, bq, bs, out, again, ws)
    assert torch.equal(again, c)


@pytest.mark.parametrize("sizes,wide", [(RAGGED, True), (BELOW, False)])
def test_nan_rows_of_large_tiles_stay_among_themselves(env, sizes, wide):
    """Also those that a tile leaves in shared memory where the next tile has no rows."""
    torch, moe = env
    n, k, g, rows = 4104, 384, len(sizes), sum(sizes)
    assert _tiling(moe, False, sizes, n, k) == (wide, 256)
    aq, as_, bq, bs = _operands(torch, sizes + [SPARE], n, k, g)
    bad = torch.arange(rows + SPARE, device="cuda") % 5 == 3
    bad[rows:] = True
    aq.view(torch.uint8)[bad] = 0x7F
    as_[torch.arange(rows + SPARE, device="cuda") % 10 == 3] = float("inf")
    want, mag = f8.product(f8.values(aq, as_, 1), f8.values(bq, bs, 128), sizes)
    c = torch.empty(rows + SPARE, n, device="cuda")
    moe.moe_gemm_fp8(g, _offsets(torch, sizes), rows + SPARE, n, k, aq, as_, bq, bs, "f32", c,
                     moe.workspace_gemm_fp8(g, rows + SPARE, n, k))
    good = ~bad[:rows]
    assert not torch.isfinite(c[:rows][bad[:rows]]).any()
    _close(c[:rows][good], want[:rows][good], mag[:rows][good] * U32 * (k + 32), "f32")


@pytest.mark.parametrize("swap", [False, True])
@pytest.mark.parametrize("sizes,wide,d,h", [(RAGGED, True, 256, 2064), (FULL, True, 272, 2048), (BELOW, False, 256, 2064),
                                            (ONE_LARGE, False, 144, 2304)])
def test_activation_codes_of_many_tiles(env, swap, sizes, wide, d, h):
    """Both orders of gate and up in memory, hidden units that end inside a block of 128."""
    torch, moe = env
    assert _tiling(moe, True, sizes, h, d, spare=5) == (wide, 256)
    _check_codes(torch, moe, sizes, d, h, swap)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,wide,d,h", [(RAGGED, True, 2320, 2064), (FULL, True, 2560, 2048),
                                            (BELOW, False, 2320, 2064), (ONE_LARGE, False, 2560, 2064)])
def test_ffn_of_many_tiles(env, out, sizes, wide, d, h):
    """Both products in the tiling."""
    torch, moe = env
    spare, g, rows = 5, len(sizes), sum(sizes)
    assert _tiling(moe, True, sizes, h, d, spare) == _tiling(moe, False, sizes, d, h, spare) == (wide, 256)
    x, xs, gq, gs = _operands(torch, sizes + [spare], h, d, g)
    _, _, uq, us = _operands(torch, [1], h, d, g)
    _, _, dq, ds = _operands(torch, [1], d, h, g)
    want, mag, flips = (t[:rows] for t in _ffn_want(torch, f8.values(x, xs, 1), f8.values(gq, gs, 128),
                                                    f8.values(uq, us, 128), f8.values(dq, ds, 128), sizes))
    y = _run(torch, moe, sizes, spare, x, xs, gq, gs, uq, us, dq, ds, out, repeats=2)
    _close(y, want, mag * 1e-5 + flips * 2.5, out)  # (flips: two steps)
    err = (y.double() - want).abs()
    near = err <= mag * 1e-5 + (want.abs() + mag * 1e-5) * HALF[out]
    assert float(near.double().mean()) >= 1 - 2 * h / 1e4


@pytest.mark.parametrize("name,wide", [("wide", True), ("swapped", False)])
def test_layer_of_many_tiles_with_a_folded_shared_expert(env, monkeypatch, name, wide):
    """The shared expert's group reads its own rows and weights, in both tilings and in both products; nothing around the
    workspace is written."""
    torch, moe = env
    # rows of the two routed groups and of the shared one; 600 tokens choose one of two experts, 500 one of eight
    tokens, e = (600, 2) if wide else (500, 8)
    monkeypatch.setitem(LAYERS, name, dict(n_tokens=tokens, d_model=2560, n_experts=e, top_k=1, d_ff=2560, d_ff_shared=2560))
    for swiglu in (True, False):
        assert moe.moe_gemm_fp8_tiling(swiglu, e + 1, True, 2 * tokens, 2560, 2560) == (wide, 256, 1)
    cfg, w, h, res, bias = _layer_case(torch, moe, name)
    i32 = dict(dtype=torch.int32, device="cuda")
    routing = dict(topk_idx=torch.empty(tokens, 1, **i32), topk_gate=torch.empty(tokens, 1, device="cuda"),
                   slot_row=torch.empty(tokens, **i32))
    size, band = moe.library().moe_workspace_size_fp8(cfg.c()), 4096
    whole = torch.full((size + 2 * band,), 0xA5, dtype=torch.uint8, device="cuda")
    ws, out = whole[band:-band], torch.empty_like(h)
    assert moe.library().moe_workspace_init(ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream) == 0
    moe.moe_layer_forward_fp8(cfg, w, h, res, bias, out, ws, routing=routing)
    assert moe.moe_check_device_error(ws)[0] == 0
    want, slack, _ = _layer_want(torch, moe, cfg, w, h, res, routing)
    _close(out, want, slack * 2.5, cfg.dtype)  # five steps, as above
    again = torch.empty_like(out)
    moe.moe_layer_forward_fp8(cfg, w, h, res, bias, again, ws)
    assert torch.equal(again, out)
    assert torch.all(whole[:band] == 0xA5) and torch.all(whole[-band:] == 0xA5)
