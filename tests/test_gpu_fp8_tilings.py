"""The tilings of the e4m3 products that only larger calls take, against plain 64-bit forms.

A call with more tiles than SM pairs takes 256 rows of a group on the MMA's M side (wide) where its groups average
256 rows or more, else chunks of up to 256 rows on the N side (swapped); calls of fewer tiles are covered elsewhere.
"""
import pytest

import fp8_helpers as f8
from test_gpu_fp8 import _offsets, _operands, _type, env  # noqa: F401 (a fixture)

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
