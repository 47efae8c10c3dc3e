"""The e4m3 operators against plain 64-bit forms on the GPU.

Tolerances.  A sum of K products accumulated in fp32 is off by at most about
K u sum|a b| (u = 2^-24) in any order; the tests allow 2^-24 * (K + 32) of the
sum of absolute products, plus half a step of the stored type.  On random signs
the real errors are far smaller.
"""
import numpy as np
import pytest

import fp8_helpers as f8
import moe_inputs as mi

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture
def env(torch_cuda):
    import sparse_mixture_experts_rmsnorm_b200 as moe
    torch_cuda.manual_seed(7)
    return torch_cuda, moe


def _type(torch, name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _close(got, want, slack, out):
    """|got - want| <= slack + half a step of the stored type (subnormals of bf16 and fp32 aside)."""
    err = (got.double() - want).abs()
    lim = slack + (want.abs() + slack) * HALF[out] + 1e-38
    bad = err > lim
    assert not bad.any(), (int(bad.sum()), float((err / lim).max()))


# ---------------------------------------------------------------- norm
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", [(0, 64), (300, 7168), (320, 4097), (2, 40001), (301, 20001), (1, 1), (1, 7168), (3, 127), (5, 128), (2, 129), (300, 1000), (64, 7168),
                                 (7, 4099), (2, 16384), (2, 49152), (2500, 256)])
@pytest.mark.parametrize("residual", [True, False])
def test_add_rmsnorm(env, dtype, n, d, residual):
    torch, moe = env
    t = _type(torch, dtype)
    x = (torch.randn(n, d, device="cuda") * torch.exp(torch.randn(n, 1, device="cuda"))).to(t)
    r = torch.randn(n, d, device="cuda").to(t) if residual else None
    w = (1 + 0.1 * torch.randn(d, device="cuda")).to(t)
    cfg = moe.Config(n, d, 1, 1, 16, dtype=dtype)
    res, xn = torch.empty_like(x), torch.empty_like(x)
    q = torch.empty(n, d, dtype=f8.E4M3, device="cuda")
    s = torch.empty(n, f8.blocks(d), device="cuda")
    moe.moe_add_rmsnorm(cfg, x, r, w, res, xn, q, s)
    if n == 0:
        return
    total = x if r is None else (x.float() + r.float()).to(t)
    assert torch.equal(res, total)
    h = total.double()
    v = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6) * w.double()
    _close(xn, v, v.abs() * 3 * U32, dtype)  # r, s r and (s r) w are each rounded to fp32
    f8.check_quantized(q, s, v, 1)
    # each output alone, and in place
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    moe.moe_add_rmsnorm(cfg, x, r, w, None, None, q2, s2)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)
    x2 = x.clone()
    moe.moe_add_rmsnorm(cfg, x2, r, w, x2, None, None, None)
    assert torch.equal(x2, res)
    x3 = x.clone()
    moe.moe_add_rmsnorm(cfg, x3, r, w, None, x3, None, None)
    assert torch.equal(x3, xn)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [(1, 1, 1, 0), (3, 3, 3, 2), (1, 2, 1, 0), (0, 0, 5, 1)])
@pytest.mark.parametrize("n,d", [(300, 1001), (297, 7), (300, 1024), (300, 30001)])
def test_norm_of_tensors_that_start_unaligned(env, dtype, at, n, d):
    """x, residual, res_out and xn start `at` elements past a 16-byte boundary, alike or not; nothing around res_out
    and xn is written."""
    torch, moe = env
    t = _type(torch, dtype)

    def place(shift, fill=None):
        whole = torch.full((n * d + 64,), 7.0, dtype=t, device="cuda")
        view = whole[8 + shift:8 + shift + n * d].view(n, d)
        if fill is not None:
            view.copy_(fill)
        return whole, view

    x, r = place(at[0], torch.randn(n, d, device="cuda"))[1], place(at[1], torch.randn(n, d, device="cuda"))[1]
    (res_all, res), (xn_all, xn) = place(at[2]), place(at[3])
    w = (1 + 0.1 * torch.randn(d, device="cuda")).to(t)
    q, s = torch.empty(n, d, dtype=f8.E4M3, device="cuda"), torch.empty(n, f8.blocks(d), device="cuda")
    moe.moe_add_rmsnorm(moe.Config(n, d, 1, 1, 16, dtype=dtype), x, r, w, res, xn, q, s)
    assert torch.equal(res, (x.float() + r.float()).to(t))
    h = res.double()
    v = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6) * w.double()
    _close(xn, v, v.abs() * 3 * U32, dtype)
    f8.check_quantized(q, s, v, 1)
    for whole, shift in ((res_all, at[2]), (xn_all, at[3])):
        assert torch.all(whole[:8 + shift] == 7.0) and torch.all(whole[8 + shift + n * d:] == 7.0)


def test_norm_bits_are_those_of_route(env):
    """xn of the fused norm equals moe_route's for h = x + residual."""
    torch, moe = env
    n, d = 70, 1024
    cfg = moe.Config(n, d, 8, 2, 64)
    x, r = torch.randn(2, n, d, device="cuda").bfloat16()
    w, wr = torch.randn(d, device="cuda").bfloat16(), torch.randn(8, d, device="cuda").bfloat16()
    xn = torch.empty_like(x)
    res = torch.empty_like(x)
    moe.moe_add_rmsnorm(cfg, x, r, w, res, xn, None, None)
    xn2 = torch.empty_like(x)
    i32 = dict(dtype=torch.int32, device="cuda")
    moe.moe_route(cfg, res, w, wr, None, xn2, None, torch.empty(n, 2, **i32), torch.empty(n, 2, device="cuda"),
                  torch.empty(8, **i32), moe.workspace(cfg))
    assert torch.equal(xn, xn2)


def test_norm_of_zero_huge_and_nan_rows(env):
    torch, moe = env
    d = 300
    x = torch.ones(4, d, device="cuda")
    x[0] = 0
    x[1] = 3e38           # squares exceed fp32: the mean is fp64
    x[2, 5] = float("nan")
    x[3, :128] = 0        # a block of zeros in an ordinary row
    cfg = moe.Config(4, d, 1, 1, 16, dtype="f32")
    w = torch.ones(d, device="cuda")
    xn, q, s = torch.empty_like(x), torch.empty(4, d, dtype=f8.E4M3, device="cuda"), torch.empty(4, 3, device="cuda")
    moe.moe_add_rmsnorm(cfg, x, None, w, None, xn, q, s)
    assert torch.all(xn[0] == 0) and torch.all(q[0].float() == 0) and torch.all(s[0] == 2.0 ** -126)
    assert torch.allclose(xn[1], torch.ones(d, device="cuda")) and torch.all(q[1].float() == 448)
    assert torch.isnan(xn[2]).all() and torch.isnan(q[2].float()).all()
    assert torch.all(q[3, :128].float() == 0) and s[3, 0] == 2.0 ** -126


# ---------------------------------------------------------------- quantisation
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("m,rows,cols", [(1, 1, 1), (2, 130, 257), (1, 128, 128), (3, 127, 120), (1, 1000, 40),
                                         (2, 300, 4096), (1, 5, 7168), (0, 4, 8), (1, 0, 8)])
def test_quantize(env, dtype, block_rows, m, rows, cols):
    torch, moe = env
    x = torch.randn(m, rows, cols, device="cuda") * torch.exp(2 * torch.randn(m, rows, 1, device="cuda"))
    if x.numel() > 500:
        x[0, 0, :40] = 0
        x[0, -1] *= 1e-42  # scales at their floor
    x = x.to(_type(torch, dtype))
    q = torch.empty(m, rows, cols, dtype=f8.E4M3, device="cuda")
    s = torch.empty(m, -(-rows // block_rows), f8.blocks(cols), device="cuda")
    moe.moe_quantize_fp8(dtype, block_rows, m, rows, cols, x, q, s)
    if x.numel():
        f8.check_quantized(q, s, x.double(), block_rows)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_every_tie_and_special(env, block_rows):
    """With a scale of exactly 1 the codes are the rounded values: every e4m3 value, every middle between
    two (ties to even), and NaN."""
    torch, moe = env
    codes = torch.arange(127, dtype=torch.uint8, device="cuda").view(f8.E4M3).float()  # 0 .. 448
    mid = (codes[1:] + codes[:-1]) / 2
    v = torch.cat([codes, mid, -codes, -mid])
    x = torch.zeros(4, 128, device="cuda")
    x.view(-1)[: len(v)] = v
    x[:, 127] = 448.0  # amax of every block
    q, s = torch.empty(4, 128, dtype=f8.E4M3, device="cuda"), torch.empty(4 if block_rows == 1 else 1, 1, device="cuda")
    moe.moe_quantize_fp8("f32", block_rows, 1, 4, 128, x, q, s)
    assert torch.all(s == 1)
    assert torch.equal(q.double(), f8.e4m3_round(x.double()))
    x[1, 3], x[2, 4] = float("nan"), float("inf")
    moe.moe_quantize_fp8("f32", block_rows, 1, 4, 128, x, q, s)
    assert torch.isnan(q.float()[1, 3]) and torch.isnan(q.float()[2, 4])
    assert torch.isinf(s.max())
    if block_rows == 1:
        assert torch.equal(q.double()[0], f8.e4m3_round(x.double()[0]))


# ---------------------------------------------------------------- products
def _operands(torch, sizes, n, k, g=None):
    g = len(sizes) if g is None else g
    rows = sum(sizes)
    a = torch.randn(rows, k, device="cuda") * torch.exp(torch.randn(rows, 1, device="cuda"))
    b = torch.randn(g, n, k, device="cuda") * 0.05 * torch.exp(torch.randn(g, 1, 1, device="cuda"))
    aq, as_ = f8.quantize(a, 1)
    bq, bs = f8.quantize(b, 128)
    return aq, as_, bq, bs


def _offsets(torch, sizes):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("rows,n,k", [(1, 1, 16), (1, 4096, 7168), (2, 7, 48), (17, 130, 144), (64, 256, 128),
                                      (128, 128, 256), (129, 384, 272), (256, 512, 1024), (257, 300, 2048),
                                      (333, 1111, 1040), (1000, 264, 640), (2048, 2048, 512), (48, 7168, 2048),
                                      (16, 257, 7168), (1, 1, 7168), (300, 256, 4096), (513, 130, 2064), (255, 512, 128),
                                      (3, 100, 16400)])
def test_gemm(env, out, rows, n, k):
    torch, moe = env
    aq, as_, bq, bs = _operands(torch, [rows], n, k)
    want, mag = f8.product(f8.values(aq, as_, 1), f8.values(bq, bs, 128), [rows])
    c = torch.full((rows, n), float("nan"), dtype=_type(torch, out), device="cuda")
    ws = moe.workspace_gemm_fp8(1, rows, n, k)
    moe.moe_gemm_fp8(1, None, rows, n, k, aq, as_, bq, bs, out, c, ws)
    _close(c, want, mag * U32 * (k + 32), out)
    assert moe.moe_check_device_error(ws)[0] == 0
    # the same bits again, in the same workspace
    c2 = torch.empty_like(c)
    moe.moe_gemm_fp8(1, None, rows, n, k, aq, as_, bq, bs, out, c2, ws)
    assert torch.equal(c, c2)


GROUPS = {
    "one of each": [1, 2, 15, 16, 17, 31, 33, 64, 65],
    "empty first and last": [0, 5, 0, 0, 300, 0],
    "all empty but one": [0, 0, 0, 77],
    "all empty": [0, 0, 0],
    "full chunks": [256, 512, 257, 255, 129],
    "one large": [3, 1500, 4, 0],
    "many small": [(7 * i) % 5 for i in range(200)],
    "the most groups": [1] * 1024,
    "large and ragged": [300, 0, 520, 257, 400],
}


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("n,k", [(256, 256), (200, 400), (130, 144)])
def test_grouped_gemm(env, out, name, n, k):
    torch, moe = env
    sizes = GROUPS[name]
    if len(sizes) == 1024 and n != 130:
        pytest.skip("one shape is enough for 1024 groups")
    spare = 9  # rows of the buffers behind the last group
    g, rows = len(sizes), sum(sizes)
    aq, as_, bq, bs = _operands(torch, sizes + [spare], n, k, g)
    want, mag = f8.product(f8.values(aq, as_, 1), f8.values(bq, bs, 128), sizes)
    c = torch.full((rows + spare, n), 7.0, dtype=_type(torch, out), device="cuda")
    ws = moe.workspace_gemm_fp8(g, rows + spare, n, k)
    moe.moe_gemm_fp8(g, _offsets(torch, sizes), rows + spare, n, k, aq, as_, bq, bs, out, c, ws)
    _close(c[:rows], want[:rows], mag[:rows] * U32 * (k + 32), out)
    assert torch.all(c[rows:] == 7.0)  # rows behind the last group are left as they were
    assert moe.moe_check_device_error(ws)[0] == 0


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,n,k", [([5, 9], 256, 2048), ([0, 3, 0], 300, 4096), ([400, 300], 200, 2048),
                                       ([0, 0], 256, 2048), ([5, 9], 256, 8192), ([0, 40, 0], 300, 6144),
                                       ([400, 300], 200, 8192)])
def test_few_tiles_cut_along_k(env, out, sizes, n, k):
    """Products of few tiles, whose parts along K meet in the workspace: the values, and the same bits every time."""
    torch, moe = env
    g, rows = len(sizes), sum(sizes) + 4
    if k >= 4096:
        assert moe.library().moe_workspace_size_gemm_fp8(g, rows, n, k) > 4096  # parts are held
    aq, as_, bq, bs = _operands(torch, sizes + [4], n, k, g)
    want, mag = f8.product(f8.values(aq, as_, 1), f8.values(bq, bs, 128), sizes)
    ws = moe.workspace_gemm_fp8(g, rows, n, k)
    c = torch.full((4, rows, n), 7.0, dtype=_type(torch, out), device="cuda")
    for i in range(4):
        moe.moe_gemm_fp8(g, _offsets(torch, sizes), rows, n, k, aq, as_, bq, bs, out, c[i], ws)
        assert torch.equal(c[i], c[0])
    m = sum(sizes)
    _close(c[0, :m], want[:m], mag[:m] * U32 * (k + 32), out)
    assert torch.all(c[:, m:] == 7.0)
    assert moe.moe_check_device_error(ws)[0] == 0


def test_offsets_past_32_bits(env):
    """Weights and results of more than 4 Gi elements: the last group's product, and the last rows."""
    torch, moe = env
    g, n, k = 300, 2048, 7168
    aq, as_, bq, bs = _operands(torch, [3], n, k)
    want, mag = f8.product(f8.values(aq, as_, 1), f8.values(bq, bs, 128), [3])
    b = torch.zeros(g, n, k, dtype=torch.uint8, device="cuda").view(f8.E4M3)
    scale = torch.ones(g, f8.blocks(n), f8.blocks(k), device="cuda")
    b[-1], scale[-1] = bq[0], bs[0]
    c = torch.empty(3, n, device="cuda")
    offs = torch.zeros(g + 1, dtype=torch.int32, device="cuda")
    offs[-1] = 3
    moe.moe_gemm_fp8(g, offs, 3, n, k, aq, as_, b, scale, "f32", c, moe.workspace_gemm_fp8(g, 3, n, k))
    _close(c, want, mag * U32 * (k + 32), "f32")
    del b, scale
    rows, n, k = 70000, 65536, 16
    aq, as_, bq, bs = _operands(torch, [rows], n, k)
    c = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    moe.moe_gemm_fp8(1, None, rows, n, k, aq, as_, bq, bs, "bf16", c, moe.workspace_gemm_fp8(1, rows, n, k))
    for r in (slice(0, 40), slice(rows - 40, rows)):
        want, mag = f8.product(f8.values(aq[r], as_[r], 1), f8.values(bq, bs, 128), [40])
        _close(c[r], want, mag * U32 * (k + 32), "bf16")
    q, s = torch.empty(rows, n, dtype=torch.uint8, device="cuda").view(f8.E4M3), torch.empty(rows, n // 128, device="cuda")
    moe.moe_quantize_fp8("bf16", 1, 1, rows, n, c, q, s)
    f8.check_quantized(q[-40:], s[-40:], c[-40:].double(), 1)


def test_a_workspace_of_other_sizes_serves(env):
    """One row with the workspace of many, and with the least there is: no room for parts, the same product."""
    torch, moe = env
    n, k = 512, 4096
    aq, as_, bq, bs = _operands(torch, [1], n, k)
    want, mag = f8.product(f8.values(aq, as_, 1), f8.values(bq, bs, 128), [1])
    assert moe.library().moe_workspace_size_gemm_fp8(1, 1, n, k) > 4096
    own = moe.workspace_gemm_fp8(1, 1, n, k)
    for ws in (own, moe.workspace_gemm_fp8(1, 100000, n, k), moe.workspace_gemm_fp8(1, 1, 64, 64)):
        c = torch.empty(1, n, device="cuda")
        moe.moe_gemm_fp8(1, None, 1, n, k, aq, as_, bq, bs, "f32", c, ws)
        _close(c, want, mag * U32 * (k + 32), "f32")
        assert moe.moe_check_device_error(ws)[0] == 0


def test_rows_that_lie_apart(env):
    """a (and the FFN's x) may be a slice of a wider buffer: the same bits as from a packed copy."""
    torch, moe = env
    rows, n, k = 200, 256, 400
    aq, as_, bq, bs = _operands(torch, [rows], n, k)
    wide = torch.full((rows, 512), 0x7F, dtype=torch.uint8, device="cuda").view(f8.E4M3)  # NaN around the slice
    wide[:, 16:16 + k] = aq
    ws = moe.workspace_gemm_fp8(1, rows, n, k)
    c = torch.empty(2, rows, n, device="cuda")
    moe.moe_gemm_fp8(1, None, rows, n, k, aq, as_, bq, bs, "f32", c[0], ws)
    moe.moe_gemm_fp8(1, None, rows, n, k, wide[:, 16:16 + k], as_, bq, bs, "f32", c[1], ws)
    assert torch.equal(c[0], c[1])
    _, _, uq, us = _operands(torch, [1], n, k)
    _, _, dq, ds = _operands(torch, [1], k, n)
    cfg = moe.Config(rows, k, 1, 1, n)
    ws = moe.workspace_fp8(cfg)
    y = torch.empty(2, rows, k, dtype=torch.bfloat16, device="cuda")
    for x, out in ((aq, y[0]), (wide[:, 16:16 + k], y[1])):
        moe.moe_expert_ffn_fp8(cfg, 1, None, rows, x, as_, bq, bs, uq, us, dq, ds, n, out, ws)
    assert torch.equal(y[0], y[1])


def test_rows_before_the_first_group_stay(env):
    torch, moe = env
    sizes, n, k = [11, 40], 64, 256
    aq, as_, bq, bs = _operands(torch, [20] + sizes, n, k, 2)
    offs = _offsets(torch, sizes) + 20
    c = torch.full((71, n), 7.0, device="cuda")
    moe.moe_gemm_fp8(2, offs, 71, n, k, aq, as_, bq, bs, "f32", c, moe.workspace_gemm_fp8(2, 71, n, k))
    assert torch.all(c[:20] == 7.0)
    want, mag = f8.product(f8.values(aq, as_, 1)[20:], f8.values(bq, bs, 128), sizes)
    _close(c[20:], want, mag * U32 * (k + 32), "f32")


def test_nonfinite_operands_stay_in_their_rows_and_columns(env):
    """A NaN code, an infinite scale and a zero scale reach the products they take part in and no others."""
    torch, moe = env
    sizes, n, k = [40, 30], 200, 384
    aq, as_, bq, bs = _operands(torch, sizes, n, k)
    au = aq.view(torch.uint8)
    au[3, 100] = 0x7F           # NaN
    as_[45, 1] = float("inf")
    as_[50] = 0.0
    bq.view(torch.uint8)[1, 77, 5] = 0x7F
    want = f8.product(f8.values(aq, as_, 1), f8.values(bq, bs, 128), sizes)[0]
    c = torch.empty(70, n, device="cuda")
    moe.moe_gemm_fp8(2, _offsets(torch, sizes), 70, n, k, aq, as_, bq, bs, "f32", c,
                     moe.workspace_gemm_fp8(2, 70, n, k))
    bad = torch.zeros(70, n, dtype=torch.bool, device="cuda")
    bad[3] = bad[45] = True
    bad[40:, 77] = True
    assert not torch.isfinite(c[3]).any() and not torch.isfinite(c[45]).any() and torch.isnan(c[40:, 77]).all()
    ok = ~bad
    assert torch.isfinite(c[ok]).all()
    assert torch.allclose(c[ok].double(), want[ok], rtol=1e-4, atol=1e-3)
    assert torch.all(c[50][ok[50]] == 0)


# ---------------------------------------------------------------- the expert FFN
def _ffn_want(torch, x, gate, up, down, sizes):
    """The FFN in 64 bits, and how far two flipped codes of its activation can move each result.

    An fp32 error of the activation (about 1e-6 of it) moves a code by one step only where it lies that close to
    a border, a few 1e-5 of the codes; a step is at most 2^-3 of the value, so a flip moves a result by at most
    2^-3 of the row's largest activation times the largest weight of the column."""
    zg, _ = f8.product(x, gate, sizes)
    zu, _ = f8.product(x, up, sizes)
    act = zg * torch.sigmoid(zg) * zu
    want, mag = f8.product(f8.values(*f8.quantize(act, 1), 1), down, sizes)
    flip = torch.zeros_like(want)
    at = 0
    for g, m in enumerate(sizes):
        if m:
            flip[at:at + m] = act[at:at + m].abs().amax(1, keepdim=True) * down[g].abs().amax(1) * 2.0 ** -3
        at += m
    return want, mag, 2 * flip


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,d,h", [([1], 128, 128), ([40], 256, 384), ([3, 0, 70, 300], 512, 256),
                                       ([5, 260, 1], 272, 208), ([700], 1024, 144), ([0, 2], 144, 16),
                                       ([(3 * i) % 4 for i in range(40)], 256, 320), ([300, 0, 520, 260], 256, 208),
                                       ([1], 7168, 256), ([300], 2048, 256), ([2, 0, 3], 2048, 128)])
def test_expert_ffn(env, out, sizes, d, h):
    torch, moe = env
    g, rows, spare = len(sizes), sum(sizes), 3
    x, xs, gq, gs = _operands(torch, sizes + [spare], h, d, g)
    _, _, uq, us = _operands(torch, [1], h, d, g)
    _, _, dq, ds = _operands(torch, [1], d, h, g)
    xv = f8.values(x, xs, 1)
    want, mag, flips = _ffn_want(torch, xv, f8.values(gq, gs, 128), f8.values(uq, us, 128), f8.values(dq, ds, 128), sizes)
    cfg = moe.Config(rows + spare, d, g, 1, h, dtype=out)
    ws = moe.workspace_fp8(cfg)
    y = torch.full((rows + spare, d), 7.0, dtype=_type(torch, out), device="cuda")
    offs = _offsets(torch, sizes) if g > 1 else None
    moe.moe_expert_ffn_fp8(cfg, g, offs, rows + (spare if g > 1 else 0), x, xs, gq, gs, uq, us, dq, ds, h, y, ws)
    # the scale of a block follows amax, off by fp32 roundings: 1e-5 of the magnitudes covers it and the sums
    _close(y[:rows], want[:rows], mag[:rows] * 1e-5 + flips[:rows], out)
    # and flips are rare: nearly all results are as near as their type allows
    err = (y[:rows].double() - want[:rows]).abs()
    near = err <= mag[:rows] * 1e-5 + (want[:rows].abs() + mag[:rows] * 1e-5) * HALF[out]
    assert float(near.double().mean()) >= 0.9 or rows * h < 4096
    assert torch.all(y[rows:] == 7.0)
    assert moe.moe_check_device_error(ws)[0] == 0


def test_a_workspace_shared_with_other_calls(env):
    """Products cut along K count their parts in the header: scratch that other calls leave behind it does not matter."""
    torch, moe = env
    n, k = 2048, 8192
    aq, as_, bq, bs = _operands(torch, [9], n, k)
    size = moe.library().moe_workspace_size_gemm_fp8(1, 9, n, k)
    assert size > 4096
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    assert moe.library().moe_workspace_init(ws.data_ptr(), size, None) == 0
    torch.cuda.synchronize()
    own, c = torch.empty(9, n, device="cuda"), torch.empty(9, n, device="cuda")
    moe.moe_gemm_fp8(1, None, 9, n, k, aq, as_, bq, bs, "f32", own, moe.workspace_gemm_fp8(1, 9, n, k))
    for fill in (0xFF, 0x00, 0x5A):
        ws[256:] = fill
        moe.moe_gemm_fp8(1, None, 9, n, k, aq, as_, bq, bs, "f32", c, ws)
        assert torch.equal(c, own)
    assert moe.moe_check_device_error(ws)[0] == 0


def test_ffn_in_a_workspace_of_more_tokens(env):
    """Fewer tokens may want more room for partial sums than more do: the call then does without."""
    torch, moe = env
    d, h, rows = 4096, 2048, 32
    small, large = moe.Config(rows, d, 1, 1, h), moe.Config(64, d, 1, 1, h)
    size = moe.library().moe_workspace_size_fp8
    assert size(small.c()) > size(large.c())
    x, xs, gq, gs = _operands(torch, [rows], h, d)
    _, _, uq, us = _operands(torch, [1], h, d)
    _, _, dq, ds = _operands(torch, [1], d, h)
    want, mag, flips = _ffn_want(torch, f8.values(x, xs, 1), *(f8.values(q, s, 128) for q, s in
                                                             ((gq, gs), (uq, us), (dq, ds))), [rows])
    for cfg in (small, large):
        ws = moe.workspace_fp8(cfg)
        y = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
        moe.moe_expert_ffn_fp8(small, 1, None, rows, x, xs, gq, gs, uq, us, dq, ds, h, y, ws)
        _close(y, want, mag * 1e-5 + flips, "bf16")
        assert moe.moe_check_device_error(ws)[0] == 0


# ---------------------------------------------------------------- the operators together, as the layer uses them
LAYERS = {
    "folded shared expert": dict(n_tokens=300, d_model=256, n_experts=8, top_k=2, d_ff=128, d_ff_shared=128),
    "separate shared expert, capacity": dict(n_tokens=200, d_model=512, n_experts=16, top_k=4, d_ff=256,
                                             d_ff_shared=144, capacity_factor=0.75),
    "tensor-core router": dict(n_tokens=520, d_model=384, n_experts=64, top_k=8, d_ff=128, d_ff_shared=128),
    "single token": dict(n_tokens=1, d_model=1024, n_experts=32, top_k=4, d_ff=256),
    "every slot dropped": dict(n_tokens=20, d_model=128, n_experts=8, top_k=1, d_ff=64, capacity_factor=0.2),
    "fp32": dict(n_tokens=90, d_model=272, n_experts=8, top_k=2, d_ff=208, d_ff_shared=208, dtype="f32"),
    "no tokens": dict(n_tokens=0, d_model=128, n_experts=8, top_k=1, d_ff=64),
}


def _layer_case(torch, moe, name, seed=3):
    cfg = moe.Config(**LAYERS[name])
    N, d, E, H, Hs = cfg.n_tokens, cfg.d_model, cfg.n_experts, cfg.d_ff, cfg.d_ff_shared
    t = _type(torch, cfg.dtype)
    torch.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    w = {"norm_w": (1 + 0.1 * rand(d)).to(t), "w_router": (rand(E, d) * 0.1).to(t)}
    shapes = {"w_gate": (E, H, d), "w_up": (E, H, d), "w_down": (E, d, H)}
    if Hs:
        shapes.update(ws_gate=(1, Hs, d), ws_up=(1, Hs, d), ws_down=(1, d, Hs))
    for m, s in shapes.items():
        x = (rand(*s) * 0.08).to(t)
        w[m] = torch.empty(s, dtype=f8.E4M3, device="cuda")
        w[m + "_scale"] = torch.empty(s[0], f8.blocks(s[1]), f8.blocks(s[2]), device="cuda")
        moe.moe_quantize_fp8(cfg.dtype, 128, s[0], s[1], s[2], x, w[m], w[m + "_scale"])
    h, res = rand(N, d).to(t), rand(N, d).to(t)
    bias = rand(E) * 0.01
    return cfg, w, h, res, bias


def _layer_want(torch, moe, cfg, w, h, res, routing):
    """The layer in 64 bits on the routing that the call returned and on moe_add_rmsnorm's codes of its rows
    (checked by themselves above), and how far each result may be off: two flipped codes of each expert's
    activation, the sums' fp32 roundings, and the storage of each expert's output (half a step of its type)."""
    N, d, E, k = cfg.n_tokens, cfg.d_model, cfg.n_experts, cfg.top_k
    s = torch.empty_like(h)
    q, qs = torch.empty(N, d, dtype=f8.E4M3, device="cuda"), torch.empty(N, f8.blocks(d), device="cuda")
    moe.moe_add_rmsnorm(cfg, h, res, w["norm_w"], s, None, q, qs)
    x = f8.values(q, qs, 1)
    mats = {m: f8.values(w[m], w[m + "_scale"], 128) for m in ("w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down")
            if m in w}
    out = s.double()
    slack = out.abs() * U32 * (k + 2)
    keep = routing["slot_row"].view(N, k) >= 0

    def add(t, gates, names, e):
        nonlocal out, slack
        y, mag, flips = _ffn_want(torch, x[t], *(mats[m][e:e + 1] for m in names), [len(t)])
        out.index_add_(0, t, y * gates)
        slack.index_add_(0, t, (mag * 2e-5 + flips + y.abs() * HALF[cfg.dtype] * 1.01) * gates)

    for e in range(E):
        t, j = torch.nonzero((routing["topk_idx"] == e) & keep, as_tuple=True)
        if len(t):
            add(t, routing["topk_gate"][t, j].double()[:, None], ("w_gate", "w_up", "w_down"), e)
    if cfg.d_ff_shared:
        add(torch.arange(N, device="cuda"), 1.0, ("ws_gate", "ws_up", "ws_down"), 0)
    return out, slack, s


@pytest.mark.parametrize("name", list(LAYERS))
@pytest.mark.parametrize("residual", [True, False])
def test_layer_forward(env, name, residual):
    torch, moe = env
    cfg, w, h, res, bias = _layer_case(torch, moe, name)
    res = res if residual else None
    N, E, k = cfg.n_tokens, cfg.n_experts, cfg.top_k
    i32 = dict(dtype=torch.int32, device="cuda")
    routing = dict(topk_idx=torch.empty(N, k, **i32), topk_gate=torch.empty(N, k, device="cuda"),
                   slot_row=torch.empty(N * k, **i32), counts=torch.empty(E, **i32))
    ws = moe.workspace_fp8(cfg)
    out = torch.empty_like(h)
    moe.moe_layer_forward_fp8(cfg, w, h, res, bias, out, ws, routing=routing)
    assert moe.moe_check_device_error(ws)[0] == 0
    if N == 0:
        return
    want, slack, s = _layer_want(torch, moe, cfg, w, h, res, routing)
    # the routing is moe_route's on h + residual (the same kernels and xn)
    c2 = moe.Config(**LAYERS[name])
    idx, gate = torch.empty(N, k, **i32), torch.empty(N, k, device="cuda")
    moe.moe_route(c2, s, w["norm_w"], w["w_router"], bias, torch.empty_like(s), None, idx, gate,
                  torch.empty(E, **i32), moe.workspace(c2))
    assert torch.equal(idx, routing["topk_idx"]) and torch.equal(gate, routing["topk_gate"])
    assert int(routing["counts"].sum()) == N * k
    _close(out, want, slack, cfg.dtype)
    # in place: out may be h, or the residual
    for alias in ("h", "res"):
        if alias == "res" and res is None:
            continue
        h2, r2 = h.clone(), None if res is None else res.clone()
        o2 = h2 if alias == "h" else r2
        moe.moe_layer_forward_fp8(cfg, w, h2, r2, bias, o2, ws)
        assert torch.equal(o2, out)


def test_layer_matches_the_bf16_layer(env):
    """The 8-bit layer stays near the bf16 layer on the same weights: each operand's e4m3 rounding is off
    by at most 2^-4 of it, on random signs far less in a sum."""
    torch, moe = env
    lc = mi.LayerConfig(name="near", n_tokens=256, d_model=512, n_experts=16, top_k=4, d_ff=256, d_ff_shared=256, seed=2)
    dev = mi.device_tensors(lc)
    cfg = moe.Config(lc.n_tokens, lc.d_model, lc.n_experts, lc.top_k, lc.d_ff, lc.d_ff_shared)
    out = torch.empty_like(dev["h"])
    moe.moe_layer_forward(cfg, {n: dev[n] for n in dev}, dev["h"], dev["bias"], out, moe.workspace(cfg))
    w = {"norm_w": dev["norm_w"], "w_router": dev["w_router"]}
    for m in ("w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down"):
        x = dev[m] if dev[m].dim() == 3 else dev[m][None]
        w[m] = torch.empty(x.shape, dtype=f8.E4M3, device="cuda")
        w[m + "_scale"] = torch.empty(x.shape[0], f8.blocks(x.shape[1]), f8.blocks(x.shape[2]), device="cuda")
        moe.moe_quantize_fp8("bf16", 128, *x.shape, x, w[m], w[m + "_scale"])
    out8 = torch.empty_like(out)
    moe.moe_layer_forward_fp8(cfg, w, dev["h"], None, dev["bias"], out8, moe.workspace_fp8(cfg))
    a, b = (out - dev["h"]).double(), (out8 - dev["h"]).double()
    # three chained roundings of relative rms about 2^-4 / sqrt(3) each, in both factors of a product: under 0.1
    assert float((a - b).norm() / a.norm()) <= 0.1


def test_tensors_off_the_current_device_are_refused(env):
    """On the host, before anything is launched."""
    torch, moe = env
    cfg = moe.Config(4, 128, 1, 1, 16)
    x, w, out = torch.ones(4, 128), torch.ones(128), torch.ones(4, 128, device="cuda")
    with pytest.raises(ValueError):
        moe.moe_add_rmsnorm(cfg, x.bfloat16(), None, w.bfloat16().cuda(), out.bfloat16(), None, None, None)
    with pytest.raises(ValueError):
        moe.moe_quantize_fp8("f32", 1, 1, 4, 128, out, torch.empty(4, 128, dtype=torch.uint8), torch.empty(4, 1).cuda())
    ws = moe.workspace_gemm_fp8(1, 4, 128, 128)
    q, s = torch.zeros(4, 128, dtype=torch.uint8, device="cuda"), torch.ones(4, 1, device="cuda")
    b, bs = torch.zeros(128, 128, dtype=torch.uint8, device="cuda"), torch.ones(1, 1)
    with pytest.raises(ValueError):
        moe.moe_gemm_fp8(1, None, 4, 128, 128, q, s, b, bs, "f32", out, ws)


# ---------------------------------------------------------------- streams, graphs, guard bands
def test_graph_capture_and_other_stream(env):
    torch, moe = env
    cfg, w, h, res, bias = _layer_case(torch, moe, "tensor-core router")
    ws = moe.workspace_fp8(cfg)
    out, ref = torch.empty_like(h), torch.empty_like(h)
    moe.moe_layer_forward_fp8(cfg, w, h, res, bias, ref, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.moe_layer_forward_fp8(cfg, w, h, res, bias, out, ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_layer_forward_fp8(cfg, w, h, res, bias, out, ws)
    _, _, h2, res2, _ = _layer_case(torch, moe, "tensor-core router", seed=9)
    h.copy_(h2)
    res.copy_(res2)
    out.zero_()
    for _ in range(3):
        graph.replay()
    moe.moe_layer_forward_fp8(cfg, w, h, res, bias, ref, ws)
    assert torch.equal(out, ref)
    assert moe.moe_check_device_error(ws)[0] == 0


def test_two_calls_at_once_and_two_graphs_on_one_workspace(env):
    """Products on two streams, each with its own workspace, and two captured graphs that share one."""
    torch, moe = env
    cases = [(1, 512, 4096), (300, 256, 2048), (700, 1024, 512)]
    ops = [_operands(torch, [r], n, k) for r, n, k in cases]
    ref = []
    for (r, n, k), o in zip(cases, ops):
        ref.append(torch.empty(r, n, device="cuda"))
        moe.moe_gemm_fp8(1, None, r, n, k, *o, "f32", ref[-1], moe.workspace_gemm_fp8(1, r, n, k))
    torch.cuda.synchronize()
    got = [torch.empty_like(x) for x in ref]
    spaces = [moe.workspace_gemm_fp8(1, *c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for (r, n, k), o, c, ws, st in zip(cases, ops, got, spaces, streams):
            moe.moe_gemm_fp8(1, None, r, n, k, *o, "f32", c, ws, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    size = max(w.numel() for w in spaces)
    shared = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert moe.library().moe_workspace_init(shared.data_ptr(), size, None) == 0
    torch.cuda.synchronize()
    graphs = []
    for (r, n, k), o, c in zip(cases, ops, got):
        c.zero_()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            moe.moe_gemm_fp8(1, None, r, n, k, *o, "f32", c, shared)
    for i in (0, 1, 2, 1, 0, 2, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("name", ["folded shared expert", "separate shared expert, capacity", "fp32"])
def test_no_write_outside_any_buffer(env, name):
    torch, moe = env
    band, fill = 4096, 0xA5
    bufs = []

    def guarded(shape, dtype):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        buf = torch.full((n + 2 * band,), fill, dtype=torch.uint8, device="cuda")
        bufs.append((buf, n))
        return buf[band:band + n].view(dtype).view(*shape)

    cfg, w, h, res, bias = _layer_case(torch, moe, name)
    N, d, H = cfg.n_tokens, cfg.d_model, cfg.d_ff
    t = _type(torch, cfg.dtype)
    ws = guarded((moe.library().moe_workspace_size_fp8(cfg.c()),), torch.uint8)
    assert moe.library().moe_workspace_init(ws.data_ptr(), ws.numel(), None) == 0
    moe.moe_layer_forward_fp8(cfg, w, h, res, bias, guarded((N, d), t), ws)
    xn, q, s = guarded((N, d), t), guarded((N, d), f8.E4M3), guarded((N, f8.blocks(d)), torch.float32)
    moe.moe_add_rmsnorm(cfg, h, res, w["norm_w"], guarded((N, d), t), xn, q, s)
    moe.moe_quantize_fp8(cfg.dtype, 1, 1, N, d, xn, guarded((N, d), f8.E4M3), guarded((N, f8.blocks(d)), torch.float32))
    moe.moe_quantize_fp8(cfg.dtype, 128, 1, N, d, xn, guarded((N, d), f8.E4M3),
                         guarded((f8.blocks(N), f8.blocks(d)), torch.float32))
    for out in ("bf16", "f32"):
        size = moe.library().moe_workspace_size_gemm_fp8(1, N, H, d)
        gws = guarded((size,), torch.uint8)
        assert moe.library().moe_workspace_init(gws.data_ptr(), size, None) == 0
        moe.moe_gemm_fp8(1, None, N, H, d, q, s, w["w_gate"], w["w_gate_scale"], out, guarded((N, H), _type(torch, out)),
                         gws)
    torch.cuda.synchronize()
    for i, (buf, n) in enumerate(bufs):
        assert torch.all(buf[:band] == fill) and torch.all(buf[band + n:] == fill), i
