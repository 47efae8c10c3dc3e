"""Values and inputs at which the e4m3 calls go wrong most easily."""
import pytest

import fp8_helpers as f8
from test_gpu_fp8 import env  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [60, 2048])
def test_activation_is_fp32_at_every_gate(env, rows):
    """silu(gate) * up from -80 to 80, through the scale of a block whose only value it is (its code is 448).

    In units of 2^-24 of the value: the exponential and the division are off by at most 2 ulp (4 units each), and
    1 + e^-g, the product with up, amax / 448 and 448 * scale are rounded once each: 12.  Gate and up are exact.  60 rows
    take the tiling with rows on the MMA's N side, 2048 the one with rows on its M side; the last row's gates of -500
    and 500 give 0 and 250000."""
    torch, moe = env
    d, h = 128, 2048
    v = torch.exp(torch.linspace(-7.0, 4.38, rows, device="cuda", dtype=torch.float64)).float()  # 0.0009 to 79.8
    v[-1] = 500.0
    x = torch.zeros(rows, d, device="cuda")
    x[:, 0] = 1.0
    gate, up = torch.zeros(2, 1, h, d, device="cuda")
    gate[0, 0::256, 0], gate[0, 128::256, 0] = -1.0, 1.0  # the first hidden unit of each block of 128
    up[0, ::128, 0] = 1.0
    down = torch.zeros(1, d, h, device="cuda")
    n = torch.arange(d, device="cuda")
    down[0, n, n % 16 * 128] = 1.0
    ones = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    cfg = moe.Config(rows, d, 1, 1, h, dtype="f32")
    y = torch.empty(rows, d, device="cuda")
    gate, up, down = (w.to(f8.E4M3) for w in (gate, up, down))
    moe.moe_expert_ffn_fp8(cfg, 1, None, rows, x.to(f8.E4M3), v[:, None].contiguous(), gate, ones(1, 16, 1), up,
                           ones(1, 16, 1), down, ones(1, 1, 16), h, y, moe.workspace_fp8(cfg))
    u = v.double()[:, None]
    g = torch.where(n % 2 == 0, -1.0, 1.0) * u
    want = g / (1.0 + torch.exp(-g)) * u
    err = (y.double() - want).abs() - want.abs() * 12 * 2.0 ** -24
    assert torch.all(y[-1, ::2] == 0)
    assert torch.all(err[:-1] <= 0) and torch.all(err[-1] <= 1e-30)


@pytest.mark.parametrize("n_tokens", [64, 600])
def test_layer_takes_router_weights_of_any_alignment(env, n_tokens):
    """Router weights that start 2 bytes off a 16-byte boundary, with out in the place of h: the layer runs as for few
    tokens instead of refusing after it has written h + residual to out."""
    torch, moe = env
    d, e, k, f = 256, 64, 4, 128
    cfg = moe.Config(n_tokens, d, e, k, f)
    w = {"norm_w": (1 + 0.1 * torch.randn(d, device="cuda")).bfloat16()}
    for name, shape in (("w_gate", (e, f, d)), ("w_up", (e, f, d)), ("w_down", (e, d, f))):
        w[name], w[name + "_scale"] = f8.quantize(torch.randn(*shape, device="cuda") * 0.08, 128)
    router = torch.randn(e, d, device="cuda").bfloat16() * 0.1
    off = torch.empty(e * d + 8, device="cuda", dtype=torch.bfloat16)[1:1 + e * d].view(e, d)
    off.copy_(router)
    assert router.data_ptr() % 16 == 0 and off.data_ptr() % 16 == 2
    h, res = (torch.randn(n_tokens, d, device="cuda").bfloat16() for _ in range(2))
    bias = torch.zeros(e, device="cuda")
    got, idx = [], []
    for r in (router, off):
        out = h.clone()
        idx.append(torch.empty(n_tokens, k, dtype=torch.int32, device="cuda"))
        ws = moe.workspace_fp8(cfg)
        moe.moe_layer_forward_fp8(cfg, {**w, "w_router": r}, out, res, bias, out, ws, routing=dict(topk_idx=idx[-1]))
        assert moe.moe_check_device_error(ws)[0] == 0
        got.append(out.double())
    # the two routers sum in different orders: a token whose scores nearly tie may choose otherwise
    same = (idx[0] == idx[1]).all(1)
    assert float(same.double().mean()) >= 0.99
    # and its gates differ by 2^-24 d of the logits' absolute sums at most, which moves a bf16 result by a step at most
    diff = (got[0] - got[1])[same].abs()
    assert torch.all(diff <= got[0][same].abs() * 2.0 ** -7 + 1e-4)


@pytest.mark.parametrize("name", ["scores", "topk_idx", "topk_gate", "counts", "offsets", "slot_row", "row_token"])
def test_layer_refuses_routing_outputs_off_the_device(env, name):
    """On the host, before anything is launched: out stays as it was."""
    torch, moe = env
    cfg = moe.Config(4, 128, 2, 1, 16)
    shapes = dict(scores=(4, 2), topk_idx=(4, 1), topk_gate=(4, 1), counts=(2,), offsets=(3,), slot_row=(4,), row_token=(4,))
    kind = torch.float32 if name in ("scores", "topk_gate") else torch.int32
    codes = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    ones = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    w = dict(norm_w=ones(128).bfloat16(), w_router=ones(2, 128).bfloat16(), w_gate=codes(2, 16, 128),
             w_gate_scale=ones(2, 1, 1), w_up=codes(2, 16, 128), w_up_scale=ones(2, 1, 1), w_down=codes(2, 128, 16),
             w_down_scale=ones(2, 1, 1))
    out = ones(4, 128).bfloat16() * 7
    with pytest.raises(ValueError):
        moe.moe_layer_forward_fp8(cfg, w, ones(4, 128).bfloat16(), None, None, out, moe.workspace_fp8(cfg),
                                  routing={name: torch.zeros(shapes[name], dtype=kind)})
    torch.cuda.synchronize()
    assert torch.all(out == 7)


def test_rows_of_a_wider_buffer_given_whole(env):
    """A contiguous matrix wider than k (or d_model) is read at its own pitch, like the slice of it."""
    torch, moe = env
    rows, n, k = 200, 256, 400
    a, sa = f8.quantize(torch.randn(rows, k, device="cuda"), 1)
    b, sb = f8.quantize(torch.randn(2, 1, n, k, device="cuda") * 0.05, 128)
    down, sd = f8.quantize(torch.randn(1, k, n, device="cuda") * 0.05, 128)
    wide = torch.full((rows, 512), 0x7F, dtype=torch.uint8, device="cuda").view(f8.E4M3)  # NaN behind the columns
    wide[:, :k] = a
    ws = moe.workspace_gemm_fp8(1, rows, n, k)
    c = torch.empty(3, rows, n, device="cuda")
    for x, out in ((a, c[0]), (wide, c[1]), (wide[:, :k], c[2])):
        moe.moe_gemm_fp8(1, None, rows, n, k, x, sa, b[0], sb[0], "f32", out, ws)
    assert torch.isfinite(c).all() and torch.equal(c[0], c[1]) and torch.equal(c[0], c[2])
    one = torch.empty(1, n, device="cuda")
    moe.moe_gemm_fp8(1, None, 1, n, k, wide[5:6], sa[5:6], b[0], sb[0], "f32", one, ws)  # one row has no pitch
    assert torch.isfinite(one).all()
    cfg = moe.Config(rows, k, 1, 1, n)
    ws = moe.workspace_fp8(cfg)
    y = torch.empty(3, rows, k, dtype=torch.bfloat16, device="cuda")
    for x, out in ((a, y[0]), (wide, y[1]), (wide[:, :k], y[2])):
        moe.moe_expert_ffn_fp8(cfg, 1, None, rows, x, sa, b[0], sb[0], b[1], sb[1], down, sd, n, out, ws)
    assert torch.isfinite(y).all() and torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])
