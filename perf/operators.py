"""Measured cases of the 8-bit serving operators, with a plain form and a 64-bit definition of each.

The operators (e4m3 is the 8-bit format with 4 exponent and 3 mantissa bits, largest value 448):

  norm      s = x + residual (stored in the layer's type), xn = s / sqrt(mean(s^2) + eps) * w, and xn in e4m3 with one
            fp32 scale for each 128 columns of a row;
  quantize  a matrix in e4m3 with one fp32 scale for each 1 x 128 or 128 x 128 block;
  gemm      rows [offsets[g], offsets[g+1]) of A times B[g]^T, both in e4m3 with block scales (1 x 128 for A,
            128 x 128 for B): one group is a plain product, many are the experts' ragged products;
  ffn       the SwiGLU experts on such operands: down(e4m3(silu(gate x) * (up x))).

A scale is max(amax / 448, 2^-126) and a value is stored as e4m3(x * (1 / scale)), rounded to nearest even and
saturated.  Where `own` is false everything is elementary torch; where it is true the library's entry points run.
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # one decode step of 64 tokens at the DeepSeek-V3-shaped width: a few microseconds, latency counts
        dict(name="norm decode 64x7168", op="norm", rows=64, d=7168, dtype="bf16", residual=True),
        # the prefill of the same layer: 8192 tokens, bound by HBM
        dict(name="norm prefill 8192x7168", op="norm", rows=8192, d=7168, dtype="bf16", residual=True),
        # fp32 activations and an odd width, no residual
        dict(name="norm f32 2048x5003", op="norm", rows=2048, d=5003, dtype="f32", residual=False),
        # activations of Mixtral-8x7B's hidden width, a scale per row and 128 columns
        dict(name="quantize rows 4096x14336", op="quantize", mats=1, rows=4096, cols=14336, block_rows=1, dtype="bf16"),
        # a stack of expert weights of the same layer, 128 x 128 blocks, once at load time
        dict(name="quantize weights 8x14336x4096", op="quantize", mats=8, rows=14336, cols=4096, block_rows=128,
             dtype="bf16"),
        # a single token through one projection: the weights are read once, latency and split count
        dict(name="gemm 1x4096x7168", op="gemm", groups=1, rows=1, n=4096, k=7168, out="bf16", spread="even"),
        # a dense projection over a prefill of 8192 tokens
        dict(name="gemm 8192x4096x7168", op="gemm", groups=1, rows=8192, n=4096, k=7168, out="bf16", spread="even"),
        # ragged groups with empty ones among them, fp32 results
        dict(name="gemm 64 groups 9001x2048x7168", op="gemm", groups=64, rows=9001, n=2048, k=7168, out="f32",
             spread="ragged"),
        # odd sizes: K ends inside a block of 128, N inside a tile
        dict(name="gemm 333x1111x1040", op="gemm", groups=1, rows=333, n=1111, k=1040, out="f32", spread="even"),
        # decode of the DeepSeek-V3-shaped layer: 64 tokens, top-8 of 256 experts, bound by the weights' bytes
        dict(name="ffn decode 512 of 256", op="ffn", groups=256, rows=512, d=7168, h=2048, out="bf16", spread="even"),
        # prefill of the same layer: 8192 tokens
        dict(name="ffn prefill 65536 of 256", op="ffn", groups=256, rows=65536, d=7168, h=2048, out="bf16",
             spread="even"),
        # Mixtral-8x7B-shaped experts, most rows on one of them
        dict(name="ffn skewed 5000 of 8", op="ffn", groups=8, rows=5000, d=4096, h=14336, out="bf16", spread="skewed"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "gemm", "gemm", "ffn", "ffn"])
    if op == "norm":
        return dict(op=op, rows=_log(rng, 1, 8192), d=_log(rng, 64, 8192), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    residual=rng.random() < 0.7)
    if op == "quantize":
        block_rows = rng.choice([1, 128])
        return dict(op=op, mats=1 if block_rows == 1 else rng.randint(1, 8), rows=_log(rng, 1, 8192),
                    cols=_log(rng, 32, 8192), block_rows=block_rows, dtype=rng.choice(["bf16", "f32"]))
    groups = rng.choice([1, _log(rng, 2, 128)])
    spread = "even" if groups == 1 else rng.choice(["even", "ragged", "skewed" if groups <= 16 else "ragged"])
    rows = _log(rng, 1, 16384 if spread != "skewed" else 4096)
    out = rng.choice(["bf16", "bf16", "f32"])
    if op == "gemm":
        return dict(op=op, groups=groups, rows=rows, n=_log(rng, 16, 4096), k=16 * _log(rng, 4, 448), out=out,
                    spread=spread)
    return dict(op=op, groups=groups, rows=rows, d=16 * _log(rng, 8, 448), h=16 * _log(rng, 4, 128), out=out,
                spread=spread)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _blocks(n):
    return (n + 127) // 128


def _store(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _quantized_weights(groups, rows, cols, gen):
    """e4m3 weights of N(0, 0.02) with 128 x 128 scales, made a few groups at a time."""
    q, s = _store((groups, rows, cols), E4M3), _store((groups, _blocks(rows), _blocks(cols)), torch.float32)
    step = max(1, (1 << 28) // (rows * cols))
    for g in range(0, groups, step):
        w = torch.randn((min(step, groups - g), rows, cols), device="cuda", generator=gen) * 0.02
        q[g:g + step], s[g:g + step] = _quantize(w, 128)
    return q, s


def _group_sizes(groups, rows, spread, gen):
    p = torch.ones(groups, device="cuda")
    if spread == "ragged":  # a third of the groups stays empty, the others differ by up to a factor of about ten
        p = torch.exp(torch.randn(groups, device="cuda", generator=gen))
        p[torch.rand(groups, device="cuda", generator=gen) < 0.33] = 0
        p[0] += 1e-3
    elif spread == "skewed":  # one group takes most rows
        p[int(torch.randint(groups, (1,), device="cuda", generator=gen))] = 9.0 * groups
    pick = torch.multinomial(p, rows, replacement=True, generator=gen)
    return torch.bincount(pick, minlength=groups)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    rand = lambda *shape: torch.randn(shape, device="cuda", generator=gen)  # noqa: E731
    op = case["op"]
    if op == "norm":
        n, d, t = case["rows"], case["d"], TYPES[case["dtype"]]
        x = rand(n, d) * torch.exp(0.5 * rand(n, 1))
        x[:, :: max(1, d // 7)] *= 8  # a few columns stand out, as in trained networks
        st = dict(x=x.to(t), residual=(rand(n, d) * 2).to(t) if case["residual"] else None,
                  w=(1 + 0.1 * rand(d)).to(t))
        st["out"] = dict(res=_store((n, d), t), xn=_store((n, d), t), q=_store((n, d), E4M3),
                         scale=_store((n, _blocks(d)), torch.float32))
    elif op == "quantize":
        m, n, k = case["mats"], case["rows"], case["cols"]
        x = _store((m, n, k), TYPES[case["dtype"]])
        for i in range(m):
            x[i] = rand(n, k) * torch.exp(rand(n, 1))
        st = dict(x=x, out=dict(q=_store((m, n, k), E4M3),
                                scale=_store((m, -(-n // case["block_rows"]), _blocks(k)), torch.float32)))
    else:
        rows, groups = case["rows"], case["groups"]
        k = case["k"] if op == "gemm" else case["d"]
        n_out = case["n"] if op == "gemm" else case["d"]
        sizes = _group_sizes(groups, rows, case["spread"], gen)
        st = dict(offsets=torch.cat([sizes.new_zeros(1), sizes.cumsum(0)]).int(), most=int(sizes.max()))
        st["a"], st["a_scale"] = (v[0] for v in _quantize((rand(rows, k) * torch.exp(0.3 * rand(rows, 1)))[None], 1))
        if op == "gemm":
            st["b"], st["b_scale"] = _quantized_weights(groups, n_out, k, gen)
        else:
            for name, (r, c) in dict(gate=(case["h"], k), up=(case["h"], k), down=(k, case["h"])).items():
                st[name], st[name + "_scale"] = _quantized_weights(groups, r, c, gen)
        st["out"] = _store((rows, n_out), TYPES[case["out"]])
    st["case"] = case
    return st


# ---------------------------------------------------------------------------
# the plain forms: fp32, rounded once at the end
# ---------------------------------------------------------------------------
def _quantize(x, block_rows):
    """x [m][rows][cols] in fp32: its e4m3 values and the scales of its blocks."""
    m, rows, cols = x.shape
    br = -(-rows // block_rows)
    bc = _blocks(cols)
    padded = x
    if rows != br * block_rows or cols != bc * 128:
        padded = torch.nn.functional.pad(x, (0, bc * 128 - cols, 0, br * block_rows - rows))
    padded = padded.view(m, br, block_rows, bc, 128)
    scale = (padded.abs().amax(dim=(2, 4)) / 448.0).clamp_min(2.0 ** -126)
    q = (padded * (1.0 / scale)[:, :, None, :, None]).clamp(-448.0, 448.0).to(E4M3)
    return q.view(m, br * block_rows, bc * 128)[:, :rows, :cols], scale


def _values(q, scale, block_rows):
    """The fp32 values that e4m3 codes [m][rows][cols] with block scales stand for."""
    m, rows, cols = q.shape
    v = q.float()
    if block_rows > 1 and rows % block_rows == 0 and cols % 128 == 0:
        v.view(m, rows // block_rows, block_rows, cols // 128, 128).mul_(scale[:, :, None, :, None])
        return v
    across = torch.arange(cols, device=q.device) // 128
    down = torch.arange(rows, device=q.device) // block_rows
    return v.mul_(scale[:, down][:, :, across])


def _rows_of_groups(st):
    """[groups][most] row numbers, and which of them exist."""
    offs = st["offsets"].long()
    at = offs[:-1, None] + torch.arange(max(1, st["most"]), device=offs.device)
    there = at < offs[1:, None]
    return torch.where(there, at, torch.zeros_like(at)), there


def _product(a, at, b):
    """[groups][most][n] products of the groups' rows of a with b [groups][n][k]."""
    return torch.bmm(a[at], b.transpose(1, 2))


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "norm":
        t = TYPES[case["dtype"]]
        s = st["x"] if st["residual"] is None else (st["x"].float() + st["residual"].float()).to(t)
        r = (1.0 / torch.sqrt(s.double().square().mean(1, keepdim=True) + EPS)).float()
        v = s.float() * r * st["w"].float()
        q, scale = _quantize(v[None], 1)
        return dict(res=s.clone(), xn=v.to(t), q=q[0], scale=scale[0])
    if op == "quantize":
        q, scale = _quantize(st["x"].float(), case["block_rows"])
        return dict(q=q, scale=scale)
    at, there = _rows_of_groups(st)
    a = _values(st["a"][None], st["a_scale"][None], 1)[0]
    if op == "gemm":
        y = _product(a, at, _values(st["b"], st["b_scale"], 128))
    else:
        gate = _product(a, at, _values(st["gate"], st["gate_scale"], 128))
        up = _product(a, at, _values(st["up"], st["up_scale"], 128))
        act = gate / (1.0 + torch.exp(-gate)) * up
        act = _values(*_quantize(act, 1), 1)
        y = torch.bmm(act, _values(st["down"], st["down_scale"], 128).transpose(1, 2))
    return y[there].to(TYPES[case["out"]])


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
_kept = {}


def _plan(case):
    """The layer config and the workspace that a user's program keeps for these sizes."""
    key = tuple(sorted((k, v) for k, v in case.items() if k != "name"))
    if key not in _kept:
        import sparse_mixture_experts_rmsnorm_b200 as moe
        if len(_kept) > 8:
            _kept.clear()
        op = case["op"]
        if op == "norm":
            _kept[key] = moe, moe.Config(case["rows"], case["d"], 1, 1, 16, dtype=case["dtype"], rms_eps=EPS), None
        elif op == "quantize":
            _kept[key] = moe, None, None
        elif op == "gemm":
            _kept[key] = moe, None, moe.workspace_gemm_fp8(case["groups"], case["rows"], case["n"], case["k"])
        else:
            cfg = moe.Config(case["rows"], case["d"], case["groups"], 1, case["h"], dtype=case["out"])
            _kept[key] = moe, cfg, moe.workspace_fp8(cfg)
    return _kept[key]


def run(st):
    if not own:
        return _plain(st)
    case, out = st["case"], st["out"]
    moe, cfg, ws = _plan(case)
    op = case["op"]
    if op == "norm":
        moe.moe_add_rmsnorm(cfg, st["x"], st["residual"], st["w"], out["res"], out["xn"], out["q"], out["scale"])
    elif op == "quantize":
        moe.moe_quantize_fp8(case["dtype"], case["block_rows"], case["mats"], case["rows"], case["cols"], st["x"],
                             out["q"], out["scale"])
    elif op == "gemm":
        offsets = st["offsets"] if case["groups"] > 1 else None
        moe.moe_gemm_fp8(case["groups"], offsets, case["rows"], case["n"], case["k"], st["a"], st["a_scale"],
                         st["b"], st["b_scale"], case["out"], out, ws)
    else:
        offsets = st["offsets"] if case["groups"] > 1 else None
        moe.moe_expert_ffn_fp8(cfg, case["groups"], offsets, case["rows"], st["a"], st["a_scale"], st["gate"],
                               st["gate_scale"], st["up"], st["up_scale"], st["down"], st["down_scale"], case["h"],
                               out, ws)
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _touched(case):
    """Groups that have rows: their expected number (weights of the others are not read)."""
    g, rows = case["groups"], case["rows"]
    if case["spread"] == "ragged":
        g = max(1.0, g * 0.67)
    if case["spread"] == "skewed":
        share = 1.0 / (9.0 * g + g - 1)
        return 1 + (g - 1) * (1 - (1 - share) ** rows)
    return g * (1 - (1 - 1.0 / g) ** rows) if g > 1 else 1


def work(case):
    op = case["op"]
    size = lambda t: 2 if t == "bf16" else 4  # noqa: E731
    if op == "norm":
        n, d, e = case["rows"], case["d"], size(case["dtype"])
        return dict(bytes=n * d * (e * (4 if case["residual"] else 3) + 1) + 4 * n * _blocks(d) + d * e,
                    flops=8 * n * d)
    if op == "quantize":
        n = case["mats"] * case["rows"] * case["cols"]
        scales = case["mats"] * -(-case["rows"] // case["block_rows"]) * _blocks(case["cols"])
        return dict(bytes=n * (size(case["dtype"]) + 1) + 4 * scales, flops=3 * n)
    rows, out = case["rows"], size(case["out"])
    if op == "gemm":
        n, k = case["n"], case["k"]
        b = n * k + 4 * _blocks(n) * _blocks(k)
        return dict(bytes=rows * (k + 4 * _blocks(k)) + _touched(case) * b + rows * n * out, flops=2 * rows * n * k)
    d, h = case["d"], case["h"]
    b = 3 * (d * h + 4 * _blocks(d) * _blocks(h))
    return dict(bytes=rows * (d + 4 * _blocks(d)) + _touched(case) * b + rows * d * out, flops=6 * rows * d * h)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_64(v):
    """v rounded to the nearest e4m3 value (ties to even, saturated at 448), in 64 bits."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3.0)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _spread_64(scale, rows, cols, block_rows):
    return scale.repeat_interleave(block_rows, -2)[..., :rows, :].repeat_interleave(128, -1)[..., :cols]


def _quantize_64(x, block_rows):
    """x [rows][cols]: (e4m3 values, scales), block by block of 128 columns."""
    rows, cols = x.shape
    br, bc = -(-rows // block_rows), -(-cols // 128)
    big = torch.zeros((br * block_rows, bc * 128), dtype=torch.float64, device=x.device)
    big[:rows, :cols] = x.abs()
    scale = big.reshape(br, block_rows, bc, 128).amax(3).amax(1).div(448.0).clamp_min(2.0 ** -126)
    return _e4m3_64(x / _spread_64(scale, rows, cols, block_rows)), scale


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        total = st["x"].double()
        if st["residual"] is not None:
            total = total + st["residual"].double()
        s = total.to(st["x"].dtype).double()  # the norm is of the sum as it is stored
        v = s * torch.rsqrt((s * s).sum(1, keepdim=True) / case["d"] + EPS) * st["w"].double()
        q, scale = _quantize_64(v, 1)
        return dict(res=total, xn=v, q=q, scale=scale)
    if op == "quantize":
        qs = [_quantize_64(m.double(), case["block_rows"]) for m in st["x"]]
        return dict(q=torch.stack([q for q, _ in qs]), scale=torch.stack([s for _, s in qs]))
    offs = st["offsets"].tolist()

    def weights(name, g):
        q = st[name][g].double()
        return q * _spread_64(st[name + "_scale"][g].double(), q.shape[0], q.shape[1], 128)

    a = st["a"].double() * _spread_64(st["a_scale"].double(), st["a"].shape[0], st["a"].shape[1], 1)
    y = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    for g in range(case["groups"]):
        x = a[offs[g]:offs[g + 1]]
        if not len(x):
            continue
        if op == "gemm":
            y[offs[g]:offs[g + 1]] = x @ weights("b", g).T
            continue
        z = x @ weights("gate", g).T
        q, scale = _quantize_64(z * torch.sigmoid(z) * (x @ weights("up", g).T), 1)
        y[offs[g]:offs[g + 1]] = (q * _spread_64(scale, q.shape[0], q.shape[1], 1)) @ weights("down", g).T
    return y
