"""The 8-bit floating point operators: what is measured, in their plain form and through the library.

* ``quantize``: e4m3 codes with a scale for each group of 128 channels of a row (activations) or for
  each 128 x 128 block (weights).
* ``norm``: RMS norm of residual + x, the sum kept as the new residual, the normalised rows as e4m3
  codes with a scale per group of 128.
* ``gemm``: the product of two such matrices, with the epilogues of a decoder layer.
* ``mlp``: the three together, as a decoder's MLP block runs them.

A group's scale is max(largest magnitude, 448 * 2^-126) / 448 and its codes are e4m3(x * (448 / that
magnitude)).  Row scales are stored group-major, [ceil(cols / 128)][rows] with the pitch a multiple of 4;
block scales are [ceil(rows / 128)][ceil(cols / 128)].
"""
import torch

own = False

E4M3 = torch.float8_e4m3fn
TOP = 448.0                    # the largest e4m3 number
TINY = TOP * 2.0 ** -126       # the smallest magnitude a group's scale stands for
GROUP = 128
EPS = 1e-5

STORE_F32, ADD_F32, SWIGLU_FP8, STORE_BF16 = 0, 1, 2, 3
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the attention output of a blended prefill's recomputed rows, before the output projection
        {"name": "quantize_rows_535x4096", "kind": "quantize", "rows": 535, "cols": 4096, "block": 1, "x": "bf16"},
        # a Yi-34B-shaped gate matrix, quantised once when a model is loaded
        {"name": "quantize_weights_20480x7168", "kind": "quantize", "rows": 20480, "cols": 7168, "block": 128, "x": "bf16"},
        # one decoded token (the smallest call: its latency counts)
        {"name": "norm_1x4096", "kind": "norm", "rows": 1, "cols": 4096, "x": "bf16", "res": "f32", "weight": False},
        # the recomputed rows of a blended Yi-34B-shaped prompt of 8320 tokens
        {"name": "norm_1357x7168", "kind": "norm", "rows": 1357, "cols": 7168, "x": "bf16", "res": "f32", "weight": False},
        # a full prefill at the Llama-70B width with a bf16 residual stream and norm weights
        {"name": "norm_8320x8192", "kind": "norm", "rows": 8320, "cols": 8192, "x": "bf16", "res": "bf16", "weight": True},
        # q, k and v of one decoded token at the Mistral-7B shape
        {"name": "gemm_1x6144x4096", "kind": "gemm", "m": 1, "n": 6144, "k": 4096, "epilogue": STORE_F32},
        # the down projection of a batch of 16 decoded tokens, added to the residual
        {"name": "gemm_16x4096x14336_add", "kind": "gemm", "m": 16, "n": 4096, "k": 14336, "epilogue": ADD_F32},
        # an odd batch at the Llama-7B shape whose last group of channels is short
        {"name": "gemm_77x11008x4112_bf16", "kind": "gemm", "m": 77, "n": 11008, "k": 4112, "epilogue": STORE_BF16},
        # gate and up of the recomputed rows of a blended Mistral-7B-shaped prompt
        {"name": "gemm_535x28672x4096_swiglu", "kind": "gemm", "m": 535, "n": 28672, "k": 4096, "epilogue": SWIGLU_FP8},
        # the down projection of the recomputed rows of a blended Yi-34B-shaped prompt
        {"name": "gemm_1357x7168x20480_add", "kind": "gemm", "m": 1357, "n": 7168, "k": 20480, "epilogue": ADD_F32},
        # gate and up of a full Yi-34B-shaped prefill
        {"name": "gemm_8320x40960x7168_swiglu", "kind": "gemm", "m": 8320, "n": 40960, "k": 7168, "epilogue": SWIGLU_FP8},
        # a whole Mistral-7B-shaped MLP block of a batch of 64 decoded tokens
        {"name": "mlp_64x4096x14336", "kind": "mlp", "m": 64, "d": 4096, "ffn": 14336},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(["quantize", "norm", "gemm", "gemm", "gemm", "mlp"])
    if kind == "quantize":
        return {"kind": kind, "rows": _log(rng, 1, 20480), "cols": 16 * _log(rng, 8, 448), "block": rng.choice([1, 128]),
                "x": rng.choice(["bf16", "f32"])}
    if kind == "norm":
        return {"kind": kind, "rows": _log(rng, 1, 8320), "cols": 16 * _log(rng, 8, 512), "x": rng.choice(["bf16", "f32"]),
                "res": rng.choice(["bf16", "f32", "none"]), "weight": rng.choice([True, False])}
    if kind == "gemm":
        return {"kind": kind, "m": _log(rng, 1, 8320), "n": 32 * _log(rng, 4, 896), "k": 16 * _log(rng, 8, 512),
                "epilogue": rng.choice([STORE_F32, ADD_F32, SWIGLU_FP8, STORE_BF16])}
    return {"kind": kind, "m": _log(rng, 1, 1024), "d": 16 * _log(rng, 32, 256), "ffn": 16 * _log(rng, 64, 896)}


# ------------------------------------------------------------------------------------- plain forms
def _amax(x, block):
    """Largest magnitude of each group of x [rows, cols]: [rows, groups] (block 1) or [row blocks, groups]."""
    rows, cols = x.shape
    g = -(-cols // GROUP)
    r = -(-rows // block)
    x = torch.nn.functional.pad(x.abs(), (0, g * GROUP - cols, 0, r * block - rows))
    return x.view(r, block, g, GROUP).amax(dim=(1, 3)).clamp(min=TINY)


def _spread(s, rows, cols, block):
    """A value per group as a value per element."""
    return s.repeat_interleave(GROUP, dim=1)[:, :cols].repeat_interleave(block, dim=0)[:rows]


def _quantize(x, block=1):
    """Codes of x (32 or 64 bits) and its scales: [groups, rows] for rows, [row blocks, groups] for blocks."""
    rows, cols = x.shape
    a = _amax(x, block)
    codes = (x * _spread(TOP / a, rows, cols, block)).clamp(-TOP, TOP).to(E4M3)
    s = a / TOP
    return codes, (s.t().contiguous() if block == 1 else s)


def _values(codes, scales, block, dtype):
    s = scales.t() if block == 1 else scales
    return codes.to(dtype) * _spread(s.to(dtype), codes.shape[0], codes.shape[1], block)


def _norm(x, res, weight):
    h = x if res is None else res + x
    y = h / torch.sqrt((h * h).mean(dim=1, keepdim=True) + EPS)
    return h, y if weight is None else y * weight


def _silu(x):
    return x / (1 + torch.exp(-x))


def _product(s, dtype):
    """The accumulators of one product: one matrix, or gate and up."""
    a = _values(s["a"], s["a_scales"], 1, dtype)
    return [a @ _values(b, bs, 128, dtype).t() for b, bs in zip(s["b"], s["b_scales"])]


# ------------------------------------------------------------------------------------------ inputs
def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, rows, cols):
    """Rows as they leave a norm or an attention: unit variance, a few channels of far larger values."""
    x = _rand(gen, rows, cols)
    loud = torch.randint(0, cols, (max(1, cols // 256),), generator=gen, device="cuda")
    x[:, loud] *= 20.0
    return x


def _weights(gen, rows, cols):
    """A weight matrix's codes and block scales (values of standard deviation 0.02)."""
    return _quantize(_rand(gen, rows, cols) * 0.02, 128)


def _row_scales(rows, cols):
    return torch.empty(-(-cols // GROUP), -(-rows // 4) * 4, dtype=torch.float32, device="cuda")[:, :rows]


def _coded(gen, rows, cols):
    """Activations as codes and scales, the scales with the pitch that the product reads."""
    codes, s = _quantize(_activations(gen, rows, cols))
    scales = _row_scales(rows, cols)
    scales.copy_(s)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind = case["kind"]
    s = {"kind": kind}
    if kind == "quantize":
        rows, cols, block = case["rows"], case["cols"], case["block"]
        x = _activations(gen, rows, cols) if block == 1 else _rand(gen, rows, cols) * 0.02
        s.update(x=x.to(DT[case["x"]]), block=block, codes=torch.empty(rows, cols, dtype=E4M3, device="cuda"))
        s["scales"] = _row_scales(rows, cols) if block == 1 else torch.empty(
            -(-rows // 128), -(-cols // GROUP), dtype=torch.float32, device="cuda")
    elif kind == "norm":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _rand(gen, rows, cols).to(DT[case["x"]])
        s["res"] = None if case["res"] == "none" else (4.0 * _activations(gen, rows, cols)).to(DT[case["res"]])
        s["weight"] = (1.0 + 0.1 * _rand(gen, cols)).to(DT[case["x"]]) if case["weight"] else None
        s["res_out"] = None if s["res"] is None else torch.empty_like(s["res"])
        s.update(codes=torch.empty(rows, cols, dtype=E4M3, device="cuda"), scales=_row_scales(rows, cols))
    elif kind == "gemm":
        m, n, k, e = case["m"], case["n"], case["k"], case["epilogue"]
        s["epilogue"] = e
        s["a"], s["a_scales"] = _coded(gen, m, k)
        width = n // 2 if e == SWIGLU_FP8 else n
        s["b"], s["b_scales"] = zip(*[_weights(gen, width, k) for _ in range(2 if e == SWIGLU_FP8 else 1)])
        s["addend"] = 4.0 * _activations(gen, m, n) if e == ADD_F32 else None
        s["c"] = torch.empty(m, width, device="cuda", dtype={SWIGLU_FP8: E4M3, STORE_BF16: torch.bfloat16}.get(e, torch.float32))
        s["c_scales"] = _row_scales(m, width) if e == SWIGLU_FP8 else None
    else:
        m, d, ffn = case["m"], case["d"], case["ffn"]
        s["x"] = _rand(gen, m, d).to(torch.bfloat16)
        s["res"] = (4.0 * _activations(gen, m, d)).to(torch.bfloat16)
        s["weight"] = (1.0 + 0.1 * _rand(gen, d)).to(torch.bfloat16)
        s["gate"], s["up"], s["down"] = _weights(gen, ffn, d), _weights(gen, ffn, d), _weights(gen, d, ffn)
        s["res_out"] = torch.empty_like(s["res"])
        s.update(codes=torch.empty(m, d, dtype=E4M3, device="cuda"), scales=_row_scales(m, d))
        s.update(mid=torch.empty(m, ffn, dtype=E4M3, device="cuda"), mid_scales=_row_scales(m, ffn))
        s["c"] = torch.empty(m, d, dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------------------------------ passes
def run(s):
    kind = s["kind"]
    if own:
        import rag_non_prefix_gb300 as cb

        if kind == "quantize":
            return cb.cb_quantize(s["x"], s["block"], s["codes"], s["scales"])
        if kind == "norm":
            codes, scales, res = cb.cb_add_rmsnorm_quantize(s["x"], s["res"], s["weight"], EPS, s["res_out"], s["codes"], s["scales"])
            return {"codes": codes, "scales": scales, "residual": res}
        if kind == "gemm":
            two = len(s["b"]) == 2
            cb.cb_gemm_scaled(s["a"], s["a_scales"], s["b"][0], s["b_scales"][0], s["c"], s["epilogue"],
                           B2=s["b"][1] if two else None, B2_scales=s["b_scales"][1] if two else None,
                           addend=s["addend"], C_scales=s["c_scales"])
            return (s["c"], s["c_scales"]) if two else s["c"]
        cb.cb_add_rmsnorm_quantize(s["x"], s["res"], s["weight"], EPS, s["res_out"], s["codes"], s["scales"])
        cb.cb_gemm_scaled(s["codes"], s["scales"], *s["gate"], s["mid"], SWIGLU_FP8, B2=s["up"][0], B2_scales=s["up"][1],
                       C_scales=s["mid_scales"])
        cb.cb_gemm_scaled(s["mid"], s["mid_scales"], *s["down"], s["c"], STORE_BF16)
        return {"out": s["c"], "residual": s["res_out"]}

    if kind == "quantize":
        return _quantize(s["x"].float(), s["block"])
    if kind in ("norm", "mlp"):
        h, y = _norm(s["x"].float(), None if s["res"] is None else s["res"].float(),
                     None if s["weight"] is None else s["weight"].float())
        codes, scales = _quantize(y)
        res = None if s["res"] is None else h.to(s["res"].dtype)
        if kind == "norm":
            return {"codes": codes, "scales": scales, "residual": res}
        a = _values(codes, scales, 1, torch.float32)
        gate, up = (a @ _values(*s[w], 128, torch.float32).t() for w in ("gate", "up"))
        mid = _values(*_quantize(_silu(gate) * up), 1, torch.float32)
        return {"out": (mid @ _values(*s["down"], 128, torch.float32).t()).to(torch.bfloat16), "residual": res}
    acc = _product(s, torch.float32)
    if s["epilogue"] == SWIGLU_FP8:
        return _quantize(_silu(acc[0]) * acc[1])
    if s["epilogue"] == ADD_F32:
        return s["addend"] + acc[0]
    return acc[0].to(s["c"].dtype)


# -------------------------------------------------------------------------------- 64-bit definition
def _blocks64(x):
    """(codes, scales) of the rows of x in 64 bits, from the definition, group by group."""
    rows, cols = x.shape
    codes, scales = torch.empty_like(x), []
    for c in range(0, cols, GROUP):
        part = x[:, c:c + GROUP]
        top = torch.maximum(part.abs().max(dim=1).values, torch.tensor(TINY, dtype=torch.float64, device=x.device))
        scales.append(top / TOP)
        q = part * TOP / top[:, None]
        # e4m3: 3 fraction bits, the smallest exponent -6; nearest, ties to even
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        codes[:, c:c + GROUP] = torch.clamp(torch.round(q / step) * step, -TOP, TOP)
    return codes, torch.stack(scales)


def _matmul64(codes, scales, b, b_scales):
    """sum over k of A B^T in 64 bits, one group of 128 channels after the other."""
    m, k = codes.shape
    out = torch.zeros(m, b.shape[0], dtype=torch.float64, device=codes.device)
    block_of = torch.arange(b.shape[0], device=b.device) // 128
    for g, c in enumerate(range(0, k, 1024)):
        e = min(k, c + 1024)
        of = torch.arange(c, e, device=b.device) // GROUP
        left = codes[:, c:e].double() * scales.double().t()[:, of]
        right = b[:, c:e].double() * b_scales.double()[block_of][:, of]
        out += left @ right.t()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind == "quantize":
        x = s["x"].double()
        if s["block"] == 1:
            return _blocks64(x)
        rows, cols = x.shape
        codes = torch.empty_like(x)
        scales = torch.empty(s["scales"].shape, dtype=torch.float64, device=x.device)
        for r in range(0, rows, 128):
            # one block of rows as one long row per group
            part = x[r:r + 128]
            g = -(-cols // GROUP)
            wide = torch.nn.functional.pad(part, (0, g * GROUP - cols)).view(-1, g, GROUP).transpose(0, 1).reshape(g, -1)
            top = torch.maximum(wide.abs().max(dim=1).values, torch.tensor(TINY, dtype=torch.float64, device=x.device))
            scales[r // 128] = top / TOP
            q = part * TOP / top.repeat_interleave(GROUP)[:cols]
            step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
            codes[r:r + 128] = torch.clamp(torch.round(q / step) * step, -TOP, TOP)
        return codes, scales
    if kind in ("norm", "mlp"):
        h = s["x"].double() + (0 if s["res"] is None else s["res"].double())
        y = h * torch.rsqrt(h.square().sum(dim=1, keepdim=True) / h.shape[1] + EPS)
        if s["weight"] is not None:
            y = y * s["weight"].double()
        codes, scales = _blocks64(y)
        res = None if s["res"] is None else h
        if kind == "norm":
            return {"codes": codes, "scales": scales, "residual": res}
        gate, up = _matmul64(codes, scales, *s["gate"]), _matmul64(codes, scales, *s["up"])
        return {"out": _matmul64(*_blocks64(gate * torch.sigmoid(gate) * up), *s["down"]), "residual": res}
    acc = [_matmul64(s["a"], s["a_scales"], b, bs) for b, bs in zip(s["b"], s["b_scales"])]
    if s["epilogue"] == SWIGLU_FP8:
        return _blocks64(acc[0] * torch.sigmoid(acc[0]) * acc[1])
    return acc[0] + s["addend"].double() if s["epilogue"] == ADD_F32 else acc[0]


# -------------------------------------------------------------------------------------------- work
def _scale_bytes(rows, cols, block=1):
    return 4 * -(-rows // block) * -(-cols // GROUP)


def work(case):
    size = {"bf16": 2, "f32": 4, "none": 0}
    kind = case["kind"]
    if kind == "quantize":
        r, c = case["rows"], case["cols"]
        return {"bytes": r * c * (size[case["x"]] + 1) + _scale_bytes(r, c, case["block"]), "flops": 3 * r * c}
    if kind == "norm":
        r, c = case["rows"], case["cols"]
        return {"bytes": r * c * (size[case["x"]] + 2 * size[case["res"]] + 1) + _scale_bytes(r, c)
                + (c * size[case["x"]] if case["weight"] else 0), "flops": 8 * r * c}
    if kind == "gemm":
        m, n, k, e = case["m"], case["n"], case["k"], case["epilogue"]
        width = n // 2 if e == SWIGLU_FP8 else n
        out = {STORE_F32: 4 * m * n, ADD_F32: 8 * m * n, SWIGLU_FP8: m * width + _scale_bytes(m, width),
               STORE_BF16: 2 * m * n}[e]
        return {"bytes": m * k + n * k + _scale_bytes(m, k) + _scale_bytes(n, k, 128) + out, "flops": 2 * m * n * k}
    m, d, f = case["m"], case["d"], case["ffn"]
    return {"bytes": 3 * d * f + 3 * _scale_bytes(f, d, 128) + m * d * 8 + 2 * d, "flops": 6 * m * d * f}
