"""Measured cases of the 4-bit tensors, the policy loss and the Muon step:
microscaled 4-bit quantisation (MXFP4, NVFP4; as it lies and transposed),
dequantisation and the product of two such tensors, the clipped policy loss
over packed sequences with its gradient, and the update of weight matrices by
their orthogonalised momentum.

``run`` computes each operator in elementary torch operations in 32 bits (64
where the sums are long), or, with ``own`` set, through the package's entry
points.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}
BLOCK = {"nvfp4": 16, "mxfp4": 32}          # elements that share a scale
FP8 = torch.float8_e4m3fn
# The quintic of the Newton-Schulz products (K. Jordan, "Muon: an optimizer
# for hidden layers in neural networks", 2024).
QUINTIC = (3.4445, -4.7750, 2.0315)
MOST_PRODUCT = 2 * 16384 * 28672 * 8192     # operations of the largest product
MOST_EXACT = 1.2e13                         # of a case that 64 bits are asked of
MOST_MUON = 2 * 5 * (4 * 4096 * 4096 * 14336 + 2 * 4096 ** 3)


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # a layer's gradient or weight before its two backward products: the
        # codes as it lies and those of its transpose, with the tensor's scale
        {"name": "fp4 quant, both ways", "op": "quant", "fmt": "nvfp4", "rows": 16384, "cols": 8192,
         "pad": 0, "dtype": "bf16", "both": True},
        # activations before one product, power-of-two scales
        {"name": "fp4 quant, activations", "op": "quant", "fmt": "mxfp4", "rows": 16384, "cols": 8192,
         "pad": 0, "dtype": "bf16", "both": False},
        # a decoding step's few rows: latency
        {"name": "fp4 quant, few rows", "op": "quant", "fmt": "nvfp4", "rows": 7, "cols": 4128,
         "pad": 8, "dtype": "f16", "both": False},
        # a whole weight back in 16 bits (a check, an export)
        {"name": "fp4 dequant, weight", "op": "dequant", "fmt": "nvfp4", "rows": 28672, "cols": 8192,
         "pad": 0, "dtype": "bf16"},
        # a small odd tensor in 32 bits
        {"name": "fp4 dequant, odd", "op": "dequant", "fmt": "mxfp4", "rows": 333, "cols": 992,
         "pad": 1, "dtype": "f32"},
        # one token through the ffn: the weight is read once
        {"name": "fp4 product, one token", "op": "product", "fmt": "nvfp4", "m": 1, "n": 28672,
         "k": 8192, "pad": 0, "dtype": "bf16"},
        # a ragged batch of sequences' tokens, 32-bit result for a sum
        {"name": "fp4 product, ragged", "op": "product", "fmt": "mxfp4", "m": 1111, "n": 4099,
         "k": 4128, "pad": 5, "dtype": "f32"},
        # the training batch through the ffn (the block-scaled FP8 product's size)
        {"name": "fp4 product, batch", "op": "product", "fmt": "nvfp4", "m": 16384, "n": 28672,
         "k": 8192, "pad": 0, "dtype": "bf16"},
        # one micro-batch of short answers: latency
        {"name": "policy loss, micro-batch", "op": "policy", "tokens": 4099, "seqs": 16,
         "reduction": "sequence", "masked": True, "per_token": False, "ref": True, "dual": 0.0,
         "grad": True},
        # a whole step's samples, long answers of very different lengths
        {"name": "policy loss, batch", "op": "policy", "tokens": 8388608, "seqs": 2048,
         "reduction": "token", "masked": True, "per_token": True, "ref": True, "dual": 3.0,
         "grad": True},
        # a small model's matrices: latency of many dependent products
        {"name": "muon, small matrices", "op": "muon", "count": 12, "rows": 256, "cols": 768,
         "grad": "f32", "copy": True, "nesterov": True, "steps": 5},
        # two ffn matrices of a layer (hidden 4096, ffn 14336)
        {"name": "muon, ffn matrices", "op": "muon", "count": 2, "rows": 14336, "cols": 4096,
         "grad": "f32", "copy": True, "nesterov": True, "steps": 5},
    ]


def _log_int(rng, lo, hi):
    """An integer from [lo, hi], uniform over the logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["quant", "dequant", "product", "product", "policy", "muon"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    fmt = rng.choice(["nvfp4", "mxfp4"])
    if op in ("quant", "dequant"):
        both = op == "quant" and rng.choice([True, False])
        cols = 32 * _log_int(rng, 1, 512)
        rows = _log_int(rng, 1, min(65536, 16384 * 8192 * 2 // (cols * BYTES[dtype])))
        if both:
            rows = -(-rows // 32) * 32
        case = {"op": op, "fmt": fmt, "rows": rows, "cols": cols, "pad": rng.choice([0, 0, 1, 8]),
                "dtype": dtype}
        return case | {"both": both} if op == "quant" else case
    if op == "product":
        k = 32 * _log_int(rng, 1, 448)
        n = _log_int(rng, 1, 32768)
        m = _log_int(rng, 1, max(1, min(32768, MOST_PRODUCT // (2 * k * n))))
        if rng.random() < 0.3:
            m, n = n, m
        return {"op": op, "fmt": fmt, "m": m, "n": n, "k": k, "pad": rng.choice([0, 0, 1, 8]),
                "dtype": rng.choice(["bf16", "f32"])}
    if op == "policy":
        tokens = _log_int(rng, 1, 8388608)
        return {"op": op, "tokens": tokens, "seqs": _log_int(rng, 1, min(tokens, 20000)),
                "reduction": rng.choice(["token", "sequence", "sum"]),
                "masked": rng.choice([True, False]), "per_token": rng.choice([True, False]),
                "ref": rng.choice([True, False]), "dual": rng.choice([0.0, 3.0]),
                "grad": rng.choice([True, True, False])}
    rows, cols = _log_int(rng, 1, 8192), _log_int(rng, 1, 14336)
    steps = rng.choice([5, 5, 6])
    most = int(MOST_MUON // _muon_flops(rows, cols, steps))
    return {"op": "muon", "count": _log_int(rng, 1, max(1, min(32, most, 3 * 10 ** 8 // (rows * cols)))),
            "rows": rows, "cols": cols, "grad": dtype, "copy": rng.choice([True, False]),
            "nesterov": rng.choice([True, False]), "steps": steps}


def _muon_flops(rows, cols, steps):
    """Of one matrix: the two symmetric products need half of their entries."""
    s, l = min(rows, cols), max(rows, cols)
    return steps * (s * (s + 1) * (l + s) + 2 * s * s * l)


# ---- inputs -----------------------------------------------------------------

class State:
    pass


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = State()
    s.case = case
    {"quant": _prepare_quant, "dequant": _prepare_dequant, "product": _prepare_product,
     "policy": _prepare_policy, "muon": _prepare_muon}[case["op"]](s, case, gen)
    return s


def _activations(gen, rows, cols, dtype):
    """Values of order one with a few hot channels, as in a residual stream."""
    hot = 1.0 + 20.0 * (torch.rand(cols, device=DEV, generator=gen) < 0.002)
    x = torch.empty(rows, cols, dtype=TYPES[dtype], device=DEV)
    step = max(1, (1 << 26) // cols)
    for r in range(0, rows, step):
        part = x[r:r + step]
        part.copy_(torch.randn(part.shape, device=DEV, generator=gen) * hot)
    return x


def _padded(rows, cols, pad, dtype):
    return torch.zeros(rows, cols + pad, dtype=TYPES[dtype], device=DEV)[:, :cols]


def _tiles(rows, cols, fmt):
    """A scale buffer's shape: tiles of 128 rows and 4 scales, as
    [row tiles, scale tiles, 32, 4, 4]."""
    return -(-rows // 128), -(-cols // (4 * BLOCK[fmt])), 32, 4, 4


def _prepare_quant(s, case, gen):
    rows, cols, fmt = case["rows"], case["cols"], case["fmt"]
    s.x = _padded(rows, cols, case["pad"], case["dtype"])
    s.x.copy_(_activations(gen, rows, cols, case["dtype"]))
    byte = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device=DEV)  # noqa: E731
    s.q, s.scales = byte(rows, cols // 2), byte(*_tiles(rows, cols, fmt))
    s.qt = s.scales_t = None
    if case["both"]:
        s.qt, s.scales_t = byte(cols, rows // 2), byte(*_tiles(cols, rows, fmt))
    s.ts = torch.zeros(1, device=DEV) if fmt == "nvfp4" else None
    s.ws = None
    if own and fmt == "nvfp4":
        import mixed_precision_numerics_gradscaler_gb300 as gs
        s.ws = torch.empty(gs.gs_ws_bytes(), dtype=torch.uint8, device=DEV)


def _prepare_dequant(s, case, gen):
    fmt = case["fmt"]
    x = _activations(gen, case["rows"], case["cols"], "bf16")
    s.ts = _tensor_scale(x) if fmt == "nvfp4" else None
    s.q, s.scales = _quantise(x, fmt, s.ts)
    s.y = _padded(case["rows"], case["cols"], case["pad"], case["dtype"])


def _prepare_product(s, case, gen):
    m, n, k, fmt = case["m"], case["n"], case["k"], case["fmt"]
    a = _activations(gen, m, k, "bf16")
    b = _activations(gen, n, k, "bf16") * 0.02
    s.ta, s.tb = (_tensor_scale(a), _tensor_scale(b)) if fmt == "nvfp4" else (None, None)
    s.qa, s.sa = _quantise(a, fmt, s.ta)
    s.qb, s.sb = _quantise(b, fmt, s.tb)
    s.d = _padded(m, n, case["pad"], case["dtype"])


def _prepare_policy(s, case, gen):
    tokens, seqs = case["tokens"], case["seqs"]
    rand = lambda n: torch.rand(n, device=DEV, generator=gen)  # noqa: E731
    randn = lambda n: torch.randn(n, device=DEV, generator=gen)  # noqa: E731
    # lengths over two orders of magnitude, empty sequences among them
    share = torch.exp(1.5 * randn(seqs)).double()
    share[rand(seqs) < 0.02] = 0
    ends = torch.cumsum(share, 0) / share.sum().clamp(min=1e-9) * tokens
    s.offsets = torch.zeros(seqs + 1, dtype=torch.int64, device=DEV)
    s.offsets[1:] = ends.round().long().clamp(max=tokens)
    s.offsets[-1] = tokens
    s.logprob = -torch.exp(0.5 + randn(tokens))
    # policies a few updates apart, some tokens far off
    gap = 0.1 * randn(tokens) * torch.where(rand(tokens) < 0.02, 10.0, 1.0)
    s.old = s.logprob - gap
    s.ref = s.logprob + 0.2 * randn(tokens) if case["ref"] else None
    s.adv = randn(tokens if case["per_token"] else seqs)
    s.targets = None
    if case["masked"]:
        s.targets = torch.randint(0, 128256, (tokens,), device=DEV, generator=gen)
        prompt = rand(tokens) < 0.3                      # prompt and tool tokens: no loss
        s.targets[prompt] = -100
        for t in (s.logprob, s.old, s.ref):
            if t is not None:
                t[prompt] = 0.0                          # as the log probabilities come
    s.dloss = torch.full((1,), 0.25, device=DEV)         # a quarter of an accumulated step
    s.loss, s.stats = torch.zeros(1, device=DEV), torch.zeros(4, device=DEV)
    s.dlogprob = torch.zeros(tokens, device=DEV) if case["grad"] else None
    s.clip_low, s.clip_high, s.kl = _f32(0.2), _f32(0.28), _f32(0.05)
    s.ws = None
    if own:
        import mixed_precision_numerics_gradscaler_gb300 as gs
        s.ws = torch.empty(gs.gs_policy_loss_ws_bytes(tokens, seqs), dtype=torch.uint8, device=DEV)


def _prepare_muon(s, case, gen):
    shape = (case["count"], case["rows"], case["cols"])
    randn = lambda *sh: torch.randn(sh, device=DEV, generator=gen)  # noqa: E731
    s.w = randn(*shape) * 0.02
    s.wb = s.w.to(torch.bfloat16) if case["copy"] else None
    # a gradient of a few strong directions over noise, and a momentum like it
    r = min(8, case["rows"], case["cols"])
    strong = randn(shape[0], shape[1], r) @ randn(shape[0], r, shape[2])
    s.g = ((randn(*shape) + 0.3 * strong) * 1e-3).to(TYPES[case["grad"]])
    s.m = (randn(*shape) + strong) * 5e-3
    s.found_inf = torch.zeros(1, dtype=torch.int32, device=DEV)
    s.grad_norm = s.g.double().square().sum().sqrt().float().reshape(1)
    s.lr, s.mu, s.wd = _f32(2e-4), _f32(0.95), _f32(0.1)
    s.max_norm = _f32(0.5 * float(s.grad_norm))          # the step is clipped
    s.list = None
    if own:
        import mixed_precision_numerics_gradscaler_gb300 as gs
        s.list = gs.gs_muon_list_create(list(s.w), list(s.g), list(s.m),
                                        None if s.wb is None else list(s.wb))


def _f32(v):
    return float(np.float32(v))


# ---- one pass ---------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"quant": _quant, "dequant": _dequant, "product": _product, "policy": _policy,
            "muon": _muon}[s.case["op"]](s)


def _run_own(s):
    import mixed_precision_numerics_gradscaler_gb300 as gs
    case = s.case
    if case["op"] == "quant":
        gs.fp4_quant(s.x, case["fmt"], s.q, s.scales, s.ts, s.ws, s.qt, s.scales_t)
        return _quant_outputs(s)
    if case["op"] == "dequant":
        gs.fp4_dequant(s.q, s.scales, case["fmt"], s.y, s.ts)
        return {"y": s.y}
    if case["op"] == "product":
        gs.fp4_gemm_block_scaled(s.qa, s.sa, s.qb, s.sb, case["fmt"], s.d, s.ta, s.tb)
        return {"d": s.d}
    if case["op"] == "policy":
        gs.gs_policy_loss(s.logprob, s.old, s.adv, s.loss, s.ws, s.dlogprob, s.stats, s.ref, s.targets,
                          s.offsets, s.dloss, s.clip_low, s.clip_high, case["dual"],
                          0.0 if s.ref is None else s.kl, case["reduction"], per_sequence=not case["per_token"])
        return {"loss": s.loss, "stats": s.stats, "dlogprob": s.dlogprob}
    gs.gs_master_update_muon(s.list, s.found_inf, s.lr, s.mu, s.wd, case["nesterov"], case["steps"],
                             "rms", s.max_norm, s.grad_norm)
    return {"w": s.w, "copy": s.wb, "m": s.m}


def _quant_outputs(s):
    """Two codes lie in a byte: bytes are compared, so that every value and
    the sign of every zero has to be the same.  Scales as what they stand for."""
    form = (lambda t: t) if s.ts is None else lambda t: None if t is None else t.view(FP8)
    return {"q": s.q, "qt": s.qt, "scales": form(s.scales), "scales_t": form(s.scales_t), "ts": s.ts}


def _tensor_scale(x):
    amax = x.float().abs().amax().reshape(1)
    ts = amax.clamp(min=1e-12) / torch.full_like(amax, 2688.0)      # 448 * 6
    return torch.where(amax.isfinite(), ts, math.nan)


def _codes(y):
    """e2m1 codes: 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    a = y.abs()
    c = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    c += 8 * torch.signbit(y).to(torch.uint8)
    return c[:, 0::2] | (c[:, 1::2] << 4)


def _to_tiles(sc, fmt):
    """Scales [rows, blocks] in tiles of 128 rows and 4 blocks, the four of
    rows r, r + 32, r + 64, r + 96 side by side; zeros past the edges."""
    rt, kt = -(-sc.shape[0] // 128), -(-sc.shape[1] // 4)
    full = torch.zeros(rt * 128, kt * 4, dtype=torch.uint8, device=sc.device)
    full[:sc.shape[0], :sc.shape[1]] = sc
    return full.view(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).contiguous()


def _from_tiles(tiles, rows, blocks):
    rt, kt = tiles.shape[:2]
    return tiles.permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:rows, :blocks]


def _quantise(x, fmt, ts):
    rows, cols = x.shape
    b = x.float().reshape(rows, cols // BLOCK[fmt], BLOCK[fmt])
    amax = b.abs().amax(dim=2)
    if fmt == "mxfp4":
        # the exponent field is floor(log2) of a normal amax; 2 is that of the largest code
        e = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - 2, -127).clamp(-127, 127)
        scale, r = (e + 127).to(torch.uint8), torch.ldexp(torch.ones_like(amax), -e)
    else:
        s8 = (amax / (ts * 6.0)).clamp(max=448.0).to(FP8)
        d = s8.float() * ts
        scale, r = s8.view(torch.uint8), torch.where(d > 0, 1.0 / d, 0.0)
    return _codes((b * r[:, :, None]).view(rows, cols)), _to_tiles(scale, fmt)


def _quant(s):
    fmt = s.case["fmt"]
    if s.ts is not None:
        s.ts = _tensor_scale(s.x)
    s.q, s.scales = _quantise(s.x, fmt, s.ts)
    if s.qt is not None:
        s.qt, s.scales_t = _quantise(s.x.t(), fmt, s.ts)
    return _quant_outputs(s)


def _decode(q, tiles, fmt, dtype):
    """The values of codes with their block scales, without the tensor's."""
    one = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=q.device, dtype=dtype)
    one = torch.cat([one, -one])
    rows, cols = q.shape[0], 2 * q.shape[1]
    v = torch.stack([one[(q & 15).int()], one[(q >> 4).int()]], dim=2).view(rows, cols // BLOCK[fmt], BLOCK[fmt])
    sc = _from_tiles(tiles, rows, cols // BLOCK[fmt])
    sc = sc.contiguous().view(FP8).to(dtype) if fmt == "nvfp4" else torch.ldexp(torch.ones_like(sc, dtype=dtype), sc.int() - 127)
    return (v * sc[:, :, None]).view(rows, cols)


def _dequant(s):
    v = _decode(s.q, s.scales, s.case["fmt"], torch.float32)
    return {"y": (v if s.ts is None else v * s.ts).to(s.y.dtype)}


def _product(s):
    fmt = s.case["fmt"]
    d = _decode(s.qa, s.sa, fmt, torch.float32) @ _decode(s.qb, s.sb, fmt, torch.float32).t()
    return {"d": (d if s.ta is None else d * (s.ta * s.tb)).to(s.d.dtype)}


def _policy(s):
    case = s.case
    tokens, seqs = case["tokens"], case["seqs"]
    at = torch.arange(tokens, device=DEV)
    seq = torch.searchsorted(s.offsets[1:], at, right=True)
    live = torch.ones_like(at, dtype=torch.bool) if s.targets is None else s.targets >= 0
    # differences near zero: the estimate of the divergence is quadratic in them
    lp, adv = s.logprob.double(), (s.adv if case["per_token"] else s.adv[seq]).double()
    ratio = torch.exp(lp - s.old)
    plain, held = ratio * adv, ratio.clamp(1 - s.clip_low, 1 + s.clip_high) * adv
    won = torch.minimum(plain, held)
    moves = plain <= held
    clipped = ~moves
    if case["dual"]:
        floor = torch.where(adv < 0, case["dual"] * adv, -math.inf)
        clipped |= won < floor
        moves &= won >= floor
        won = torch.maximum(won, floor)
    slope = torch.where(moves, -plain, 0.0)
    kl = torch.zeros_like(lp)
    if s.ref is not None:
        away = s.ref - lp
        kl = torch.expm1(away) - away
        slope = slope - s.kl * torch.expm1(away)
    n = live.sum()
    if case["reduction"] == "sequence":
        each = torch.zeros(seqs, dtype=torch.int64, device=DEV).scatter_add_(0, seq, live.long())
        weight = 1.0 / ((each > 0).sum() * each.clamp(min=1))[seq].double()
    else:
        weight = torch.where(n > 0, 1.0 / n, 0.0) if case["reduction"] == "token" else torch.ones((), device=DEV)
    mean = lambda v: torch.where(live, v, 0.0).sum() / n.clamp(min=1)  # noqa: E731
    loss = torch.where(live, weight * (s.kl * kl - won), 0.0).sum().reshape(1)
    out = {"loss": loss.float(), "dlogprob": None,
           "stats": torch.stack([n.double(), mean(ratio), mean(clipped.double()), mean(kl)]).float()}
    if case["grad"]:
        out["dlogprob"] = torch.where(live, s.dloss * weight * slope, 0.0).float()
    return out


def _muon(s):
    case = s.case
    coef = torch.where(s.grad_norm > s.max_norm, s.max_norm / s.grad_norm, 1.0)
    g = s.g.float() * coef
    s.m.copy_(s.m * s.mu + g)
    u = g + s.m * s.mu if case["nesterov"] else s.m
    norm = u.double().square().sum(dim=(1, 2), keepdim=True).sqrt()
    x = (u / (norm + 1e-30)).float()
    wide = case["rows"] <= case["cols"]
    x = x if wide else x.transpose(1, 2)
    a, b, c = QUINTIC
    for _ in range(case["steps"]):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    x = x if wide else x.transpose(1, 2)
    step = s.lr * 0.2 * math.sqrt(max(case["rows"], case["cols"]))
    s.w.copy_(s.w * (1 - s.lr * s.wd) - step * x)
    if s.wb is not None:
        s.wb.copy_(s.w)
    return {"w": s.w, "copy": s.wb, "m": s.m}


# ---- bytes and operations ---------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("quant", "dequant"):
        n, e = case["rows"] * case["cols"], BYTES[case["dtype"]]
        codes = n // 2 + n // BLOCK[case["fmt"]]
        return {"bytes": n * e + codes * (2 if case.get("both") else 1), "flops": 4 * n}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        codes = (m + n) * (k // 2 + k // BLOCK[case["fmt"]])
        return {"bytes": codes + m * n * BYTES[case["dtype"]], "flops": 2 * m * n * k}
    if op == "policy":
        t = case["tokens"]
        each = 8 + 4 * case["ref"] + 8 * case["masked"] + 4 * case["grad"]
        return {"bytes": t * each + 4 * (t if case["per_token"] else case["seqs"]) + 8 * case["seqs"],
                "flops": 20 * t}
    n = case["count"] * case["rows"] * case["cols"]
    return {"bytes": n * (16 + BYTES[case["grad"]] + (2 if case["copy"] else 0)),
            "flops": case["count"] * _muon_flops(case["rows"], case["cols"], case["steps"])}


# ---- the definitions in 64 bits ---------------------------------------------

def exact(case, seed):
    if work(case)["flops"] > MOST_EXACT or case["op"] == "quant" and case["fmt"] == "mxfp4":
        return None                                      # too long, or whole numbers alone
    s = prepare(case, seed)
    return {"quant": _exact_quant, "dequant": _exact_dequant, "product": _exact_product,
            "policy": _exact_policy, "muon": _exact_muon}[case["op"]](s, case)


def _values(q, tiles, ts, fmt):
    """What codes and scales stand for, from the formats' fields: sign, two
    bits of exponent (bias 1), one of mantissa."""
    code = torch.stack([q & 15, q >> 4], dim=2).flatten(1).long()
    e, m = (code >> 1) & 3, (code & 1).double()
    v = torch.where(e == 0, 0.5 * m, torch.exp2((e - 1).double()) * (1 + 0.5 * m)) * (1 - 2 * (code >> 3)).double()
    rows, cols = v.shape
    r, c = torch.arange(rows, device=DEV)[:, None], (torch.arange(cols, device=DEV) // BLOCK[fmt])[None]
    # byte (r, c): tile (r / 128, c / 4), then (r % 32) * 16 + (r % 128 / 32) * 4 + c % 4
    place = ((r // 128) * tiles.shape[1] + c // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + c % 4
    byte = tiles.flatten()[place].long()
    if fmt == "mxfp4":
        return v * torch.exp2((byte - 127).double())
    e, m = byte >> 3, (byte & 7).double()
    return v * torch.where(e == 0, m * 2.0 ** -9, torch.exp2((e - 7).double()) * (1 + m / 8)) * ts.double()


def _exact_quant(s, case):
    """The scales before they are rounded; whole bytes have no such value."""
    out = {"q": None, "qt": None, "scales": None, "scales_t": None, "ts": None}
    top = max(float(s.x.double().abs().max()), 1e-12)
    out["ts"] = torch.tensor([top / 448 / 6], dtype=torch.float64, device=DEV)

    def scales(x, like):
        full = torch.zeros(like.shape[0] * 128, like.shape[1] * 4, dtype=torch.float64, device=DEV)
        part = x.double().abs().unflatten(1, (-1, 16)).amax(2) / 6 / out["ts"]
        full[:part.shape[0], :part.shape[1]] = part
        return full.unflatten(0, (-1, 4, 32)).unflatten(3, (-1, 4)).permute(0, 3, 2, 1, 4)

    out["scales"] = scales(s.x, s.scales)
    out["scales_t"] = None if s.qt is None else scales(s.x.t(), s.scales_t)
    return out


def _exact_dequant(s, case):
    return {"y": _values(s.q, s.scales, s.ts, case["fmt"])}


def _exact_product(s, case):
    return {"d": torch.einsum("mk,nk->mn", _values(s.qa, s.sa, s.ta, case["fmt"]),
                              _values(s.qb, s.sb, s.tb, case["fmt"]))}


def _exact_policy(s, case):
    tokens, seqs = case["tokens"], case["seqs"]
    lengths = s.offsets.diff()
    of = torch.repeat_interleave(torch.arange(seqs, device=DEV), lengths)
    keep = torch.ones(tokens, device=DEV, dtype=torch.float64)
    if s.targets is not None:
        keep = (s.targets >= 0).double()
    d = s.logprob.double() - s.old.double()
    adv = (s.adv if case["per_token"] else s.adv[of]).double()
    ratio = d.exp()
    # where the objective no longer follows the ratio, by the sign of the advantage
    high, low = math.inf, -math.inf
    if case["dual"]:
        high = case["dual"]
    top = torch.where(adv > 0, 1.0 + s.clip_high, high)
    bottom = torch.where(adv < 0, 1.0 - s.clip_low, low)
    out_of = ((ratio > top) | (ratio < bottom)) & (adv != 0)
    value = torch.minimum(torch.maximum(ratio, bottom), top) * adv
    value = torch.where(adv == 0, 0.0, value)
    grad = torch.where(out_of, 0.0, -ratio * adv)
    kl = torch.zeros_like(ratio)
    if s.ref is not None:
        x = s.ref.double() - s.logprob.double()
        kl = torch.where(x.abs() < 1e-3, x * x * (0.5 + x * (1 / 6 + x * (1 / 24 + x / 120))), x.exp() - 1 - x)
        grad = grad + s.kl * (1 - x.exp())
    n = float(keep.sum())
    if case["reduction"] == "sum":
        w = keep
    elif case["reduction"] == "token":
        w = keep / max(n, 1.0)
    else:
        counts = torch.zeros(seqs, dtype=torch.float64, device=DEV).index_add_(0, of, keep)
        w = keep / counts.clamp(min=1)[of] / max(1.0, float((counts > 0).sum()))
    mean = lambda v: (keep * v).sum() / max(n, 1.0)  # noqa: E731
    return {"loss": (w * (s.kl * kl - value)).sum().reshape(1),
            "stats": torch.stack([keep.sum(), mean(ratio), mean(out_of.double()), mean(kl)]),
            "dlogprob": float(s.dloss) * w * grad if case["grad"] else None}


def _exact_muon(s, case):
    norm = float(s.grad_norm)
    g = s.g.double() * min(1.0, s.max_norm / norm) if norm > 0 else s.g.double()
    m = s.mu * s.m.double() + g
    u = g + s.mu * m if case["nesterov"] else m
    u = u / torch.linalg.vector_norm(u, dim=(1, 2), keepdim=True)
    tall = case["rows"] > case["cols"]
    if tall:
        u = u.mT
    a, b, c = QUINTIC
    for _ in range(case["steps"]):
        gram = torch.einsum("bik,bjk->bij", u, u)
        u = torch.baddbmm(u, torch.baddbmm(gram, gram, gram, beta=b, alpha=c), u, beta=a)
    if tall:
        u = u.mT
    w = s.w.double()
    w = w - s.lr * (s.wd * w + 0.2 * max(case["rows"], case["cols"]) ** 0.5 * u)
    return {"w": w, "copy": w if s.wb is not None else None, "m": m}
