"""The operators of a mixed-precision training step around the cast-and-scale
path, as measured cases: layer norm (forward, backward), log probabilities of
given tokens with entropy and top alternatives (forward, backward under a loss
scale), and the AdamW step over a list of tensors with 32-bit or 8-bit states.

``run`` computes each operator in elementary torch operations in 32 bits, or,
with ``own`` set, through the package's entry points.  ``exact`` gives the same
outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}
FP8 = torch.float8_e4m3fn
M32 = 0xFFFFFFFF

# One transformer layer's matrices and norm vectors and a quarter of the
# output head, at the sizes of this repository's gradient-list workload
# (hidden 4096, kv 1024, ffn 14336, vocabulary 128256).
LAYER = "16777216*2,4194304*2,58720256*3,4096*2"
HEAD_QUARTER = "131334144"
# The small odd-sized list of the same workload family (2^20 elements).
SMALL_LIST = "300007,200003,150001,131071,100000,80000,50000,37494"


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # the norm before the output head for a handful of rows: latency
        {"name": "norm fwd, 8 rows", "op": "norm_fwd", "rows": 8, "cols": 4096, "pad": 0,
         "dtype": "bf16", "w": "bf16"},
        # a training batch's activations (the 1x128 quantiser's workload)
        {"name": "norm fwd, batch", "op": "norm_fwd", "rows": 16384, "cols": 8192, "pad": 0,
         "dtype": "bf16", "w": "f32"},
        # fp16 activations cut out of a wider buffer, odd width
        {"name": "norm bwd, odd width", "op": "norm_bwd", "rows": 4099, "cols": 1023, "pad": 2,
         "dtype": "f16", "w": "f32"},
        # the batch's backward pass
        {"name": "norm bwd, batch", "op": "norm_bwd", "rows": 16384, "cols": 8192, "pad": 0,
         "dtype": "bf16", "w": "f32"},
        # scoring the tokens of one decoding step, with alternatives
        {"name": "logprob, decode", "op": "logprob", "rows": 4, "cols": 128256, "pad": 0,
         "dtype": "bf16", "top": 20, "entropy": True},
        # scoring a batch of sampled sequences
        {"name": "logprob, batch", "op": "logprob", "rows": 4096, "cols": 128256, "pad": 0,
         "dtype": "bf16", "top": 8, "entropy": True},
        # the loss's gradient, fp16 under a loss scale, odd vocabulary, with
        # an entropy bonus
        {"name": "logprob bwd, odd vocabulary", "op": "logprob_bwd", "rows": 1021, "cols": 32003,
         "pad": 0, "dtype": "f16", "out": "f16", "entropy": True},
        # the gradient of a training batch
        {"name": "logprob bwd, batch", "op": "logprob_bwd", "rows": 8192, "cols": 128256, "pad": 0,
         "dtype": "bf16", "out": "bf16", "entropy": False},
        # a small model's update, or one shard's norms and biases: latency
        {"name": "adamw 32-bit, small list", "op": "adamw", "sizes": SMALL_LIST, "states": 32,
         "grad": "f32", "copy": True, "packed": True},
        # an update of two layers and a part of the head
        {"name": "adamw 32-bit, layers", "op": "adamw",
         "sizes": LAYER + "," + LAYER + "," + HEAD_QUARTER, "states": 32, "grad": "f32",
         "copy": True, "packed": False},
        # the same with 8-bit states
        {"name": "adamw 8-bit, small list", "op": "adamw", "sizes": SMALL_LIST, "states": 8,
         "grad": "bf16", "copy": True, "packed": False},
        {"name": "adamw 8-bit, layers", "op": "adamw",
         "sizes": LAYER + "," + LAYER + "," + HEAD_QUARTER, "states": 8, "grad": "f32",
         "copy": True, "packed": False},
    ]


def _log_int(rng, lo, hi):
    """An integer from [lo, hi], uniform over the logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "logprob", "logprob_bwd", "adamw", "adamw"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    if op in ("norm_fwd", "norm_bwd"):
        cols = _log_int(rng, 32, 16384)
        rows = _log_int(rng, 1, min(65536, 16384 * 8192 * 2 // (cols * BYTES[dtype])))
        return {"op": op, "rows": rows, "cols": cols, "pad": rng.choice([0, 0, 1, 8]),
                "dtype": dtype, "w": rng.choice(["f32", dtype])}
    if op in ("logprob", "logprob_bwd"):
        cols = _log_int(rng, 100, 200000)
        most = 4096 * 128256 if op == "logprob" else 8192 * 128256
        rows = _log_int(rng, 1, min(16384, most * 2 // (cols * BYTES[dtype])))
        case = {"op": op, "rows": rows, "cols": cols, "pad": rng.choice([0, 0, 1, 8]),
                "dtype": dtype, "entropy": rng.choice([True, False])}
        if op == "logprob":
            case["top"] = rng.choice([0, 1, 5, 20, 32])
        else:
            case["out"] = rng.choice([dtype, "f16"])
        return case
    states = rng.choice([32, 8])
    count = _log_int(rng, 1, 40)
    total = _log_int(rng, 1000, 400000000)
    shares = [rng.random() + 0.02 for _ in range(count)]
    sizes = [max(1, int(total * s / sum(shares))) for s in shares]
    return {"op": "adamw", "sizes": ",".join(str(n) for n in sizes), "states": states,
            "grad": rng.choice(["f32", "bf16", "f16"]), "copy": rng.choice([True, False]),
            "packed": states == 32 and rng.choice([True, False])}


# ---- inputs -----------------------------------------------------------------

class State:
    pass


def _numels(case):
    sizes = []
    for part in case["sizes"].split(","):
        n, _, times = part.partition("*")
        sizes += [int(n)] * int(times or 1)
    return sizes


def _rows(gen, rows, cols, pad, dtype, fill):
    """A [rows, cols] view of a buffer whose rows are `pad` elements longer."""
    buf = torch.empty(rows, cols + pad, dtype=TYPES[dtype], device=DEV)
    step = max(1, (1 << 26) // (cols + pad))
    for r in range(0, rows, step):
        part = buf[r:r + step]
        part.copy_(fill(torch.randn(part.shape, device=DEV, generator=gen)))
    return buf[:, :cols]


def _like(x, dtype=None):
    """An output buffer laid out as x, rows and padding."""
    rows, ld = x.shape[0], x.stride(0)
    return torch.zeros(rows, max(ld, x.shape[1]), dtype=dtype or x.dtype, device=DEV)[:, :x.shape[1]]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = State()
    s.case = case
    if case["op"] in ("norm_fwd", "norm_bwd"):
        _prepare_norm(s, case, gen)
    elif case["op"] in ("logprob", "logprob_bwd"):
        _prepare_logprob(s, case, gen)
    else:
        _prepare_adamw(s, case, gen)
    return s


def _prepare_norm(s, case, gen):
    rows, cols, pad, dtype = case["rows"], case["cols"], case["pad"], case["dtype"]
    # activations with an offset and a few hot channels, as a residual stream has
    hot = 1.0 + 20.0 * (torch.rand(cols + pad, device=DEV, generator=gen) < 0.002)
    s.x = _rows(gen, rows, cols, pad, dtype, lambda v: v * hot + 0.1)
    s.gamma = (1 + 0.1 * torch.randn(cols, device=DEV, generator=gen)).to(TYPES[case["w"]])
    s.beta = (0.1 * torch.randn(cols, device=DEV, generator=gen)).to(TYPES[case["w"]])
    s.eps = 1e-5
    if case["op"] == "norm_fwd":
        s.y = _like(s.x)
        s.mean = torch.empty(rows, device=DEV)
        s.rstd = torch.empty(rows, device=DEV)
        return
    # gradients under a loss scale are of order one, not of the loss's size
    s.dy = _rows(gen, rows, cols, pad, dtype, lambda v: v * 0.5)
    s.dx = _like(s.x)
    var, mean = torch.var_mean(s.x.double(), dim=1, unbiased=False)
    s.mean = mean.float()
    s.rstd = (var + s.eps).rsqrt().float()
    s.dgamma = torch.empty(cols, device=DEV)
    s.dbeta = torch.empty(cols, device=DEV)
    s.ws = None
    if own:
        import mixed_precision_numerics_gradscaler_gb300 as gs
        s.ws = torch.empty(gs.gs_layernorm_ws_bytes(rows, cols), dtype=torch.uint8, device=DEV)


def _prepare_logprob(s, case, gen):
    rows, cols, pad, dtype = case["rows"], case["cols"], case["pad"], case["dtype"]
    s.logits = _rows(gen, rows, cols, pad, dtype, lambda v: v * 2.5)
    s.targets = torch.randint(0, cols, (rows,), device=DEV, generator=gen)
    # the target and one rival stand out, as they do after some training
    at = torch.arange(rows, device=DEV)
    s.logits[at, s.targets] += (6 * torch.rand(rows, device=DEV, generator=gen)).to(s.logits.dtype)
    rival = torch.randint(0, cols, (rows,), device=DEV, generator=gen)
    s.logits[at, rival] += 8
    if rows >= 4:
        s.targets[rows // 3] = -100                      # a prompt token: no loss
        s.logits[rows // 2, cols // 2:] = -math.inf      # a constrained vocabulary
    if rows >= 100:
        s.logits[rows - 2] = -math.inf                   # nothing is allowed
    s.logprob = torch.empty(rows, device=DEV)
    s.lse = torch.empty(rows, device=DEV)
    s.entropy = torch.empty(rows, device=DEV) if case["entropy"] else None
    if case["op"] == "logprob":
        k = min(case["top"], cols)
        s.top_ids = torch.empty(rows, k, dtype=torch.int32, device=DEV) if k else None
        s.top_logprob = torch.empty(rows, k, device=DEV) if k else None
        return
    s.dlogits = _like(s.logits, TYPES[case["out"]])
    s.dlogprob = -(0.5 + torch.rand(rows, device=DEV, generator=gen)) / rows
    s.dentropy = torch.full((rows,), -0.01 / rows, device=DEV) if case["entropy"] else None
    s.loss_scale = torch.full((1,), 4096.0, device=DEV)
    step = max(1, (1 << 27) // cols)
    for r in range(0, rows, step):
        x = s.logits[r:r + step].double()
        lse = torch.logsumexp(x, dim=1)
        s.lse[r:r + step] = lse.float()
        if case["entropy"]:
            s.entropy[r:r + step] = torch.special.entr((x - _finite(lse)[:, None]).exp()).sum(1).float()


def _prepare_adamw(s, case, gen):
    sizes = _numels(case)
    pad = 1 if case["packed"] else 128
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += -(-n // pad) * pad
    live = torch.zeros(total, dtype=torch.bool, device=DEV)
    for at, n in zip(starts, sizes):
        live[at:at + n] = True

    def flat(make, dtype=torch.float32):
        return torch.where(live, make(), 0).to(dtype)

    randn = lambda: torch.randn(total, device=DEV, generator=gen)  # noqa: E731
    s.w = flat(lambda: randn() * 0.02)
    s.wb = s.w.to(torch.bfloat16) if case["copy"] else None
    # gradients over several orders of magnitude
    s.g = flat(lambda: randn() * torch.exp2(-8 * torch.rand(total, device=DEV, generator=gen)) * 1e-2,
               TYPES[case["grad"]])
    m = flat(lambda: randn() * 1e-3)
    r = flat(lambda: (randn().abs() + 0.05) * 3e-3)
    if case["states"] == 8:
        # an earlier step's states, rounded to nearest
        s.m, s.m_scale = _to_codes(m)
        s.v, s.v_scale = _to_codes(r)
    else:
        s.m, s.v, s.m_scale, s.v_scale = m, r * r, None, None
    s.step = torch.full((1,), 999, dtype=torch.int64, device=DEV)
    s.found_inf = torch.zeros(1, dtype=torch.int32, device=DEV)
    s.grad_norm = s.g.double().square().sum().sqrt().float().reshape(1)
    # betas as the 32-bit numbers that the step works with
    s.lr, s.wd, s.eps = _f32(1e-3), _f32(0.1), _f32(1e-8)
    s.beta1, s.beta2 = _f32(0.9), _f32(0.999)
    s.max_norm = _f32(0.5 * float(s.grad_norm))           # the step is clipped
    s.seed = 1234
    s.list = None
    if own:
        import mixed_precision_numerics_gradscaler_gb300 as gs
        cut = lambda t: None if t is None else [t[at:at + n] for at, n in zip(starts, sizes)]  # noqa: E731
        blocks = lambda t: None if t is None else [  # noqa: E731
            t[at // 128:at // 128 + -(-n // 128)] for at, n in zip(starts, sizes)]
        s.list = gs.gs_adamw_list_create(cut(s.w), cut(s.g), cut(s.m), cut(s.v), blocks(s.m_scale),
                                         blocks(s.v_scale), cut(s.wb))


def _f32(v):
    return float(np.float32(v))


def _finite(lse):
    """lse where it can be subtracted, 0 for a row with nothing allowed."""
    return torch.where(lse == -math.inf, torch.zeros_like(lse), lse)


def _to_codes(x):
    blocks = x.view(-1, 128)
    amax = blocks.abs().amax(dim=1).clamp(min=1e-30)
    scale = amax / torch.full_like(amax, 448.0)
    return (blocks / scale[:, None]).to(FP8).view(torch.uint8).view(-1), scale


# ---- one pass ---------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "logprob": _logprob,
            "logprob_bwd": _logprob_bwd, "adamw": _adamw}[s.case["op"]](s)


def _run_own(s):
    import mixed_precision_numerics_gradscaler_gb300 as gs
    op = s.case["op"]
    if op == "norm_fwd":
        gs.gs_layernorm_fwd(s.x, s.gamma, s.beta, s.y, s.mean, s.rstd, s.eps)
        return {"y": s.y, "mean": s.mean, "rstd": s.rstd}
    if op == "norm_bwd":
        gs.gs_layernorm_bwd(s.dy, s.x, s.gamma, s.mean, s.rstd, s.dx, s.dgamma, s.dbeta, s.ws)
        return {"dx": s.dx, "dgamma": s.dgamma, "dbeta": s.dbeta}
    if op == "logprob":
        gs.gs_token_logprob(s.logits, s.targets, s.logprob, s.lse, s.entropy, s.top_ids, s.top_logprob)
        return {"logprob": s.logprob, "lse": s.lse, "entropy": s.entropy, "top_ids": s.top_ids,
                "top_logprob": s.top_logprob}
    if op == "logprob_bwd":
        gs.gs_token_logprob_bwd(s.logits, s.targets, s.lse, s.dlogprob, s.dlogits, s.entropy,
                                s.dentropy, s.loss_scale)
        return {"dlogits": s.dlogits}
    gs.gs_master_update_adamw(s.list, s.step, s.found_inf, s.lr, s.beta1, s.beta2, s.eps, s.wd,
                              s.max_norm, s.grad_norm, s.seed)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    out = {"w": s.w, "copy": s.wb, "step": s.step}
    if s.m_scale is None:
        return out | {"m": s.m, "v": s.v}
    return out | {"m": s.m.view(FP8), "v": s.v.view(FP8), "m_scale": s.m_scale, "v_scale": s.v_scale}


def _norm_fwd(s):
    x = s.x.float()
    mean = x.mean(dim=1)
    xc = x - mean[:, None]
    rstd = torch.rsqrt((xc * xc).mean(dim=1) + s.eps)
    y = xc * rstd[:, None] * s.gamma.float() + s.beta.float()
    return {"y": y.to(s.x.dtype), "mean": mean, "rstd": rstd}


def _norm_bwd(s):
    xh = (s.x.float() - s.mean[:, None]) * s.rstd[:, None]
    dy = s.dy.float()
    dxh = dy * s.gamma.float()
    dx = (dxh - dxh.mean(dim=1, keepdim=True) - xh * (dxh * xh).mean(dim=1, keepdim=True)) * s.rstd[:, None]
    return {"dx": dx.to(s.x.dtype), "dgamma": (dy * xh).sum(dim=0), "dbeta": dy.sum(dim=0)}


def _logprob(s):
    x = s.logits.float()
    d = x - _finite(x.amax(dim=1))[:, None]
    e = torch.exp(d)
    total = e.sum(dim=1)
    lse = _finite(x.amax(dim=1)) + torch.log(total)
    valid = s.targets >= 0
    at = x.gather(1, s.targets.clamp(min=0)[:, None])[:, 0]
    logprob = torch.where(valid, torch.where(lse == -math.inf, lse, at - lse), 0.0)
    out = {"logprob": logprob, "lse": lse, "entropy": None, "top_ids": None, "top_logprob": None}
    if s.entropy is not None:
        t = torch.where(e > 0, e * d, 0.0).sum(dim=1)
        out["entropy"] = torch.where(total > 0, torch.log(total) - t / total, 0.0)
    if s.top_ids is not None:
        # one whole number for the value's order and, below it, the lowest index first
        n = x.shape[1]
        bits = (x + 0.0).view(torch.int32).long()
        order = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF) - 1)
        key = order * (1 << 20) + (n - 1 - torch.arange(n, device=x.device))
        ids = (n - 1) - (key.topk(s.top_ids.shape[1], dim=1).values & ((1 << 20) - 1))
        out["top_ids"] = ids.int()
        out["top_logprob"] = torch.where((lse == -math.inf)[:, None], -math.inf,
                                         x.gather(1, ids) - lse[:, None])
    return out


def _logprob_bwd(s):
    x = s.logits.float()
    logp = x - _finite(s.lse)[:, None]
    p = torch.exp(logp)
    live = (s.targets >= 0) & (s.lse > -math.inf)
    dlp = torch.where(live, s.dlogprob, 0.0)
    d = -dlp[:, None] * p
    at = torch.arange(x.shape[0], device=x.device)
    d[at, s.targets.clamp(min=0)] += dlp
    if s.dentropy is not None:
        d -= torch.where(p > 0, s.dentropy[:, None] * p * (logp + s.entropy[:, None]), 0.0)
    return {"dlogits": (d * s.loss_scale).to(s.dlogits.dtype)}


def _mix(x):
    """A 32-bit mixer of two multiplications (multipliers from C. Wellons'
    2018 search for low-bias mixers), in 64-bit integers."""
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & M32
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & M32
    return x ^ (x >> 16)


def _random(n, seed, step):
    """32 random bits per element of the list, from the seed, the step's
    number and the element's place."""
    i = torch.arange(n, device=DEV)
    key = _mix((seed + 0x9E3779B9 * step + 0x85EBCA6B * (i >> 32)) & M32)
    return _mix((i & M32) ^ key)


def _round_codes(x, r16):
    """x (blocks of 128) as E4M3 codes and scales, rounded up or down at
    random: 16 random bits below the three kept bits of the significand,
    carried into them, the rest cut off.  Below 2^-6 the spacing stays 2^-9,
    which adding 2^-6 makes that of the first binade."""
    blocks = x.view(-1, 128)
    amax = blocks.abs().amax(dim=1).clamp(min=1e-30)
    top = torch.full_like(amax, 448.0)
    t = blocks * (top / amax)[:, None]
    a = t.abs()
    low = a < 2.0 ** -6
    b = torch.where(low, a + 2.0 ** -6, a).view(torch.int32)
    b = ((b + (r16.view(-1, 128) << 4).int()) & -(1 << 20)).view(torch.float32)
    b = torch.where(low, b - 2.0 ** -6, b).clamp(max=448.0)
    return torch.copysign(b, t), amax / top


def _adamw(s):
    coef = torch.where(s.grad_norm > s.max_norm,
                       torch.full_like(s.grad_norm, s.max_norm) / s.grad_norm, 1.0)
    g = s.g.float() * coef
    if s.m_scale is None:
        m, v = s.m, s.v
    else:
        m = (s.m.view(FP8).float().view(-1, 128) * s.m_scale[:, None]).view(-1)
        r = (s.v.view(FP8).float().view(-1, 128) * s.v_scale[:, None]).view(-1)
        v = r * r
    m = m * s.beta1 + g * (1 - s.beta1)
    v = v * s.beta2 + (g * (1 - s.beta2)) * g
    r = torch.sqrt(v)
    s.step += 1
    step = s.step.float()
    c1 = s.lr / -torch.expm1(step * math.log(s.beta1))
    c2 = torch.rsqrt(-torch.expm1(step * math.log(s.beta2)))
    s.w.copy_(s.w * (1 - s.lr * s.wd) - (m * c1) / (r * c2 + s.eps))
    if s.wb is not None:
        s.wb.copy_(s.w)
    if s.m_scale is None:
        s.m.copy_(m)
        s.v.copy_(v)
        return _adamw_outputs(s)
    h = _random(m.numel(), s.seed, s.step)
    q, scale = _round_codes(m, h & 0xFFFF)
    s.m.copy_(q.to(FP8).view(torch.uint8).view(-1))
    s.m_scale.copy_(scale)
    q, scale = _round_codes(r, h >> 16)
    q = torch.where((r.view(-1, 128) > 0) & (q == 0), 2.0 ** -9, q)  # never below the least value
    s.v.copy_(q.to(FP8).view(torch.uint8).view(-1))
    s.v_scale.copy_(scale)
    return _adamw_outputs(s)


# ---- bytes and operations ---------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        n, e = case["rows"] * case["cols"], BYTES[case["dtype"]]
        w, rows = case["cols"] * BYTES[case["w"]], case["rows"] * 8
        if op == "norm_fwd":
            return {"bytes": 2 * n * e + 2 * w + rows, "flops": 8 * n}
        return {"bytes": 3 * n * e + w + rows + case["cols"] * 8, "flops": 14 * n}
    if op in ("logprob", "logprob_bwd"):
        n, rows = case["rows"] * case["cols"], case["rows"]
        ent = 4 if case["entropy"] else 0
        if op == "logprob":
            return {"bytes": n * BYTES[case["dtype"]] + rows * (8 + 8 + ent + 8 * case["top"]),
                    "flops": (6 if ent else 4) * n}
        return {"bytes": n * (BYTES[case["dtype"]] + BYTES[case["out"]]) + rows * (8 + 8 + 2 * ent),
                "flops": (7 if ent else 4) * n}
    n = sum(_numels(case))
    each = 8 + (2 if case["copy"] else 0) + BYTES[case["grad"]]
    states = 16 if case["states"] == 32 else 4 + 16 / 128
    return {"bytes": n * (each + states), "flops": 20 * n}


# ---- the definitions in 64 bits ---------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        var, mean = torch.var_mean(s.x.double(), dim=1, unbiased=False)
        rstd = (var + s.eps) ** -0.5
        y = torch.addcmul(s.beta.double(), (s.x.double() - mean[:, None]) * rstd[:, None], s.gamma.double())
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        mean, rstd, n = s.mean.double()[:, None], s.rstd.double()[:, None], case["cols"]
        dy, xh = s.dy.double(), (s.x.double() - mean) * rstd
        gdy = dy * s.gamma.double()
        dx = rstd / n * (n * gdy - gdy.sum(1, keepdim=True) - xh * (gdy * xh).sum(1, keepdim=True))
        return {"dx": dx, "dgamma": torch.einsum("rc,rc->c", dy, xh), "dbeta": dy.sum(0)}
    if op == "logprob":
        return _exact_logprob(s)
    if op == "logprob_bwd":
        x, rows = s.logits.double(), case["rows"]
        p = torch.exp(x - _finite(s.lse.double())[:, None])
        keep = (s.targets >= 0) & (s.lse > -math.inf)
        d = torch.zeros_like(p)
        d[torch.arange(rows, device=DEV)[keep], s.targets[keep]] = 1.0
        d = (d - p) * (s.dlogprob.double() * keep)[:, None]
        if s.dentropy is not None:
            # dH/dx = -p (log p + H), with -p log p as one function of p
            d += s.dentropy.double()[:, None] * (torch.special.entr(p) - p * s.entropy.double()[:, None])
        return {"dlogits": d * s.loss_scale.double()}
    return _exact_adamw(s)


def _exact_logprob(s):
    x = s.logits.double()
    lse = torch.logsumexp(x, dim=1)
    at = x.gather(1, s.targets.clamp(min=0)[:, None])[:, 0]
    some = lse > -math.inf
    out = {"logprob": torch.where(s.targets < 0, 0.0, torch.where(some, at - lse, -math.inf)),
           "lse": lse, "entropy": None, "top_ids": None, "top_logprob": None}
    if s.entropy is not None:
        out["entropy"] = torch.special.entr((x - _finite(lse)[:, None]).exp()).sum(1)
    if s.top_ids is not None:
        vals, ids = [], []
        for r in range(0, x.shape[0], 512):
            v, i = torch.sort(s.logits[r:r + 512].float(), dim=1, descending=True, stable=True)
            vals.append(v[:, :s.top_ids.shape[1]].double())
            ids.append(i[:, :s.top_ids.shape[1]].int())
        out["top_ids"] = torch.cat(ids)
        out["top_logprob"] = torch.where(some[:, None], torch.cat(vals) - lse[:, None], -math.inf)
    return out


def _exact_adamw(s):
    scale = min(1.0, s.max_norm / float(s.grad_norm))
    g = s.g.double() * scale
    if s.m_scale is None:
        m, v = s.m.double(), s.v.double()
    else:
        m = (s.m.view(FP8).double().view(-1, 128) * s.m_scale.double()[:, None]).view(-1)
        v = (s.v.view(FP8).double().view(-1, 128) * s.v_scale.double()[:, None]).view(-1) ** 2
    m = s.beta1 * m + (1 - s.beta1) * g
    v = s.beta2 * v + (1 - s.beta2) * g ** 2
    t = int(s.step) + 1
    mh, vh = m / (1 - s.beta1 ** t), v / (1 - s.beta2 ** t)
    w = s.w.double()
    w = w - s.lr * (mh / (vh.sqrt() + s.eps) + s.wd * w)
    out = {"w": w, "copy": w if s.wb is not None else None, "step": torch.tensor([t], device=DEV)}
    if s.m_scale is None:
        return out | {"m": m, "v": v}
    h = _random(m.numel(), s.seed, t)
    for name, x, bits in (("m", m, h & 0xFFFF), ("v", v.sqrt(), h >> 16)):
        b = x.view(-1, 128)
        amax = b.abs().amax(dim=1).clamp(min=1e-30)
        q = b.abs() * (448.0 / amax)[:, None]
        step = torch.exp2(torch.floor(torch.log2(q.clamp(min=2.0 ** -6))) - 3)
        up = torch.floor(q / step + bits.view(-1, 128).double() / 65536.0) * step
        up = up.clamp(max=448.0)
        if name == "v":
            up = torch.where((b > 0) & (up == 0), 2.0 ** -9, up)
        out[name] = (up * torch.sign(b)).view(-1)
        out[name + "_scale"] = amax / 448.0
    return out
