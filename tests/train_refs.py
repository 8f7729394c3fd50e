"""Plain 64-bit restatements of layer norm, token log probabilities and the
AdamW step for the tests, and the bit-level rule of the 8-bit moments in
numpy fp32 (test infrastructure; no code of the package)."""
import math

import numpy as np
import torch

EPS24 = 2.0 ** -24   # half an ulp of 1 in fp32
INF = math.inf


# ---- layer norm -------------------------------------------------------------

def layernorm(x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1) + eps)
    y = xc * rstd[:, None]
    if gamma is not None:
        y = y * gamma.double()
    if beta is not None:
        y = y + beta.double()
    return y, mean, rstd


def layernorm_bwd(dy, x, gamma, mean, rstd):
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    xh = (x - mean) * rstd
    d = dy if gamma is None else dy * gamma.double()
    dx = rstd * (d - d.mean(1, keepdim=True) - xh * (d * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


# ---- token log probabilities ------------------------------------------------

def _log_softmax(x):
    """(x - max - log sum, max, log sum) in float64, an empty row -Inf."""
    m = x.amax(1)
    m0 = torch.where(m.abs() == INF, 0.0, m)
    ls = torch.log(torch.exp(x - m0[:, None]).sum(1))
    none = m == -INF
    logp = x - m0[:, None] - torch.where(none, 0.0, ls)[:, None]
    return logp, m0, ls, none


def token_logprob(logits, targets, k=0):
    """(logprob, lse, entropy, top_ids, top_logprob) in float64, with the
    rules for masked, empty and NaN rows."""
    x = logits.double()
    V = x.shape[1]
    bad = torch.isnan(x).any(1) | (x == INF).any(1)
    logp, m, ls, none = _log_softmax(x)
    entropy = torch.where(bad, math.nan, torch.special.entr(torch.exp(logp)).sum(1))
    lse = torch.where(bad, math.nan, torch.where(none, -INF, m + ls))
    logp = torch.where(bad[:, None], math.nan, logp)
    logprob = logp.gather(1, targets.clamp(0, V - 1)[:, None])[:, 0]
    logprob = torch.where(targets < 0, 0.0, torch.where(targets >= V, math.nan, logprob))
    ids = tlp = None
    if k:
        key = torch.where(torch.isnan(x), INF, x)
        nan_first = torch.isnan(x).double()
        # stable sorts: by value, then NaN before everything
        o = torch.argsort(key, dim=1, descending=True, stable=True)
        o = o.gather(1, torch.argsort(nan_first.gather(1, o), dim=1, descending=True, stable=True))
        ids = o[:, :k]
        tlp = logp.gather(1, ids)
    return logprob, lse, entropy, ids, tlp


def token_logprob_bwd(logits, targets, dlogprob, entropy=None, dentropy=None, scale=1.0):
    x = logits.double()
    V = x.shape[1]
    bad = torch.isnan(x).any(1) | (x == INF).any(1)
    logp, _, _, none = _log_softmax(x)
    p = torch.exp(logp)
    g = torch.where(targets < 0, 0.0, dlogprob.double())
    hot = torch.zeros_like(x)
    ok = (targets >= 0) & (targets < V)
    hot[torch.arange(x.shape[0], device=x.device)[ok], targets[ok]] = 1.0
    d = g[:, None] * (hot - p)
    if dentropy is not None:
        d = d - torch.where(p > 0, dentropy.double()[:, None] * p * (logp + entropy.double()[:, None]), 0.0)
    d = torch.where(none[:, None], 0.0, d) * scale
    return torch.where(((targets >= V) | bad)[:, None], math.nan, d)


# ---- AdamW ------------------------------------------------------------------

def adamw(w, g, m, v, t, lr, beta1, beta2, eps, wd, coef=1.0):
    """One step in float64; beta1, beta2 etc. as fp32 values."""
    g = g.double() * coef
    m = beta1 * m.double() + (1 - beta1) * g
    v = beta2 * v.double() + (1 - beta2) * g * g
    w = w.double()
    return w - lr * wd * w - adamw_update(m, torch.sqrt(v), t, lr, beta1, beta2, eps), m, v


def adamw_update(m, r, t, lr, beta1, beta2, eps):
    """What a step subtracts, from the new first moment and the root of the
    second."""
    mh, rh = m.double() / (1 - beta1 ** t), r.double() / math.sqrt(1 - beta2 ** t)
    return lr * mh / (rh + eps)


F = np.float32


def moments_f32(g, m, v, beta1, beta2, coef=1.0):
    """The new moments with every operation rounded to fp32 (numpy)."""
    g = g.astype(F) * F(coef)
    m = m * F(beta1) + g * F(1.0 - float(F(beta1)))
    v = v * F(beta2) + (g * F(1.0 - float(F(beta2)))) * g
    return m, v, np.sqrt(v)


def _mix(x):
    x = x.astype(np.uint32)
    x = x ^ (x >> np.uint32(16))
    x = x * np.uint32(0x7FEB352D)
    x = x ^ (x >> np.uint32(15))
    x = x * np.uint32(0x846CA68B)
    return x ^ (x >> np.uint32(16))


def random_bits(place, n, seed, t):
    i = place + np.arange(n, dtype=np.int64)
    key = ((seed + 0x9E3779B9 * t) % 2 ** 32 + 0x85EBCA6B * (i >> 32)) & 0xFFFFFFFF
    return _mix((i & 0xFFFFFFFF).astype(np.uint32) ^ _mix(key))


def e4m3_values():
    """The value of every E4M3 code."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    mag = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    mag = np.where((c & 127) == 127, np.nan, mag)
    return np.where(c >= 128, -mag, mag)


def round_block(x, r16, keep_positive=False):
    """One tensor's moments (fp32) -> (codes, scales): the scale and the
    product rounded to fp32, the rounding between neighbouring values decided
    by exact arithmetic on the E4M3 grid."""
    n = x.size
    pad = -n % 128
    b = np.pad(x.astype(F), (0, pad)).reshape(-1, 128)
    a = np.maximum(np.abs(b).max(1), F(1e-30))
    scale = a / F(448.0)
    t = (b * (F(448.0) / a)[:, None]).reshape(-1)[:n]
    grid = e4m3_values()[:127]
    mag = np.abs(t.astype(np.float64))
    lo = np.clip(np.searchsorted(grid, mag, side="right") - 1, 0, 126)
    hi = np.minimum(lo + 1, 126)
    gap = np.where(hi > lo, grid[hi] - grid[lo], 32.0)
    # the fraction of the gap in units of its 20 dropped significand bits
    # (exact for values at or above 2^-6; below, the sum with 2^-6 is rounded)
    low = mag < 2.0 ** -6
    magr = np.where(low, (mag.astype(F) + F(2.0 ** -6)).astype(np.float64) - 2.0 ** -6, mag)
    lo = np.where(low, np.clip(np.searchsorted(grid, magr, side="right") - 1, 0, 126), lo)
    frac = np.floor((magr - grid[lo]) / gap * 2.0 ** 20)
    up = frac + r16.astype(np.float64) * 16 >= 2.0 ** 20
    code = np.minimum(np.where(up, lo + 1, lo), 126)
    if keep_positive:
        code = np.where((x > 0) & (code == 0), 1, code)
    return (code | np.where(np.signbit(t), 128, 0)).astype(np.uint8), scale
