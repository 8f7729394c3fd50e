"""Plain restatements of the 4-bit tensors, the policy loss and the update by
orthogonalised momentum for the tests (test infrastructure; no code of the
package): the quantisers step by step in numpy fp32, the rest in float64."""
import math

import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
BLOCK = {"nvfp4": 16, "mxfp4": 32}
QUINTIC = (3.4445, -4.7750, 2.0315)


def e4m3_table():
    """The 127 finite values from 0 to 448, by their fields."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, 2.0 ** (e - 7.0) * (1 + m / 8))


def nearest(table, v):
    """Codes of the table's values nearest to v >= 0, ties to the even code,
    the last one beyond."""
    mid = (table[:-1] + table[1:]) / 2
    at = np.searchsorted(mid, v, side="left")              # v <= mid: the lower one
    tie = (at < len(mid)) & (mid[np.minimum(at, len(mid) - 1)] == v)
    return np.where(tie & (at % 2 == 1), at + 1, at).astype(np.uint8)


# ---- 4-bit tensors ----------------------------------------------------------

def tensor_scale(x):
    a = np.abs(x).max() if x.size else np.float32(0)
    if not np.isfinite(a):
        return np.float32(np.nan)
    return np.float32(np.maximum(np.float32(a), np.float32(1e-12)) / np.float32(2688))


def quantise(x, fmt, ts=None):
    """(codes [R, C], one per element, scale bytes [R, C / block]) of float32 x."""
    R, C = x.shape
    n = BLOCK[fmt]
    b = x.reshape(R, C // n, n)
    with np.errstate(all="ignore"):
        amax = np.abs(b).max(2) if x.size else np.zeros((R, C // n), np.float32)
        fine = np.isfinite(amax)
        if fmt == "mxfp4":
            _, e = np.frexp(np.where(fine, amax, 1).astype(np.float64))
            e = np.where(amax > 0, np.clip(e - 1 - 2, -127, 127), -127)
            s = np.where(fine, e + 127, 255).astype(np.uint8)
            r = np.ldexp(np.float32(1), -e).astype(np.float32)
        else:
            fine = fine & bool(2.0 ** -100 <= float(ts) <= 2.0 ** 120)
            u = (amax / (np.float32(6) * np.float32(ts))).astype(np.float32)
            s = np.where(fine, nearest(e4m3_table(), np.where(fine, u, 0).astype(np.float64)), 0x7F).astype(np.uint8)
            v = e4m3_table()[np.minimum(s, 126)].astype(np.float32)
            r = np.where(v > 0, np.float32(1) / (v * np.float32(ts)), 0).astype(np.float32)
        y = (b * r[:, :, None]).astype(np.float32)
    c = nearest(E2M1, np.where(np.isfinite(b), np.abs(y), 6).astype(np.float64))
    c = c | (np.signbit(y).astype(np.uint8) << 3)
    c = np.where(fine[:, :, None], c, 0)
    return c.reshape(R, C).astype(np.uint8), s


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(q):
    return np.stack([q & 15, q >> 4], 2).reshape(q.shape[0], -1)


def tiles(s, fmt):
    """Scale bytes [R, K] at their places, zeros past the edges, as one run."""
    R, K = s.shape
    rt, kt = -(-R // 128), -(-K // 4)
    out = np.zeros(rt * kt * 512, np.uint8)
    r, k = np.arange(R)[:, None], np.arange(K)[None]
    out[((r // 128) * kt + k // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + k % 4] = s
    return out


def values(codes, s, fmt, ts=None):
    """What codes and scale bytes stand for, in float64."""
    v = E2M1[codes & 7] * np.where(codes >> 3, -1.0, 1.0)
    if fmt == "mxfp4":
        f = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
    else:
        f = np.where(s == 127, np.nan, e4m3_table()[np.minimum(s, 126)]) * float(ts)
    return v * np.repeat(f, BLOCK[fmt], 1)


# ---- policy loss ------------------------------------------------------------

def policy_loss(lp, old, adv, ref=None, targets=None, offsets=None, clip_low=0.2, clip_high=0.2,
                dual=0.0, kl=0.0, reduction="token", dloss=1.0):
    """(loss, stats, gradient (NaN for tokens in no sequence), per-token error
    scale) in float64; adv per token or per sequence."""
    T = lp.numel()
    offsets = torch.tensor([0, T]) if offsets is None else offsets.cpu()
    S = offsets.numel() - 1
    lp, old, adv = lp.cpu().double(), old.cpu().double(), adv.cpu().double()
    seq = torch.full((T,), -1, dtype=torch.long)
    for s in range(S):
        seq[int(offsets[s]):int(offsets[s + 1])] = s
    live = seq >= 0
    if targets is not None:
        live &= targets.cpu() >= 0
    if adv.numel() != T:
        adv = adv[seq.clamp(min=0)]
    idx = live.nonzero().flatten()
    d = lp[idx] - old[idx]
    a = adv[idx]
    rho = torch.exp(d)
    held = ((a > 0) & (rho > 1 + clip_high)) | ((a < 0) & (rho < 1 - clip_low))
    if dual:
        held |= (a < 0) & (rho > dual)
    f64 = lambda v: torch.tensor(v, dtype=torch.float64)  # noqa: E731
    top = torch.where(a < 0, f64(dual if dual else math.inf), f64(1 + clip_high))
    low = torch.where(a < 0, f64(1 - clip_low), f64(-math.inf))
    obj = torch.where(a == 0, 0.0, torch.minimum(torch.maximum(rho, low), top) * a)
    slope = torch.where(held, 0.0, -rho * a)
    k = torch.zeros_like(rho)
    ey = torch.ones_like(rho)
    if ref is not None:
        y = ref.cpu().double()[idx] - lp[idx]
        k, ey = torch.expm1(y) - y, torch.exp(y)
        slope = slope - kl * torch.expm1(y)
    n = len(idx)
    w = torch.ones(n, dtype=torch.float64)
    if reduction == "token":
        w /= max(1, n)
    elif reduction == "sequence":
        counts = torch.bincount(seq[idx], minlength=S)
        w /= counts[seq[idx]] * max(1, int((counts > 0).sum()))
    grad = torch.full((T,), math.nan, dtype=torch.float64)
    grad[seq >= 0] = 0.0
    grad[idx] = dloss * w * slope
    # what the terms are rounded by: their sizes before any cancels
    size = torch.zeros(T, dtype=torch.float64)
    size[idx] = w * ((2 + d.abs()) * rho * a.abs() + abs(kl) * (ey + 1))
    mean = lambda v: float(v.sum()) / max(1, n)  # noqa: E731
    stats = [float(n), mean(rho), mean(held.double()), mean(k)]
    return float((w * (kl * k - obj)).sum()), stats, grad, size


# ---- orthogonalised momentum ------------------------------------------------

def orthogonalise(u, steps):
    """The quintic's products in float64; a matrix of zeros stays one."""
    u = u.double()
    norm = torch.linalg.norm(u)
    if float(norm) == 0.0:
        return u
    x = u / norm
    if u.shape[0] > u.shape[1]:
        x = x.t()
    a, b, c = QUINTIC
    for _ in range(steps):
        g = x @ x.t()
        x = a * x + (b * g + c * g @ g) @ x
    return x.t() if u.shape[0] > u.shape[1] else x


def muon(w, g, m, lr, mu, wd=0.0, nesterov=True, steps=5, scale="rms", clip=1.0):
    """(w, m) after one step, in float64."""
    R, C = w.shape
    g = g.double() * clip
    m = mu * m.double() + g
    x = orthogonalise(g + mu * m if nesterov else m, steps)
    f = 0.2 * math.sqrt(max(R, C)) if scale == "rms" else math.sqrt(max(1.0, R / C))
    return w.double() * (1 - lr * wd) - lr * f * x, m
