"""The restatements the GPU tests compare with, pinned on the CPU: gradients
against central differences, the 8-bit rounding against its definition."""
import math

import numpy as np
import pytest
import torch

import train_refs as tr


def _numeric(f, x, h=1e-5):
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        e = torch.zeros_like(x).view(-1)
        e[i] = h
        e = e.view_as(x)
        g.view(-1)[i] = (f(x + e) - f(x - e)) / (2 * h)
    return g


def test_layernorm_gradients_against_differences():
    torch.manual_seed(1)
    x, dy = torch.randn(3, 7, dtype=torch.float64), torch.randn(3, 7, dtype=torch.float64)
    g, b = torch.randn(7, dtype=torch.float64), torch.randn(7, dtype=torch.float64)
    loss = lambda x, g, b: float((tr.layernorm(x, g, b, 1e-5)[0] * dy).sum())  # noqa: E731
    _, mean, rstd = tr.layernorm(x, g, b, 1e-5)
    dx, dg, db = tr.layernorm_bwd(dy, x, g, mean, rstd)
    # central differences: truncation ~ h^2 times third derivatives of order 1
    assert torch.allclose(dx, _numeric(lambda v: loss(v, g, b), x), atol=1e-7)
    assert torch.allclose(dg, _numeric(lambda v: loss(x, v, b), g), atol=1e-7)
    assert torch.allclose(db, _numeric(lambda v: loss(x, g, v), b), atol=1e-7)


@pytest.mark.parametrize("entropy", [False, True])
def test_token_logprob_gradient_against_differences(entropy):
    torch.manual_seed(2)
    x = torch.randn(4, 6, dtype=torch.float64)
    x[2, 1:3] = -math.inf
    targets = torch.tensor([0, -1, 5, 3])
    dlp, dh = torch.randn(4, dtype=torch.float64), torch.randn(4, dtype=torch.float64)

    def loss(v):
        lp, _, h, _, _ = tr.token_logprob(v, targets)
        return float((lp * dlp).sum() + ((h * dh).sum() if entropy else 0.0))

    _, _, h, _, _ = tr.token_logprob(x, targets)
    d = tr.token_logprob_bwd(x, targets, dlp, h if entropy else None, dh if entropy else None, 8.0)
    assert torch.allclose(d, 8.0 * _numeric(loss, x), atol=1e-6)


def test_token_logprob_rules():
    inf, nan = math.inf, math.nan
    x = torch.tensor([[1.0, 3.0, 3.0, -inf], [-inf] * 4, [nan, 1.0, inf, 0.0], [0.0, -0.0, 0.0, -1.0]])
    lp, lse, h, ids, tlp = tr.token_logprob(x, torch.tensor([1, 2, 1, -5]), 3)
    assert ids.tolist() == [[1, 2, 0], [0, 1, 2], [0, 2, 1], [0, 1, 2]]
    assert lp[1] == -inf and lse[1] == -inf and h[1] == 0 and (tlp[1] == -inf).all()
    assert torch.isnan(torch.stack([lp[2], lse[2], h[2]])).all() and lp[3] == 0
    assert math.isclose(float(lp[0]), 3 - math.log(math.e + 2 * math.e ** 3))
    low = torch.full((1, 8), torch.finfo(torch.float32).min)   # uniform, however low
    lp, lse, h, _, _ = tr.token_logprob(low, torch.tensor([3]))
    assert math.isclose(float(lp[0]), -math.log(8)) and math.isclose(float(h[0]), math.log(8))


def test_adamw_step_against_scalar_formula():
    rng = np.random.default_rng(3)
    w, g, m, v = (torch.from_numpy(rng.standard_normal(5)) for _ in range(4))
    v = v * v
    w1, m1, v1 = tr.adamw(w, g, m, v, 7, 1e-2, 0.9, 0.99, 1e-6, 0.1, 0.5)
    for i in range(5):
        gi = 0.5 * float(g[i])
        mi, vi = 0.9 * float(m[i]) + 0.1 * gi, 0.99 * float(v[i]) + 0.01 * gi * gi
        wi = float(w[i]) * (1 - 1e-2 * 0.1) - 1e-2 * (mi / (1 - 0.9 ** 7)) / (
            math.sqrt(vi / (1 - 0.99 ** 7)) + 1e-6)
        assert math.isclose(wi, float(w1[i]), rel_tol=1e-12)


def test_e4m3_table_matches_the_oracle(orc):
    codes = np.arange(256, dtype=np.uint8)
    want = orc.dequant(codes.reshape(2, 128), np.ones((2, 1), np.float32), 1, 128, orc.E4M3).ravel()
    assert np.array_equal(tr.e4m3_values().astype(np.float32), want, equal_nan=True)


def test_random_rounding_is_between_neighbours_and_unbiased():
    rng = np.random.default_rng(4)
    x = np.abs(rng.standard_normal(128).astype(np.float32)) * np.exp2(-rng.uniform(0, 20, 128)).astype(np.float32)
    grid = tr.e4m3_values()
    total = np.zeros(128)
    for s in range(4096):
        r = tr.random_bits(0, 128, s, 1)
        q, scale = tr.round_block(x, r & 0xFFFF)
        y = grid[q] * float(scale[0])
        t = x / scale[0]
        lo = np.clip(np.searchsorted(grid[:127], t, side="right") - 1, 0, 126)
        assert ((q == lo) | (q == np.minimum(lo + 1, 126))).all()
        total += y
    gap = np.maximum(np.exp2(np.floor(np.log2(np.maximum(x / scale[0], 2.0 ** -6))) - 3), 2.0 ** -9) * float(scale[0])
    # the mean of 4096 draws: standard deviation at most gap / 2 / 64; six of them
    assert (np.abs(total / 4096 - x) <= gap * 6 / 128).all()


def test_random_bits_look_uniform():
    r = tr.random_bits(1 << 33, 1 << 16, 9, 12)
    for bit in range(32):
        ones = int(((r >> np.uint32(bit)) & 1).sum())
        assert abs(ones - (1 << 15)) < 6 * 128   # six standard deviations of 2^16 fair bits
    assert np.unique(r).size > (1 << 16) - 40
    assert not np.array_equal(r, tr.random_bits(0, 1 << 16, 9, 12))
