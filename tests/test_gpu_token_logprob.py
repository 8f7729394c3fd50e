"""Token log probabilities, entropy, alternatives and their gradient against
64-bit restatements.

Tolerances, with d = x - max and E[.] the mean under the softmax: a term
e^d is computed with relative error (8 + 4 |d|) 2^-24, a sum adds at most
n = V / 32 + 16 more; so the sum s is off by (n + 8 + 4 E|d|) 2^-24 and
log s by as much and 2^-23 (1 + |log s|), lse by that and
2^-23 (|max| + |lse|), a log probability d - log s by log s's error and
2^-23 |d|.  t / s is off by (n + 16) E|d| + E[(8 + 4 |d|) |d|] + its share of
s.  A gradient's p has relative error (8 + 4 |x - lse|) 2^-24, and that of
the sum where it is formed anew, on top of lse's rounding, 2^-23 |lse| where
|lse| <= 256."""
import math

import pytest
import torch

import train_refs as tr
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
E = tr.EPS24
INF = math.inf


@pytest.fixture(scope="module")
def gs():
    import mixed_precision_numerics_gradscaler_gb300 as gs
    torch.cuda.set_device(0)
    return gs


def check(got, want, tol, what):
    got, want = got.double(), want.double()
    fin = torch.isfinite(want)
    same = torch.where(fin, (got - want).abs() <= tol, (got == want) | (got.isnan() & want.isnan()))
    bad = ~same
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4].tolist(), want[bad][:4].tolist())


def view(R, V, pad, dtype, offset, fill=7.0):
    buf = torch.full((offset + R * (V + pad) + 8,), fill, dtype=dtype, device=DEV)
    return buf.as_strided((R, V), (V + pad, 1), offset), buf


def gaps_kept(buf, x, offset, fill=7.0):
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask.as_strided(x.shape, x.stride(), offset).fill_(False)
    return bool((buf[mask] == fill).all())


def make(R, V, dtype, pad=0, offset=0, scale=2.5, kind="random"):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(R * 31 + V)
    x, _ = view(R, V, pad, dtype, offset)
    v = torch.randn(R, V, device=DEV, generator=gen) * scale
    if kind == "peaked":
        v[torch.arange(R, device=DEV), torch.randint(0, V, (R,), device=DEV, generator=gen)] += 30
    elif kind == "rising":
        v = v.sort(dim=1).values
    elif kind == "falling":
        v = v.sort(dim=1, descending=True).values
    elif kind == "equal":
        v = torch.full_like(v, 1.5)
    elif kind == "few values":
        v = v.round()
    elif kind == "masked":
        v[torch.rand(R, V, device=DEV, generator=gen) < 0.95] = -INF
    elif kind == "lowest":
        v[torch.rand(R, V, device=DEV, generator=gen) < 0.95] = torch.finfo(dtype).min
    elif kind == "large":
        v = v * 400
    elif kind == "one thread's":   # the largest ones a fixed distance apart
        v[:, ::1024] += 50
    x.copy_(v.clamp(torch.finfo(dtype).min, torch.finfo(dtype).max) if kind != "masked" else v)
    t = torch.randint(0, V, (R,), device=DEV, generator=gen)
    if R > 3:
        t[1], t[3] = -100, -1
    return x, t, gen


def fwd_check(gs, x, t, k):
    R, V = x.shape
    f = lambda: torch.full((R,), 9.0, device=DEV)  # noqa: E731
    lp, lse, h = f(), f(), f()
    ids = torch.full((R, k), -9, dtype=torch.int32, device=DEV) if k else None
    tlp = torch.full((R, k), 9.0, device=DEV) if k else None
    gs.gs_token_logprob(x, t, lp, lse, h, ids, tlp)
    wlp, wlse, wh, wids, wtlp = tr.token_logprob(x, t, k)
    xd = x.double()
    m = xd.amax(1)
    m0 = torch.where(m.abs() == INF, 0.0, m)
    p = torch.exp(xd - m0[:, None])
    p = p / p.sum(1, keepdim=True).clamp(min=1.0)
    d = torch.where(p > 0, (xd - m0[:, None]).abs(), 0.0)
    ed, ed2 = (p * d).sum(1), (p * d * d).sum(1)
    n = V / 32 + 16
    es = (n + 8 + 4 * ed) * E
    ls = torch.where(torch.isfinite(wlse), wlse - m0, 0.0).abs()
    es = es + 2 * E * (1 + ls)
    check(lse, wlse, es + 2 * E * (m0.abs() + torch.nan_to_num(wlse, 0.0, 0.0, 0.0).abs()), "lse")
    check(lp, wlp, es + 4 * E * torch.nan_to_num(wlp, 0.0, 0.0, 0.0).abs(), "logprob")
    eh = es + ((n + 16) * ed + 8 * ed + 4 * ed2 + ed * (n + 8 + 4 * ed)) * E + 4 * E * (1 + ed)
    check(h, wh, eh, "entropy")
    if k:
        assert torch.equal(ids.long(), wids), "top ids"
        check(tlp, wtlp, es[:, None] + 4 * E * torch.nan_to_num(wtlp, 0.0, 0.0, 0.0).abs(), "top logprob")
    # without the optional outputs: the same values
    lp2, ids2 = f(), None if ids is None else torch.empty_like(ids)
    gs.gs_token_logprob(x, t, lp2)
    check(lp2, lp, 0.0, "logprob alone")
    if k:
        gs.gs_token_logprob(x, None, None, None, None, ids2, torch.empty_like(tlp))
        assert torch.equal(ids2, ids)


VOCABS = [1, 2, 3, 7, 31, 33, 100, 255, 257, 1000, 1024, 4097, 8192, 32003, 50000, 128256, 200001]


@pytest.mark.parametrize("V", VOCABS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_forward_sizes(gs, V, dtype):
    for R in (1, 5, 40):
        x, t, _ = make(R, V, TYPES[dtype])
        fwd_check(gs, x, t, min(V, 20))


@pytest.mark.parametrize("R", [2, 8, 17, 75, 150, 310, 640, 2000])
def test_forward_row_counts(gs, R):
    for V in (1003, 20001):
        x, t, _ = make(R, V, torch.bfloat16)
        fwd_check(gs, x, t, 8)


@pytest.mark.parametrize("kind", ["peaked", "rising", "falling", "equal", "few values", "masked",
                                  "lowest", "large", "one thread's"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_forward_distributions(gs, kind, dtype):
    for R, V in ((3, 32003), (6, 700), (200, 5001), (2, 200001)):
        x, t, _ = make(R, V, TYPES[dtype], kind=kind)
        for k in (1, 5, 32):
            fwd_check(gs, x, t, k)


@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (3, 5), (8, 8), (13, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_forward_strides_and_alignment(gs, pad, offset, dtype):
    for V in (5, 1000, 32003):
        x, t, _ = make(9, V, TYPES[dtype], pad, offset)
        fwd_check(gs, x, t, min(V, 6))


def special_rows(V, dtype):
    x = torch.randn(12, V, device=DEV).to(dtype)
    t = torch.arange(12, device=DEV) % V
    x[1] = -INF                       # nothing allowed
    x[2] = -INF
    x[2, V // 2] = 3.0                # one allowed
    x[3, V - 1] = math.nan
    x[4, 0] = INF
    x[5] = torch.finfo(dtype).min     # the lowest value everywhere: uniform
    x[6, t[6]] = -INF                 # the target itself masked
    x[7] = -INF
    x[7, 0] = torch.finfo(dtype).min  # one at the lowest value, the rest masked
    t[8], t[9] = V, V + 10 ** 12      # beyond the vocabulary
    t[10] = -(1 << 40)
    x[11] = torch.where(torch.arange(V, device=DEV) % 2 == 0, 0.0, -0.0)
    return x, t


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [40, 1001, 70000])
def test_special_rows(gs, V, dtype):
    x, t = special_rows(V, TYPES[dtype])
    fwd_check(gs, x, t, 12)
    lp, lse, h = (torch.empty(12, device=DEV) for _ in range(3))
    gs.gs_token_logprob(x, t, lp, lse, h)
    bwd_check(gs, x, t, lse, h, TYPES[dtype], True)
    bwd_check(gs, x, t, lse, h, torch.float32, False)


def bwd_check(gs, x, t, lse, h, out, entropy, pad=0, offset=0, scale=512.0):
    R, V = x.shape
    gen = torch.Generator(device=DEV)
    gen.manual_seed(V)
    g = torch.randn(R, device=DEV, generator=gen)
    ge = torch.randn(R, device=DEV, generator=gen) * 0.3 if entropy else None
    S = torch.full((1,), scale, device=DEV)
    d, buf = view(R, V, pad, out, offset)
    gs.gs_token_logprob_bwd(x, t, lse, g, d, h if entropy else None, ge, S)
    want = tr.token_logprob_bwd(x, t, g, h, ge, scale)
    l = torch.nan_to_num(lse.double(), 0.0, 0.0, 0.0)[:, None]
    logp = tr._log_softmax(x.double())[0]
    a = torch.where(torch.isfinite(logp), logp.abs(), 0.0)
    p = torch.exp(logp).nan_to_num(0.0)
    again = (V / 32 + 16 + 4 * (p * a).sum(1, keepdim=True)) * (l.abs() > 256)
    ep = (8 + 4 * a + 2 * l.abs().clamp(max=256.0) + again) * E * p
    ga = g.double().abs()[:, None]
    tol = scale * ga * (ep + 4 * E * (want != 0))
    if entropy:
        hb = h.double().abs()[:, None].nan_to_num(0.0)
        tol = tol + scale * ge.double().abs()[:, None] * (ep * (a + hb) + p * 8 * E * (a + hb + l.abs().clamp(max=256.0) + again))
    tol = tol + want.abs().nan_to_num(0.0) * HALF_ULP[out] * 1.01
    if out == torch.float16:
        tol = tol + 2.0 ** -25
        want = torch.where(want.abs() >= 65520, torch.sign(want) * INF, want)
    else:
        tol = tol + 2.0 ** -126   # results below the normal range may be flushed
    check(d, want, tol, "dlogits")
    assert gaps_kept(buf, d, offset)
    if out == x.dtype:   # in place, the logits' own layout
        y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=DEV)
        y.copy_(x)
        gs.gs_token_logprob_bwd(y, t, lse, g, y, h if entropy else None, ge, S)
        check(y, d, 0.0, "in place")


@pytest.mark.parametrize("V", VOCABS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_backward_sizes(gs, V, dtype):
    for R, out in ((1, dtype), (5, "f16"), (33, "f32")):
        x, t, _ = make(R, V, TYPES[dtype])
        _, lse, h, _, _ = tr.token_logprob(x, t)
        bwd_check(gs, x, t, lse.float(), h.float(), TYPES[out], R != 5)


@pytest.mark.parametrize("pad,offset,opad,ooff", [(1, 0, 1, 0), (0, 1, 0, 1), (3, 5, 0, 0), (8, 8, 3, 2),
                                                  (0, 0, 1, 1)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("f32", "f16"),
                                       ("bf16", "f32")])
def test_backward_strides_and_alignment(gs, pad, offset, opad, ooff, dtype, out):
    for V in (5, 1000, 32003):
        x, t, _ = make(9, V, TYPES[dtype], pad, offset)
        _, lse, h, _, _ = tr.token_logprob(x, t)
        bwd_check(gs, x, t, lse.float(), h.float(), TYPES[out], True, opad, ooff)


@pytest.mark.parametrize("kind", ["peaked", "masked", "lowest", "large", "equal"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_backward_distributions(gs, kind, dtype):
    for R, V in ((3, 32003), (6, 700), (200, 5001)):
        x, t, _ = make(R, V, TYPES[dtype], kind=kind)
        _, lse, h, _, _ = tr.token_logprob(x, t)
        bwd_check(gs, x, t, lse.float(), h.float(), TYPES[dtype], True)
        bwd_check(gs, x, t, lse.float(), h.float(), torch.float32, False)


def test_backward_overflow_is_infinite(gs):
    x, t, _ = make(6, 1000, torch.float16)
    _, lse, h, _, _ = tr.token_logprob(x, t)
    bwd_check(gs, x, t, lse.float(), h.float(), torch.float16, False, scale=2.0 ** 24)


def test_backward_without_scale_and_many_rows(gs):
    x, t, _ = make(70000, 17, torch.bfloat16)
    _, lse, _, _, _ = tr.token_logprob(x, t)
    g = torch.ones(70000, device=DEV)
    d = torch.empty(70000, 17, device=DEV)
    gs.gs_token_logprob_bwd(x, t, lse.float(), g, d)
    want = tr.token_logprob_bwd(x, t, g)
    assert (d.double() - want).abs().max() <= 64 * 2.0 ** -24
    fwd_check(gs, x, t, 3)


def test_rows_beyond_32_bit_offsets(gs):
    V, ld = 5000, (1 << 31) + 8
    for off in (0, 1):
        big = torch.empty(2 * ld + V + 8, dtype=torch.float16, device=DEV)
        x = big.as_strided((3, V), (ld, 1), off)
        x.copy_(torch.randn(3, V, device=DEV))
        t = torch.tensor([3, 4999, 77], device=DEV)
        fwd_check(gs, x, t, 4)
        near = x.contiguous()
        _, lse, _, _, _ = tr.token_logprob(near, t)
        g = torch.ones(3, device=DEV)
        want = torch.empty_like(near)
        gs.gs_token_logprob_bwd(near, t, lse.float(), g, want)
        gs.gs_token_logprob_bwd(x, t, lse.float(), g, x)
        assert torch.equal(x.contiguous(), want)
        del big, x
        torch.cuda.empty_cache()


def test_runs_on_the_given_stream_and_in_a_graph(gs):
    x, t, _ = make(10, 32003, torch.bfloat16)
    lp, lse, h = (torch.empty(10, device=DEV) for _ in range(3))
    gs.gs_token_logprob(x, t, lp, lse, h)
    g, d, want = torch.ones(10, device=DEV), torch.empty_like(x), torch.empty_like(x)
    gs.gs_token_logprob_bwd(x, t, lse, g, want)
    wanted = [v.clone() for v in (lp, lse, h)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lp.zero_()
    torch.cuda.synchronize()
    gs.gs_token_logprob(x, t, lp, lse, h, stream=side)
    side.synchronize()
    assert torch.equal(lp, wanted[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gs.gs_token_logprob(x, t, lp, lse, h)
        gs.gs_token_logprob_bwd(x, t, lse, g, d)
    for v in (lp, lse, h, d):
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((lp, lse, h, d), (*wanted, want)))


def test_refusals(gs):
    x, t, _ = make(4, 100, torch.float32)
    lp = torch.empty(4, device=DEV)
    ids, tlp = torch.empty(4, 33, dtype=torch.int32, device=DEV), torch.empty(4, 33, device=DEV)
    with pytest.raises(gs.GsError):
        gs.gs_token_logprob(x, t, lp, top_ids=ids, top_logprob=tlp)          # beyond GS_MAX_TOP
    with pytest.raises(gs.GsError):
        gs.gs_token_logprob(x[:, :4], t, lp, top_ids=ids[:, :5].contiguous(),
                            top_logprob=tlp[:, :5].contiguous())               # beyond V
    with pytest.raises(gs.GsError):
        gs.gs_token_logprob(x, None, lp)
    with pytest.raises(gs.GsError):
        gs.gs_token_logprob(x, t, lp, lse=lp)                                 # outputs overlap
    with pytest.raises(gs.GsError):
        gs.gs_token_logprob(x[:, :0], t, lp)
    with pytest.raises(ValueError):
        gs.gs_token_logprob(x, t.int(), lp)
    with pytest.raises(ValueError):
        gs.gs_token_logprob(x, t[:3], lp)
    with pytest.raises(ValueError):
        gs.gs_token_logprob(x.t(), t, lp)
    with pytest.raises(gs.GsError):
        gs.gs_token_logprob(x.cpu(), t, lp)
    g, d = torch.ones(4, device=DEV), torch.empty_like(x)
    with pytest.raises(gs.GsError):
        gs.gs_token_logprob_bwd(x, t, lp, g, d, entropy=lp)                   # without dentropy
    with pytest.raises(gs.GsError):
        gs.gs_token_logprob_bwd(x[:3], t[:3], lp[:3], g[:3], x[1:])           # overlaps, not in place
    with pytest.raises(ValueError):
        gs.gs_token_logprob_bwd(x, t, lp, g, d[:, :99])
    # no rows: nothing to do
    gs.gs_token_logprob(x[:0], t[:0], lp[:0])
    gs.gs_token_logprob_bwd(x[:0], t[:0], lp[:0], g[:0], d[:0])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [700, 32003, 128256, 200001, 1000003, 16000001])
def test_backward_sum_of_many_equal_terms(gs, V, dtype):
    """|lse| > 256 and equal logits: p = 1 / V.  The row's sum is formed anew to
    be closer than lse's own rounding; equal terms added one after another
    in fp32 would all round alike (1e-5 off at V = 128256, 1e-3 at 16 M).
    Tolerance, in 2^-24: the two products with log2 e and the difference from
    log s round d = ln V three times, two exponentials by 8 in all, blocks of
    terms and the threads' join by 16, independently of V."""
    tol = (3 * math.log(V) + 24) * E
    rows = 3 if V < 1 << 20 else 1
    for value, pad in ((300.0, 0), (-300.0, 1), (1000.0, 5)):
        x, _ = view(rows, V, pad, TYPES[dtype], 0)
        x.fill_(value)
        t = torch.full((rows,), -1, device=DEV)
        t[0] = V // 2
        lse = torch.full((rows,), value + math.log(V), dtype=torch.float64, device=DEV).float()
        g = torch.ones(rows, device=DEV)
        outs = [torch.empty(rows, V, device=DEV)]
        gs.gs_token_logprob_bwd(x, t, lse, g, outs[0], loss_scale=torch.full((1,), -float(V), device=DEV))
        if dtype == "f32":
            gs.gs_token_logprob_bwd(x, t, lse, g, x, loss_scale=torch.full((1,), -float(V), device=DEV))
            outs.append(x)
        for d in outs:
            d = d.double()
            d[0, V // 2] += V
            assert ((d[0] - 1).abs() <= tol + V * E * (torch.arange(V, device=DEV) == V // 2)).all()
            assert (d[1:] == 0).all()          # no target, no gradient


# rows and columns that take every number of CTAs per row and of threads per CTA
ONE_BY_ONE = [(400, 100), (300, 1536), (300, 1537), (64, 4097), (2, 8192), (40, 12289), (900, 12288), (5, 32003),
              (150, 32003), (1, 128256), (16, 128256), (40, 128256), (100, 128256), (420, 128256), (900, 50001),
              (3, 200001), (800, 32003)]


def telling_columns(V):
    """The first and last ones, those about the edges of vectors, blocks and parts,
    and some others (all of a short row)."""
    gen = torch.Generator()
    gen.manual_seed(V)
    if V <= 1537:
        return torch.randperm(V, generator=gen)
    edges = torch.cat([torch.arange(0, V + 1, 2048)] +
                      [torch.arange(0, p + 1) * ((-(-V // p) + 7) // 8 * 8) for p in (2, 4, 8)])
    near = (edges[:, None] + torch.tensor([-9, -8, -1, 0, 1, 7, 8])).flatten()
    some = torch.cat([torch.arange(40), torch.arange(V - 40, V), near, torch.randint(0, V, (200,), generator=gen)])
    some = some[(some >= 0) & (some < V)].unique()
    return some[torch.randperm(some.numel(), generator=gen)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,V", ONE_BY_ONE)
def test_every_logit_counts_once(gs, R, V, dtype):
    """Rows of -Inf but two equal logits: lse - x = entropy = ln 2, each log
    probability -ln 2, each p one half.  A logit left out or read twice makes
    that 0 or ln 3, whatever V is.  With x = 0, and with x = 300, where the
    gradient forms the sum itself; tolerance: a few roundings of 300."""
    columns = telling_columns(V)
    ln2 = math.log(2.0)
    at = torch.arange(R, device=DEV)
    x, _ = view(R, V, 1, TYPES[dtype], 0)
    x.fill_(-INF)
    d, _ = view(R, V, 1, torch.float32, 0)
    f = lambda: torch.empty(R, device=DEV)  # noqa: E731
    lp, lse, h, tlp = f(), f(), f(), torch.empty(R, 3, device=DEV)
    ids = torch.empty(R, 3, dtype=torch.int32, device=DEV)
    for k, first in enumerate(range(0, columns.numel(), R)):
        value, tol = ((0.0, 4 * E), (300.0, 2048 * E))[k % 2]
        c = columns[(torch.arange(R) + first) % columns.numel()].to(DEV)
        o = (c + V // 2) % V
        x[at, c] = x[at, o] = value
        gs.gs_token_logprob(x, c, lp, lse, h, ids, tlp)
        gs.gs_token_logprob_bwd(x, c, lse, torch.ones(R, device=DEV), d)
        x[at, c] = x[at, o] = -INF
        for got, want in ((lse - value, ln2), (h, ln2), (lp, -ln2), (tlp[:, :2], -ln2)):
            assert ((got.double() - want).abs() <= tol).all()
        assert torch.equal(ids[:, :2].long(), torch.stack([torch.minimum(c, o), torch.maximum(c, o)], 1))
        assert (tlp[:, 2] == -INF).all()
        assert ((d[at, c].double() - 0.5).abs() <= tol).all() and ((d[at, o].double() + 0.5).abs() <= tol).all()
        d[at, c] = d[at, o] = 0
        assert (d == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", VOCABS)
def test_equal_logits_are_all_counted(gs, V, dtype):
    """Equal logits: every term is 1 and the sum V exactly, so that lse - x is ln V
    within its own rounding: 2^-22 of it, less than one logit's share."""
    for R in (1, 5, 40, 150):
        x, _ = view(R, V, 3, TYPES[dtype], 1)
        x.fill_(0.0)
        lse, h = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
        gs.gs_token_logprob(x, None, None, lse, h)
        want = math.log(V)
        assert V == 1 or want * 2.0 ** -22 < 0.75 / V
        for got in (lse, h):
            assert ((got.double() - want).abs() <= want * 2.0 ** -22).all()
