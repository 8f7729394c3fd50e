"""The update by orthogonalised momentum against float64.

Tolerance: each of a step's three products rounds its operand or result to fp16
once, an error of at most 2^-11 / sqrt(3) = 2.8e-4 of it in the mean; the
polynomial carries an error on with a factor that, relative to what it makes of the
singular values, stays below 3 (its slope is at most 3.45, where it grows them
as much).  Five steps' 15 roundings in quadrature: sqrt(15) 2.8e-4 3 = 3.3e-3 of
|X| in the 2-norm, n steps' 3.3e-3 sqrt(n / 5).  That is a mean over many
entries: G and P of fewer than 32 rows have so few that matter that a rounding can
be near its bound, 2^-11 of what it rounds, in all of them: sqrt(15) 2^-11 3 =
5.7e-3 there.  Momenta are a product and a sum in fp32; weights are held to X's
share and two roundings."""
import math

import pytest
import torch

import more_refs as mr
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def gs():
    import mixed_precision_numerics_gradscaler_gb300 as gs
    torch.cuda.set_device(0)
    return gs


def make(shapes, dtype="f32", seed=0, offset=0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed + 1)

    def flat(scale, dt=torch.float32):
        out = []
        for s in shapes:
            n = s[0] * s[1]
            buf = torch.full((n + offset + 8,), 5.0, dtype=dt, device=DEV)
            buf[offset:offset + n] = (torch.randn(n, device=DEV, generator=gen) * scale).to(dt)
            out.append((buf[offset:offset + n].view(s), buf))
        return out

    return [flat(0.02), flat(1e-3, TYPES[dtype]), flat(5e-3), flat(1.0, torch.bfloat16)]


def views(ts):
    return [[v for v, _ in t] for t in ts]


def step(gs, w, g, m, wb, lr=0.02, found=0, max_norm=0.0, norm=1.0, **k):
    li = gs.gs_muon_list_create(w, g, m, wb)
    f = torch.full((1,), found, dtype=torch.int32, device=DEV)
    gs.gs_master_update_muon(li, f, lr, max_norm=max_norm, grad_norm=torch.full((1,), norm, device=DEV), **k)
    torch.cuda.synchronize()
    return li


def check(gs, shapes, dtype="f32", offset=0, steps=5, nesterov=True, scale="rms", copy=True, wd=0.1, lr=0.02,
          max_norm=0.0, norm=1.0, seed=0):
    ts = make(shapes, dtype, seed, offset)
    w, g, m, wb = views(ts)
    before = [[t.clone() for t in v] for v in (w, m)]
    li = step(gs, w, g, m, wb if copy else None, lr, 0, max_norm, norm, momentum=0.95, weight_decay=wd,
              nesterov=nesterov, ns_steps=steps, scale=scale)
    f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    clip = f32(f32(max_norm) / f32(norm)) if 0 < max_norm < norm else 1.0
    for i, s in enumerate(shapes):
        ww, wm = mr.muon(before[0][i], g[i], before[1][i], f32(lr), f32(0.95), f32(wd), nesterov, steps, scale, clip)
        assert bool(((m[i].double() - wm).abs() <= (before[1][i].double().abs() + g[i].double().abs() * clip) * 2.0 ** -22).all())
        moved = torch.linalg.norm(ww - before[0][i].double() * (1 - f32(lr) * f32(wd)))
        part = 3.3e-3 if min(s) >= 32 else 5.7e-3
        tol = part * math.sqrt(max(steps, 5) / 5) * float(moved) + float(torch.linalg.norm(ww)) * 2.0 ** -22
        assert float(torch.linalg.norm(w[i].double() - ww)) <= tol, (s, float(torch.linalg.norm(w[i].double() - ww)), tol)
        if copy:
            assert torch.equal(wb[i], w[i].bfloat16())
    for t in ts:
        for (v, buf) in t:                               # nothing beside the matrices
            assert bool((buf[:offset] == 5.0).all()) and bool((buf[offset + v.numel():] == 5.0).all())
    assert gs.gs_device_status() == gs.GS_OK
    return li


@pytest.mark.parametrize("shape", [(1, 1), (1, 50), (50, 1), (7, 9), (64, 64), (65, 63), (100, 1000), (1000, 100), (256, 256),
                                   (257, 255), (300, 2000), (2000, 300), (513, 769), (1024, 2050)])
def test_one_matrix(gs, shape):
    check(gs, [shape])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("scale", ["rms", "aspect"])
def test_types_and_settings(gs, dtype, nesterov, scale):
    check(gs, [(300, 520), (520, 300)], dtype, nesterov=nesterov, scale=scale, copy=nesterov, max_norm=0.5, norm=2.0)


@pytest.mark.parametrize("offset", [1, 2, 3])
def test_lists_of_many_shapes_unaligned(gs, offset):
    gen = torch.Generator()
    gen.manual_seed(offset)
    shapes = [tuple(torch.randint(1, 400, (2,), generator=gen).tolist()) for _ in range(20)]
    check(gs, shapes, "bf16", offset)


def test_more_matrices_than_the_table_in_shared_memory(gs):
    check(gs, [(5 + i % 40, 3 + i % 23) for i in range(300)])


@pytest.mark.parametrize("steps", [1, 2, 7])
def test_steps(gs, steps):
    check(gs, [(200, 700), (700, 200)], steps=steps)


def test_skipped_when_found_inf_is_set(gs):
    w, g, m, wb = views(make([(90, 140)]))
    keep = [t.clone() for t in (w[0], m[0], wb[0])]
    g[0][3, 3] = math.inf
    step(gs, w, g, m, wb, found=1)
    assert all(torch.equal(a, b) for a, b in zip(keep, (w[0], m[0], wb[0])))


def test_zero_momentum_and_non_finite_gradients(gs):
    w, g, m, wb = views(make([(40, 60), (60, 40), (30, 30)]))
    g[0].zero_(), m[0].zero_()
    g[1][2, 2] = math.nan
    keep = w[0].clone()
    step(gs, w, g, m, wb, weight_decay=0.5)
    f = 1 - float(torch.tensor(0.02)) * 0.5
    assert torch.allclose(w[0], keep * f, rtol=2.0 ** -22) and bool(w[1].isnan().all())
    assert bool(torch.isfinite(w[2]).all())              # one matrix's NaN stays its own


@pytest.mark.parametrize("shape", [(257, 255), (255, 257), (61, 333), (3, 5)])
def test_a_list_forgets_a_step_of_nan(gs, shape):
    """After a step whose gradients were NaN, and the state put back, the list
    does as a new one: nothing of its workspace, rows' paddings among it, counts."""
    w, g, m, wb = views(make([shape]))
    state = [t[0].clone() for t in (w, g, m)]
    g[0].fill_(math.nan)
    li = step(gs, w, g, m, wb)
    assert bool(w[0].isnan().all())
    for t, s in zip((w, g, m), state):
        t[0].copy_(s)
    gs.gs_master_update_muon(li, torch.zeros(1, dtype=torch.int32, device=DEV), 0.02)
    w2, g2, m2, wb2 = views(make([shape]))
    step(gs, w2, g2, m2, wb2)
    assert torch.equal(w[0], w2[0]) and torch.equal(m[0], m2[0])


def test_scales_of_gradients_do_not_matter(gs):
    """X = u / |u|: a power of two on gradient and momentum changes nothing."""
    outs = []
    for e in (0, -40, 30):
        w, g, m, wb = views(make([(120, 333)]))
        g[0].mul_(2.0 ** e), m[0].mul_(2.0 ** e)
        step(gs, w, g, m, wb)
        outs.append(w[0].clone())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_empty_lists_and_matrices(gs):
    step(gs, [], [], [], None)
    w, g, m, wb = views(make([(0, 5), (4, 0), (6, 7)]))
    keep = w[2].clone()
    step(gs, w, g, m, wb)
    assert not torch.equal(w[2], keep)


def test_overlaps_are_refused(gs):
    w, g, m, _ = views(make([(8, 8), (8, 8)]))
    for bad in (([w[0], w[0]], g, m, None), (w, [m[0], g[1]], m, None), (w, g, [w[1], m[1]], None)):
        with pytest.raises(gs.GsError):
            gs.gs_muon_list_create(*bad)


def test_repeated_and_captured_calls_on_two_lists(gs):
    """Two lists' steps, captured into two graphs and replayed in turn and on
    two streams at once, do as single calls in their order do."""
    def lists():
        a = views(make([(130, 300), (300, 130)], seed=3))
        b = views(make([(260, 200)], seed=4))
        return a, b

    def update(li, f):
        gs.gs_master_update_muon(li, f, 0.02, weight_decay=0.1)

    f = torch.zeros(1, dtype=torch.int32, device=DEV)
    (a, b) = lists()
    la, lb = (gs.gs_muon_list_create(*v) for v in (a, b))
    for _ in range(3):
        update(la, f), update(lb, f)
    torch.cuda.synchronize()
    want = [t.clone() for v in (a, b) for x in v for t in x]
    (a, b) = lists()
    la, lb = (gs.gs_muon_list_create(*v) for v in (a, b))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = []
    for li, s in zip((la, lb), streams):
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            update(li, f)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    got = [t for v in (a, b) for x in v for t in x]
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert gs.gs_device_status() == gs.GS_OK


def test_waits_run_out_and_the_list_recovers(gs):
    """No loads (the test hook): the products give up after about 2 s, report it
    and free what they hold; the same list then works."""
    w, g, m, wb = views(make([(300, 600)]))
    li = gs.gs_muon_list_create(w, g, m, wb)
    f = torch.zeros(1, dtype=torch.int32, device=DEV)
    one = torch.ones(1, device=DEV)
    q, s, d = torch.zeros(64, 64, dtype=torch.uint8, device=DEV), None, torch.zeros(64, 64, device=DEV)
    s = torch.zeros(gs.fp4_scale_bytes(64, 128, "nvfp4"), dtype=torch.uint8, device=DEV)
    gs.gs_test_set_stall(True)
    try:
        gs.gs_master_update_muon(li, f, 0.02)
        assert gs.gs_device_status() == gs.GS_ERR_TIMEOUT
        gs.fp4_gemm_block_scaled(q, s, q, s, "nvfp4", d, one, one)
        assert gs.gs_device_status() == gs.GS_ERR_TIMEOUT
        gs.fp4_gemm_block_scaled(q[:3], s, q, s, "nvfp4", d[:3], one, one)
        assert gs.gs_device_status() == gs.GS_ERR_TIMEOUT
    finally:
        gs.gs_test_set_stall(False)
    assert gs.gs_device_status() == gs.GS_OK
    w2, g2, m2, wb2 = views(make([(300, 600)]))
    m[0].copy_(m2[0]), w[0].copy_(w2[0])
    gs.gs_master_update_muon(li, f, 0.02)
    gs.gs_master_update_muon(gs.gs_muon_list_create(w2, g2, m2, wb2), f, 0.02)
    torch.cuda.synchronize()
    assert torch.equal(w[0], w2[0]) and torch.equal(m[0], m2[0])
    assert gs.gs_device_status() == gs.GS_OK
