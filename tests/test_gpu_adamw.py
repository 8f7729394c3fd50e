"""The AdamW step: moments bit for bit against a numpy fp32 restatement (8-bit
codes and scales too), weights against float64 from those moments (the step
defines them rounded to fp32; m may be a difference of two near products).

Tolerance of a weight: w (1 - lr wd) is off by 2 units of 2^-24 of |w|, the
update by 2^-20 of itself (the two corrections from expm1, the products and a
2-ulp division), the difference by 2^-24 of the result: |error| <= 2^-22 |w| + 2^-19 |update|."""
import numpy as np
import pytest
import torch

import train_refs as tr
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def f32(v):
    return float(np.float32(v))


@pytest.fixture(scope="module")
def gs():
    import mixed_precision_numerics_gradscaler_gb300 as gs
    torch.cuda.set_device(0)
    return gs


class Params:
    """A list of tensors, each a view `off` elements into its own buffer."""

    def __init__(self, gs, sizes, e4m3, grad="f32", copy=True, off=0, decay=None, zero=False, seed=0):
        gen = torch.Generator(device=DEV)
        gen.manual_seed(seed + 17)
        self.sizes, self.e4m3, self.decay = sizes, e4m3, decay
        self.bufs = []

        def new(n, dtype, fill):
            b = torch.full((n + off + 16,), 77, dtype=dtype, device=DEV)
            b[off:off + n] = fill
            self.bufs.append((b, off, n))
            return b[off:off + n]

        rn = lambda n: torch.randn(n, device=DEV, generator=gen)  # noqa: E731
        wide = lambda n: rn(n) * torch.exp2(-18 * torch.rand(n, device=DEV, generator=gen))  # noqa: E731
        self.w = [new(n, torch.float32, rn(n) * 0.1) for n in sizes]
        self.wb = [new(n, torch.bfloat16, 0) for n in sizes] if copy else None
        self.g = [new(n, TYPES[grad], (wide(n) * 0.3).to(TYPES[grad])) for n in sizes]
        if e4m3:
            codes = lambda n, top: torch.randint(0, top, (n,), device=DEV, generator=gen)  # noqa: E731
            sign = lambda n: 128 * torch.randint(0, 2, (n,), device=DEV, generator=gen)  # noqa: E731
            nb = lambda n: -(-n // 128)  # noqa: E731
            z = 0 if zero else 1
            self.m = [new(n, torch.uint8, (codes(n, 127) + sign(n)) * z) for n in sizes]
            self.v = [new(n, torch.uint8, codes(n, 127) * z) for n in sizes]
            self.ms = [new(nb(n), torch.float32, 1e-4 * z * (rn(nb(n)).abs() + 0.1)) for n in sizes]
            self.vs = [new(nb(n), torch.float32, 1e-4 * z * (rn(nb(n)).abs() + 0.1)) for n in sizes]
        else:
            z = 0.0 if zero else 1.0
            self.m = [new(n, torch.float32, wide(n) * 0.1 * z) for n in sizes]
            self.v = [new(n, torch.float32, (wide(n) * 0.1 * z) ** 2) for n in sizes]
            self.ms = self.vs = None
        self.step = torch.zeros(1, dtype=torch.int64, device=DEV)
        self.found = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.list = gs.gs_adamw_list_create(self.w, self.g, self.m, self.v, self.ms, self.vs,
                                            self.wb, decay)

    def state(self):
        return [[t.clone() for t in ts] for ts in (self.w, self.g, self.m, self.v, self.ms or [],
                                                   self.vs or [], self.wb or [])]

    def guards_kept(self):
        return all((b[:o] == 77).all() and (b[o + n:] == 77).all() for b, o, n in self.bufs)


HP = dict(lr=f32(1e-2), beta1=f32(0.9), beta2=f32(0.999), eps=f32(1e-8), weight_decay=f32(0.1))


def run_and_check(gs, p, hp=HP, coef=None, norm=None, max_norm=0.0, seed=5):
    w0, g0, m0, v0, ms0, vs0, _ = p.state()
    t = int(p.step) + 1
    gs.gs_master_update_adamw(p.list, p.step, p.found, max_norm=max_norm,
                              grad_norm=norm, seed=seed, **hp)
    assert int(p.step) == t
    assert p.guards_kept(), "written outside the tensors"
    coef = 1.0 if coef is None else coef
    place = 0
    grid = tr.e4m3_values().astype(np.float32)
    for i, n in enumerate(p.sizes):
        if n == 0:
            continue
        g = g0[i].float().cpu().numpy()
        if p.e4m3:
            blk = np.arange(n) // 128
            m = grid[m0[i].cpu().numpy()] * ms0[i].cpu().numpy()[blk]
            r = grid[v0[i].cpu().numpy()] * vs0[i].cpu().numpy()[blk]
            v = r * r
        else:
            m, v = m0[i].cpu().numpy(), v0[i].cpu().numpy()
        nm, nv, nr = tr.moments_f32(g, m, v, hp["beta1"], hp["beta2"], coef)
        if p.e4m3:
            bits = tr.random_bits(place, n, seed, t)
            for got, got_s, x, r16, keep in ((p.m[i], p.ms[i], nm, bits & 0xFFFF, False),
                                             (p.v[i], p.vs[i], nr, bits >> np.uint32(16), True)):
                code, scale = tr.round_block(x, r16, keep)
                assert np.array_equal(got_s.cpu().numpy(), scale), (i, "scales")
                bad = got.cpu().numpy() != code
                assert not bad.any(), (i, "codes", np.flatnonzero(bad)[:5])
        else:
            assert np.array_equal(p.m[i].cpu().numpy(), nm), (i, "m")
            assert np.array_equal(p.v[i].cpu().numpy(), nv), (i, "v")
        wd = hp["weight_decay"] * (p.decay[i] if p.decay else 1.0)
        keep = w0[i].cpu().double() * (1 - hp["lr"] * wd)
        want = keep - tr.adamw_update(torch.from_numpy(nm), torch.from_numpy(nr), t, hp["lr"],
                                      hp["beta1"], hp["beta2"], hp["eps"])
        tol = 2.0 ** -22 * w0[i].cpu().double().abs() + 2.0 ** -19 * (want - keep).abs() + 2.0 ** -126
        bad = (p.w[i].cpu().double() - want).abs() > tol
        assert not bad.any(), (i, "w", int(bad.sum()))
        if p.wb is not None:
            assert torch.equal(p.wb[i], p.w[i].bfloat16()), (i, "copy")
        place += -(-n // 128) * 128


SIZES = [1, 127, 128, 129, 0, 1000, 8191, 8192, 8193, 20011, 3]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("grad", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("copy", [False, True])
def test_three_steps(gs, e4m3, grad, copy):
    p = Params(gs, SIZES, e4m3, grad, copy)
    for _ in range(3):
        run_and_check(gs, p)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("off", [1, 2, 3, 4, 8, 16])
def test_alignment(gs, e4m3, off):
    p = Params(gs, [5, 130, 9000, 16384], e4m3, "bf16", True, off)
    run_and_check(gs, p)


@pytest.mark.parametrize("e4m3", [False, True])
def test_first_step_from_zero_moments(gs, e4m3):
    run_and_check(gs, Params(gs, [1000, 8192], e4m3, zero=True))


@pytest.mark.parametrize("e4m3", [False, True])
def test_betas_of_zero_and_no_decay(gs, e4m3):
    hp = dict(lr=f32(1e-3), beta1=0.0, beta2=0.0, eps=f32(1e-6), weight_decay=0.0)
    run_and_check(gs, Params(gs, [1000, 300], e4m3), hp)


@pytest.mark.parametrize("e4m3", [False, True])
def test_later_steps_and_decay_factors(gs, e4m3):
    p = Params(gs, [513, 40, 8200], e4m3, decay=[1.0, 0.0, 0.5])
    for t in (9, 999, 10 ** 6, 10 ** 10):
        p.step.fill_(t)
        run_and_check(gs, p)


@pytest.mark.parametrize("e4m3", [False, True])
def test_clipping(gs, e4m3):
    p = Params(gs, [700, 9000], e4m3)
    norm = torch.tensor([3.7], device=DEV)
    run_and_check(gs, p, norm=norm, max_norm=f32(1.1), coef=float(np.float32(1.1) / np.float32(3.7)))
    run_and_check(gs, p, norm=norm, max_norm=5.0)       # below the limit: unchanged
    run_and_check(gs, p, norm=norm, max_norm=0.0)       # no clipping


@pytest.mark.parametrize("e4m3", [False, True])
def test_many_tensors(gs, e4m3):
    rng = np.random.default_rng(1)
    run_and_check(gs, Params(gs, [int(n) for n in rng.integers(1, 700, 900)], e4m3, "bf16"))


@pytest.mark.parametrize("e4m3", [False, True])
def test_large_tensors(gs, e4m3):
    run_and_check(gs, Params(gs, [3000001, 128, 1 << 21], e4m3, "bf16"))


@pytest.mark.parametrize("e4m3", [False, True])
def test_skipped_step_changes_nothing(gs, e4m3):
    p = Params(gs, [1000, 8200], e4m3)
    before = p.state()
    p.found.fill_(1)
    gs.gs_master_update_adamw(p.list, p.step, p.found, **HP)
    after = p.state()
    assert int(p.step) == 0
    assert all(torch.equal(a, b) for x, y in zip(before, after) for a, b in zip(x, y))
    p.found.zero_()
    run_and_check(gs, p)


@pytest.mark.parametrize("e4m3", [False, True])
def test_empty_list_counts_the_step(gs, e4m3):
    p = Params(gs, [], e4m3)
    gs.gs_master_update_adamw(p.list, p.step, p.found, **HP)
    assert int(p.step) == 1


def test_zero_blocks_and_tiny_and_huge_moments(gs):
    p = Params(gs, [128 * 6], True, zero=True)
    g = p.g[0].view(6, 128)
    g[0] = 0                       # stays zero
    g[1] = torch.randn(128, device=DEV) * 1e-30
    g[2] = torch.randn(128, device=DEV) * 1e-18
    g[3] = torch.randn(128, device=DEV) * 1e15
    g[4] = 0
    g[4, 77] = 1.0                 # one value: the others' roots stay zero
    g[5] = 1e-6
    g[5, 3] = 1.0                  # roots far below the block's largest: not zero
    for _ in range(2):
        run_and_check(gs, p)
    v = p.v[0].view(6, 128)
    assert (v[0] == 0).all() and (v[4] != 0).sum() == 1 and (v[5] != 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nonfinite_gradients_show_in_the_states(gs, bad):
    for e4m3 in (False, True):
        p = Params(gs, [512], e4m3)
        p.g[0][200] = bad
        gs.gs_master_update_adamw(p.list, p.step, p.found, **HP)
        w = p.w[0]
        assert not torch.isfinite(w[200]) and torch.isfinite(w[:128]).all()
        if e4m3:
            assert not torch.isfinite(p.ms[0][1]) and not torch.isfinite(p.vs[0][1])
            assert torch.isfinite(p.ms[0][[0, 2, 3]]).all()
        else:
            assert not torch.isfinite(p.m[0][200]) and torch.isfinite(p.m[0][:200]).all()


def test_root_of_every_significand(gs):
    """The step's square root is its own: beta2 = 0 and gradients g make v the
    rounded product g * g, whose root must be the IEEE one (numpy's).  With
    g = s * 2^k, s every 2^-12th significand, over the whole range of v, in
    both element types' kernels."""
    s = (1 + np.arange(4096) / 4096).astype(np.float32)
    g = np.concatenate([s * np.float32(2.0 ** k) for k in (-60, -49, -48, -47, -20, -1, 0, 7, 47, 48, 49, 60)])
    rng = np.random.default_rng(2)
    g = np.concatenate([g, np.exp2(rng.uniform(-62, 62, 1 << 20)).astype(np.float32)])
    hp = dict(lr=0.0, beta1=0.0, beta2=0.0, eps=f32(1e-8), weight_decay=0.0)
    for e4m3 in (False, True):
        p = Params(gs, [g.size], e4m3, "f32", False, zero=True)
        p.g[0].copy_(torch.from_numpy(g))
        gs.gs_master_update_adamw(p.list, p.step, p.found, seed=5, **hp)
        _, v, r = tr.moments_f32(g, 0 * g, 0 * g, 0.0, 0.0)
        if e4m3:
            code, scale = tr.round_block(r, tr.random_bits(0, g.size, 5, 1) >> np.uint32(16), True)
            assert np.array_equal(p.vs[0].cpu().numpy(), scale)
            assert np.array_equal(p.v[0].cpu().numpy(), code)
        else:
            assert np.array_equal(p.v[0].cpu().numpy(), v)


def test_codes_read_back_through_fp8_dequant(gs):
    p = Params(gs, [1024], True)
    gs.gs_master_update_adamw(p.list, p.step, p.found, **HP)
    y = torch.empty(1, 1024, device=DEV)
    gs.fp8_dequant(p.m[0].view(1, 1024), p.ms[0], 1, 128, "e4m3", y)
    grid = tr.e4m3_values().astype(np.float32)
    want = grid[p.m[0].cpu().numpy()] * np.repeat(p.ms[0].cpu().numpy(), 128)
    assert np.array_equal(y.cpu().numpy()[0], want)


def test_place_beyond_32_bits(gs):
    """Two tensors, the first past 2^32 elements: the second's random bits
    use the place's high word, and the first's far end is updated."""
    n = (1 << 32) + 300
    w = torch.zeros(n, device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    m, v = (torch.zeros(n, dtype=torch.uint8, device=DEV) for _ in range(2))
    ms, vs = (torch.zeros(-(-n // 128), device=DEV) for _ in range(2))
    cut = (1 << 32) - 512
    tail = slice(cut, n)
    g[tail] = torch.randn(n - cut, device=DEV).bfloat16()
    w2, g2 = torch.zeros(1000, device=DEV), torch.randn(1000, device=DEV).bfloat16()
    m2, v2 = (torch.zeros(1000, dtype=torch.uint8, device=DEV) for _ in range(2))
    ms2, vs2 = (torch.zeros(8, device=DEV) for _ in range(2))
    al = gs.gs_adamw_list_create([w, w2], [g, g2], [m, m2], [v, v2], [ms, ms2], [vs, vs2])
    step, found = torch.zeros(1, dtype=torch.int64, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    gs.gs_master_update_adamw(al, step, found, seed=3, **HP)
    for gg, mm, vv, place in ((g[tail], m[tail], v[tail], cut), (g2, m2, v2, -(-n // 128) * 128)):
        gn = gg.float().cpu().numpy()
        z = np.zeros_like(gn)
        nm, nv, nr = tr.moments_f32(gn, z, z, HP["beta1"], HP["beta2"])
        bits = tr.random_bits(place, gn.size, 3, 1)
        assert np.array_equal(mm.cpu().numpy(), tr.round_block(nm, bits & 0xFFFF)[0])
        assert np.array_equal(vv.cpu().numpy(), tr.round_block(nr, bits >> np.uint32(16), True)[0])
    assert (w[cut:] != 0).sum() >= n - cut - 2 and (w[:cut] == 0).all()


def test_graph_replays_advance_the_step(gs):
    for e4m3 in (False, True):
        a, b = (Params(gs, [5000, 77], e4m3, seed=8) for _ in range(2))
        for _ in range(3):
            gs.gs_master_update_adamw(a.list, a.step, a.found, seed=1, **HP)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            gs.gs_master_update_adamw(b.list, b.step, b.found, seed=1, **HP)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        assert int(b.step) == 3
        assert all(torch.equal(x, y) for u, v in zip(a.state(), b.state()) for x, y in zip(u, v))


def test_8_bit_moments_follow_a_falling_second_moment(gs):
    """Gradients shrink a hundredfold and stay there: the stored root has to
    come down with beta2's decay (nearest rounding would keep every code of a
    block whose largest element does not shrink)."""
    n = 128 * 64
    p = Params(gs, [n], True, zero=True)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(4)
    hp = dict(HP, beta2=f32(0.99), lr=0.0, weight_decay=0.0)
    big = torch.randn(n, device=DEV, generator=gen)
    big.view(-1, 128)[:, 0] = 3.0
    v = np.zeros(n)
    for s in range(600):
        scale = 1.0 if s < 200 else 0.01
        gn = big * scale
        gn.view(-1, 128)[:, 0] = 3.0
        p.g[0].copy_(gn)
        gs.gs_master_update_adamw(p.list, p.step, p.found, seed=2, **hp)
        v = v * 0.99 + 0.01 * gn.cpu().numpy().astype(np.float64) ** 2
    r = tr.e4m3_values()[p.v[0].cpu().numpy()] * np.repeat(p.vs[0].cpu().numpy(), 128)
    rest = np.arange(n) % 128 != 0
    # root mean square over the elements: within the noise of rounding up or
    # down (E4M3's gap is up to 1/8) and the bias its variance gives r^2
    got, want = np.sqrt((r[rest] ** 2).mean()), np.sqrt(v[rest].mean())
    assert 0.8 < got / want < 1.25, (got, want)


def test_refusals(gs):
    w, g, m, v = (torch.zeros(300, device=DEV) for _ in range(4))
    step, found = torch.zeros(1, dtype=torch.int64, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    with pytest.raises(gs.GsError):
        gs.gs_adamw_list_create([w], [w], [m], [v])          # gradients overlap the master
    with pytest.raises(gs.GsError):
        gs.gs_adamw_list_create([w], [g], [m], [m])
    with pytest.raises(gs.GsError):
        gs.gs_adamw_list_create([w, w[100:200]], [g, g[:100]], [m, m[:100]], [v, v[:100]])
    with pytest.raises(gs.GsError):
        gs.gs_adamw_list_create([w], [g], [m], [v], decay=[-1.0])
    with pytest.raises(ValueError):
        gs.gs_adamw_list_create([w], [g], [m], [v[:299]])
    with pytest.raises(ValueError):
        gs.gs_adamw_list_create([w], [g], [m], [v.byte()])
    with pytest.raises(ValueError):
        gs.gs_adamw_list_create([w], [g], [m.byte()], [v.byte()], [torch.zeros(2, device=DEV)],
                                [torch.zeros(3, device=DEV)])
    with pytest.raises(gs.GsError):
        gs.gs_adamw_list_create([w.cpu()], [g], [m], [v])
    al = gs.gs_adamw_list_create([w], [g], [m], [v])
    for bad in (dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=float("inf")),
                dict(weight_decay=-0.1), dict(max_norm=1.0), dict(max_norm=float("nan"))):
        with pytest.raises(gs.GsError):
            gs.gs_master_update_adamw(al, step, found, **{"lr": 1e-3, **bad})
    torch.cuda.synchronize()
    assert int(step) == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("off", [0, 1])
def test_eps_whose_reciprocal_is_no_normal_number(gs, e4m3, off):
    """eps below 2^-126, where the divisor is eps alone (v = 0, with m = 0 and
    with m small enough for v to underflow), and above 2^126."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(21)
    for eps in (1e-45, 1e-41, 1.1e-38, 1.2e-38):
        p = Params(gs, [1000, 8192], e4m3, off=off, zero=True)
        for g in p.g:
            g.copy_(torch.randn(g.numel(), device=DEV, generator=gen) * 1e-25)
            g[::3] = 0
        for _ in range(2):
            run_and_check(gs, p, dict(HP, eps=f32(eps)))
    for eps in (1e38, 3.4e38):
        p = Params(gs, [1000, 8192], e4m3, off=off, zero=True)
        for g in p.g:
            g.copy_((torch.rand(g.numel(), device=DEV, generator=gen) - 0.5) * 4e18)
        run_and_check(gs, p, dict(HP, lr=f32(1e20), eps=f32(eps), weight_decay=0.0))
        assert (p.w[0].abs() > 0.01).any()


def root_bits(gs, bits):
    """The bits of the 8-bit step's roots of the numbers with these bits."""
    v = torch.from_numpy(bits.view(np.int32)).to(DEV).view(torch.float32)
    r = torch.full_like(v, 7.0)
    gs.gs_test_adamw_root(v, r)
    return r.cpu().numpy().view(np.uint32)


@pytest.mark.parametrize("exponent", [0, -96, 94])
def test_root_of_every_significand_of_two_binades(gs, exponent):
    """[2^e, 2^(e + 2)) whole, in the middle and at both ends of the range
    that has the step's own root: the bits of the IEEE root (numpy's)."""
    first = (127 + exponent) << 23
    bits = np.arange(first, first + (1 << 24), dtype=np.uint32)
    want = np.sqrt(bits.view(np.float32)).view(np.uint32)
    assert np.array_equal(root_bits(gs, bits), want)
    # paired otherwise: each number's root is its own lane's
    order = np.random.default_rng(exponent + 100).permutation(bits.size)[:1 << 22]
    assert np.array_equal(root_bits(gs, bits[order]), want[order])


def test_roots_over_the_whole_type(gs):
    """Random pairs over every exponent, both kinds of number in a pair
    included, and zeros, subnormals and infinities: the IEEE root's bits; NaN
    for NaN."""
    rng = np.random.default_rng(11)
    bits = rng.integers(0, 0x7F800001, 1 << 22, dtype=np.uint32)
    ends = np.array([0, 1, 2, 0x007FFFFF, 0x00800000, 0x7F7FFFFF, 0x7F800000,
                     (127 - 96) << 23, ((127 - 96) << 23) - 1, (127 + 96) << 23, ((127 + 96) << 23) + 1], np.uint32)
    bits = np.concatenate([bits, np.repeat(ends, ends.size), np.tile(ends, ends.size), ends, ends])
    bits = np.concatenate([bits, np.stack([np.repeat(ends, ends.size), np.tile(ends, ends.size)], 1).ravel()])
    want = np.sqrt(bits.view(np.float32)).view(np.uint32)
    assert np.array_equal(root_bits(gs, bits), want)
    nan = np.array([0x7FC00000, 0x3F800000, 0x3F800000, 0x7FC00000, 0x7FC00000, 0], np.uint32)
    got = root_bits(gs, nan).view(np.float32)
    assert np.array_equal(np.isnan(got), np.isnan(nan.view(np.float32))) and got[1] == got[2] == 1 and got[5] == 0


def test_root_refusals(gs):
    v = torch.ones(64, device=DEV)
    with pytest.raises(gs.GsError):
        gs.gs_test_adamw_root(v[:63], torch.empty(63, device=DEV))
    with pytest.raises(gs.GsError):
        gs.gs_test_adamw_root(v, v)
    with pytest.raises(ValueError):
        gs.gs_test_adamw_root(v, torch.empty(62, device=DEV))
    with pytest.raises(gs.GsError):
        gs.gs_test_adamw_root(v.cpu(), torch.empty(64, device=DEV))
