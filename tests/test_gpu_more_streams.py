"""The 4-bit tensors and the policy loss captured into graphs and replayed on new
inputs, and called by several threads on streams of their own: the same bits as
single calls in order."""
import threading

import pytest
import torch

from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gs():
    import mixed_precision_numerics_gradscaler_gb300 as gs
    torch.cuda.set_device(0)
    return gs


class Work:
    """One of each operator on buffers of its own."""

    def __init__(self, gs, R, C, N, T, S, fmt):
        self.gs, self.fmt, self.T, self.S = gs, fmt, T, S
        u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)  # noqa: E731
        nv = fmt == "nvfp4"
        one = lambda: torch.zeros(1, device=DEV) if nv else None  # noqa: E731
        self.x, self.w = torch.zeros(R, C, device=DEV).bfloat16(), torch.zeros(N, C, device=DEV)
        self.q, self.s = u8(R, C // 2), u8(gs.fp4_scale_bytes(R, C, fmt))
        self.qt, self.st = u8(C, R // 2), u8(gs.fp4_scale_bytes(C, R, fmt))
        self.wq, self.ws = u8(N, C // 2), u8(gs.fp4_scale_bytes(N, C, fmt))
        self.ta, self.tb = one(), one()
        self.space = u8(gs.gs_ws_bytes()) if nv else None
        self.y, self.d = torch.zeros(R, C, device=DEV), torch.zeros(R, N, device=DEV)
        f = lambda: torch.zeros(T, device=DEV)  # noqa: E731
        self.lp, self.old, self.ref, self.grad = f(), f(), f(), f()
        self.adv, self.tg = torch.zeros(S, device=DEV), torch.zeros(T, dtype=torch.int64, device=DEV)
        self.off = torch.linspace(0, T, S + 1, device=DEV).long()
        self.loss, self.stats = torch.zeros(1, device=DEV), torch.zeros(4, device=DEV)
        self.lws = torch.full((gs.gs_policy_loss_ws_bytes(T, S),), 0x77, dtype=torch.uint8, device=DEV)

    def fill(self, seed):
        gen = torch.Generator(device=DEV)
        gen.manual_seed(seed)
        rnd = lambda t: t.copy_(torch.randn(t.shape, device=DEV, generator=gen))  # noqa: E731
        for t in (self.x, self.w, self.lp, self.old, self.ref, self.adv):
            rnd(t)
        self.tg.copy_(torch.randint(-2, 9, (self.T,), device=DEV, generator=gen))

    def run(self):
        gs = self.gs
        gs.fp4_quant(self.x, self.fmt, self.q, self.s, self.ta, self.space, self.qt, self.st)
        gs.fp4_quant(self.w, self.fmt, self.wq, self.ws, self.tb, self.space)
        gs.fp4_gemm_block_scaled(self.q, self.s, self.wq, self.ws, self.fmt, self.d, self.ta, self.tb)
        gs.fp4_dequant(self.q, self.s, self.fmt, self.y, self.ta)
        gs.gs_policy_loss(self.lp, self.old, self.adv, self.loss, self.lws, self.grad, self.stats, self.ref, self.tg,
                          self.off, kl_coef=0.1, reduction="sequence")

    def out(self):
        ts = (self.q, self.s, self.qt, self.st, self.ta, self.d, self.y, self.grad, self.loss, self.stats)
        return [t.clone() for t in ts if t is not None]


SIZES = [(1024, 512, 700, 30000, 40, "nvfp4"), (32, 96, 33, 900, 7, "nvfp4"), (1056, 544, 130, 6000, 3000, "mxfp4"),
         (32, 4096, 5000, 5121, 2, "nvfp4")]


@pytest.mark.parametrize("size", SIZES)
def test_captured_calls_replay_on_new_inputs(gs, size):
    w = Work(gs, *size)
    want = []
    for seed in (1, 2):
        w.fill(seed)
        w.run()
        want.append(w.out())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        w.run()
    for seed in (2, 1, 2):
        w.fill(seed)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(w.out(), want[seed - 1]))
    assert gs.gs_device_status() == gs.GS_OK


def test_threads_on_streams_of_their_own(gs):
    works = [Work(gs, *s) for s in SIZES]
    want = []
    for i, w in enumerate(works):
        w.fill(i)
        w.run()
        want.append(w.out())
    torch.cuda.synchronize()
    failed = []

    def go(w, want):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    w.run()
                got = w.out()
            s.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want)):
                failed.append("differs")
        except Exception as e:  # a thread's failure is the test's
            failed.append(e)

    threads = [threading.Thread(target=go, args=a) for a in zip(works, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    assert gs.gs_device_status() == gs.GS_OK
