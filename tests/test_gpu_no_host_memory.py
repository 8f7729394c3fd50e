"""Entry points called when the host has no memory left: nothing is thrown
across the C interface.  A child process preloads an operator new that throws
on request; the library's first launch of a kernel, which remembers its
occupancy on the heap, must work all the same, and a list, which needs
memory, must be refused."""
import os
import subprocess
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu

_NEW = r'''
#include <cstdlib>
#include <new>
static thread_local int failing = 0, failed = 0;
extern "C" void fail_new(int on) { failing = on; }
extern "C" int failed_news() { return failed; }
void* operator new(std::size_t n) {
  void* p = failing ? nullptr : std::malloc(n ? n : 1);
  if (failing) ++failed;
  if (!p) throw std::bad_alloc();
  return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }
'''

_SCRIPT = r'''
import ctypes, sys
import torch
sys.path.insert(0, sys.argv[1])
import mixed_precision_numerics_gradscaler_gb300 as gs
host = ctypes.CDLL(None)
lib, vp, i64 = gs._lib, ctypes.c_void_p, ctypes.c_int64
dev = "cuda:0"

def failing(call):
    before = host.failed_news()
    host.fail_new(1)
    status = call()
    host.fail_new(0)
    assert host.failed_news() > before, "the preloaded operator new was not reached"
    return status

x, dy = (torch.randn(4096, 9000, device=dev).bfloat16() for _ in range(2))
y, dx = torch.zeros_like(x), torch.zeros_like(x)
mean, rstd = torch.zeros(4096, device=dev), torch.zeros(4096, device=dev)
gs.gs_layernorm_fwd(x[:8].float(), None, None, torch.empty(8, 9000, device=dev))   # the runtime is up
torch.cuda.synchronize()
R, C = x.shape
p = lambda t: t.data_ptr()
for rows, cols in ((4096, 9000), (4096, 4096)):      # a cluster's rows, and a CTA's
    args = (p(x), C, gs.GS_BF16, rows, cols, None, None, gs.GS_F32, 1e-5, p(y), C, p(mean), p(rstd), 0)
    assert failing(lambda: lib.gs_layernorm_fwd(*args)) == gs.GS_OK
    args = (p(dy), C, p(x), C, gs.GS_BF16, rows, cols, None, gs.GS_F32, p(mean), p(rstd), p(dx), C, None, None,
            gs.GS_F32, None, 0)
    assert failing(lambda: lib.gs_layernorm_bwd(*args)) == gs.GS_OK
    xd, dd = x[:, :cols].double(), dy[:, :cols].double()
    xh = (xd - xd.mean(1, keepdim=True)) / (xd.var(1, unbiased=False, keepdim=True) + 1e-5).sqrt()
    assert (y[:, :cols].double() - xh).abs().max() < 0.03
    want = (dd - dd.mean(1, keepdim=True) - xh * (dd * xh).mean(1, keepdim=True)) * rstd.double()[:, None]
    assert (dx[:, :cols].double() - want).abs().max() < 0.03
ptr = (vp * 1)(p(mean))
other = [(vp * 1)(p(t)) for t in (rstd, torch.zeros(64, device=dev), torch.zeros(64, device=dev))]
out, n = vp(), (i64 * 1)(64)
assert failing(lambda: lib.gs_adamw_list_create(ptr, None, other[0], gs.GS_F32, gs.GS_MOMENTS_F32, other[1],
                                                other[2], None, None, None, n, 1, ctypes.byref(out))) == gs.GS_ERR_ARG
assert not out.value and gs.gs_device_status() == gs.GS_OK
print("ok")
'''


def test_nothing_is_thrown_when_memory_runs_out(tmp_path):
    src, so = tmp_path / "new.cpp", tmp_path / "libnew.so"
    src.write_text(_NEW)
    subprocess.run(["g++", "-shared", "-fPIC", "-O1", "-o", str(so), str(src)], check=True, timeout=120)
    r = subprocess.run([sys.executable, "-c", _SCRIPT, ROOT], capture_output=True, text=True, timeout=300,
                       env={**os.environ, "LD_PRELOAD": str(so)})
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), (r.returncode, r.stdout, r.stderr[-2000:])
