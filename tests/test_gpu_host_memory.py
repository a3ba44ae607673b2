"""A host allocation that fails inside an entry point ends neither the process nor the
call: the library's caches of kernel attributes are filled by the next one (GPU; in a
child process whose operator new fails on demand)."""
import os
import shutil
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))

SHIM = r"""
#include <cstdlib>
#include <new>
extern "C" { int starkv_test_fail = 0; int starkv_test_failed = 0; }
void* operator new(std::size_t n) {
  if (starkv_test_fail) { ++starkv_test_failed; throw std::bad_alloc(); }
  void* p = std::malloc(n ? n : 1);
  if (!p) throw std::bad_alloc();
  return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }
"""

CHILD = r"""
import ctypes, sys
sys.path[:0] = [sys.argv[2], sys.argv[3]]
import numpy as np, torch
import rank_compressed_kv_star_b200 as S
from group_common import Layer, make_cross, to_device, call, reference
shim = ctypes.CDLL(sys.argv[1])
fail, failed = (ctypes.c_int.in_dll(shim, "starkv_test_" + x) for x in ("fail", "failed"))
L = Layer(1, 8, 2, 64, 48, 192)
c = make_cross(L, [(70, 3)])
lib, ref = S.load_library(), reference(L, c)
desc = S.layer_desc(L.H, L.d, L.r, L.R, c["nb"], c["tables"].shape[1], num_kv_heads=L.Hkv)
args = (ctypes.byref(desc), 1, 3, 70)
torch.cuda.init()
fail.value = 1                                   # nothing of this call is in the caches yet
nbytes = lib.starkv_cross_workspace_bytes(*args)
fail.value = 0
assert failed.value > 0 and nbytes == lib.starkv_cross_workspace_bytes(*args), (failed.value, nbytes)
g = to_device(L, c)
call(L, c, g)
assert S.starkv_decode_check(g["ws"]) == (0, 0)
got = g["out"].float().cpu().numpy()
assert all((np.abs(got[b] - ref[0][b]) <= ref[1][b]).all() for b in ref[0])
print("done")
"""


def test_a_failed_host_allocation_is_not_an_abort(cuda_ok, tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, so = tmp_path / "shim.cpp", tmp_path / "shim.so"
    src.write_text(SHIM)
    subprocess.run([cxx, "-O1", "-std=c++17", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    child = subprocess.run([sys.executable, "-c", CHILD, str(so), os.path.dirname(HERE), HERE], capture_output=True, text=True,
                           timeout=300, env=dict(os.environ, LD_PRELOAD=str(so)))
    assert child.returncode == 0 and "done" in child.stdout, (child.returncode, child.stderr[-2000:])
