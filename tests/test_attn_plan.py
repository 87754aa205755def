"""What qmv_attend launches, over the sizes that it takes: on the CPU, by a launch function
that notes its arguments and starts nothing."""
import json
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STUB = r"""
typedef struct { unsigned x, y, z; } dim3;
int launches;
unsigned grid[2];
unsigned turns;        /* of the join, the second launch: its seventh argument */
int hipLaunchKernel(const void* f, dim3 g, dim3 b, void** args, unsigned long lds, void* stream)
{
    if (launches < 2) grid[launches] = g.x * g.y * g.z;
    if (launches == 1) turns = *(unsigned*)args[6];
    ++launches;
    return 0;
}
"""

# The library finds the stub's function before HIP's own, since that is loaded first and for all.
CHILD = r"""
import ctypes, itertools, json, sys
stub = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[2])
from bit_quantized_gemv_amd import ops
L = ops._load()
n, grid, turns = (t.in_dll(stub, s) for t, s in ((ctypes.c_int, "launches"), (ctypes.c_uint * 2, "grid"), (ctypes.c_uint, "turns")))
at = lambda i: (1 << 20) + (i << 44)
joins = 0
for B, more, Hq, Hkv, D, new, length, window, out in itertools.product(
        (1, 3, 64, 255, 1024, 1025, 2048, 4097, 9000, 65535), (0, 1, 17, 512, 4096), (1, 2, 8, 16), (1, 2, 8), (8, 64, 128, 256),
        (1, 16, 17, 513), (0, 64, 512, 4096, 131072), (0, 1000), (0, 2)):
    if Hq % Hkv:
        continue
    T = min(B, 1 << 22) + more
    c = ops.Cache(k=at(5), v=at(6), k_page=16 * Hkv * D, k_slot=Hkv * D, k_head=D, v_page=16 * Hkv * D, v_slot=Hkv * D, v_head=D, pages=at(7),
                  starts=at(8), lengths=at(9), pages_row=1 << 13, n_pages=50, page_size=16, n_seqs=B, max_pages=1 << 13, heads=Hkv, head_size=D, dt=2)
    sizes = (new, length, window, 3)
    case = (B, T, Hq, Hkv, D, *sizes, out)
    need = L.qmv_attend_workspace(ctypes.byref(c), T, Hq, *sizes)
    n.value = 0
    print(case, file=sys.stderr)          # what a call that ends the process was
    e = L.qmv_attend(ctypes.byref(c), at(20), at(23), at(24), need, T, Hq, Hq * D, D, *sizes, 0.1, out, None)
    assert e == 0, (case, e)
    assert need >= 0 and n.value in (1, 2) and grid[0] > 0, case
    assert need == 0 or out == 0 or n.value == 2, case
    if n.value == 2:
        joins += 1
        assert grid[1] > 0 and turns.value > 0, case
print(json.dumps(joins))
"""


@pytest.fixture(scope="module")
def stub(tmp_path_factory):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    from bit_quantized_gemv_amd import qmv
    if not os.path.exists(qmv.library_path()):
        from bit_quantized_gemv_amd import build
        build.build()
    d = tmp_path_factory.mktemp("stub")
    (d / "stub.c").write_text(STUB)
    subprocess.run([cc, "-shared", "-fPIC", "-O1", "-o", str(d / "stub.so"), str(d / "stub.c")], check=True)
    return str(d / "stub.so")


def test_launches(stub):
    """Every call is launched, and joined by one workgroup or more where its keys are shared."""
    r = subprocess.run([sys.executable, "-c", CHILD, stub, ROOT], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, (r.returncode, r.stderr[-600:])
    assert json.loads(r.stdout.strip().splitlines()[-1]) > 1000
