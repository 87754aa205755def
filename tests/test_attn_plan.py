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
unsigned long shared;  /* bytes of LDS of the first */
int hipLaunchKernel(const void* f, dim3 g, dim3 b, void** args, unsigned long lds, void* stream)
{
    if (launches < 2) grid[launches] = g.x * g.y * g.z;
    if (launches == 0) shared = lds;
    if (launches == 1) turns = *(unsigned*)args[6];
    ++launches;
    return 0;
}
"""

# The library finds the stub's functions before HIP's own, since that is loaded first and for all.
BEGIN = r"""
import ctypes, itertools, json, sys
stub = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[2])
from bit_quantized_gemv_amd import ops
L = ops._load()
n, grid, turns, shared = (t.in_dll(stub, s) for t, s in ((ctypes.c_int, "launches"), (ctypes.c_uint * 2, "grid"), (ctypes.c_uint, "turns"),
                                                         (ctypes.c_ulong, "shared")))
at = lambda i: (1 << 20) + (i << 44)

def call(B, T, Hq, Hkv, D, new, length, window=0, sinks=3, dt=2, out=2):
    c = ops.Cache(k=at(5), v=at(6), k_page=16 * Hkv * D, k_slot=Hkv * D, k_head=D, v_page=16 * Hkv * D, v_slot=Hkv * D, v_head=D, pages=at(7),
                  starts=at(8), lengths=at(9), pages_row=1 << 13, n_pages=50, page_size=16, n_seqs=B, max_pages=1 << 13, heads=Hkv, head_size=D, dt=dt)
    need = L.qmv_attend_workspace(ctypes.byref(c), T, Hq, new, length, window, sinks)
    n.value = 0
    print((B, T, Hq, Hkv, D, new, length, window, dt, out), file=sys.stderr)          # what a call that ends the process was
    return L.qmv_attend(ctypes.byref(c), at(20), at(23), at(24), need, T, Hq, Hq * D, D, new, length, window, sinks, 0.1, out, None), need
"""

SIZES = BEGIN + r"""
joins = 0
for B, more, Hq, Hkv, D, new, length, window, out in itertools.product(
        (1, 3, 64, 255, 1024, 1025, 2048, 4097, 9000, 65535), (0, 1, 17, 512, 4096), (1, 2, 8, 16), (1, 2, 8), (8, 64, 128, 256),
        (1, 16, 17, 513), (0, 64, 512, 4096, 131072), (0, 1000), (0, 2)):
    if Hq % Hkv:
        continue
    e, need = call(B, min(B, 1 << 22) + more, Hq, Hkv, D, new, length, window, out=out)
    assert e == 0 and need >= 0 and n.value in (1, 2) and grid[0] > 0, e
    assert need == 0 or out == 0 or n.value == 2
    if n.value == 2:
        joins += 1
        assert grid[1] > 0 and turns.value > 0
print(json.dumps(joins))
"""

# 256 workgroups a share of the keys, and 256 of blocks beside them, of one tile of rows and of two
ROUNDS = BEGIN + r"""
found = []
for D, dt, out, (T, Hq, Hkv) in itertools.product((64, 96, 128, 192, 256), (1, 2), (0, 2), ((2048, 16, 16), (1024, 32, 1))):
    T *= 1 + (D > 192)
    e, _ = call(1, T, Hq, Hkv, D, T, 16 * 16384 // (64 if D <= 64 else 128 if D <= 128 else 256), dt=dt, out=out)
    assert e == 0
    found.append((D, Hq, dt, out, grid[0] / 256 - 1, shared.value))
print(json.dumps(found))
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


def child(stub, program):
    r = subprocess.run([sys.executable, "-c", program, stub, ROOT], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, (r.returncode, r.stderr[-600:])
    return json.loads(r.stdout.strip().splitlines()[-1])


def test_launches(stub):
    """Every call is launched, and joined by one workgroup or more where its keys are shared."""
    assert child(stub, SIZES) > 1000


def test_shares_fit(stub):
    """A chunk's keys are cut into no more shares than run at once: by the LDS that the launch asks for, of 160 KB in pieces of 1280 bytes."""
    for D, Hq, dt, out, shares, lds in child(stub, ROUNDS):
        assert 1 <= shares <= 128 // -(-lds // 1280), (D, Hq, dt, out, shares, lds)
