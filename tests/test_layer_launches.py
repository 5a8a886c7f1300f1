"""What the layer operators launch, recorded on the host: a process of its own loads
libgdn.so behind a stand-in for hipLaunchKernel that notes every launch and runs nothing, so
the largest problems need no GPU and no memory.  A launch has fewer than 2^32 threads."""
import ctypes
import json
import os
import subprocess
import sys

import pytest

import chunked_gated_delta_prepare_amd as gdn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STAND_IN = r"""
#include <string.h>
typedef struct { unsigned x, y, z; } dims;
int noted = 0;
unsigned grids[4096], blocks[4096];
unsigned char params[4096][48];
int hipLaunchKernel(const void *fn, dims grid, dims block, void **args, unsigned long lds, void *stream) {
    if (noted < 4096) {
        grids[noted] = grid.x * grid.y * grid.z;
        blocks[noted] = block.x * block.y * block.z;
        memcpy(params[noted], args[0], 48);
        ++noted;
    }
    return 0;
}
"""
CHILD = r"""
import ctypes, json, sys
sys.path.insert(0, %r)
stand_in = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
import chunked_gated_delta_prepare_amd as gdn
from chunked_gated_delta_prepare_amd import layer_abi as A
lib = gdn.load_library()
out = []
FAKE = 0x10000
for name, kind, fields, args in json.loads(sys.argv[2]):
    ctypes.c_int.in_dll(stand_in, "noted").value = 0
    pr = getattr(A, kind)(**fields)
    st = getattr(lib, name)(ctypes.byref(pr), *args, None)
    n = ctypes.c_int.in_dll(stand_in, "noted").value
    get = lambda what, t: (t * 4096).in_dll(stand_in, what)
    out.append([st, [[get("grids", ctypes.c_uint)[i], get("blocks", ctypes.c_uint)[i], list(get("params", ctypes.c_uint64 * 6)[i])] for i in range(n)]])
print(json.dumps(out))
""" % ROOT

FAKE, BIG = 1 << 16, 1 << 50


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    """launches([(function, problem's kind, fields, arguments), ...]): (status, [(workgroups, threads
    of one, the parameters' first six 64-bit words)]) of each call."""
    if not os.path.exists(gdn.LIB_PATH):
        from chunked_gated_delta_prepare_amd import build
        build.build()
    d = tmp_path_factory.mktemp("launches")
    (d / "stand_in.c").write_text(STAND_IN)
    so = str(d / "stand_in.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", so, str(d / "stand_in.c")], check=True)

    def run(calls):
        r = subprocess.run([sys.executable, "-c", CHILD, so, json.dumps(calls)], capture_output=True, text=True, cwd=ROOT)
        assert r.returncode == 0, r.stderr[-2000:]
        return json.loads(r.stdout.strip().splitlines()[-1])

    return run


def small(found):
    return all(grid * block < 1 << 32 for _, calls in found for grid, block, _ in calls)


def gate_norm_backward(T, H, D, each=1, dbias=True):
    pr = dict(T=T, H=H, D=D, x_stride_t=H * D, x_stride_h=D, z_stride_t=H * D, z_stride_h=D, dz_stride_t=H * D, dz_stride_h=D,
              io_dtype=1, w_dtype=1, each=each, gate_first=0, center=1, act=0, eps=1e-5)
    return "gdn_gate_norm_backward", "GateNormProblem", pr, [FAKE] * 8 + [FAKE if dbias else None, FAKE, BIG]


def test_sums_of_the_weights_gradients(launches):
    """Weights of each of many wide heads: the sums' launches are as many as they need, and
    take all classes between them, in order."""
    sizes = [(1, 4096, 8192, True), (1, 4096, 8192, False), (2, 65536, 4096, True), (3, 65535, 4095, False), (2, 8, 1024, True)]
    found = launches([gate_norm_backward(T, H, D, 1, b) for T, H, D, b in sizes])
    assert small(found)
    for (T, H, D, both), (status, calls) in zip(sizes, found):
        assert status == 0
        cols, done = -(-D // 16), 0
        for grid, block, (part, dw, db, d, rows, c) in calls[1:]:
            classes = grid // (cols * (1 + both))
            assert block == 1024 and grid == classes * cols * (1 + both) and (d, rows, c) == (D, 1, cols)
            assert part == FAKE + done * rows * 2 * D * 4 and dw == FAKE + done * D * 4 and db == (FAKE + done * D * 4 if both else 0)
            done += classes
        assert done == H
    assert len(found[-1][1]) == 2
