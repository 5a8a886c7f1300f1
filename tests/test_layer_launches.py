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


def glr(name, B, T, D, io=1, grads=True):
    pr = dict(B=B, T=T, D=D, n_seqs=0, io_dtype=io, g_dtype=io, form=2, scale=2)
    for k in ("x", "g", "dy", "dx", "dg"):
        pr[k + "_stride_b"], pr[k + "_stride_t"] = T * D, D
    if name == "gdn_glr_forward":
        args = [FAKE] * 5 + [None, FAKE, FAKE, FAKE, BIG]
    else:
        args = [FAKE] * 6 + [None] + [FAKE] * 3 + [FAKE if grads else None] * 2 + [FAKE, FAKE, BIG]
    return name, "GlrProblem", pr, args


def test_gradients_of_very_many_short_sequences(launches):
    """Two to seven tiles of 32 tokens a sequence: the launch of the states at the tiles' borders
    has no more threads than the tiles'."""
    sizes = [(1 << 21, 33, 1), (1 << 22, 33, 64), ((1 << 23) - 1, 33, 64), (1 << 21, 224, 64), (1 << 15, 513, 640), (2, 8192, 4096)]
    found = launches([glr("gdn_glr_backward", *s) for s in sizes])
    assert small(found)
    for (B, T, D), (status, calls) in zip(sizes, found):
        tiles, groups = -(-T // 32), -(-D // 64)
        if B * D >= 1 << 29 or tiles * B * groups * 256 >= 1 << 32:
            assert status == 3 and not calls
            continue
        assert status == 0 and [c[:2] for c in calls[:3]] == [[tiles * B * groups, 256], [2 * B * groups, 64 * min(tiles, 16)],
                                                              [tiles * B * groups, 256]]
    # whatever is enqueued is enqueued whole
    found = launches([glr("gdn_glr_backward", 1 << k, T, 1) for k in range(19, 25) for T in (1, 32, 33, 64, 65, 97, 225, 481, 513)])
    assert small(found) and all((status == 0) == bool(calls) for status, calls in found)


def test_very_many_short_prompts(launches):
    """A wave for each of 2^24 prompts of some tokens, four waves for 2^23 of some more; with
    eight waves each the launch would be too large, and is refused."""
    sizes = [(1 << 24, 16, 1, 64), (1 << 23, 64, 63, 64), (1 << 23, 200, 1, 256), (1 << 23, 513, 1, 0), ((1 << 23) - 1, 513, 1, 512), (1, 37, 1030, 512)]
    found = launches([glr("gdn_glr_forward", B, T, D) for B, T, D, _ in sizes])
    assert small(found)
    for (B, T, D, threads), (status, calls) in zip(sizes, found):
        if not threads:
            assert status == 3 and not calls
        else:
            assert status == 0 and [c[:2] for c in calls] == [[B * -(-D // 64), threads]]


def test_pieces_of_the_moves(launches):
    """(sequences, tokens, channels, fp32, workgroups of the moves and of y): fp32 rows of
    several segments before the last are not cut in two or three pieces; long ones in twice as many of eight tiles, unless they are packed."""
    sizes = [(1, 8192, 4096, 0, 3 * 64 * 2, 256), (1, 8192, 4096, 1, 3 * 64, 256), (1, 12288, 4096, 0, 3 * 64 * 3, 256),
             (1, 12288, 4096, 1, 3 * 64, 256), (1, 65536, 4096, 0, 3 * 64 * 8, 256), (1, 32768, 4096, 1, 3 * 64 * 4, 256),
             (2, 8192, 4096, 1, 128 * 4, 256), (2, 4096, 4096, 1, 128 * 2, 256), (1, 2048, 1024, 1, 16 * 4, 32), (1, 2048, 1024, 0, 16 * 4, 32)]
    found = launches([glr("gdn_glr_forward", B, T, D, 0 if f else 1) for B, T, D, f, _, _ in sizes])
    assert small(found)
    for (*size, moves, y), (status, calls) in zip(sizes, found):
        assert status == 0 and [c[:2] for c in calls] == [[moves, 512], [y, 512]], (size, calls)
    packed = glr("gdn_glr_forward", 1, 65536, 4096)
    packed[2]["n_seqs"], packed[3][5] = 9, FAKE
    status, calls = launches([packed])[0]
    assert status == 0 and [c[:2] for c in calls] == [[3 * 64 * 4, 512], [256, 512]]
