"""Every kernel source of the package is built: a file that no build unit reaches is a
second, stale copy of a kernel to whoever reads or searches the sources."""
import os
import re

from chunked_gated_delta_prepare_amd import build

PACKAGE = os.path.dirname(os.path.abspath(build.__file__))


def test_every_source_is_reached_by_a_build_unit():
    found = {os.path.join(d, f) for d, _, files in os.walk(PACKAGE) for f in files if f.endswith((".hip", ".h", ".cpp", ".c"))}
    todo, reached = [os.path.join(build.CSRC, unit) for unit in build.UNITS], set()
    while todo:
        path = todo.pop()
        if path in reached:
            continue
        assert os.path.exists(path), path
        reached.add(path)
        with open(path) as f:
            for name in re.findall(r'^\s*#\s*include\s+"([^"]+)"', f.read(), re.M):
                todo.append(os.path.normpath(os.path.join(os.path.dirname(path), name)))
    assert not found - reached, sorted(os.path.relpath(p, PACKAGE) for p in found - reached)
