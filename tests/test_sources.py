"""The kernels' sources: every header is included by a source that is built."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp8_delayed_scaling_03_b200", "csrc")


def test_every_header_is_included():
    seen, todo = set(), sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    while todo:
        path = todo.pop()
        if path in seen or not os.path.exists(path):
            continue
        seen.add(path)
        todo += [os.path.join(CSRC, h) for h in re.findall(r'#include "([^"]+)"', open(path).read())]
    headers = {p for p in glob.glob(os.path.join(CSRC, "*")) if p.endswith((".h", ".cuh"))}
    assert headers <= seen, sorted(os.path.basename(p) for p in headers - seen)
