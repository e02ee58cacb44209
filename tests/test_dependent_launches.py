"""Kernels that may start while the one before them on the stream still runs read global memory by ordinary (coherent) loads: the
read-only path (__ldg, ld.global.nc, const __restrict__ pointers) is specified for memory that nobody writes during the
kernel's life, and such a kernel's life begins before its wait.  A wrong load gives no wrong result that a run would
show every time, so the sources are read (CPU only)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "zeroth_order_transformer_b200", "csrc")


def _code(path):
    src = open(path).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", src, flags=re.S)


def test_dependent_kernels_do_not_read_through_the_read_only_path():
    shared = _code(os.path.join(CSRC, "dust_device.cuh"))
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        code = _code(path)
        if "dependent_launch(" not in code:
            continue
        found.append(os.path.basename(path))
        for text in (code, shared):
            bad = re.findall(r"[^\n]*(?:__ldg\b|__restrict__|ld\.global(?:\.\w+)*\.nc)[^\n]*", text)
            assert not bad, (os.path.basename(path), bad)
    assert {"dust_embed.cu", "dust_linear.cu"} <= set(found)
