"""Sources of the kernels that are launched close to the previous one: a grid that may be resident while
the stream's previous kernel still writes has no read-only memory (CPU only)."""
import glob
import os
import re

from speculative_decoding_verify_sv_gb300 import build as svbuild


def _code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_no_non_coherent_loads_behind_the_wait():
    sources = {p: _code(p) for p in glob.glob(os.path.join(svbuild.CSRC, "*.cu*"))}
    close = [p for p, s in sources.items() if p.endswith(".cu") and "wait_previous()" in s]
    names = {os.path.basename(p) for p in close}
    assert {"tables.cu", "qk_norm_rope.cu", "window_attention.cu", "window_attention_f32.cu"} <= names
    # (the helpers that they share, too: a tree's parents may come from the previous kernel)
    for p in close + [os.path.join(svbuild.CSRC, n) for n in ("sv_common.cuh", "cluster.cuh")]:
        found = re.findall(r"__ldg|__ldcs|__ldca|__ldlu|ld\.global\.nc", sources[p])
        assert not found, (os.path.basename(p), found)
