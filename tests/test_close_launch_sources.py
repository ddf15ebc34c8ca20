"""All sources of the kernels that are launched close to the previous one, the headers with their bodies among them: such a
grid may be resident while the stream's previous kernel still writes, so that nothing of it is read-only memory
(CPU only)."""
import glob
import os
import re

import pytest

from speculative_decoding_verify_sv_gb300 import build as svbuild

LOADS = r"__ldg|__ldcs|__ldca|__ldlu|ld\.global\.nc"
# where the bodies of the kernels are that wait for the previous one
BODIES = {"tables.cu", "qk_norm_rope.cu", "window_attention.cu", "window_attention_f32.cu", "stacked_attention.cu", "pages.cu",
          "page_scores_tc.cu", "unit_attention.cuh", "warp_units.cuh", "stacked_keys.cuh", "sv_common.cuh", "cluster.cuh"}


def sources():
    out = {}
    for path in glob.glob(os.path.join(svbuild.CSRC, "*")):
        with open(path) as f:
            out[os.path.basename(path)] = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    return out


def reached(code, name):
    """The file and all that it includes."""
    seen, todo = set(), [name]
    while todo:
        n = todo.pop()
        if n in code and n not in seen:
            seen.add(n)
            todo += re.findall(r'#include\s+"([^"]+)"', code[n])
    return seen


def close_sources(code):
    """The .cu files with kernels that wait for the previous one, by themselves or in a header, with their headers."""
    out = set()
    for name in code:
        files = reached(code, name) if name.endswith(".cu") else set()
        if any(re.search(r"wait_previous\(\);", code[n]) for n in files):
            out |= files
    return out


def offending(code):
    return sorted(n for n in close_sources(code) if re.search(LOADS, code[n]))


def test_no_non_coherent_loads_in_any_of_them():
    code = sources()
    scanned = close_sources(code)
    assert BODIES <= scanned, BODIES - scanned
    assert {"joined_units.cu", "own_units.cu", "listed_units.cu", "warp_units.cu", "own_warps.cu"} <= scanned
    assert offending(code) == []


@pytest.mark.parametrize("name", sorted(BODIES))
def test_a_load_in_any_of_them_is_found(name):
    code = sources()
    code[name] += "\n__device__ int planted(const int *p) { return __ldg(p); }\n"
    assert name in offending(code)
