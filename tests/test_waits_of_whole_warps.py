"""Sources of the kernels with waits that can give up: what a wait says is decided by the warp before it parts, since
behind it are operations (tcgen05.ld, votes, __syncwarp) that wait for all of its lanes without a limit (CPU only)."""
import os
import re

import pytest

from speculative_decoding_verify_sv_gb300 import build as svbuild

# file -> the name of its wait
SOURCES = {"stacked_attention.cu": "stack_wait", "unit_attention.cuh": "limited_wait", "warp_units.cuh": "limited_wait"}


def statements(name):
    with open(os.path.join(svbuild.CSRC, name)) as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    return re.split(r"[;{}]", code)


def parting(source, wait):
    """The statements that call `wait` in several lanes without a vote."""
    bad = []
    for s in source:
        s = " ".join(s.split())
        if not re.search(rf"\b{wait}\(", s) or re.search(rf"\bbool {wait}\(", s):
            continue
        voted = len(re.findall(rf"__all_sync\(0xFFFFFFFFu, {wait}\(", s)) == len(re.findall(rf"\b{wait}\(", s))
        one_lane = re.search(r"\blane == 0\b|\belect_one\(\)", s)
        if not voted and not one_lane:
            bad.append(s)
    return bad


@pytest.mark.parametrize("name", SOURCES)
def test_a_warp_decides_as_a_whole(name):
    code = statements(name)
    assert any(SOURCES[name] + "(" in s for s in code)
    assert not parting(code, SOURCES[name])


def test_a_wait_of_each_lane_is_found():
    assert parting(["if (!stack_wait(&full[sv], 0, abort_flag, limit)) ", "ok = ok && stack_wait(bar, 0, a, l)"], "stack_wait") != []
    assert parting(["if (copied >= ST && lane == 0) ok = stack_wait(&empty[st], 0, a, l)",
                    "return __all_sync(0xFFFFFFFFu, stack_wait(bar, 0, a, l))"], "stack_wait") == []


def part(name, begin, end=None):
    """The code of a file from one text to another."""
    with open(os.path.join(svbuild.CSRC, name)) as f:
        text = f.read()
    assert text.count(begin) == 1, begin
    text = text[text.index(begin):]
    text = text[:text.index(end)] if end else text
    return re.split(r"[;{}]", re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S))


def test_the_lm_heads_epilogue_decides_as_a_whole():
    code = part("lm_head.cu", "---- epilogue")
    assert any("mbar_wait_warp(" in s for s in code)
    assert not parting(code, "mbar_wait")
