"""The tcgen05 attention kernel's warps are whole where an instruction is the whole warp's (``.sync.aligned``: loads, stores and waits of
tensor memory, its allocation, register splits, named barriers).

A statement that only some lanes of a warp run may leave the others in front of such an instruction.  So each of them has the
warp's meeting as the next statement of its own block - a lambda or a helper must not leave that to whoever calls it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lossless_bf16_weight_exponent_gb300", "csrc")
SOME_LANES = re.compile(r"\bif \((?P<c>(?:[^()]|\((?:[^()]|\([^()]*\))*\))*)\)")
OF_A_LANE = re.compile(r"\blane == 0\b|\bleader\b|\brow == 0\b|\bin\b|\bthreadIdx\.x == 0\b")
MEETING = re.compile(r"__sync(warp|threads)\(\);")


def code(text):
    return re.sub(r"//[^\n]*", "", text)


def statement_end(text, at):
    """Behind the statement that begins at `at`: a block, or up to its semicolon."""
    while text[at].isspace():
        at += 1
    if text[at] == "{":
        depth = 0
        for i in range(at, len(text)):
            depth += (text[i] == "{") - (text[i] == "}")
            if depth == 0:
                return i + 1
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] in "({[") - (text[i] in ")}]")
        if text[i] == ";" and depth == 0:
            return i + 1
    raise AssertionError("no end")


def without_meeting(text):
    text = code(text)
    bad, found = [], 0
    for m in SOME_LANES.finditer(text):
        if not OF_A_LANE.search(m["c"]):
            continue
        found += 1
        end = statement_end(text, m.end())
        if not MEETING.match(text[end:].lstrip()):
            bad.append(text[m.start():end].strip())
    return bad, found


def test_the_check_itself():
    assert without_meeting("auto f = [&] { __syncwarp(); if (lane == 0) go(b); };")[0] == ["if (lane == 0) go(b);"]
    assert without_meeting("if (lane == 0) go(b);\n // as above\n __syncwarp();")[0] == []
    assert without_meeting("if (in) { x(); y(); } load();")[0] == ["if (in) { x(); y(); }"]
    assert without_meeting("if (!wait(&d[0], 0) && lane == 0) put(a, 1); free();") == (["if (!wait(&d[0], 0) && lane == 0) put(a, 1);"], 1)
    assert without_meeting("if (ok) go(); load();") == ([], 0)


def test_every_branch_of_some_lanes_meets():
    text = open(os.path.join(CSRC, "k_attend_tc.cu")).read()
    bad, found = without_meeting(text[text.index("attend_tc_kernel"):])
    assert found > 10
    assert not bad, "\n".join(bad)


def test_named_barriers_meet_first():
    text = code(open(os.path.join(CSRC, "k_attend_tc.cu")).read())
    body = re.search(r"void tile_sync\(int t\)\s*\{(.*?)\n\}", text, re.S) or re.search(r"void tile_sync\(int t\) \{(.*)\}", text)
    assert MEETING.match(body[1].strip())


@pytest.mark.parametrize("what", ["tcgen05.dealloc.cta_group::1.sync.aligned"])
def test_tensor_memory_is_freed_by_a_whole_warp(what):
    text = code(open(os.path.join(CSRC, "k_attend_tc.cu")).read())
    at = text.index(what)
    assert "__syncwarp();" in text[text.rindex("__syncthreads();", 0, at):at]


WHOLE = re.compile(r"\btmem_(?:ld|st)\d+\((?!uint32_t)|tcgen05\.(?:ld|dealloc)\.|\bbar\.sync|\bcolumns\((?!uint32_t)")


@pytest.mark.parametrize("name", ["k_group_tc.cu", "k_tc4.cu", "k_tc.cu"])
def test_whole_warps_in_the_other_tensor_memory_kernels(name):
    """Their waits and rows left out let lanes go one by one: a meeting stands in the lines in front of each instruction of a warp."""
    lines = code(open(os.path.join(CSRC, name)).read()).split("\n")
    text = "\n".join(lines)
    sites = [text[:m.start()].count("\n") for m in WHOLE.finditer(text)]
    sites = [i for i in sites if "[=]" not in lines[i] and "[&](uint32_t" not in lines[i]]
    assert len(sites) >= 4
    for i in sites:
        if "columns(run" in lines[i] or "tmem_st16(run" in lines[i] or "tmem_ld16(acc, u)" in lines[i]:
            continue  # behind the loads or the output of the same columns, which the whole warp has just done
        assert any("__syncwarp();" in lines[j] for j in range(max(0, i - 6), i)), (i, lines[i])
