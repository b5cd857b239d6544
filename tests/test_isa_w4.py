"""Static check of the assembly of the products with 4-bit weights (CPU only).  Their loops hold the codes that are on
the way from memory, the sums of a group and the totals in registers: a kernel that spills one of them to memory is
several times slower, so none may; and the loop over K (the one with the most products; the others finish what is left
of K) may not drain its loads, which would wait for the ones that were asked for ahead."""
import concurrent.futures
import os
import re
import subprocess
import tempfile

import pytest

from tests.test_isa_hazards import CSRC, INCLUDE, _blocks, _hipcc, _vmcnt

SOURCES = ("gemm_w4_bf16", "gemm_w4_bf16_zeros", "gemm_w4_f16", "gemm_w4_f16_zeros")
KERNEL = re.compile(r"^(_ZN3tbg\d+gemm_w4_(?:panel_)?kernel\S*):", re.M)


def inner_loops(lines):
    """The instructions of the loops that hold no other loop, by their backward branches."""
    bl = _blocks(lines)
    at = {b[0]: i for i, b in enumerate(bl) if b[0]}
    spans = set()
    for i, (_, ins) in enumerate(bl):
        for t in ins:
            m = re.match(r"s_c?branch\w* (\.LBB\d+_\d+)", t)
            if m and at[m.group(1)] <= i:
                spans.add((at[m.group(1)], i))
    inner = [s for s in spans if not any(o != s and s[0] <= o[0] and o[1] <= s[1] for o in spans)]
    return [[t for b in bl[a:z + 1] for t in b[1]] for a, z in inner]


def test_inner_loops_on_small_listings():
    body = ["v_mov_b32 v1, v2", ".LBB0_1:", "s_nop 0", ".LBB0_2:", "v_mfma_f32 a", "s_waitcnt vmcnt(0)",
            "s_cbranch_scc1 .LBB0_2", "s_cbranch_scc1 .LBB0_1", "s_endpgm"]
    (loop,) = inner_loops(body)
    assert loop[:2] == ["v_mfma_f32 a", "s_waitcnt vmcnt(0)"]


def _products(instructions):
    return sum(t.startswith("v_mfma") for t in instructions)


def _problems(src):
    out = tempfile.NamedTemporaryFile(suffix=".s", delete=False).name
    try:
        r = subprocess.run([_hipcc(), "--offload-arch=gfx950", "-O3", "-std=c++17", "-Wno-unused-command-line-argument",
                            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", INCLUDE, "-I", CSRC,
                            "--cuda-device-only", "-S", os.path.join(CSRC, src + ".hip"), "-o", out],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        text = open(out).read()
    finally:
        os.unlink(out)
    problems, heads = [], list(KERNEL.finditer(text))
    for i, h in enumerate(heads):
        body = text[h.end():heads[i + 1].start() if i + 1 < len(heads) else len(text)]
        body = body[:body.find(".Lfunc_end")]
        if "scratch_" in body:
            problems.append(f"{h.group(1)}: spills")
        main = max(inner_loops(body.splitlines()), key=_products)
        if _products(main) < 8:
            problems.append(f"{h.group(1)}: no loop over K found")
        if any(_vmcnt(t) == 0 for t in main):
            problems.append(f"{h.group(1)}: the loop over K drains its loads")
    return len(heads), problems


@pytest.mark.skipif(_hipcc() is None, reason="hipcc not found")
def test_products_neither_spill_nor_drain_their_loads():
    with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as ex:
        results = list(ex.map(_problems, SOURCES))
    assert [n for n, _ in results] == [18, 18, 18, 18]
    assert not [p for _, ps in results for p in ps]
