"""Static check of the ragged, weight-gradient and 4-bit rings' AMD assembly (CPU only), as
tests/test_isa_hazards.py makes it for the dense rings: the hand-counted waits hold only if the copy
atoms are the only vector-memory instructions in flight between a kernel's first copy and its drain
(the loads of the group offsets complete before), and every barrier there must wait for one of the
intended counts: 0, the atoms of S-2 tiles or those of S-1.  The kernel that walks several tiles stores
one while the next one's copies are in flight: there only the barriers are checked, and that it
spills nothing to memory."""
import concurrent.futures
import os
import re
import subprocess
import tempfile

import pytest

from tests.test_isa_hazards import CSRC, INCLUDE, _blocks, _hipcc, _vmcnt

KERNEL = re.compile(r"^(_ZN3tbg(?:19gemm_grouped_kernel|17gemm_wgrad_kernel|15gemm_mx4_kernel|20gemm_mx4_walk_kernel)"
                    r"I((?:Li\d+E)+)\S*):", re.M)
SOURCES = ("gemm_grouped_64", "gemm_grouped_128", "gemm_grouped_256", "gemm_mx4")


def _is_copy(t):
    return t.startswith("buffer_load_dwordx4") and t.endswith(" lds")


def walk(lines):
    """From the first copy atom on, over every path up to the drain (a vmcnt(0) wait that a barrier
    follows): the other vector-memory instructions met, and the vmcnt each barrier waits for (None
    when no vmcnt wait precedes it since the last barrier on that path)."""
    bl = _blocks(lines)
    at = {b[0]: i for i, b in enumerate(bl) if b[0]}
    start = next((i, j) for i, b in enumerate(bl) for j, t in enumerate(b[1]) if _is_copy(t))
    stray, waits = [], set()
    seen, todo = set(), [(start[0], start[1], None, False)]
    while todo:
        i, j0, wait, only = todo.pop()
        if (i, j0, wait) in seen:
            continue
        seen.add((i, j0, wait))
        ins, done = bl[i][1], False
        for t in ins[j0:]:
            if _vmcnt(t) is not None:
                wait = _vmcnt(t) if wait is None else min(wait, _vmcnt(t))
            elif t == "s_barrier":
                waits.add(wait)
                wait = None
            elif re.match(r"(buffer|global|flat|scratch)_", t) and not _is_copy(t):
                # stores of the epilogue follow the drain's barrier, the last one a path meets
                if t.startswith(("global_store", "global_load")) and 0 in waits:
                    done = True
                    break
                stray.append(t)
        last = ins[-1] if ins else ""
        if done or last.startswith("s_endpgm"):
            continue
        m = re.match(r"s_(c?)branch\w* (\.LBB\d+_\d+)", last)
        if m:
            todo.append((at[m.group(2)], 0, wait, only))
        if not m or m.group(1):
            if i + 1 < len(bl):
                todo.append((i + 1, 0, wait, only))
    return stray, waits


def test_walk_on_small_listings():
    copy = "buffer_load_dwordx4 v1, s[8:11], 0 offen lds"
    head = ["global_load_dword v1, v[2:3], off", "s_waitcnt vmcnt(0)", copy, copy]
    loop = [".LBB0_1:", copy, "s_waitcnt vmcnt(8) lgkmcnt(0)", "v_add_u32 v1, v1, v2", "s_barrier", "s_cbranch_scc1 .LBB0_1"]
    end = ["s_waitcnt vmcnt(0) lgkmcnt(0)", "s_barrier", "global_store_dwordx4 v[2:3], v[4:7], off nt", "s_endpgm"]
    assert walk(head + loop + end) == ([], {8, 0})
    spill = head + loop[:2] + ["scratch_store_dword off, v5, s0 offset:16"] + loop[2:] + end
    assert walk(spill)[0] == ["scratch_store_dword off, v5, s0 offset:16"]
    none = head + [x for x in loop if "waitcnt" not in x] + end
    assert None in walk(none)[1]


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
        args, walks = [int(a) for a in re.findall(r"Li(\d+)E", h.group(2))], "walk" in h.group(1)
        bm, bn, s = (args[0], args[0], args[1]) if walks else args[:3]
        atoms = bm // 32 + bn // 32
        body = text[h.end():heads[i + 1].start() if i + 1 < len(heads) else len(text)]
        if walks and "scratch_" in body[:body.find(".Lfunc_end")]:
            problems.append(f"{h.group(1)}: spills")
        stray, waits = walk(body[:body.find(".Lfunc_end")].splitlines())
        if stray and not walks:
            problems.append(f"{h.group(1)}: {stray[:3]} among the copies")
        if not waits <= {0, atoms * (s - 2), atoms * (s - 1)} or atoms * (s - 1) not in waits:
            problems.append(f"{h.group(1)}: barriers wait for {waits}")
    return len(heads), problems


@pytest.mark.skipif(_hipcc() is None, reason="hipcc not found")
def test_only_copies_are_in_flight_and_barriers_wait_for_the_intended_counts():
    with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as ex:
        results = list(ex.map(_problems, SOURCES))
    assert [n for n, _ in results] == [24, 24, 24, 24]
    problems = [p for _, ps in results for p in ps]
    assert not problems, "\n".join(problems[:20])
