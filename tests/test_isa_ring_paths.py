"""Static checks of the ragged, weight-gradient and 4-bit rings' AMD assembly (CPU only) that need the
paths a wave can take, not the listing's order.

Copies.  The hand-counted waits hold only if the copy atoms are the only vector-memory instructions in
flight from a kernel's first copy to its drain.  The drain is the barrier that waits for vmcnt(0) and
behind which no path leads to another copy (two-stage rings wait for 0 at every barrier of their loop,
so the count alone does not tell it).  The kernel that walks several tiles stores one while the next
one's copies are in flight and is left to tests/test_isa_grouped.py.

Products.  A matrix product may read a vector register two wait states after a vector instruction
wrote it, not before.  The compiler sees to that for its builtins and cannot for products written as
assembly, so here every product is checked: no vector instruction on any path within two wait
states (each instruction counts 1, s_nop N counts N + 1) before it may write one of its registers."""
import concurrent.futures
import os
import re
import subprocess

import pytest

from tests.test_isa_grouped import KERNEL, SOURCES, _is_copy
from tests.test_isa_hazards import CSRC, INCLUDE, _blocks, _hipcc, _vmcnt

WAIT_STATES = 2


def successors(bl):
    """Blocks that may follow each block."""
    at = {b[0]: i for i, b in enumerate(bl) if b[0]}
    out = []
    for i, (_, ins) in enumerate(bl):
        last, nxt = ins[-1] if ins else "", []
        m = re.match(r"s_(c?)branch\w* (\.LBB\d+_\d+)", last)
        if m:
            nxt.append(at[m.group(2)])
        if not last.startswith("s_endpgm") and (not m or m.group(1)) and i + 1 < len(bl):
            nxt.append(i + 1)
        out.append(nxt)
    return out


def stray_vmem(lines):
    """Vector-memory instructions other than copies on a path from the first copy to a drain, and the
    number of drains."""
    bl = _blocks(lines)
    succ = successors(bl)
    copies = [any(map(_is_copy, ins)) for _, ins in bl]
    reach = list(copies)  # a copy in the block or after it
    for _ in bl:
        new = [c or any(reach[n] for n in s) for c, s in zip(copies, succ)]
        if new == reach:
            break
        reach = new
    first = next(i for i, c in enumerate(copies) if c)
    start = next(j for j, t in enumerate(bl[first][1]) if _is_copy(t))
    stray, drains, seen, todo = [], set(), set(), [(first, start, None)]
    while todo:
        i, j0, wait = todo.pop()
        if (i, j0, wait) in seen:
            continue
        seen.add((i, j0, wait))
        ins, done = bl[i][1], False
        for j in range(j0, len(ins)):
            t = ins[j]
            if _vmcnt(t) is not None:
                wait = _vmcnt(t) if wait is None else min(wait, _vmcnt(t))
            elif t == "s_barrier":
                if wait == 0 and not any(map(_is_copy, ins[j:])) and not any(reach[n] for n in succ[i]):
                    drains.add((i, j))
                    done = True
                    break
                wait = None
            elif re.match(r"(buffer|global|flat|scratch)_", t) and not _is_copy(t):
                stray.append(t)
        if not done:
            todo += [(n, 0, wait) for n in succ[i]]
    return stray, len(drains)


def _vregs(tok):
    """Vector registers a operand names: v5, a7, v[0:3]."""
    m = re.match(r"([va])(?:(\d+)|\[(\d+):(\d+)\])$", tok.strip())
    if not m:
        return set()
    lo, hi = (m.group(2), m.group(2)) if m.group(2) else (m.group(3), m.group(4))
    return {f"{m.group(1)}{r}" for r in range(int(lo), int(hi) + 1)}


def _operands(t):
    rest = re.sub(r"\s(op_sel|op_sel_hi|cbsz|blgp|abid|neg_lo|neg_hi|quad_perm|row_\w+|row_mask|bank_mask|bound_ctrl)\b.*$", "",
                  t.partition(" ")[2])
    return [o for o in re.split(r",\s*(?![^\[]*\])", rest)]


def _writes(t):
    """Vector registers a vector instruction other than a product writes."""
    if not t.startswith("v_") or t.startswith(("v_mfma", "v_cmp", "v_readfirstlane", "v_readlane", "v_nop")):
        return set()
    ops = _operands(t)
    two = t.startswith(("v_swap", "v_permlane16_swap", "v_permlane32_swap"))
    return _vregs(ops[0]) | (_vregs(ops[1]) if two else set())


def early_reads(lines):
    """(product, vector instruction that wrote one of its registers, wait states between), closer than
    WAIT_STATES on some path; and the number of products."""
    bl = _blocks(lines)
    pred = [[] for _ in bl]
    for i, nxt in enumerate(successors(bl)):
        for n in nxt:
            pred[n].append(i)
    found, products = [], 0

    def back(i, j, need, states, t, seen):
        while j > 0 and states < WAIT_STATES:
            j -= 1
            p = bl[i][1][j]
            if _writes(p) & need:
                found.append((t, p, states))
                return
            m = re.match(r"s_nop (\d+)", p)
            states += int(m.group(1)) + 1 if m else 1
        if states < WAIT_STATES:
            for q in pred[i]:
                if (q, states) not in seen:
                    seen.add((q, states))
                    back(q, len(bl[q][1]), need, states, t, seen)

    for i, (_, ins) in enumerate(bl):
        for j, t in enumerate(ins):
            if t.startswith("v_mfma"):
                products += 1
                back(i, j, set().union(*map(_vregs, _operands(t)[1:])), 0, t, set())
    return found, products


COPY = "buffer_load_dwordx4 v1, s[8:11], 0 offen lds"


def test_stray_vmem_on_small_listings():
    """A two-stage ring whose every barrier waits for 0: the loop's loads and stores are reported, the
    epilogue's are not, also where it is laid out ahead of the remainder that ends in the drain."""
    load, store = "global_load_dword v9, v[2:3], off", "global_store_dwordx4 v[2:3], v[4:7], off nt"
    wait = ["s_waitcnt vmcnt(0) lgkmcnt(0)", "s_barrier"]
    head = [load, "s_waitcnt vmcnt(0)", COPY, COPY, "s_waitcnt vmcnt(4)", "s_barrier"]
    loop = [".LBB0_1:", "ds_read_b128 v[4:7], v8", *wait, COPY, "s_cbranch_scc1 .LBB0_1"]
    end = [*wait, store, "s_endpgm"]
    assert stray_vmem(head + loop + end) == ([], 1)
    for bad in (load, store, "scratch_store_dword off, v5, s0 offset:16", "buffer_load_dword v1, off, s[0:3], 0"):
        assert stray_vmem(head + loop[:4] + [bad] + loop[4:] + end)[0] == [bad]
        assert stray_vmem(head + loop[:2] + [bad] + loop[2:] + end)[0] == [bad]
    assert stray_vmem(head + loop + [store] + end)[0] == [store]
    laid_out = head + loop + ["s_branch .LBB0_3", ".LBB0_2:", store, load, "s_endpgm", ".LBB0_3:", COPY, *wait,
                              "s_branch .LBB0_2"]
    assert stray_vmem(laid_out) == ([], 1)
    assert stray_vmem([t if t != "s_branch .LBB0_3" else "s_cbranch_scc0 .LBB0_3" for t in laid_out])[0] == [store, load]
    assert stray_vmem(head + loop + [store, "s_endpgm"]) == ([store], 0)


def test_early_reads_on_small_listings():
    product = "v_mfma_scale_f32_16x16x128_f8f6f4 a[0:3], v[4:7], v[8:11], a[0:3], v12, v13 op_sel_hi:[0,0,0] cbsz:4 blgp:4"
    assert early_reads(["v_and_b32_e32 v12, v1, v2", product])[0] == [(product, "v_and_b32_e32 v12, v1, v2", 0)]
    assert early_reads(["v_and_b32_e32 v13, v1, v2", "s_nop 0", product])[0][0][2] == 1
    assert early_reads(["v_mov_b64_e32 v[6:7], v[2:3]", "s_mov_b32 s1, s2", product])[0][0][2] == 1
    assert early_reads(["v_accvgpr_write_b32 a2, 0", product])[0][0][2] == 0
    assert early_reads(["v_swap_b32 v1, v12", product])[0][0][2] == 0
    for far in (["v_and_b32_e32 v12, v1, v2", "s_nop 1"], ["v_and_b32_e32 v12, v1, v2", "s_nop 0", "s_mov_b32 s1, s2"],
                ["v_and_b32_e32 v14, v12, v13"], ["v_cmp_lt_i32_e32 vcc, v12, v13"], ["v_readfirstlane_b32 s12, v12"]):
        assert early_reads(far + [product]) == ([], 1)
    looped = [".LBB0_1:", product, "v_add_u32_e32 v9, 1, v9", "s_cbranch_scc1 .LBB0_1", "s_endpgm"]
    assert early_reads(looped)[0] == [(product, "v_add_u32_e32 v9, 1, v9", 1)]


def _listing(src, tmp):
    out = os.path.join(tmp, src + ".s")
    r = subprocess.run([_hipcc(), "--offload-arch=gfx950", "-O3", "-std=c++17", "-Wno-unused-command-line-argument",
                        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", INCLUDE, "-I", CSRC,
                        "--cuda-device-only", "-S", os.path.join(CSRC, src + ".hip"), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = open(out).read()
    kernels, heads = [], list(KERNEL.finditer(text))
    for i, h in enumerate(heads):
        body = text[h.end():heads[i + 1].start() if i + 1 < len(heads) else len(text)]
        kernels.append((h.group(1), body[:body.find(".Lfunc_end")].splitlines()))
    return kernels


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if _hipcc() is None:
        pytest.skip("hipcc not found")
    tmp = str(tmp_path_factory.mktemp("isa"))
    with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as ex:
        found = [k for ks in ex.map(lambda s: _listing(s, tmp), SOURCES) for k in ks]
    assert len(found) == 96
    return found


def test_only_copies_are_in_flight_up_to_the_drain(kernels):
    problems = []
    for name, lines in kernels:
        if "walk" not in name:
            stray, drains = stray_vmem(lines)
            if stray or not drains:
                problems.append(f"{name}: {stray[:3]} among the copies, {drains} drains")
    assert not problems, "\n".join(problems[:20])


def test_no_product_reads_a_register_that_was_just_written(kernels):
    problems = []
    for name, lines in kernels:
        found, products = early_reads(lines)
        assert products, name
        problems += [f"{name}: {t!r} {n} wait states after {p!r}" for t, p, n in found[:2]]
    assert not problems, "\n".join(problems[:20])
