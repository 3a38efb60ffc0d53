"""The counted waits of the 4-bit product's kernels that load rows straight into LDS, checked on
the CPU in the device assembly the build keeps (`_build/fp4_gemm-gfx950.s`).

Such a kernel waits for `vmcnt(2 WT)` before each barrier: of the wave's vector-memory operations,
which retire in order, all but the 2 WT newest are done.  What has to be done is every load into
LDS of the slab to be read, and what may still be under way are that slab's weights, WT loads of
codes and WT of scales, issued behind them.  So on every way through the code that leads to such a
wait the 2 WT newest operations are loads into registers, and the TT before them (a wave's share
of 16 TT rows, four rows a load) are those into LDS."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ASM = os.path.join(ROOT, "_build", "fp4_gemm-gfx950.s")

NAME = re.compile(r"^(_ZN\S*k_fp4_tiledILi(\d+)ELi(\d+)ELi(\d+)ELb[01]ELb([01])E\S*):")
VMEM = re.compile(r"(buffer|global|flat|scratch)_(load|store|atomic)")
WAIT = re.compile(r"s_waitcnt vmcnt\((\d+)\) lgkmcnt\(0\)$")


class Violation(AssertionError):
    pass


def functions(text):
    """(name, WT, TT, KS, DMA, code lines) of the tiled kernels."""
    name, lines = None, []
    for line in text.splitlines():
        m = NAME.match(line)
        if m:
            name, lines = m.groups(), []
        elif name and line.startswith(".Lfunc_end"):
            yield name[0], *(int(v) for v in name[1:]), lines
            name = None
        elif name:
            code = line.split(";")[0].strip()
            if code:
                lines.append(code)


def before(lines):
    """For each line, the lines that can come right before it."""
    at = {l[:-1]: i for i, l in enumerate(lines) if l.endswith(":")}
    prev = [[] for _ in lines]
    for i, l in enumerate(lines):
        op = l.split()[0]
        if op.startswith(("s_branch", "s_cbranch")):
            prev[at[l.split()[1]]].append(i)
        if i + 1 < len(lines) and op not in ("s_branch", "s_endpgm"):
            prev[i + 1].append(i)
        assert not op.startswith(("s_setpc", "s_swappc", "s_call", "s_cbranch_i_fork"))
    return prev


def check(lines, WT, TT):
    """Number of counted waits, all of them sound."""
    prev, waits = before(lines), 0
    for i, l in enumerate(lines):
        if l != "s_barrier":
            continue
        m = WAIT.match(lines[i - 1])
        if not m or prev[i] != [i - 1]:
            raise Violation(f"a barrier without its wait: {lines[i - 1]}")
        if int(m.group(1)) != 2 * WT:
            raise Violation(f"{lines[i - 1]} for {WT} weight tiles")
        waits += 1
        todo, seen, reached = [(i - 1, 0)], set(), 0
        while todo:
            at, n = todo.pop()
            if (at, n) in seen:
                continue
            seen.add((at, n))
            if not prev[at]:
                raise Violation(f"{n} operations before a wait, {2 * WT + TT} expected")
            for p in prev[at]:
                k = n
                if VMEM.match(lines[p]):
                    lds = lines[p].endswith(" lds")
                    if "load" not in lines[p] or lds != (k >= 2 * WT):
                        raise Violation(f"operation {k} before a wait for {2 * WT}: {lines[p]}")
                    k += 1
                if k == 2 * WT + TT:
                    reached += 1
                else:
                    todo.append((p, k))
        assert reached
    return waits


@pytest.mark.skipif(not os.path.exists(ASM), reason="device assembly not built "
                    "(python lora_expert_gemm_amd/build.py)")
def test_loads_are_in_the_order_that_the_waits_count():
    seen = set()
    for name, WT, TT, KS, dma, lines in functions(open(ASM).read()):
        if not dma:
            assert not any(l.endswith(" lds") for l in lines), name
            continue
        assert KS == 1
        # both halves of the loop and the odd last step
        assert check(lines, WT, TT) == 3, name
        seen.add((WT, TT, name))
    assert {s[:2] for s in seen} == {(2, 2), (4, 4)} and len(seen) == 4, seen


# a kernel of one weight tile and one group of rows: prologue, a step of the loop, the last one
STEP = ["s_waitcnt vmcnt(2) lgkmcnt(0)", "s_barrier", "buffer_load_dwordx4 v1, s[4:7], s0 offen lds",
        "buffer_load_dwordx4 v[4:7], v2, s[8:11], s0 offen", "buffer_load_dword v8, v3, s[12:15], s0 offen",
        "v_mfma_f32_16x16x32_bf16 v[0:3], v[4:7], v[4:7], v[0:3]"]
KERNEL = STEP[2:5] + [".LBB0_1:"] + STEP + ["s_cbranch_scc1 .LBB0_1"] + STEP[:3] + ["s_endpgm"]


def test_the_check_finds_planted_mistakes():
    assert check(KERNEL, 1, 1) == 2

    def planted(at, *put, cut=0):
        lines = KERNEL[:at] + list(put) + KERNEL[at + cut:]
        with pytest.raises(Violation):
            check(lines, 1, 1)

    loop = KERNEL.index(".LBB0_1:") + 1
    planted(loop, "s_waitcnt vmcnt(3) lgkmcnt(0)", cut=1)             # one more under way than counted
    planted(loop, "s_waitcnt vmcnt(2)", cut=1)                        # LDS reads not waited for
    planted(0, cut=1)                                                 # nothing loaded for the first step
    planted(loop + 2, *STEP[3:5], STEP[2], cut=3)                     # weights first
    planted(loop + 4, cut=1)                                          # scales not loaded: rows under way
    planted(loop + 5, "scratch_load_dword v9, off, s32")              # a reload from scratch, not counted
    planted(loop + 5, "global_store_dword v[0:1], v2, off")
