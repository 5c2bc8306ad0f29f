"""Wait states around the matrix instructions that csrc/gemm.h writes as inline
assembly. The compiler puts none around those by itself (it does around its own),
so copies that it places next to them could read or overwrite a register too
early. The sources that use them are compiled to assembly here, and every path of
up to 18 wait states before each instruction is looked over:
  * a vector register written by a VALU instruction is not read by such an MFMA
    within 2 wait states;
  * its result is not read or overwritten by anything but an MFMA within 18 (a
    16x16x32 MFMA itself takes 4 of them).
"""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from convolution_conv2d_nhwc_amd import build

VALU_TO_MFMA, MFMA_TO_OTHER, MFMA_ISSUE = 2, 18, 4
SOURCES = ["head_loss.hip", "ortho.hip"]
INLINE = "inline "  # before the name of an MFMA between the compiler's marks of inline assembly


def regs(token):
    m = re.match(r"^([va])\[(\d+):(\d+)\]$", token) or re.match(r"^([va])(\d+)$", token)
    return {(m.group(1), i) for i in range(int(m.group(2)), int(m.groups()[-1]) + 1)} if m else set()


def functions(text):
    """(name, [(opcode, operands)], {index: its predecessors}) of a listing's functions."""
    name, ins, labels, inline = None, [], {}, False
    for line in text.split("\n") + ["_Z:"]:
        m = re.match(r"^(_Z\w*):", line)
        if m:
            if name and ins:
                at, jumps = {}, {}
                for i, (op, args) in enumerate(ins):
                    if op.startswith(("s_branch", "s_cbranch")):
                        jumps.setdefault(args[0], []).append(i)
                for label, i in labels.items():
                    at.setdefault(i, []).extend(jumps.get(label, []))
                pred = {i: at.get(i, []) + ([i - 1] if i and ins[i - 1][0] not in ("s_branch", "s_endpgm") else [])
                        for i in range(len(ins))}
                yield name, ins, pred
            name, ins, labels = m.group(1), [], {}
            continue
        m = re.match(r"^(\.LBB\w+):", line)
        if m:
            labels[m.group(1)] = len(ins)
            continue
        if "#ASMSTART" in line or "#ASMEND" in line:
            inline = "#ASMSTART" in line
        m = re.match(r"^\t(\w+)[ \t]*([^;]*)", line)
        if m and name:
            mark = INLINE if inline and m.group(1).startswith("v_mfma") else ""
            ins.append((mark + m.group(1), [a.strip() for a in m.group(2).split(",")] if m.group(2).strip() else []))


def found_before(ins, pred, i, states, mfma_states, hit):
    """An instruction that hit() takes fewer than `states` wait states before i."""
    todo, seen = [(i, states)], {}
    while todo:
        at, left = todo.pop()
        if left <= 0 or seen.get(at, 0) >= left:
            continue
        seen[at] = left
        for p in pred[at]:
            op, args = ins[p]
            if hit(op, args):
                return ins[p]
            cost = int(args[0], 0) + 1 if op == "s_nop" else mfma_states if "v_mfma" in op else 1
            todo.append((p, left - cost))
    return None


def problems(text):
    """(number of inline MFMAs, what is wrong)."""
    count, bad = 0, []
    for name, ins, pred in functions(text):
        for i, (op, args) in enumerate(ins):
            if op.startswith(INLINE):
                count += 1
                reads = regs(args[1]) | regs(args[2]) | regs(args[3])
                by = found_before(ins, pred, i, VALU_TO_MFMA, 1, lambda o, a: o.startswith("v_") and a and
                                  not o.startswith(("v_cmp", "v_readfirstlane", "v_readlane")) and regs(a[0]) & reads)
            elif "v_mfma" not in op and op.startswith(("v_", "ds_", "global_", "buffer_", "flat_", "scratch_")):
                uses = set().union(*(regs(a) for a in args)) if args else set()
                by = uses and found_before(ins, pred, i, MFMA_TO_OTHER, MFMA_ISSUE,
                                           lambda o, a: o.startswith(INLINE) and regs(a[0]) & uses)
            else:
                continue
            if by:
                bad.append((name, i, op, args, "too soon after", by))
    return count, bad


PLAIN = "\tv_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]\n"
MFMA = "\t;;#ASMSTART\n" + PLAIN + "\t;;#ASMEND\n"


@pytest.mark.parametrize("body,ok", [
    ("\tv_mov_b32_e32 v5, v9\n" + MFMA, False),
    ("\tv_mov_b32_e32 v5, v9\n\ts_nop 0\n" + MFMA, False),
    ("\tv_mov_b32_e32 v5, v9\n\ts_nop 1\n" + MFMA, True),
    ("\tv_mov_b32_e32 v8, v9\n" + MFMA, True),
    ("\tv_accvgpr_write_b32 a2, v9\n" + MFMA, False),
    ("\tv_mov_b32_e32 v5, v9\n\ts_cbranch_scc1 .LBB0_1\n\ts_nop 4\n.LBB0_1:\n" + MFMA, False),
    (MFMA + "\tv_accvgpr_read_b32 v9, a1\n", False),
    (MFMA + "\ts_nop 12\n\tv_accvgpr_read_b32 v9, a1\n", False),
    (MFMA + "\ts_nop 15\n\ts_nop 3\n\tv_accvgpr_read_b32 v9, a1\n", True),
    (MFMA + "\tglobal_store_dwordx4 v[10:11], a[0:3], off\n", False),
    (MFMA + MFMA.replace("a[0:3]", "a[4:7]") * 5 + "\tv_accvgpr_read_b32 v9, a1\n", True),
    (MFMA + MFMA, True),
    (PLAIN + "\tv_accvgpr_read_b32 v9, a1\n", True),  # the compiler's own: its to see to
])
def test_planted_hazards_are_found(body, ok):
    count, bad = problems("_Zf:\n" + body + "\ts_endpgm\n")
    assert count == body.count("#ASMEND") and (not bad) == ok, bad


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")
def test_no_mfma_reads_or_is_read_too_soon(tmp_path):
    def listing(name):
        out = str(tmp_path / (name + ".s"))
        cmd = [build.HIPCC] + build.CFLAGS + ["--cuda-device-only", "-S", os.path.join(build.CSRC, name), "-o", out]
        subprocess.run(cmd, check=True, stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
        return open(out).read()
    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        for name, text in zip(SOURCES, ex.map(listing, SOURCES)):
            count, bad = problems(text)
            assert count > 100, name  # the listing was understood
            assert not bad, (name, len(bad), bad[:3])
