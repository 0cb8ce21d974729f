"""What the compiler emits for the 8-bit product's tiles, followed along every edge of its control flow, without a GPU.

The matrix instructions stand there as assembly.  Each writes its last sums 18 wait states on (an instruction
of 16 passes), and nothing but another of them may touch those before; an instruction is one state at
least, s_nop N is N + 1.  What is still to be written at a block's beginning is the most of what is at the ends of
the blocks that lead there."""
import re

import numpy as np
import pytest

from zero_dp_sharded_amd import build

STATES = 18
SUMS = 256


def blocks_of(body):
    """[(label or None, instructions, where it goes)]: the next block is None in a list, others by label."""
    blocks, label, lines = [], None, []

    def end(goes):
        nonlocal label, lines
        blocks.append((label, lines, goes))
        label, lines = None, []

    for line in body.splitlines():
        ins = line.split(";")[0].strip()
        if not ins:
            continue
        m = re.match(r"(\.L\w+):$", ins)
        if m:
            if lines or label:
                end([None])
            label = m.group(1)
        elif not ins.startswith("."):
            lines.append(ins)
            m = re.match(r"s_(c?)branch\S*\s+(\S+)", ins)
            if m:
                end([m.group(2)] + ([None] if m.group(1) else []))
            elif ins.startswith("s_endpgm"):
                end([])
            else:
                assert not re.match(r"s_(setpc|swappc|call|subvector)", ins), ins
    if lines or label:
        end([])
    return blocks


def registers(ins):
    found = {int(x) for x in re.findall(r"\ba(\d+)\b", ins)}
    for lo, hi in re.findall(r"\ba\[(\d+):(\d+)\]", ins):
        found.update(range(int(lo), int(hi) + 1))
    return sorted(found)


def early(body):
    """Instructions that touch sums which a matrix instruction before them, on some way, has yet to write."""
    blocks = blocks_of(body)
    at = {label: k for k, (label, _, _) in enumerate(blocks) if label}
    parsed = []
    for _, lines, _ in blocks:
        steps = []
        for ins in lines:
            nop = re.match(r"s_nop (\d+)", ins)
            mfma = ins.startswith("v_mfma")
            touched = registers(ins.split(",")[0]) if mfma else registers(ins)
            steps.append((ins, mfma, touched, int(nop.group(1)) + 1 if nop else 1))
        parsed.append(steps)
    begin = [None] * len(blocks)
    begin[0] = np.zeros(SUMS, np.int16)
    todo, wrong = [0], set()
    while todo:
        k = todo.pop()
        left = begin[k].copy()
        for ins, mfma, touched, states in parsed[k]:
            if not mfma and any(left[r] > 0 for r in touched):
                wrong.add(ins)
            np.maximum(left - states, 0, out=left)
            if mfma:
                left[touched] = STATES
        for goes in blocks[k][2]:
            n = at[goes] if goes else k + 1
            if n >= len(blocks):
                continue
            if begin[n] is None:
                begin[n] = left.copy()
            elif (left > begin[n]).any():
                begin[n] = np.maximum(begin[n], left)
            else:
                continue
            todo.append(n)
    return sorted(wrong), sum(mfma for steps in parsed for _, mfma, _, _ in steps)


MFMA = "\tv_mfma_scale_f32_16x16x128_f8f6f4 a[4:7], v[0:7], v[8:15], a[4:7], v16, v17 op_sel_hi:[0,0,0]\n"
READ = "\tv_accvgpr_read_b32 v20, a5\n"
END = "\ts_endpgm\n"


@pytest.mark.parametrize("listing,is_early", [
    (MFMA + READ + END, True),
    (MFMA + "\ts_nop 15\n" + "\ts_nop 0\n" + "\tv_mov_b32_e32 v1, v2\n" + READ + END, False),           # 16 + 1 + 1 states
    (MFMA + "\ts_nop 15\n" + "\ts_nop 0\n" + READ + END, True),
    (MFMA + ".LBB0_1:\n" + READ + END, True),                                                           # falls into the next block
    (MFMA + "\ts_branch .LBB0_2\n.LBB0_1:\n" + END + ".LBB0_2:\n" + READ + END, True),                  # goes there
    ("\ts_cbranch_scc1 .LBB0_2\n" + MFMA + ".LBB0_2:\n" + READ + END, True),                            # on one of two ways
    (".LBB0_1:\n" + READ + MFMA + "\ts_cbranch_scc1 .LBB0_1\n" + END, True),                            # round a loop
    (".LBB0_1:\n" + READ + MFMA + "\ts_nop 15\n\ts_nop 15\n\ts_cbranch_scc1 .LBB0_1\n" + END, False),
    (MFMA + "\ts_nop 15\n\ts_nop 15\n.LBB0_1:\n" + READ + END, False),
    (MFMA + MFMA + "\tv_accvgpr_read_b32 v20, a8\n" + END, False),                                      # other sums, or more products
    (MFMA + "\ts_cbranch_execz .LBB0_3\n\tglobal_store_dwordx4 v[0:1], a[0:3], off\n.LBB0_3:\n" + END, False),
    (MFMA + "\ts_cbranch_execz .LBB0_3\n" + END + ".LBB0_3:\n\tglobal_store_dwordx4 v[0:1], a[4:7], off\n" + END, True),
    (MFMA + "\tv_accvgpr_write_b32 a7, 0\n" + END, True),
])
def test_the_check_itself(listing, is_early):
    wrong, seen = early(listing)
    assert bool(wrong) == is_early and seen >= 1


def test_no_sum_is_touched_before_it_is_written_on_any_way():
    asm = build.device_asm("ops_product.hip")
    kernels = re.findall(r"^(_Z\S*tile_kernel\S*):", asm, re.M)
    assert len(kernels) == 12
    for name in kernels:
        start = asm.index("\n" + name + ":") + len(name) + 2
        wrong, seen = early(asm[start:asm.index(".Lfunc_end", start)])
        assert not wrong, (name, wrong[:5])
        assert seen > 0
