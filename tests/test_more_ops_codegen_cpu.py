"""What the compiler emits for the 8-bit product's tiles, checked without a GPU.

Their matrix instructions are written out as assembly, so that their sums stay in place; the
compiler does not know them as such.  It must not touch the sums between them (a move right behind
an instruction of 16 passes would read what it has not written yet), and the kernel waits
for the last ones itself before it reads them.  And no packed fp32 arithmetic."""
import re

import pytest

from zero_dp_sharded_amd import build


@pytest.fixture(scope="module")
def asm():
    return build.device_asm("ops_product.hip")


def functions(asm, word):
    for m in re.finditer(r"^(_Z\S*" + word + r"\S*):", asm, re.M):
        yield m.group(1), asm[m.end():asm.index(".Lfunc_end", m.end())]


def test_the_sums_are_left_alone_between_the_instructions(asm):
    kernels = list(functions(asm, "tile_kernel"))
    assert len(kernels) == 12                    # fp16 and bf16, three tiles, both forms of scales
    for name, body in kernels:
        seen = 0
        for block in re.split(r"^\.LBB\S+:", body, flags=re.M):
            pending = set()                      # sums that may still be written
            for line in block.splitlines():
                ins = line.split(";")[0].strip()
                if ins.startswith("v_mfma"):
                    m = re.match(r"v_mfma_scale_f32_16x16x128_f8f6f4 (a\[(\d+):(\d+)\]), v\[\d+:\d+\], v\[\d+:\d+\], \1, v\d+, v\d+ ", ins)
                    assert m, (name, ins)
                    pending.update(range(int(m.group(2)), int(m.group(3)) + 1))
                    seen += 1
                elif ins == "s_nop 15":
                    pending.clear()
                else:
                    touched = {int(x) for x in re.findall(r"\ba(\d+)", ins)}
                    for lo, hi in re.findall(r"\ba\[(\d+):(\d+)\]", ins):
                        touched.update(range(int(lo), int(hi) + 1))
                    assert not (touched & pending), (name, ins)
        assert seen > 0


def test_every_instruction_waits_for_what_a_move_before_it_wrote(asm):
    for name, body in functions(asm, "tile_kernel"):
        lines = [line.split(";")[0].strip() for line in body.splitlines()]
        lines = [x for x in lines if x and not x.startswith(".")]
        for before, ins in zip(lines, lines[1:]):
            if ins.startswith("v_mfma"):
                assert before == "s_nop 1", (name, before, ins)


def test_no_packed_fp32_and_no_spills_in_the_loops(asm):
    assert not re.search(r"^\s*v_pk_(add|mul|fma)_f32", asm, re.M)
    for name, body in functions(asm, "tile_kernel"):
        assert "scratch_" not in body, name
