"""The tiled product's hand-written instructions in the built library, no GPU: the
compiler does not see what a matrix instruction or a load to LDS in inline assembly
needs around it, so the listing of every kernel that has them is looked through.

Matrix instructions: none of their operands is written by a vector instruction in the
two places before, and no other instruction touches an accumulator within eleven
places after it was written (wait states; s_nop n counts n + 1).  Loads to LDS: M0
holds the place that the instruction before set, and nothing else is in it."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "tensor_adamw_optimizer_amd", "libapexw.so")
OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
MFMA = re.compile(r"v_mfma_f32_16x16x32_bf16 a\[(\d+):(\d+)\], (v\[\d+:\d+\]), (v\[\d+:\d+\]), a\[\1:\2\]$")
SETTLED, FRESH = 11, 2


def _registers(text):
    """The vector registers that an operand list names."""
    out = set()
    for kind, one, lo, hi in re.findall(r"\b([va])(?:(\d+)\b|\[(\d+):(\d+)\])", text):
        out |= {kind + str(i) for i in (range(int(lo), int(hi) + 1) if lo else (int(one),))}
    return out


def faults(lines):
    """What is wrong with one kernel's instructions, as (place, instruction, why)."""
    wrong = []
    wrote, settled, m0 = {}, {}, None    # by register: the place of a vector write, of an MFMA's
    at = 0
    for text in lines:
        m = MFMA.match(text)
        op, _, args = text.partition(" ")
        regs = _registers(args)
        if m:
            for r in sorted(regs):
                if at - wrote.get(r, -FRESH - 1) <= FRESH:
                    wrong.append((at, text, "%s written right before" % r))
            settled.update((r, at) for r in _registers("a[%s:%s]" % m.groups()[:2]))
        else:
            for r in sorted(regs):
                if at - settled.get(r, -SETTLED - 1) <= SETTLED:
                    wrong.append((at, text, "%s written by a matrix instruction right before" % r))
            if op.startswith("v_") and not op.startswith("v_mfma"):
                first = args.split(",")[0]
                wrote.update((r, at) for r in _registers(first))
        if re.search(r"\bm0\b", args):
            if op != "s_add_i32" or not args.startswith("m0,"):
                wrong.append((at, text, "M0 in another use"))
            m0 = at
        elif op.startswith("buffer_load") and text.endswith(" lds"):
            if m0 is None:
                wrong.append((at, text, "M0 not set"))
            m0 = None
        elif m0 is not None and op != "s_nop":
            wrong.append((at, text, "between M0 and its load"))
        at += int(args.split()[0], 0) + 1 if op == "s_nop" else 1
    return wrong


def _kernels(tmp_path):
    """{name: instructions} of the library's device code."""
    if not os.path.exists(LIB):
        pytest.skip("the library is not built")
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    lib = shutil.copy(LIB, str(tmp_path))
    subprocess.check_call([OBJDUMP, "--offloading", lib], stdout=subprocess.DEVNULL, cwd=str(tmp_path))
    out, lines = {}, None
    for name in sorted(os.listdir(str(tmp_path))):
        if "amdgcn" not in name:
            continue
        text = subprocess.check_output([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr",
                                        str(tmp_path / name)], text=True)
        for line in text.splitlines():
            m = re.match(r"<(\S+)>:$", line)
            if m:
                lines = out.setdefault(name + " " + m.group(1), [])
            elif lines is not None and line.strip():
                lines.append(line.split("//")[0].strip())
    return out


def test_every_kernel_with_hand_written_instructions(tmp_path):
    kernels = _kernels(tmp_path)
    loads = {n: k for n, k in kernels.items() if any(x.endswith(" lds") for x in k)}
    large = {n: k for n, k in loads.items() if "IDF16b" in n and "ELi256ELi256E" in n}
    assert len(loads) > 50 and len(large) >= 16
    for name, lines in loads.items():
        # (only the large bf16 tile's matrix instructions are hand-written)
        wrong = faults(lines if name in large else [x for x in lines if not x.startswith("v_mfma")])
        assert not wrong, (name, len(wrong), wrong[:4])
        if name in large:
            # two steps of 32 in a slice
            assert sum(bool(MFMA.match(x)) for x in lines) >= 64, name


@pytest.mark.parametrize("lines,why", [
    (["v_mov_b32 v8, v1", "s_nop 0", "v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[8:11], a[0:3]"], "v8"),
    (["v_accvgpr_write_b32 a2, 0", "v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[8:11], a[0:3]"], "a2"),
    (["v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[8:11], a[0:3]", "s_nop 9",
      "v_accvgpr_read_b32 v1, a3"], "a3"),
    (["v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[8:11], a[0:3]", "ds_write_b128 v1, a[0:3]"], "a0"),
    (["s_add_i32 m0, s4, 0", "s_mov_b32 s3, m0", "buffer_load_dwordx4 v1, s[0:3], 0 offen lds"], "M0"),
    (["buffer_load_dwordx4 v1, s[0:3], 0 offen lds"], "M0"),
])
def test_the_look_finds_what_it_looks_for(lines, why):
    assert why in faults(lines)[0][2]


def test_the_look_passes_what_is_right():
    assert not faults(["v_accvgpr_write_b32 a2, 0", "s_nop 1", "s_nop 15",
                       "v_mfma_f32_16x16x32_bf16 a[0:3], v[4:7], v[8:11], a[0:3]",
                       "v_mfma_f32_16x16x32_bf16 a[0:3], v[12:15], v[8:11], a[0:3]",
                       "s_add_i32 m0, s4, 0", "s_nop 0", "buffer_load_dwordx4 v1, s[0:3], 0 offen lds",
                       "s_nop 15", "v_accvgpr_read_b32 v1, a3"])
