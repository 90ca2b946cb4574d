"""CPU: no matrix product's result is read before it is there.

A matrix instruction writes its registers some cycles after it issues, and nothing in the hardware makes another
instruction wait for them: the compiler puts enough instructions, or s_nop, in between.  Where a branch follows the
products, the compiler that builds this library has been seen to count the instructions that the branch skips.  This test
walks every path behind each matrix instruction of the compiled kernels and counts issue slots up to the first
instruction other than a matrix instruction that touches the result (between matrix instructions the hardware waits)."""
import os
import re
import subprocess

import pytest

from selective_state_space_55_amd import build as hipbuild

# slots that a result takes: 4 passes (16x16x32) and 8 passes (32x32x16), and the largest for others
SLOTS = (("32x32x16", 11), ("16x16x32", 7))
SOURCES = ["linear_attention.hip", "ssd_fwd.hip", "ssd_varlen.hip"]


def early_reads(text):
    found, products = [], 0
    for func in re.split(r"\n(?=_Z\S+:)", text):
        ins, labels = [], {}
        for line in func.split("\n")[1:]:
            s = line.split(";")[0].strip()
            m = re.match(r"(\.?LBB\w+):", s)
            if m:
                labels[m.group(1)] = len(ins)
            elif s and not s.startswith(".") and not s.endswith(":"):
                ins.append(s)

        def following(i):
            s = ins[i]
            if s.startswith("s_endpgm"):
                return []
            if s.startswith("s_branch"):
                return [labels[s.split()[1]]]
            then = [i + 1] if i + 1 < len(ins) else []
            return then + [labels[s.split()[1]]] if s.startswith("s_cbranch") else then

        regs = [[(k, int(a), int(b or a)) for k, a, b in re.findall(r"\b([av])\[?(\d+)(?::(\d+))?\]?", s)] for s in ins]
        for i, s in enumerate(ins):
            m = re.match(r"v_mfma_f32_(\w+) ([av])\[(\d+):(\d+)\]", s)
            if not m:
                continue
            products += 1
            need = next((n for shape, n in SLOTS if m.group(1).startswith(shape)), 19)
            kind, lo, hi = m.group(2), int(m.group(3)), int(m.group(4))
            least, stack = {}, [(j, 0) for j in following(i)]
            while stack:
                j, slots = stack.pop()
                if slots >= need or least.get(j, need) <= slots:
                    continue
                least[j] = slots
                if any(k == kind and not (b < lo or a > hi) for k, a, b in regs[j]):
                    if not ins[j].startswith("v_mfma"):
                        found.append((func.split(":")[0], s, slots, need, ins[j]))
                    continue
                took = int(ins[j].split()[1], 0) + 1 if ins[j].startswith("s_nop") else 1
                stack += [(k, slots + took) for k in following(j)]
    return found, products


@pytest.mark.parametrize("src", SOURCES)
def test_results_are_there_when_read(src, tmp_path):
    path = str(tmp_path / "k.s")
    flags = [f for f in hipbuild.flags() if f not in ("-shared", "-fPIC")]
    subprocess.run([hipbuild.hipcc()] + flags + ["--cuda-device-only", "-S", "-o", path, os.path.join(hipbuild.CSRC, src)],
                   check=True, capture_output=True)
    text = open(path).read()
    found, products = early_reads(text)
    assert products > 100
    assert not found, found[:5]
    # and no spills: a register in memory costs these kernels a quarter of their time and more
    if src == "linear_attention.hip":
        sizes = [int(x) for x in re.findall(r"\.private_segment_fixed_size:\s+(\d+)", text)]
        assert sizes and max(sizes) == 0
        assert not re.findall(r"\bv_pk_(add|mul|fma)_f32\b", text)


def test_a_read_behind_a_skipped_block_is_found():
    text = """
_Z1kv:
	v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], 0
	s_cbranch_vccnz .LBB0_2
	v_add_f32_e32 v8, v9, v10
	v_add_f32_e32 v8, v9, v10
	v_add_f32_e32 v8, v9, v10
	v_add_f32_e32 v8, v9, v10
	v_add_f32_e32 v8, v9, v10
	v_add_f32_e32 v8, v9, v10
	v_add_f32_e32 v8, v9, v10
.LBB0_2:
	%sv_accvgpr_read_b32 v11, a3
	s_endpgm
"""
    found, products = early_reads(text % "")
    assert products == 1 and [f[2] for f in found] == [1]
    assert early_reads(text % "s_nop 7\n\t")[0] == []
