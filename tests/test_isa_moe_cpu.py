"""Resources and instructions of libgba_moe's kernels, read from the built library.

  * every kernel: no scratch, no spilled vector registers, LDS within the 160 KiB of a CU;
  * the products use the 8-bit matrix instruction; the staged kernels load straight to LDS;
  * the staged kernels' main loops neither copy accumulators nor move them between register files;
  * no packed fp32 instruction anywhere.
"""
import os
import re
import subprocess
from collections import defaultdict

import pytest

from tests import test_isa_cpu as isa
from tests.test_isa_experts_cpu import early_writes, kinds, registers
from tiled_dense_gemm_bias_amd import moe

pytestmark = isa.pytestmark
MFMA = "v_mfma_f32_16x16x128_f8f6f4"
PRODUCTS = ("grouped_ring_kernel", "f8_persist_kernel", "f8_stream_kernel")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """(name -> metadata, name -> instructions as lists of an opcode and its operands)"""
    with pytest.MonkeyPatch.context() as m:
        m.setattr(isa.gba, "LIB_PATH", moe.MOE_LIB_PATH)
        paths = isa._code_objects(str(tmp_path_factory.mktemp("co")))
    meta, code = {}, defaultdict(list)
    for path in paths:
        notes = subprocess.run([os.path.join(isa.LLVM, "llvm-readelf"), "--notes", path],
                               capture_output=True, text=True, check=True).stdout
        # A kernel's entries stand in alphabetical order: some come before its name.
        for entry in re.split(r"^  - \.agpr_count", notes, flags=re.M)[1:]:
            entry = "    .agpr_count" + entry
            name = re.search(r"^    \.name:\s+(\S+)$", entry, flags=re.M).group(1)
            meta[name] = {k: int(v) for k, v in re.findall(r"^    \.(\w+):\s+(\d+)$", entry, flags=re.M)}
        dis = subprocess.run([os.path.join(isa.LLVM, "llvm-objdump"), "-d", "--mcpu=gfx950", "--no-show-raw-insn", path],
                             capture_output=True, text=True, check=True).stdout
        sym = None
        for line in dis.splitlines():
            m = re.match(r"^[0-9a-f]+ <(\S+)>:$", line)
            if m:
                sym = m.group(1)
            elif sym:
                t = line.split("//")[0].replace(",", " ").split()
                if t and re.match(r"^[a-z_][a-z0-9_]*$", t[0]):
                    code[sym].append(t)
    assert meta
    return meta, code


def test_the_kernels_and_their_resources(kernels):
    meta, _ = kernels
    known = PRODUCTS + ("grouped_reduce_kernel", "route_kernel", "route_grad_kernel", "count_kernel", "sort_kernel", "dispatch_kernel",
                        "combine_kernel", "combine_grad_kernel", "quantize_rows_kernel", "quantize_weights_kernel")
    for k in known:
        assert kinds(meta, k), k
    for n, m in meta.items():
        assert any(k in n for k in known), n
        assert m["private_segment_fixed_size"] == 0 and m["vgpr_spill_count"] == 0, (n, m)
        assert m["group_segment_fixed_size"] <= 160 * 1024, (n, m)
        # a block's waves fit a CU's registers: 512 a lane and SIMD, in all
        waves_a_simd = -(-m["max_flat_workgroup_size"] // 256)
        assert m["vgpr_count"] * waves_a_simd <= 512, (n, m)


def test_products_use_the_matrix_cores(kernels):
    meta, code = kernels
    names = [n for k in PRODUCTS for n in kinds(meta, k)]
    for n in names:
        assert {t[0] for t in code[n] if t[0].startswith("v_mfma")} == {MFMA}, n
        to_lds = any(t[0] == "buffer_load_dwordx4" and t[-1] == "lds" for t in code[n])
        assert to_lds == ("f8_stream" not in n), n
    for n in meta:
        if n not in names:
            assert not any(t[0].startswith("v_mfma") for t in code[n]), n


def test_no_packed_fp32(kernels):
    _, code = kernels
    for n, ops in code.items():
        assert not {t[0] for t in ops} & {"v_pk_add_f32", "v_pk_mul_f32", "v_pk_fma_f32"}, n


def test_main_loops_leave_accumulators_alone(kernels):
    meta, code = kernels
    for n in kinds(meta, "f8_persist") + kinds(meta, "grouped_ring"):
        ops = [t[0] for t in code[n]]
        mf = [i for i, o in enumerate(ops) if o.startswith("v_mfma")]
        bad = {o for o in ops[mf[0]:mf[-1]] if o.startswith(("v_accvgpr", "scratch_"))}
        assert not bad, (n, bad)


def test_operands_of_matrix_instructions_are_written_in_time(kernels):
    """The persistent kernel's additions are inline assembly beside the compiler's matrix instructions: none of them, or
    of any other vector instruction, writes a matrix instruction's operand in the two instructions before it."""
    meta, code = kernels
    for n in kinds(meta, "f8_persist"):
        assert not early_writes(code[n]), (n, early_writes(code[n])[:3])


def early_reads(code):
    """Vector instructions that read a matrix instruction's sums too soon: fewer than LAG others stand between (each waits
    for the one before, 32 cycles), and fewer than 18 wait states of instructions and s_nop."""
    lag, bad, written, states, count = 3, [], {}, 0, 0
    for t in code:
        if t[0] == "s_nop":
            states += int(t[1], 0) + 1
            continue
        if t[0].startswith("v_") and not t[0].startswith("v_mfma"):
            read = t[1:] if t[0].startswith("v_fmac") else t[2:]
            for x in read:
                for r in registers(x):
                    if r in written and count - written[r][0] < lag and states - written[r][1] < 18:
                        bad.append((" ".join(t), count - written[r][0], states - written[r][1]))
            for r in registers(t[1]) if len(t) > 1 else ():
                written.pop(r, None)
        states += 1
        if t[0].startswith("v_mfma"):
            count += 1
            for r in registers(t[1]):
                written[r] = (count, states)
    return bad


def test_sums_of_matrix_instructions_are_read_late_enough(kernels):
    meta, code = kernels
    product = ["v_mfma_f32_16x16x128_f8f6f4", "v[0:3]", "v[8:15]", "v[16:23]", "0"]
    other = ["v_mfma_f32_16x16x128_f8f6f4", "v[4:7]", "v[8:15]", "v[16:23]", "0"]
    add = ["v_fmac_f32_e32", "v30", "v2", "v31"]
    assert early_reads([product, other, other, add]) and not early_reads([product, other, other, other, add])
    assert not early_reads([product, ["s_nop", "7"], ["s_nop", "7"], ["s_nop", "7"], add])
    for n in kinds(meta, "f8_persist"):
        adds = [t for t in code[n] if t[0].startswith("v_fmac_f32")]
        assert len(adds) >= 128 and not early_reads(code[n]), (n, len(adds), early_reads(code[n])[:3])
