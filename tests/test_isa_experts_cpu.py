"""Resources and instructions of libgba_experts' kernels, read from the built library.

  * every kernel: no scratch, LDS within the 160 KiB of a CU;
  * the products use the matrix instruction of their operands and load straight to LDS;
  * the main loops neither copy accumulators nor move them between register files;
  * no vector instruction writes a matrix instruction's operand within the two
    instructions before it: the persistent kernels' matrix instructions are inline
    assembly, for which the compiler places no wait states.
"""
import os
import re
import subprocess
from collections import defaultdict

import pytest

from tests import test_isa_cpu as isa
from tiled_dense_gemm_bias_amd import experts

pytestmark = isa.pytestmark
OPS = {0: "v_mfma_f32_16x16x32_f16", 1: "v_mfma_f32_16x16x32_bf16", 2: "v_mfma_scale_f32_16x16x128_f8f6f4"}


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """(name -> metadata, name -> instructions as lists of an opcode and its operands)"""
    paths = None
    with pytest.MonkeyPatch.context() as m:
        m.setattr(isa.gba, "LIB_PATH", experts.EXPERTS_LIB_PATH)
        paths = isa._code_objects(str(tmp_path_factory.mktemp("co")))
    meta, code = {}, defaultdict(list)
    for path in paths:
        notes = subprocess.run([os.path.join(isa.LLVM, "llvm-readelf"), "--notes", path],
                               capture_output=True, text=True, check=True).stdout
        cur = None
        for line in notes.splitlines():
            m = re.match(r"\s+\.(\w+):\s+(.*)$", line)
            if m and m.group(1) == "name" and not m.group(2).endswith(".kd"):
                cur = meta.setdefault(m.group(2).strip(), {})
            elif m and cur is not None and m.group(2).strip().isdigit():
                cur[m.group(1)] = int(m.group(2))
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


def kinds(meta, kind):
    return [n for n in meta if kind in n]


def test_the_kernels_and_their_resources(kernels):
    meta, _ = kernels
    known = ("grouped_ring_kernel", "grouped_persist_kernel", "grouped_reduce_kernel", "column_sums_kernel",
             "mx4_quantize_kernel", "mx4_dequantize_kernel")
    for k in known:
        assert kinds(meta, k), k
    for n, m in meta.items():
        assert any(k in n for k in known), n
        assert m.get("private_segment_fixed_size", 0) == 0 and m.get("vgpr_spill_count", 0) == 0, (n, m)
        assert m.get("group_segment_fixed_size", 0) <= 160 * 1024, n
        assert m.get("vgpr_count", 0) <= (256 if "ring" in n else 512), n


def test_products_use_the_matrix_cores_and_load_to_lds(kernels):
    meta, code = kernels
    for n in kinds(meta, "grouped_ring") + kinds(meta, "grouped_persist"):
        a = isa._targs(n)
        op = a[5] if "ring" in n else a[0]
        used = {t[0] for t in code[n] if t[0].startswith("v_mfma")}
        assert used == {OPS[op]}, (n, used)
        assert any(t[0] == "buffer_load_dwordx4" and t[-1] == "lds" for t in code[n]), n


def test_main_loops_leave_accumulators_alone(kernels):
    """Between the first and the last matrix instruction (the ring kernel: of each stage's slice)."""
    meta, code = kernels
    for n in kinds(meta, "grouped_persist"):
        ops = [t[0] for t in code[n]]
        mf = [i for i, o in enumerate(ops) if o.startswith("v_mfma")]
        for lo in range(0, len(mf) - 63, 64):
            bad = {o for o in ops[mf[lo]:mf[lo + 63]] if o.startswith(("v_accvgpr", "scratch_"))}
            assert not bad, (n, bad)
    for n in kinds(meta, "grouped_ring"):
        ops = [t[0] for t in code[n]]
        mf = [i for i, o in enumerate(ops) if o.startswith("v_mfma")]
        bad = {o for o in ops[mf[0]:mf[-1]] if o.startswith(("v_accvgpr", "scratch_"))}
        assert not bad, (n, bad)


def registers(token):
    m = re.match(r"^([va])(?:(\d+)|\[(\d+):(\d+)\])$", token)
    if not m:
        return set()
    lo = int(m.group(2) or m.group(3))
    return {(m.group(1), i) for i in range(lo, int(m.group(4) or lo) + 1)}


def early_writes(code):
    """Matrix instructions with an operand that one of the two instructions before wrote."""
    bad, last = [], []
    for t in code:
        if t[0].startswith("v_mfma"):
            use = set().union(*(registers(x) for x in t[2:]))
            bad += [(o, " ".join(t)) for o, dst in last[-2:] if dst & use]
            last.append((t[0], set()))
        elif t[0] == "s_nop":
            last += [("s_nop", set())] * (int(t[1], 0) + 1)
        else:
            last.append((t[0], registers(t[1]) if t[0].startswith("v_") and len(t) > 1 else set()))
    return bad


def test_operands_of_matrix_instructions_are_written_in_time(kernels):
    meta, code = kernels
    planted = [["v_mov_b32_e32", "v4", "v9"], ["s_nop", "0"], ["v_mfma_f32_16x16x32_f16", "a[0:3]", "v[4:7]", "v[8:11]", "a[0:3]"]]
    assert early_writes(planted)
    for n in kinds(meta, "grouped_persist"):
        assert not early_writes(code[n]), (n, early_writes(code[n])[:3])
