"""Wait states after matrix instructions, in the machine code of the built library.

The hardware does not hold an instruction back that reads or overwrites what a
matrix instruction has yet to write: the compiler has to put enough wait states
between them. Where paths join behind a branch it may count along a path longer
than the one taken and put too few: a form of delta_qk_grad_kernel that left the
products above the diagonal out by a branch read, on the path of the second row
block, an accumulator 2 wait states after the instruction that writes it (7 are
needed) and gave sums that varied from run to run. So every path from every
matrix instruction is walked here."""

import os
import re
import shutil
import subprocess

import pytest

from retnet_retention_amd import binding

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
# wait states until another instruction may touch the destination
NEEDED = {"v_mfma_f32_16x16x32_bf16": 7, "v_mfma_f32_32x32x16_bf16": 11, "v_mfma_f32_16x16x4_f32": 10,
          "v_mfma_f32_32x32x2_f32": 18}
REG = re.compile(r"\b([va])(?:(\d+)\b|\[(\d+):(\d+)\])")


def registers(text):
    out = set()
    for kind, one, low, high in REG.findall(text):
        out.update((kind, i) for i in (range(int(low), int(high) + 1) if low else (int(one),)))
    return out


class Kernel:
    """Instructions of a kernel: (operation, operands, index of a branch's target or None)."""

    def __init__(self, lines):
        where, rows = {}, []
        for ln in lines:
            m = re.match(r"\s+(\S+)\s*(.*?)\s*//\s*([0-9A-F]+):", ln)
            if m:
                where[int(m.group(3), 16)] = len(rows)
                rows.append((m.group(1), m.group(2), int(m.group(3), 16)))
        self.rows = []
        for op, args, at in rows:
            to = None
            if op == "s_branch" or op.startswith("s_cbranch"):
                step = int(args)
                to = where.get(at + 4 + 4 * (step - 65536 if step > 32767 else step))
            self.rows.append((op, args, to))
        self.regs = [registers(args) if op[0] != "s" else set() for op, args, _ in self.rows]

    def shortfalls(self):
        """(found, needed, matrix instruction, the one too near) over all paths."""
        for i, (op, args, _) in enumerate(self.rows):
            if not op.startswith("v_mfma"):
                continue
            assert op in NEEDED, f"no count of wait states for {op}"
            need, dst = NEEDED[op], registers(args.split(",")[0])
            best, paths = {}, [(i + 1, 0)]
            while paths:
                j, d = paths.pop()
                while j is not None and j < len(self.rows) and d < need and best.get(j, need) > d:
                    best[j] = d
                    op2, args2, to = self.rows[j]
                    if op2 == "s_endpgm":
                        break
                    if op2 == "s_nop":
                        d += int(args2, 0)
                    elif op2 == "s_branch":
                        j, d = to, d + 1
                        continue
                    elif op2.startswith("s_cbranch") and op2 != "s_cbranch_execz":  # (no lane, no access)
                        paths.append((to, d + 1))
                    elif op2.startswith("v_mfma"):
                        o = [registers(x) for x in args2.split(",")[:4]]
                        if (o[1] | o[2]) & dst:
                            yield d, need, f"{op} {args}", f"{op2} {args2}"
                            break
                        if o[0] & dst or o[3] & dst:  # accumulates on it: handed on by the hardware
                            break
                    elif self.regs[j] & dst:
                        yield d, need, f"{op} {args}", f"{op2} {args2}"
                        break
                    j, d = j + 1, d + 1


def kernels(listing):
    """{name: Kernel} of an objdump listing."""
    parts = re.split(r"^[0-9a-f]+ <(\S+)>:$", listing, flags=re.M)
    return {name: Kernel(body.splitlines()) for name, body in zip(parts[1::2], parts[2::2])}


def test_a_read_behind_a_branch_is_found():
    """Four matrix instructions with ways out between them, all to one place: the
    read there is far enough from the second on the long way, not on the short one."""
    body = """
0000000000000000 <k>:
	v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]    // 000000000000: 00000000
	s_cbranch_vccnz 10                                         // 000000000008: 00000000 <k+0x34>
	v_mfma_f32_16x16x32_bf16 a[4:7], v[0:3], v[8:11], a[4:7]   // 00000000000C: 00000000
	s_cbranch_scc1 7                                           // 000000000014: 00000000 <k+0x34>
	v_mfma_f32_16x16x32_bf16 a[8:11], v[0:3], v[4:7], a[8:11]  // 000000000018: 00000000
	s_nop 6                                                    // 000000000020: 00000000
	s_nop 0                                                    // 000000000024: 00000000
	s_nop 0                                                    // 000000000028: 00000000
	s_nop 0                                                    // 00000000002C: 00000000
	s_nop 0                                                    // 000000000030: 00000000
	ds_read_b128 v[20:23], v30                                 // 000000000034: 00000000
	v_accvgpr_read_b32 v12, a4                                 // 00000000003C: 00000000
	s_endpgm                                                   // 000000000044: 00000000
"""
    found = list(kernels(body)["k"].shortfalls())
    assert found == [(2, 7, "v_mfma_f32_16x16x32_bf16 a[4:7], v[0:3], v[8:11], a[4:7]", "v_accvgpr_read_b32 v12, a4")]
    assert not list(kernels(body.replace("ds_read_b128 v[20:23], v30", "s_nop 5"))["k"].shortfalls())


@pytest.mark.timeout(300)
def test_every_path_of_the_built_kernels_waits(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("llvm-objdump not found")
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("libretention.so not built (run __graft_entry__.build())")
    lib = tmp_path / "lib.so"
    shutil.copy(binding.LIB_PATH, lib)
    run = lambda *a: subprocess.run([OBJDUMP, *a], capture_output=True, text=True, check=True, cwd=tmp_path)  # noqa: E731
    run("--offloading", str(lib))
    matrix, bad = 0, []
    for f in sorted(tmp_path.glob("lib.so.*gfx950*")):
        for name, k in kernels(run("-d", str(f)).stdout).items():
            n = sum(op.startswith("v_mfma") for op, _, _ in k.rows)
            matrix += n > 0
            bad += [(name, *x) for x in (k.shortfalls() if n else ())]
    assert matrix > 50, "the kernels' code was not found"
    assert not bad, "\n".join(map(str, bad[:20]))
