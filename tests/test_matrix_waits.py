"""The waits between matrix instructions and the readers of their results, in the built library (CPU only).

The hardware does not hold back a vector instruction, store or LDS write that reads a matrix instruction's result too early: the
compiler has to put enough instructions or s_nop between the two.  It does so along every way through a kernel but some: behind a
uniform branch around a load it has been seen to count the longer of two ways (test_the_walk_finds_a_short_wait holds such a
kernel).  So the built code itself is walked: from every matrix instruction along every way until its result's wait is over or
somebody reads it.

A pass is four cycles; a unit makes 512 products a cycle in 16 bits (1024 in 8 bits), so 16x16x32 has 4 passes, 32x32x16 and
16x16x128 of 8-bit operands 8.  Needed are 4 wait states more than passes.  Each instruction between counts one, s_nop N counts
N + 1 (a matrix instruction issues in more than one: taken as one).
"""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "bit_quantized_moe_permute_amd", "libmoe2bit.so")
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

WAITS = {"16x16x32": 8, "32x32x16": 12, "16x16x128": 12}
REGISTERS = re.compile(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+)\b)")


def registers(text):
    out = set()
    for kind, first, last, one in REGISTERS.findall(text):
        out.update((kind, i) for i in (range(int(first), int(last) + 1) if first else [int(one)]))
    return out


class Instruction:
    __slots__ = ("op", "operands", "target")

    def __init__(self, text):
        self.op, _, rest = text.partition(" ")
        self.operands = rest.split(", ") if rest else []
        self.target = self.operands[-1].strip() if self.op.startswith(("s_branch", "s_cbranch")) else None

    def stores(self):
        return "store" in self.op or self.op.startswith("ds_write") or "atomic" in self.op

    def reads(self):
        keep = self.operands if self.stores() or self.op.startswith("v_cmp") else self.operands[1:]
        return registers(" ".join(keep)) | (registers(self.operands[0]) if re.match(r"v_(fmac|mac|dot\w*c)", self.op) else set())

    def writes(self):
        return set() if self.stores() or not self.operands else registers(self.operands[0])


def kernels(lines):
    """(name, instructions, label -> index) of every function of a disassembly."""
    name, code, labels = None, [], {}
    for line in lines:
        line = line.split("//", 1)[0].rstrip()
        if line.startswith("\t"):
            code.append(Instruction(line.strip()))
            continue
        m = re.match(r"(?:[0-9a-f]+ )?<(\S+)>:$", line)
        if not m:
            continue
        if re.fullmatch(r"L\d+", m[1]):
            labels[m[1]] = len(code)
        else:
            if name:
                yield name, code, labels
            name, code, labels = m[1], [], {}
    if name:
        yield name, code, labels


def short_waits(code, labels):
    """Number of matrix instructions, and (matrix instruction, reader, wait states between them, needed) of those read too early."""
    count, bad = 0, []
    for i, ins in enumerate(code):
        if not ins.op.startswith(("v_mfma", "v_smfma")):
            continue
        count += 1
        need = next(n for shape, n in WAITS.items() if f"_{shape}_" in ins.op)
        result = ins.writes()
        ways, least = [(i + 1, 0)], {}
        while ways:
            j, waited = ways.pop()
            if j >= len(code) or waited >= need or least.get(j, need) <= waited:
                continue
            least[j] = waited
            o = code[j]
            if o.op == "s_endpgm":
                continue
            if o.op.startswith("v_mfma"):
                # the sum goes on in the same registers without a wait; anything else of it is a reader
                if (registers(" ".join(o.operands[1:3])) & result
                        or (registers(o.operands[3]) & result and registers(o.operands[3]) != result)):
                    bad.append((i, j, waited, need))
                    continue
                if o.writes() & result:
                    continue
            elif (o.reads() | o.writes()) & result:
                bad.append((i, j, waited, need))
                continue
            if o.target:
                ways.append((labels[o.target], waited + 1))
                if o.op == "s_branch":
                    continue
            ways.append((j + 1, waited + (int(o.operands[0], 0) + 1 if o.op == "s_nop" else 1)))
    return count, bad


def disassembly(binary, folder):
    """Lines of the gfx950 code in a library or object that hipcc built."""
    copy = os.path.join(folder, "built")
    shutil.copy(binary, copy)
    subprocess.run([OBJDUMP, "--offloading", "built"], cwd=folder, check=True, capture_output=True)
    parts = [f for f in sorted(os.listdir(folder)) if f.startswith("built.") and f.endswith("gfx950")]
    assert parts, "no gfx950 code found"
    for part in parts:
        with subprocess.Popen([OBJDUMP, "-d", "--no-show-raw-insn", "--symbolize-operands", part], cwd=folder, text=True,
                              stdout=subprocess.PIPE) as p:
            yield from p.stdout
        assert p.returncode == 0


needs_objdump = pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")


@needs_objdump
def test_every_way_from_a_matrix_instruction_waits(tmp_path):
    if not os.path.exists(LIB):
        pytest.skip("libmoe2bit.so not built")
    total, found = 0, []
    for name, code, labels in kernels(disassembly(LIB, str(tmp_path))):
        n, bad = short_waits(code, labels)
        total += n
        found += [f"{name}: {code[i].op} read by {code[j].op} after {w} of {need} wait states" for i, j, w, need in bad]
    print(f"{total} matrix instructions")
    assert total > 1000
    assert not found, f"{len(found)} short waits:\n" + "\n".join(found[:20])


SHORT = r"""
#include <hip/hip_runtime.h>
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
__global__ void k_straight(const bf16x8 *a, const bf16x8 *b, float *o) {
    const int l = threadIdx.x;
    f32x4 d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[l], b[l], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
    o[l] = d[0] + d[1] + d[2] + d[3];
}
"""


@needs_objdump
@pytest.mark.skipif(not os.path.exists(HIPCC), reason="no hipcc")
def test_a_straight_kernel_has_its_wait(tmp_path):
    (tmp_path / "k.hip").write_text(SHORT)
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-shared", "-fPIC", "k.hip", "-o", "k.so"], cwd=tmp_path, check=True,
                   capture_output=True)
    found = [short_waits(code, labels) for name, code, labels in kernels(disassembly(str(tmp_path / "k.so"), str(tmp_path)))
             if "k_straight" in name]
    assert found == [(1, [])]


def test_the_walk_finds_a_short_wait():
    """What the compiler made of a uniform branch around a load: 8 wait states behind the load, 5 past it."""
    text = """
0000000000001000 <k_branch>:
\tv_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], 0 // 0
\ts_cmp_eq_u32 s0, 0
\ts_cbranch_scc1 L0
\tglobal_load_dword v7, v[4:5], off offset:256
\ts_waitcnt vmcnt(0)
\tv_add_f32_e32 v6, v6, v7
<L0>:
\ts_nop 2
\tv_fma_f32 v0, 2.0, v0, v1
\ts_endpgm
"""
    (name, code, labels), = kernels(text.splitlines())
    assert name == "k_branch"
    n, bad = short_waits(code, labels)
    assert n == 1 and [(code[j].op, w) for _, j, w, _ in bad] == [("v_fma_f32", 5)]
    longer = text.replace("s_nop 2", "s_nop 5")
    (_, code, labels), = kernels(longer.splitlines())
    assert short_waits(code, labels) == (1, [])


@pytest.mark.parametrize("reader,early", [
    ("global_store_dword v[20:21], v2, off", True), ("ds_write_b128 v20, v[0:3]", True), ("v_mov_b32_e32 v2, 0", True),
    ("v_fmac_f32_e32 v3, v8, v9", True), ("v_add_f32_e32 v8, v9, v10", False), ("global_load_dword v1, v[20:21], off", True),
    ("v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]", False),
    ("v_mfma_f32_16x16x32_bf16 v[4:7], v[8:11], v[12:15], v[0:3]", False),
    ("v_mfma_f32_16x16x32_bf16 v[4:7], v[0:3], v[12:15], 0", True),
    ("v_mfma_f32_32x32x16_bf16 v[16:31], v[8:11], v[12:15], v[2:17]", True)])
def test_the_walk_knows_readers(reader, early):
    text = f"<k>:\n\tv_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], 0\n\t{reader}\n\ts_nop 15\n\ts_endpgm\n"
    (_, code, labels), = kernels(text.splitlines())
    assert bool(short_waits(code[:2], labels)[1]) == early
