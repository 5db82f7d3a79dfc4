"""A rule of the instruction set that the compiler keeps in its own code but
not inside inline asm, checked in the built library's gfx950 code: between a
vector instruction that writes a scalar register and a vector memory
instruction that reads it there are five wait states (another instruction is
one, s_nop n is n + 1). Runs without a GPU."""
import os
import re
import shutil
import subprocess

import pytest

import collective_window_put_amd as vr

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
NEED = 5


def _registers(operand):
    """Scalar registers that an operand names."""
    m = re.fullmatch(r"-?\|?s(\d+)\|?", operand)
    if m:
        return {int(m.group(1))}
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    return {operand} if operand in ("vcc", "vcc_lo", "vcc_hi") else set()


def _written(name, ops):
    """Scalar registers that a vector instruction writes."""
    if name.startswith(("v_readfirstlane", "v_readlane", "v_cmp_")):
        return _registers(ops[0])
    if "_co_" in name or name.startswith(("v_div_scale", "v_mad_u64_u32", "v_mad_i64_i32")):
        return _registers(ops[1])
    return set()


def _wait_states(name, ops):
    return int(ops[0], 0) + 1 if name == "s_nop" else 1


def hazards(text):
    """(function, memory instruction, writing instruction, wait states between) of every place in a disassembly that
    breaks the rule, along every path that leads to the memory instruction."""
    bad, reads = [], 0
    for body in re.split(r"\n(?=[0-9a-f]+ <)", text):
        head = re.match(r"[0-9a-f]+ <(.+)>:", body.lstrip("\n"))
        if not head:
            continue
        code, at = [], {}
        for line in body.splitlines()[1:]:
            m = re.match(r"\s+(\S+)\s*(.*?)\s*// ([0-9A-F]+):(.*)", line)
            if not m:
                continue
            at[int(m.group(3), 16)] = len(code)
            code.append((m.group(1), [o.strip() for o in re.split(r",\s*|\s+", m.group(2)) if o.strip()], m.group(4)))
        before = [[] for _ in code]  # the instructions that may run right before each
        start = min(at, default=0)
        for i, (name, ops, rest) in enumerate(code):
            if i + 1 < len(code) and name not in ("s_branch", "s_endpgm", "s_setpc_b64"):
                before[i + 1].append(i)
            if name.startswith(("s_branch", "s_cbranch")):
                to = re.search(r"\+0x([0-9a-f]+)>", rest)
                before[at[start + (int(to.group(1), 16) if to else 0)]].append(i)
        for i, (name, ops, _) in enumerate(code):
            if not name.startswith(("global_", "buffer_", "flat_", "scratch_")):
                continue
            used = set().union(*map(_registers, ops)) if ops else set()
            if not used:
                continue
            reads += 1
            todo, seen = [(j, 0) for j in before[i]], set()
            while todo:
                j, states = todo.pop()
                if states >= NEED or (j, states) in seen:
                    continue
                seen.add((j, states))
                n, o, _ = code[j]
                if n.startswith("v_") and _written(n, o) & used:
                    bad.append((head.group(1), f"{name} {' '.join(ops)}", f"{n} {' '.join(o)}", states))
                    continue
                todo += [(k, states + _wait_states(n, o)) for k in before[j]]
    return bad, reads


SAMPLE = """
0000000000001000 <k>:
\tv_readfirstlane_b32 s4, v1                                 // 000000001000: 7E080501
{gap}\tglobal_load_lds_dwordx4 v12, s[4:5]                        // 000000001010: DDF48000 0004000C
\ts_endpgm                                                   // 000000001018: BF810000
"""


@pytest.mark.parametrize("gap,broken", [("", True), ("\ts_mov_b32 m0, s9  // 000000001004: BEFC0009\n\ts_nop 0  // 000000001008: BF800000\n", True),
                                        ("\ts_mov_b32 m0, s9  // 000000001004: BEFC0009\n\ts_nop 2  // 000000001008: BF800002\n", True),
                                        ("\ts_mov_b32 m0, s9  // 000000001004: BEFC0009\n\ts_nop 3  // 000000001008: BF800003\n", False)])
def test_the_check_counts_wait_states(gap, broken):
    bad, reads = hazards(SAMPLE.format(gap=gap))
    assert reads == 1 and bool(bad) is broken


@pytest.fixture(scope="module")
def disassembly(tmp_path_factory):
    """The library's device code, one text per source file."""
    if not os.path.exists(vr.LIB_PATH):
        from collective_window_put_amd.build import build
        build()
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    work = tmp_path_factory.mktemp("code")
    lib = shutil.copy(vr.LIB_PATH, work)
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=work, check=True, capture_output=True)
    objects = sorted(p for p in work.iterdir() if p.name.endswith("gfx950"))
    assert objects
    return [subprocess.run([OBJDUMP, "-d", str(p)], check=True, capture_output=True, text=True).stdout for p in objects]


def test_scalar_bases_are_ready_before_vector_memory_reads_them(disassembly):
    total = 0
    for text in disassembly:
        bad, reads = hazards(text)
        total += reads
        assert not bad, (len(bad), bad[:4])
    assert total > 1000
