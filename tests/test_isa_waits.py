"""Wait states that nothing inserts inside inline assembly, in the built
library's own gfx950 code (CPU only).

The kernels issue their loads into LDS as inline assembly, where the compiler
sees no hazards.  Two rules of the instruction set concern them:
* a scalar instruction that writes M0 and a load into LDS, which takes its LDS
  address from M0, need one instruction (or s_nop 0) between them;
* a vector instruction that writes a scalar register and a vector memory
  instruction that reads it need five.
Checked along the straight order of the code, for every vector memory
instruction.
"""
import re
import shutil
import subprocess

import pytest

import fp8_gemm_backward_amd as lp

OBJDUMP = shutil.which("llvm-objdump", path="/opt/rocm/llvm/bin") or shutil.which("llvm-objdump")
WAITS = 5


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    """[(function, instruction)] of every kernel in the library."""
    if OBJDUMP is None:
        pytest.skip("no llvm-objdump")
    at = tmp_path_factory.mktemp("code")
    shutil.copy(lp.LIB_PATH, at / "liblp.so")
    subprocess.run([OBJDUMP, "--offloading", "liblp.so"], cwd=at, check=True, capture_output=True)
    images = sorted(at.glob("*gfx950*"))
    assert len(images) > 10
    out = []
    for image in images:
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(image)], check=True, capture_output=True, text=True).stdout
        name = ""
        for line in text.splitlines():
            m = re.match(r"[0-9a-f]+ <(\w+)>:", line)
            if m:
                name = m[1]
            elif line.startswith("\t"):
                out.append((name, line.split("//")[0].strip()))
    return out


def scalars(operand: str) -> set:
    """The scalar registers an operand names."""
    m = re.match(r"s\[(\d+):(\d+)\]", operand) or re.match(r"s(\d+)()\b", operand)
    if not m:
        return {"vcc"} if operand.startswith("vcc") else set()
    return set(range(int(m[1]), int(m[2] or m[1]) + 1))


def breaches(code) -> list:
    """(function, writer, reader) of every read that comes too early."""
    found, written, m0, here, last = [], {}, None, None, ""       # register -> (wait states since, writer)
    for name, line in code:
        if name != here or re.match(r"s_(branch|endpgm|setpc|swappc)", last):     # (what follows is reached from elsewhere)
            written, m0, here = {}, None, name
        last = line
        op, _, rest = line.partition(" ")
        operands = [o.strip() for o in rest.split(",")]
        memory = op.startswith(("buffer_", "global_", "flat_", "scratch_"))
        if memory:
            used = set().union(*(scalars(o.split(" ")[0]) for o in operands))
            found += [(name, w, line) for r, (n, w) in written.items() if r in used]
            if op.startswith("buffer_load") and line.endswith("lds") and m0 is not None:
                found.append((name, m0, line))
        waits = int(operands[0], 0) + 1 if op == "s_nop" else 1
        written = {r: (n + waits, w) for r, (n, w) in written.items() if n + waits < WAITS}
        target = operands[0] if op.startswith(("s_", "v_")) and not op.startswith(("s_nop", "s_waitcnt", "s_cmp", "s_branch", "s_cbranch")) else ""
        m0 = line if op.startswith("s_") and target == "m0" else None
        if op.startswith("s_"):
            for r in scalars(target):
                written.pop(r, None)
        elif op.startswith("v_"):
            for o in operands[:2]:                      # (the second result of a carry-out addition)
                if o is operands[0] or "_co_" in op:
                    for r in scalars(o):
                        written[r] = (0, line)
    return found


def test_planted_breaches_are_seen():
    def check(*lines):
        return bool(breaches([("f", line) for line in lines]))
    load = "buffer_load_dwordx4 v1, s[4:7], s9 offen lds"
    assert check("s_mov_b32 m0, s3", load) == 1 and check("s_mov_b32 m0, s3", "s_nop 0", load) == 0
    assert check("s_mov_b32 m0, s3", "buffer_load_dwordx4 v[1:4], v5, s[4:7], 0 offen") == 0
    for reg in ("s4", "s7", "s9"):
        for gap in range(7):
            assert check(f"v_readfirstlane_b32 {reg}, v1", *["v_mov_b32_e32 v8, v9"] * gap, "s_nop 0", load) == (gap + 1 < WAITS)
    assert check("v_readlane_b32 s9, v1, 3", "s_add_i32 s9, s9, s2", load) == 0      # (scalar reads wait by themselves)
    assert check("v_readlane_b32 s8, v1, 3", load) == 0
    assert check("v_cmp_lt_i32_e64 s[6:7], v1, v2", "s_nop 3", load) == 1
    assert check("v_cmp_lt_i32_e64 s[6:7], v1, v2", "s_nop 4", load) == 0
    assert check("v_cmp_lt_i32_e64 s[6:7], v1, v2", "s_branch 32", load) == 0


def test_loads_wait_for_the_scalars_they_read(code):
    loads = sum(line.endswith("lds") and line.startswith("buffer_load") for _, line in code)
    assert loads > 1000
    found = breaches(code)
    assert not found, f"{len(found)} of {loads}, e.g. {found[:3]}"
