"""The wait states that gfx950 asks for before a copy into LDS, checked on the
CPU in the library's own machine code.  The hardware does not hold such an
instruction back by itself, and the compiler adds the wait states only to what it
can see, which an asm string is not:
  * one between a scalar write of m0 and a load that lands at m0;
  * five between a vector instruction's write of a scalar register (a
    readfirstlane, a comparison) and a memory instruction that reads it, unless
    a scalar instruction writes the register after it."""
import os
import re
import shutil
import subprocess

import pytest

import fp8_block_scaled_bias_amd as M

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
REG = re.compile(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b|\b(m0|vcc)\b")
LINE = re.compile(r"^\s+([a-z][a-z0-9_]*)\s*(.*?)\s*// ([0-9A-F]{12}):")
M0_STATES, SGPR_STATES = 1, 5


def scalars(text):
    """Scalar registers of an operand."""
    out = set()
    for a, b, c, name in REG.findall(text):
        out |= {name} if name else {f"s{i}" for i in (range(int(a), int(b) + 1) if a else [int(c)])}
    return out


def operands(text):
    return [p.strip() for p in re.split(r",\s*(?![^\[]*\])", text)]


def is_copy(name, text):
    return name.startswith(("buffer_load", "global_load", "scratch_load")) and (
        "_lds" in name or text.split()[-1:] == ["lds"])


class Instruction:
    def __init__(self, name, text, addr):
        self.name, self.text, self.addr = name, text.split("//")[0], addr
        ops = operands(self.text)
        # (a carry-out, the scaled quotient's flag: the second operand)
        two = re.match(r"v_(add|sub|subrev|addc|subb|subbrev)_co_|v_div_scale|v_mad_[iu]64_", name)
        self.valu_sgprs = scalars(",".join(ops[:2 if two else 1])) if name.startswith("v_") else set()
        self.writes_m0 = name.startswith("s_") and ops[:1] == ["m0"]
        self.copy = is_copy(name, self.text)
        self.salu_sgprs = scalars(ops[0]) if name.startswith("s_") and not name.startswith(("s_cmp", "s_bitcmp")) else set()
        self.reads = scalars(self.text) if self.copy else set()
        self.states = int(ops[0], 0) + 1 if name == "s_nop" else 1


def functions(listing):
    """Per function its instructions and each one's predecessors."""
    code, targets, start = [], [], 0

    def done():
        at = {i.addr: n for n, i in enumerate(code)}
        before = [[n - 1] if n and not (code[n - 1].name in ("s_branch", "s_endpgm", "s_setpc_b64")) else []
                  for n in range(len(code))]
        for n, i in enumerate(code):
            if i.name == "s_branch" or i.name.startswith("s_cbranch"):
                to = re.search(r"\+0x([0-9a-f]+)>", targets[n])
                before[at[start + int(to.group(1), 16) if to else start]].append(n)
        return code, before

    for line in listing.splitlines():
        head = re.match(r"^([0-9a-f]+) <(.*)>:", line)
        if head:
            if code:
                yield name, *done()
            code, targets, start, name = [], [], int(head.group(1), 16), head.group(2)
            continue
        m = LINE.match(line)
        if m:
            code.append(Instruction(m.group(1), m.group(2), int(m.group(3), 16)))
            targets.append(line)
    if code:
        yield name, *done()


def too_close(code, before, n):
    """What copy n waits too little for: (register, writer)."""
    found, seen, todo = [], set(), [(p, 0, frozenset(code[n].reads | {"m0"})) for p in before[n]]
    while todo:
        p, states, regs = todo.pop()
        if states >= SGPR_STATES or (p, states, regs) in seen:
            continue
        seen.add((p, states, regs))
        w = code[p]
        if w.writes_m0 and states < M0_STATES:
            found.append(("m0", w))
        for r in w.valu_sgprs & regs:
            found.append((r, w))
        todo += [(q, states + w.states, regs - w.salu_sgprs) for q in before[p]]
    return found


def test_the_check_finds_what_it_looks_for():
    listing = """
0000000000000100 <f>:
\tv_readfirstlane_b32 s4, v0   // 000000000100: 00
\ts_mov_b32 m0, s9   // 000000000104: 00
\tbuffer_load_dwordx4 v1, s[4:7], s8 offen lds   // 000000000108: 00
\ts_mov_b32 m0, s9   // 00000000010C: 00
\ts_nop 0   // 000000000110: 00
\tglobal_load_lds_dword v[2:3], off   // 000000000114: 00
\tv_cmp_gt_i64_e64 s[6:7], s[2:3], v[4:5]   // 000000000118: 00
\ts_nop 3   // 00000000011C: 00
\tbuffer_load_dword v1, s[4:7], s8 offen lds   // 000000000120: 00
\tv_readfirstlane_b32 s8, v0   // 000000000124: 00
\ts_nop 4   // 000000000128: 00
\tbuffer_load_dword v1, s[4:7], s8 offen lds   // 00000000012C: 00
\ts_cbranch_scc1 65530   // 000000000130: 00 <f+0x8>
\tv_mad_u64_u32 v[2:3], s[8:9], v4, s1, v[6:7]   // 000000000134: 00
\ts_mov_b32 s8, 0   // 000000000138: 00
\ts_add_u32 m0, s2, 0x400   // 00000000013C: 00
\ts_nop 0   // 000000000140: 00
\tbuffer_load_dwordx4 v1, s[4:7], s8 offen lds   // 000000000144: 00
\tbuffer_load_dwordx4 v1, s[4:7], s9 offen lds   // 000000000148: 00
\ts_endpgm   // 00000000014C: 00
"""
    (name, code, before), = functions(listing)
    found = {code[n].addr: {r for r, _ in too_close(code, before, n)} for n in range(len(code)) if code[n].copy}
    assert found == {0x108: {"s4", "m0"}, 0x114: set(), 0x120: {"s6", "s7"}, 0x12C: set(), 0x144: set(), 0x148: {"s9"}}
    assert 12 in before[2] and before[12] == [11]


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="needs ROCm's llvm-objdump")
def test_copies_into_lds_wait(tmp_path):
    if not os.path.exists(M._lib.LIB_PATH):
        pytest.skip("the library is not built")
    shutil.copy(M._lib.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    files = [f for f in os.listdir(tmp_path) if f.endswith("gfx950")]
    assert files
    copies, bad = 0, []
    for f in files:
        out = subprocess.run([OBJDUMP, "-d", f], cwd=tmp_path, check=True, capture_output=True, text=True).stdout
        for name, code, before in functions(out):
            for n, i in enumerate(code):
                if not i.copy:
                    continue
                copies += 1
                bad += [f"{name}+{i.addr:#x}: {r} of {w.name} {w.text}" for r, w in too_close(code, before, n)]
    assert copies > 500
    assert not bad, f"{len(bad)} of {copies}: " + "; ".join(bad[:5])
