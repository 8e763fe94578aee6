"""Build-time check of the direct loads into LDS (buffer_load ... lds).

A vector instruction that writes a scalar register (a lane read that brings a
spilled descriptor back, a comparison) has to be at least five wait states
before a vector memory instruction that reads the register; with fewer it may
read the old value, another tile's descriptor say.  The compiler keeps that
distance for its own loads but does not look into inline assembly, where the
BF16 products make theirs.  Five wait states in each such load would cost these
products 1 to 3 per cent, so the built code is checked instead: from every
direct load back along every path that leads to it.
"""
import os
import re
import shutil
import subprocess
import tempfile

WAIT_STATES = 5
OBJDUMP = os.environ.get("LLVM_OBJDUMP", "/opt/rocm/llvm/bin/llvm-objdump")

_FUNC = re.compile(r"^([0-9a-f]+) <(\S+)>:$")
_INST = re.compile(r"^\s+(\S.*?)\s*// ([0-9A-F]+): ((?:[0-9A-F]{8} ?)+)")
_LOAD = re.compile(r"^buffer_load_dword\S*\s.*\blds$")
_SREG = re.compile(r"\b(vcc_lo|vcc_hi|vcc|m0|s\d+|s\[\d+:\d+\])(?![\w\[])")
_NO_FALL = ("s_branch", "s_endpgm", "s_setpc_b64", "s_trap")


def _sregs(operands):
    """The scalar registers that a list of operands names."""
    out = set()
    for r in _SREG.findall(operands):
        if r == "vcc":
            out |= {"vcc_lo", "vcc_hi"}
        elif r.startswith("s["):
            a, b = r[2:-1].split(":")
            out |= {f"s{i}" for i in range(int(a), int(b) + 1)}
        else:
            out.add(r)
    return out


def _split(text):
    op, _, rest = text.partition(" ")
    return op, [o.strip() for o in rest.split(",")]


def _valu_writes(text):
    """The scalar registers that a vector ALU instruction writes (none of another instruction)."""
    op, ops = _split(text)
    if not op.startswith("v_"):
        return set()
    w = _sregs(ops[0])
    if len(ops) > 1 and re.match(r"v_(add|sub|subrev|addc|subb|subbrev)_co_|v_div_scale_|v_mad_[ui]64_", op):
        w |= _sregs(ops[1])          # their second result: the carry, or the flag
    return w


def violations(listing):
    """Of a disassembly of one code object: (direct loads, [description of each that follows too closely])."""
    found, loads = [], 0
    name, code = None, []            # of the function being read: (address, size, text)

    def end():
        nonlocal loads
        at = {a: i for i, (a, _, _) in enumerate(code)}
        before = [[] for _ in code]
        for i, (a, size, text) in enumerate(code):
            op, ops = _split(text)
            if op.startswith(("s_cbranch", "s_branch")):
                n = int(ops[-1])
                to = a + 4 + 4 * (n - 65536 if n >= 32768 else n)
                if to in at:
                    before[at[to]].append(i)
            if i + 1 < len(code) and not op.startswith(_NO_FALL):
                before[i + 1].append(i)
        for i, (a, _, text) in enumerate(code):
            if not _LOAD.match(text):
                continue
            loads += 1
            need = _sregs(",".join(_split(text)[1][1:])) | {"m0"}
            todo, seen = [(j, 0, frozenset(need)) for j in before[i]], set()
            while todo:
                j, states, regs = todo.pop()
                if (j, states, regs) in seen or states >= WAIT_STATES:
                    continue
                seen.add((j, states, regs))
                t = code[j][2]
                hit = _valu_writes(t) & regs
                if hit:
                    found.append(f"{name}: '{text}' at {a:x}, {states} wait states after '{t}'")
                    continue
                op, ops = _split(t)
                if op == "s_mov_b32" and ops[0] == "m0":
                    regs = regs - {"m0"}      # (written anew by the scalar ALU)
                n = int(ops[0]) + 1 if op == "s_nop" else 1
                todo += [(k, states + n, regs) for k in before[j]]

    for line in listing.splitlines():
        m = _FUNC.match(line)
        if m:
            end()
            name, code = m.group(2), []
            continue
        m = _INST.match(line)
        if m:
            code.append((int(m.group(2), 16), 4 * len(m.group(3).split()), m.group(1)))
    end()
    return loads, found


def check(lib):
    """Raise if a direct load of the library's code objects follows too closely; -> how many loads were checked."""
    if not os.path.exists(OBJDUMP):
        raise RuntimeError(f"{OBJDUMP}: needed to check the built code (set LLVM_OBJDUMP)")
    tmp = tempfile.mkdtemp(prefix="moe4_check_")
    try:
        shutil.copy(lib, os.path.join(tmp, "lib"))
        subprocess.run([OBJDUMP, "--offloading", "lib"], cwd=tmp, check=True, stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
        total, bad = 0, []
        for f in sorted(os.listdir(tmp)):
            if "amdgcn" not in f:
                continue
            text = subprocess.run([OBJDUMP, "-d", f], cwd=tmp, check=True, capture_output=True, text=True).stdout
            n, found = violations(text)
            total += n
            bad += found
    finally:
        shutil.rmtree(tmp, ignore_errors=True)
    if bad:
        raise RuntimeError("direct loads too close behind a write of their scalar registers:\n" + "\n".join(bad))
    return total
