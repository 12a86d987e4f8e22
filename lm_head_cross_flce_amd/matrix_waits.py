"""Checks compiled kernels for the waits that their matrix instructions need.

A matrix instruction must not issue within two wait states of a vector instruction that wrote one of its operands, nor
within four of one that wrote the execution mask; the hardware does not hold it back.  The compiler sees to that for its
own matrix instructions, but not for those in inline assembly, whose waits rest on where the register allocator puts
copies.  The build therefore reads each object's own gfx950 code and fails if any matrix instruction, on any way to it,
comes too soon.
"""

from __future__ import annotations

import os
import re
import subprocess
import tempfile
from typing import Dict, List, NamedTuple, Set, Tuple

OPERAND_WAITS, MASK_WAITS = 2, 4

_FUNCTION = re.compile(r"^[0-9a-f]+ <(.+)>:$")
_REGISTER = re.compile(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+)\b)")
_ADDRESS = re.compile(r"//\s*([0-9A-Fa-f]+):")
_TARGET = re.compile(r"<(.+?)(?:\+0x([0-9a-f]+))?>\s*$")


class Instruction(NamedTuple):
    op: str
    operands: str
    target: int    # a branch's address, or -1


def _registers(text: str) -> Set[Tuple[str, int]]:
    out = set()
    for kind, first, last, one in _REGISTER.findall(text):
        out.update((kind, i) for i in (range(int(first), int(last) + 1) if first else (int(one),)))
    return out


def functions(listing: str) -> Dict[str, Dict[int, Instruction]]:
    """Instructions by address, in order, of each function of an llvm-objdump listing."""
    out: Dict[str, Dict[int, Instruction]] = {}
    start: Dict[str, int] = {}
    here = name = None
    for line in listing.splitlines():
        m = _FUNCTION.match(line)
        if m:
            name, here = m[1], out.setdefault(m[1], {})
            start[name] = int(line.split(" ", 1)[0], 16)
            continue
        m = _ADDRESS.search(line)
        if here is None or not m:
            continue
        op, _, operands = line[:m.start()].strip().partition(" ")
        target = -1
        if op.startswith(("s_branch", "s_cbranch")):
            t = _TARGET.search(line)
            if t is None:
                raise ValueError(f"a branch without a target: {line.strip()}")
            target = start[t[1]] + int(t[2] or "0", 16)
        here[int(m[1], 16)] = Instruction(op, operands, target)
    return out


def _is_matrix(op: str) -> bool:
    return op.startswith(("v_mfma", "v_smfmac"))


def _writes(i: Instruction) -> Set[Tuple[str, int]]:
    """Vector registers that a vector instruction writes."""
    if not i.op.startswith("v_") or _is_matrix(i.op):
        return set()
    parts = re.split(r",\s*(?![^\[]*\])", i.operands)
    return _registers(" ".join(parts[:2] if "swap" in i.op else parts[:1]))


def _waits(i: Instruction) -> int:
    return int(i.operands.split()[0], 0) + 1 if i.op == "s_nop" else 1


def too_soon(listing: str) -> Tuple[int, List[str]]:
    """The number of matrix instructions, and a line for each that comes too soon after what it depends on."""
    count, found = 0, []
    for name, code in functions(listing).items():
        at = list(code)
        if not any(_is_matrix(code[a].op) for a in at):
            continue
        before: Dict[int, List[int]] = {a: [] for a in at}
        for prev, a in zip(at, at[1:]):
            if code[prev].op not in ("s_branch", "s_endpgm", "s_setpc_b64"):
                before[a].append(prev)
        for a in at:
            if code[a].target in before:
                before[code[a].target].append(a)
        for a in at:
            if not _is_matrix(code[a].op):
                continue
            count += 1
            reads = _registers(code[a].operands)   # the destination too: the accumulator is tied to it
            ways, seen = [(p, 0) for p in before[a]], {}
            while ways:
                p, waited = ways.pop()
                if waited >= MASK_WAITS or seen.get(p, MASK_WAITS) <= waited:
                    continue
                seen[p] = waited
                i = code[p]
                if (waited < OPERAND_WAITS and _writes(i) & reads) or i.op.startswith("v_cmpx"):
                    found.append(f"{name}: {i.op} {i.operands.strip()} {waited} wait states before "
                                 f"{code[a].op} {code[a].operands.strip()} at {a:#x}")
                    break
                ways.extend((q, waited + _waits(i)) for q in before[p])
    return count, found


def listing_of(obj: str, arch: str = "gfx950") -> str:
    """The device code of an object that hipcc has made from one of this package's sources ("": it has none)."""
    tools = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")
    with tempfile.TemporaryDirectory(prefix="flce_waits_") as tmp:
        bundle, code = os.path.join(tmp, "bundle"), os.path.join(tmp, "code")
        for cmd in ([os.path.join(tools, "llvm-objcopy"), "--dump-section", f".hip_fatbin={bundle}", obj,
                     os.path.join(tmp, "copy")],
                    [os.path.join(tools, "clang-offload-bundler"), "--type=o", "--unbundle", f"--input={bundle}",
                     f"--targets=hipv4-amdgcn-amd-amdhsa--{arch}", f"--output={code}"]):
            r = subprocess.run(cmd, capture_output=True, text=True)
            if "section '.hip_fatbin' not found" in r.stderr:
                return ""
            if r.returncode != 0:
                raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n{r.stdout}{r.stderr}")
        r = subprocess.run([os.path.join(tools, "llvm-objdump"), "-d", "--no-show-raw-insn", code], capture_output=True,
                           text=True)
        if r.returncode != 0:
            raise RuntimeError(f"llvm-objdump failed:\n{r.stderr}")
        return r.stdout


def check(obj: str) -> int:
    """Raises if a matrix instruction of the object comes too soon; returns how many it has."""
    count, found = too_soon(listing_of(obj))
    if found:
        raise RuntimeError(f"{len(found)} matrix instructions come too soon after a write of an operand:\n"
                           + "\n".join(found[:10]))
    return count
