"""The wait states in front of hand-written loads, checked on the built code.

A memory instruction may read a scalar register that a vector instruction wrote
(v_readlane, v_readfirstlane, a comparison) only 5 wait states later.  The
compiler sees to that for the instructions it makes itself, but does not look
into assembly statements, and it may bring a load's descriptor back from a
vector register in front of any of them.  Waiting inside each statement costs
the largest tile of the 8-bit float products, whose loads go out between its
matrix instructions, 1.5 to 2.5% (8192^3 427 -> 437 us).  So the build looks at
what the compiler made instead, and leaves no library where a wait is missing.

Every path is followed, loops included.  An instruction is one wait state,
s_nop N is N + 1.
"""
from __future__ import annotations

import os
import re
import struct
import subprocess
import tempfile

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
NEEDED = 5
MEMORY = ("buffer_", "global_", "scratch_", "flat_")

_LINE = re.compile(r"\t(\S+) *(.*?) *// ([0-9A-F]+):")
_HEAD = re.compile(r"[0-9a-f]+ <(.+)>:$")
_SCALAR = re.compile(r"\bs(?:\[(\d+):(\d+)\]|(\d+)\b)")


def code_objects(data: bytes):
    """The gfx950 code objects in a library's bytes: behind the magic a count,
    and for each entry its offset, size and target's name."""
    at = data.find(MAGIC)
    while at >= 0:
        p = at + len(MAGIC)
        count, = struct.unpack_from("<Q", data, p)
        p += 8
        for _ in range(count):
            off, size, n = struct.unpack_from("<QQQ", data, p)
            if b"gfx950" in data[p + 24:p + 24 + n] and size:
                yield data[at + off:at + off + size]
            p += 24 + n
        at = data.find(MAGIC, p)


def functions(code: bytes):
    """(name, [(address, operation, operands as a text)]) of a code object."""
    with tempfile.NamedTemporaryFile(suffix=".co") as f:
        f.write(code)
        f.flush()
        text = subprocess.run([OBJDUMP, "-d", f.name], check=True, capture_output=True, text=True).stdout
    name, body = None, []
    for line in text.splitlines():
        m = _LINE.match(line)
        if m:
            body.append((int(m[3], 16), m[1], m[2]))
            continue
        m = _HEAD.match(line)
        if m:
            if body:
                yield name, body
            name, body = m[1], []
    if body:
        yield name, body


def scalars(text: str):
    found = set()
    for m in _SCALAR.finditer(text):
        lo, hi = (m[1], m[2]) if m[1] else (m[3], m[3])
        found.update(range(int(lo), int(hi) + 1))
    return found


def _written(op: str, text: str):
    """The scalar registers that a vector instruction writes: its first operand,
    or the second where that is a carry."""
    args = text.split(",")
    found = scalars(args[0])
    if len(args) > 1 and ("_co_" in op or "div_scale" in op or op.startswith(("v_mad_u64", "v_mad_i64"))):
        found |= scalars(args[1])
    return found


def _targets(body, i):
    """The indexes that may follow instruction i."""
    at, op, text = body[i]
    if op == "s_endpgm":
        return []
    if op == "s_branch" or op.startswith("s_cbranch"):
        step = int(text.split()[0])
        to = at + 4 + 4 * (step - 0x10000 if step >= 0x8000 else step)
        return ([] if op == "s_branch" else [i + 1]) + [_index(body, to)]
    if op == "s_setpc_b64":
        # a far jump: s_getpc, s_add_u32, s_addc_u32 with the distance
        before = body[max(0, i - 3):i]
        if [b[1] for b in before] != ["s_getpc_b64", "s_add_u32", "s_addc_u32"]:
            raise RuntimeError(f"a jump to an unknown place at {at:#x}")
        start, step = before[0][0], int(before[1][2].split(",")[2], 0) & 0xFFFFFFFF
        return [_index(body, start + 4 + (step - (1 << 32) if step >= 1 << 31 else step))]
    if op.startswith(("s_swappc", "s_call")):
        raise RuntimeError(f"a call at {at:#x}")
    return [i + 1] if i + 1 < len(body) else []


def _index(body, address):
    lo, hi = 0, len(body)
    while lo < hi:
        mid = (lo + hi) // 2
        if body[mid][0] < address:
            lo = mid + 1
        else:
            hi = mid
    if lo == len(body) or body[lo][0] != address:
        raise RuntimeError(f"a jump to {address:#x}, which is no instruction")
    return lo


def faults(body):
    """[(address, operation, operands)] of the memory instructions of a function
    that come too soon behind a vector instruction that writes one of their
    scalar registers, on any path."""
    after = [_targets(body, i) for i in range(len(body))]
    heads = {0} | {t for i, ts in enumerate(after) for t in ts if ts != [i + 1]}
    bad, come = set(), {0: {}}          # come: register -> wait states since it was written, at a block's head
    work = [0]
    while work:
        i = work.pop()
        ages = dict(come[i])
        while True:
            _, op, text = body[i]
            if op.startswith(MEMORY) and ages and scalars(text) & ages.keys():
                bad.add(i)
            if ages:
                n = int(text, 0) + 1 if op == "s_nop" else 1
                ages = {r: a + n for r, a in ages.items() if a + n < NEEDED}
            if op.startswith("v_"):
                ages.update(dict.fromkeys(_written(op, text), 0))
            follow = after[i]
            if len(follow) == 1 and follow[0] == i + 1 and i + 1 not in heads:
                i += 1
                continue
            for t in follow:
                old = come.get(t)
                new = dict(ages) if old is None else {r: min(a, ages.get(r, NEEDED), old.get(r, NEEDED))
                                                      for r, a in {**old, **ages}.items()}
                if new != old:
                    come[t] = new
                    work.append(t)
            break
    return [body[i] for i in sorted(bad)]


def check(library: str) -> int:
    """Raises RuntimeError where a wait is missing in a built library; the
    number of functions that were looked at."""
    with open(library, "rb") as f:
        data = f.read()
    if not os.path.exists(OBJDUMP):
        raise RuntimeError(f"{OBJDUMP} is not there: the built loads' wait states cannot be checked")
    bad, seen = [], 0
    for code in code_objects(data):
        for name, body in functions(code):
            seen += 1
            bad += [(name, hex(at), op, text) for at, op, text in faults(body)]
    if bad:
        raise RuntimeError(f"{len(bad)} loads come too soon behind the vector instruction that writes their descriptor: "
                           + "; ".join(map(str, bad[:3])))
    return seen
