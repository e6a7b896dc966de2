"""The gfx950 instructions of the built library, and the wait states that its
hand-written ones need.  The compiler inserts waits around the instructions it
makes itself, but does not look into assembly statements, so what those rely
on is checked on the code that was built.

Wait states: an instruction is one, s_nop N is N + 1.
"""
import os
import re
import struct
import subprocess

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects(library):
    """The gfx950 code objects inside a shared library, as bytes: after the
    magic a count, and for each entry its offset, size and target's name."""
    data = open(library, "rb").read()
    at = data.find(MAGIC)
    while at >= 0:
        p = at + len(MAGIC)
        count, = struct.unpack_from("<Q", data, p)
        p += 8
        for _ in range(count):
            off, size, n = struct.unpack_from("<QQQ", data, p)
            name = data[p + 24:p + 24 + n]
            p += 24 + n
            if b"gfx950" in name and size:
                yield data[at + off:at + off + size]
        at = data.find(MAGIC, p)


def kernels(library, tmp):
    """{symbol: [(operation, [operands])]} of every function in the library."""
    out = {}
    for i, code in enumerate(code_objects(library)):
        path = os.path.join(str(tmp), f"{i}.co")
        with open(path, "wb") as f:
            f.write(code)
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", path], check=True,
                              capture_output=True, text=True).stdout
        body = None
        for line in text.splitlines():
            m = re.match(r"(?:[0-9a-f]+ )?<(.+)>:$", line)
            if m:
                body = out.setdefault(m[1], [])
                continue
            line = line.split("//")[0].strip()
            if body is None or not line:
                continue
            op, *rest = line.split(None, 1)
            body.append((op, [a.strip() for a in rest[0].split(",")] if rest else []))
    return out


def registers(operand):
    """The registers of an operand: {("v", 3), ...}."""
    found = set()
    for m in re.finditer(r"\b([vas])(?:\[(\d+):(\d+)\]|(\d+)\b)", operand):
        lo, hi = (m[2], m[3]) if m[2] else (m[4], m[4])
        found |= {(m[1], i) for i in range(int(lo), int(hi) + 1)}
    return found


def states(op, args):
    return int(args[0], 0) + 1 if op == "s_nop" else 1


def m0_faults(body):
    """Loads into the LDS that do not come right behind the setting of M0, their LDS address,
    with one wait state between: an s_nop 0, or an MFMA of the same statement."""
    bad = []
    for i, (op, args) in enumerate(body):
        if op.startswith("buffer_load") and any("lds" in a.split() for a in args):
            before = [(o, a[:1]) for o, a in body[max(0, i - 2):i]]
            if before[0] not in (("s_mov_b32", ["m0"]), ("s_add_u32", ["m0"])) or not (before[-1] == ("s_nop", ["0"]) or before[-1][0].startswith("v_mfma")):
                bad.append((i, before, op))
    return bad


# A vector instruction's result is there for an MFMA after 2 wait states, and
# an MFMA's for anything but the MFMA that adds to the same registers after 18
# (the longest ones; those of 16 x 16 take fewer).  A scalar register that a
# vector instruction wrote is there for a memory instruction after 5.
VALU_TO_MFMA, MFMA_TO_OTHERS, VALU_SGPR_TO_MEMORY = 2, 18, 5


def _all(args):
    return set().union(*map(registers, args)) if args else set()


def mfma_faults(body):
    """MFMAs too soon behind a vector instruction that writes an operand, and
    instructions that touch an MFMA's result too soon."""
    bad, now, written, results = [], 0, {}, {}
    for i, (op, args) in enumerate(body):
        if op.startswith("v_mfma"):
            for r in _all(args[1:4]):
                if now - written.get(r, -100) < VALU_TO_MFMA:
                    bad.append((i, op, r))
            # the exact accumulator may follow itself; another overlap may not
            for r in _all(args[1:4]) & results.keys():
                t, whole = results[r]
                if now - t < MFMA_TO_OTHERS and not (r in registers(args[3]) and whole == args[3] == args[0]):
                    bad.append((i, op, r))
            now += 1
            results.update(dict.fromkeys(registers(args[0]), (now, args[0])))
            continue
        for r in _all(args) & results.keys():
            if now - results[r][0] < MFMA_TO_OTHERS:
                bad.append((i, op, r))
        now += states(op, args)
        if op.startswith("v_") and args:
            written.update(dict.fromkeys(registers(args[0]), now))
    return bad


def sgpr_faults(body):
    """Buffer instructions too soon behind a vector instruction that writes
    one of their scalar registers."""
    bad, now, written = [], 0, {}
    for i, (op, args) in enumerate(body):
        if op.startswith("buffer_"):
            for r in _all(args):
                if now - written.get(r, -100) < VALU_SGPR_TO_MEMORY:
                    bad.append((i, op, r))
        now += states(op, args)
        if op.startswith("v_") and args:
            written.update(dict.fromkeys([r for r in registers(args[0]) if r[0] == "s"], now))
    return bad
