"""CPU tests of the check that every build makes of its loads' wait states
(block_scaled_gemm_02_amd/wait_states.py)."""
import os
import stat

import pytest

import block_scaled_gemm_02_amd as bsg
from block_scaled_gemm_02_amd import build, wait_states

LOAD = ("buffer_load_dwordx4", "v1, s[4:7], 0 offen lds")
FILL = ("v_add_f32_e32", "v2, v3, v4")
END = ("s_endpgm", "")


def body(*code):
    """Instructions of 4 bytes each; a branch names the index it goes to."""
    out = []
    for i, (op, text) in enumerate(code):
        if op == "s_branch" or op.startswith("s_cbranch"):
            text = f"{(text - i - 1) & 0xFFFF} <somewhere>"
        out.append((0x100 + 4 * i, op, text))
    return out


def found(*code):
    return [(at - 0x100) // 4 for at, _, _ in wait_states.faults(body(*code))]


@pytest.mark.parametrize("write", [("v_readlane_b32", "s5, v9, 3"), ("v_readfirstlane_b32", "s7, v9"),
                                   ("v_cmp_lt_u32_e64", "s[6:7], v0, v1"), ("v_addc_co_u32_e64", "v0, s[4:5], v1, v2, vcc")])
def test_five_wait_states(write):
    for n in range(7):
        assert found(write, *[FILL] * n, LOAD, END) == ([n + 1] if n < 5 else [])
    assert found(write, ("s_nop", "3"), LOAD, END) == [2] and found(write, ("s_nop", "4"), LOAD, END) == []
    assert found(write, ("s_nop", "2"), ("s_mov_b32", "m0, s2"), ("s_nop", "0"), LOAD, END) == []


def test_what_is_no_fault():
    assert found(("v_readlane_b32", "s8, v9, 3"), LOAD, END) == []            # another register
    assert found(("s_mov_b32", "s5, s1"), LOAD, END) == []                    # a scalar instruction wrote it
    assert found(("v_writelane_b32", "v9, s5, 3"), LOAD, END) == []           # read, not written
    assert found(("v_readlane_b32", "s5, v9, 3"), END, LOAD, END) == []       # never comes there


def test_around_a_loop():
    """The write at a loop's end, the load at its beginning."""
    loop = [FILL, LOAD, *[FILL] * 8, ("v_readlane_b32", "s5, v9, 3"), ("s_cbranch_scc1", 0), END]
    assert found(*loop) == [1]
    assert found(*[FILL] * 3, *loop[1:11], ("s_cbranch_scc1", 0), END) == [3]
    assert found(*[FILL] * 4, *loop[1:11], ("s_cbranch_scc1", 0), END) == []


def test_the_shorter_path_counts():
    assert found(("v_readlane_b32", "s5, v9, 3"), ("s_cbranch_vccz", 4), ("s_nop", "7"), FILL, LOAD, END) == [4]
    assert found(("s_cbranch_vccz", 3), ("v_readlane_b32", "s5, v9, 3"), ("s_branch", 5), ("s_nop", "7"), FILL, LOAD, END) == [5]
    assert found(("v_readlane_b32", "s5, v9, 3"), ("s_branch", 3), LOAD, FILL, FILL, FILL, LOAD, END) == [6]
    assert found(("v_readlane_b32", "s5, v9, 3"), ("s_branch", 3), LOAD, FILL, FILL, FILL, FILL, LOAD, END) == []


def test_far_jumps_are_followed():
    def jump(distance):
        return found(("v_readlane_b32", "s5, v9, 3"), ("s_getpc_b64", "s[10:11]"), ("s_add_u32", f"s10, s10, {distance}"),
                     ("s_addc_u32", "s11, s11, 0"), ("s_setpc_b64", "s[10:11]"), END, FILL, LOAD, END)

    assert jump("0x14") == [7]          # from 0x108 to the load: four instructions between
    assert jump("0x10") == []           # to the one before it
    assert jump("0x18") == []           # past it
    with pytest.raises(RuntimeError):
        found(FILL, FILL, FILL, FILL, ("s_setpc_b64", "s[10:11]"), END)
    with pytest.raises(RuntimeError):
        found(("s_setpc_b64", "s[10:11]"), END)
    with pytest.raises(RuntimeError):
        found(("s_swappc_b64", "s[0:1], s[2:3]"), END)


@pytest.mark.skipif(not os.path.exists(wait_states.OBJDUMP), reason="no disassembler")
def test_built_library():
    assert wait_states.check(bsg.LIB_PATH) > 300


def linker(path):
    """A compiler that links a library of nothing."""
    path.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\necho nothing > "$2"\n')
    path.chmod(path.stat().st_mode | stat.S_IXUSR)
    return str(path)


def test_a_build_with_a_fault_leaves_no_library(tmp_path, monkeypatch):
    monkeypatch.setattr(build, "HIPCC", linker(tmp_path / "cc"))
    monkeypatch.setattr(build, "sources", lambda: ["nothing"])
    monkeypatch.setattr(build, "_compile", lambda src: src)
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "b"))
    out = tmp_path / "lib.so"
    monkeypatch.setattr(build, "OUT", str(out))
    assert build.build(verbose=False) == str(out) and out.exists()
    out.unlink()
    bad = body(("v_readlane_b32", "s5, v9, 3"), LOAD, END)
    monkeypatch.setattr(wait_states, "code_objects", lambda data: [b""])
    monkeypatch.setattr(wait_states, "functions", lambda code: [("f", bad)])
    with pytest.raises(RuntimeError, match="1 loads come too soon"):
        build.build(verbose=False)
    assert not out.exists()
    monkeypatch.setattr(wait_states, "OBJDUMP", str(tmp_path / "none"))
    with pytest.raises(RuntimeError, match="cannot be checked"):
        build.build(verbose=False)
