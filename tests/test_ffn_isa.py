"""CPU tests of the feed-forward tiles' built instructions (isa.py)."""
import os

import pytest

import block_scaled_gemm_02_amd as bsg
import isa

pytestmark = pytest.mark.skipif(not os.path.exists(isa.OBJDUMP), reason="no disassembler")
TILES = ("k_i8I", "k_gluI", "k_dxI", "k_dwI", "k_dxwI")


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    """The instructions of every kernel built on the tile."""
    found = {n: b for n, b in isa.kernels(bsg.LIB_PATH, tmp_path_factory.mktemp("code")).items()
             if "3ffn" in n and any(t in n for t in TILES)}
    for t in TILES:
        assert any(t in n for n in found), t
    for name, body in found.items():
        assert any(op.startswith("v_mfma") for op, _ in body), name
    return found


def test_loads_set_their_own_m0(tiles):
    """A load into the LDS takes its address from M0.  Nothing may come
    between the two, since the compiler is free to use M0 itself."""
    bad = {n: isa.m0_faults(b) for n, b in tiles.items()}
    assert not any(bad.values()), [(n, len(v), v[0]) for n, v in bad.items() if v][:3]


def test_mfmas_wait_for_their_operands(tiles):
    """The MFMAs are assembly, whose operands and results the compiler does
    not put wait states around."""
    bad = {n: isa.mfma_faults(b) for n, b in tiles.items()}
    assert not any(bad.values()), [(n, len(v), v[0]) for n, v in bad.items() if v][:3]


def test_loads_wait_for_their_descriptor(tiles):
    bad = {n: isa.sgpr_faults(b) for n, b in tiles.items()}
    assert not any(bad.values()), [(n, len(v), v[0]) for n, v in bad.items() if v][:3]


def code(text):
    return [(line.split(None, 1)[0], [a.strip() for a in line.split(None, 1)[1].split(",")] if " " in line.strip() else [])
            for line in map(str.strip, text.strip().splitlines())]


MFMA = "v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]\n"
LDS = "buffer_load_dwordx4 v9, s[4:7], 0 offen lds\n"


@pytest.mark.parametrize("check,text,faults", [
    # M0 and the load
    (isa.m0_faults, "s_mov_b32 m0, s1\ns_nop 0\n" + LDS, 0),
    (isa.m0_faults, "s_add_u32 m0, s1, 0x400\n" + MFMA + LDS, 0),
    (isa.m0_faults, "s_mov_b32 m0, s1\n" + LDS, 1),
    (isa.m0_faults, "s_mov_b32 m0, s1\n" + MFMA + "ds_read_b128 v[8:11], v1\n" + LDS, 1),
    (isa.m0_faults, "buffer_load_dwordx4 v[8:11], v9, s[4:7], 0 offen\n", 0),
    # a source written one or two wait states before
    (isa.mfma_faults, "v_add_u32_e32 v5, v8, v9\ns_nop 1\n" + MFMA, 0),
    (isa.mfma_faults, "v_add_u32_e32 v5, v8, v9\ns_nop 0\n" + MFMA, 1),
    (isa.mfma_faults, "v_accvgpr_write_b32 a2, v8\n" + MFMA, 1),
    (isa.mfma_faults, "v_add_u32_e32 v8, v8, v9\n" + MFMA, 0),
    # a result read too soon; the same accumulator may follow at once
    (isa.mfma_faults, MFMA + MFMA, 0),
    (isa.mfma_faults, MFMA + "v_accvgpr_read_b32 v8, a3\n", 1),
    (isa.mfma_faults, MFMA + "s_nop 15\ns_nop 1\nv_accvgpr_read_b32 v8, a3\n", 0),
    (isa.mfma_faults, MFMA + "v_mfma_f32_16x16x32_bf16 a[2:5], v[0:3], v[4:7], a[2:5]\n", 2),
    (isa.mfma_faults, MFMA + "v_mfma_f32_16x16x32_bf16 a[4:7], v[0:3], a[0:3], a[4:7]\n", 4),
    # a descriptor written by a vector instruction
    (isa.sgpr_faults, "v_readfirstlane_b32 s6, v1\ns_nop 4\n" + LDS, 0),
    (isa.sgpr_faults, "v_readfirstlane_b32 s6, v1\ns_nop 3\n" + LDS, 1),
    (isa.sgpr_faults, "s_mov_b32 s6, s1\n" + LDS, 0)])
def test_the_checks_find_what_they_look_for(check, text, faults):
    assert len(check(code(text))) == faults
