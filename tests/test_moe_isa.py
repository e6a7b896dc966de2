"""CPU tests of the built instructions of the 8-bit float tiles (isa.py).  Their
loads into the LDS are assembly, which the compiler puts no wait states
around; their MFMAs are the compiler's own, and an empty assembly statement
that keeps each in its place must not hide a result from the waits for it."""
import os

import pytest

import block_scaled_gemm_02_amd as bsg
import isa

pytestmark = pytest.mark.skipif(not os.path.exists(isa.OBJDUMP), reason="no disassembler")


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    found = {n: b for n, b in isa.kernels(bsg.LIB_PATH, tmp_path_factory.mktemp("code")).items()
             if "3moe" in n and "k_fp8I" in n}
    # two formats of A, two types of C; three shapes in turn, two in runs, one in parts
    assert len(found) == 2 * 2 * 6
    for name, body in found.items():
        assert any(op.startswith("v_mfma_f32_16x16x128") for op, _ in body), name
    return found


def test_loads_set_their_own_m0(tiles):
    bad = {n: isa.m0_faults(b) for n, b in tiles.items()}
    assert not any(bad.values()), [(n, len(v), v[0]) for n, v in bad.items() if v][:3]


def test_loads_wait_for_their_descriptor(tiles):
    bad = {n: isa.sgpr_faults(b) for n, b in tiles.items()}
    assert not any(bad.values()), [(n, len(v), v[0]) for n, v in bad.items() if v][:3]


def test_results_are_read_when_they_are_there(tiles, monkeypatch):
    """A 16x16x128 MFMA is 8 passes long: its result is there after 12 wait states."""
    monkeypatch.setattr(isa, "MFMA_TO_OTHERS", 12)
    bad = {n: isa.mfma_faults(b) for n, b in tiles.items()}
    assert not any(bad.values()), [(n, len(v), v[0]) for n, v in bad.items() if v][:3]


def test_nothing_in_the_main_loop_goes_to_memory(tiles):
    """No register is spilled between the MFMAs of a tile's loop: scratch
    accesses count as loads, which the loop's waits count by number."""
    for name, body in tiles.items():
        mfmas = [i for i, (op, _) in enumerate(body) if op.startswith("v_mfma")]
        inside = [op for op, _ in body[mfmas[0]:mfmas[-1]] if op.startswith("scratch_")]
        assert not inside, (name, inside[:3])
