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
