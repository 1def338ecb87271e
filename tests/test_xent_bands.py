"""Index arithmetic of the kept logits, compiled for the CPU from the header that the kernels include."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_gemm_elementwise_gb300", "csrc")
SOURCE = """
#include "xent_bands.h"
extern "C" {
int64_t band_of(int64_t V, int64_t units) { return ge::band_of(V, units); }
int64_t piece_of(int64_t T, int64_t V, int64_t bytes) { return ge::piece_of(T, V, bytes); }
int64_t slots_of(int64_t V, int64_t band, int64_t bn) { return ge::slots_of(V, band, bn); }
int slot_of(int c, int N, int band, int band_tiles, int bn) { return ge::slot_of(c, N, band, band_tiles, bn); }
int keeps(int n0, int c0, int width, int keep_cols) { return ge::keeps(n0, c0, width, keep_cols); }
}
"""
BN, PART = 128, 32  # columns of a band's tile, at most, and of what is kept together


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("bands")
    src, so = d / "bands.cpp", d / "bands.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-O2", "-Wall", "-fPIC", "-shared", "-I", CSRC, "-o", str(so), str(src)], check=True)
    L = ctypes.CDLL(str(so))
    for f, n in ((L.band_of, 2), (L.piece_of, 3), (L.slots_of, 3)):
        f.restype, f.argtypes = ctypes.c_int64, [ctypes.c_int64] * n
    L.slot_of.argtypes = [ctypes.c_int] * 5
    L.keeps.argtypes = [ctypes.c_int] * 4
    return L


def tiles(V, band):
    """(unit, first column, width) of every tile of every band, as the kernel deals them."""
    for unit in range(-(-V // band)):
        for i in range(-(-min(band, V - unit * band) // BN)):
            yield unit, unit * band + i * BN, min(BN, band - i * BN)


VOCABULARIES = [1, 31, 300, 1024, 4864, 5000, 10000, 10240, 32000, 32768, 50257, 51200, 65536, 131072, 262144]


def shapes(lib, units):
    """(V, band, piece) of 64 rows over real and odd vocabularies, with the default buffer, none, and a small one."""
    for V in VOCABULARIES:
        for bytes_ in (1 << 29, 1, 128 * 2 * 1024):
            yield V, lib.band_of(V, units), lib.piece_of(64, V, bytes_)


@pytest.mark.parametrize("units", [1, 5, 6, 19, 148, 152])
def test_kept_columns_stay_in_their_row_and_are_written_once(lib, units):
    for V, band, piece in shapes(lib, units):
        check_kept(lib, units, V, band, piece)


def check_kept(lib, units, V, band, piece):
    assert band % PART == 0 and band * units >= V and piece % 256 == 0 and piece * -(-V // piece) >= V
    keep_cols = min(piece, -(-V // 256) * 256)
    seen = set()
    for _, n0, width in tiles(V, band):
        for c0 in range(0, BN, PART):
            if lib.keeps(n0, c0, width, keep_cols):
                assert n0 + c0 + PART <= piece, (n0, c0, width, piece)
                assert n0 + c0 not in seen
                seen.add(n0 + c0)
    assert seen >= set(range(0, min(V, keep_cols), PART))


@pytest.mark.parametrize("units", [0, 1, 5, 6, 19, 148, 152])
def test_every_column_has_the_range_its_tile_left(lib, units):
    """units 0: no bands, tiles of 128 and of 256 columns."""
    for V, band, piece in shapes(lib, max(units, 1)):
        for bn in (BN,) if units else (BN, 256):
            band = band if units else 0
            slots, per = lib.slots_of(V, band, bn), -(-band // bn)
            N = min(piece, V)  # columns of the piece; whole multiples of 256 are converted, a lane's 8 at a time
            for c in range(0, -(-N // 256) * 256, 8):
                slot = lib.slot_of(c, N, band, per, bn)
                assert 0 <= slot < slots, (V, band, bn, c)
                if c < N:
                    unit, of = (c // band, c % band) if band else (0, c)
                    assert slot == 2 * (unit * per + of // bn) + of // 64 % 2
