"""CPU walk over the tiled kernel's copies of the feed-forward operators (no GPU).

csrc/tile_copy.hpp holds the address arithmetic of those copies as plain constexpr C++.  It is
compiled here and every lane's 16 bytes of every tile and k-tile (those past the sum's end,
which the pipeline also asks for, among them) are checked against the operand:

  * no dword that the buffer resource lets through lies outside the operand.  The resource of
    register-staged rows starts 16 bytes before a tile's first row, so in front of the operand
    it is the offsets alone that keep the loads inside;
  * register-staged chunks, after their shift, hold the row's bytes and zeros past its end.
"""

import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

DRIVER = r"""
#include "tile_copy.hpp"
using namespace spg;

static const int64_t kBase = (int64_t)1 << 40;

static uint8_t byte_at(int64_t i) { return (uint8_t)(1 + i % 251); }

// one lane: 0 if every dword that is let through lies in [0, size), else 1; got: the 16 bytes
static int load(const Win& w, uint32_t off, int64_t size, uint8_t* got) {
    for (int d = 0; d < 16; d += 4) {
        for (int e = 0; e < 4; ++e) got[d + e] = 0;
        const uint32_t o = off + (uint32_t)d;
        if (off >= kMasked || o >= w.n) continue;
        const int64_t at = (int64_t)(w.p + o) - kBase;
        if (at < 0 || at + 4 > size) return 1;
        for (int e = 0; e < 4; ++e) got[d + e] = byte_at(at + e);
    }
    return 0;
}

static void shift_down(uint8_t* b, uint32_t bits) {
    const int n = (int)bits / 8;
    for (int i = 0; i < 16; ++i) b[i] = i + n < 16 ? b[i + n] : 0;
}

// An operand of `rows` rows along the reduction: `segments` segments of `bytes` bytes (`skip`
// bytes from one to the next), rows `pitch` bytes apart.  0, or 1: outside, 2: wrong bytes.
template <bool REG, bool WHOLE>
static int rows_of(int64_t rows, int64_t bytes, int64_t skip, int segments, int64_t pitch, int tile) {
    using C = RowCopy<REG, WHOLE>;
    // direct copies read whole words: rows of whole words, or laid out again
    const int64_t row_bytes = WHOLE ? pitch : REG ? bytes : (bytes + 3) / 4 * 4;
    const int64_t size = (rows - 1) * pitch + row_bytes;
    const int seg_kt = (int)((bytes + 127) / 128), tail = (int)(bytes - (seg_kt - 1) * 128);
    if (segments > 1 && skip != seg_kt * 128) return 3;
    for (int64_t m0 = 0; m0 < rows; m0 += tile) {
        const int64_t here = rows - m0 < tile ? rows - m0 : tile;
        const uint64_t at = (uint64_t)(kBase + m0 * pitch) - C::kBack;
        const uint32_t all = (uint32_t)((here - 1) * pitch + row_bytes) + C::kBack;
        for (int kt = 0; kt < seg_kt * segments + 4; ++kt) {
            const bool in = kt < seg_kt * segments;
            const int lim = C::limit(WHOLE ? kt : kt % seg_kt, seg_kt, tail);
            const Win w = C::window(at, all, kt, in);
            for (int r = 0; r < tile; ++r)
                for (int pos = 0; pos < 128; pos += 16) {
                    uint8_t got[16];
                    const uint32_t off = C::offset((uint32_t)r * (uint32_t)pitch + (uint32_t)pos + C::kBack, pos, lim);
                    if (load(w, off, size, got)) return 1;
                    if (!REG || !in || r >= here) continue;
                    shift_down(got, C::shift(pos, lim));
                    for (int e = 0; e < 16; ++e) {
                        const int64_t src = (m0 + r) * pitch + (int64_t)kt * 128 + pos + e;
                        if (got[e] != (pos + e < lim ? byte_at(src) : 0)) return 2;
                    }
                }
        }
    }
    return 0;
}

// `rows` rows across the reduction of `cols` 16-bit columns, `pitch` bytes apart, the operand
// `first` bytes into its memory (the second half of a two-part matrix)
template <bool REG>
static int columns_of(int64_t rows, int64_t cols, int64_t pitch, int64_t first, int tile) {
    using C = ColumnCopy<REG>;
    const int64_t end = first ? rows * pitch : (rows - 1) * pitch + (REG ? cols * 2 : (cols * 2 + 3) / 4 * 4);
    const int nkt = (int)((rows + 63) / 64);
    for (int64_t n0 = 0; n0 < cols; n0 += tile)
        for (int kt = 0; kt < nkt + 4; ++kt) {
            const Win w = C::window((uint64_t)(kBase + first), (uint32_t)pitch, (int)rows, kt, kt < nkt);
            for (int r = 0; r < 64; ++r)
                for (int col = 0; col < tile; col += 8) {
                    uint8_t got[16];
                    const int over = C::over((int)n0 + col, (int)cols);
                    const uint32_t off = C::offset(r, (uint32_t)pitch, (int)n0 + col, over);
                    if (load(w, off, end, got)) return 1;
                    if (!REG || kt * 64 + r >= rows || over >= 8) continue;
                    shift_down(got, C::shift(over));
                    for (int e = 0; e < 16; ++e) {
                        const int64_t c = (n0 + col) * 2 + e;
                        if (got[e] != (c < cols * 2 ? byte_at(first + (int64_t)(kt * 64 + r) * pitch + c) : 0)) return 2;
                    }
                }
        }
    return 0;
}

extern "C" int walk_rows(int reg, int whole, int64_t rows, int64_t bytes, int64_t skip, int segments, int64_t pitch, int tile) {
    if (reg) return whole ? rows_of<true, true>(rows, bytes, skip, segments, pitch, tile)
                          : rows_of<true, false>(rows, bytes, skip, segments, pitch, tile);
    return whole ? rows_of<false, true>(rows, bytes, skip, segments, pitch, tile)
                 : rows_of<false, false>(rows, bytes, skip, segments, pitch, tile);
}

extern "C" int walk_columns(int reg, int64_t rows, int64_t cols, int64_t pitch, int64_t first, int tile) {
    return reg ? columns_of<true>(rows, cols, pitch, first, tile) : columns_of<false>(rows, cols, pitch, first, tile);
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("tile_copy")
    src, out = d / "walk.cpp", d / "walk.so"
    src.write_text(DRIVER)
    inc = os.path.join(ROOT, "software_pipelined_tiled_gemm_amd", "csrc")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-shared", "-fPIC", "-I", inc, str(src), "-o", str(out)], check=True)
    L = ctypes.CDLL(str(out))
    i, q = ctypes.c_int, ctypes.c_int64
    L.walk_rows.argtypes = [i, i, q, q, q, i, q, i]
    L.walk_columns.argtypes = [i, q, q, q, q, i]
    return L


def up(v, a):
    return (v + a - 1) // a * a


LENGTHS = list(range(1, 20)) + [31, 33, 63, 64, 65, 71, 72, 127, 128, 130, 200]
TILES = (64, 128, 256)


@pytest.mark.parametrize("reg", [0, 1])
def test_slopes_as_the_two_segment_operand(walk, reg):
    # dG and dU side by side, N from 1: rows of 2 np elements, each half padded to a k-tile
    for N in LENGTHS:
        np_ = up(N, 64)
        for M in (1, 9, 64, 130):
            for tile in TILES:
                assert walk.walk_rows(reg, 1, M, N * 2, np_ * 2, 2, np_ * 4, tile) == 0, (N, M, tile)


def test_the_walk_finds_loads_in_front_of_the_operand(walk):
    # as ordinary rows the slopes' first chunk of N < 8 would be moved to before the matrix
    for N in range(1, 8):
        assert walk.walk_rows(1, 0, 9, N * 2, 128, 2, 256, 64) == 1, N
    assert walk.walk_rows(1, 0, 9, 16, 0, 1, 16, 64) == 0


@pytest.mark.parametrize("reg", [0, 1])
def test_rows_along_the_reduction(walk, reg):
    # X, the weights and int8 operands: rows from the 16 bytes that the tiled kernels take; on
    # any byte when staged, on words (with their padding, when laid out again) when copied
    for bytes_ in [n + 15 for n in LENGTHS] + [256, 257, 258]:
        for rows in (1, 3, 64, 70, 259):
            for tile in TILES:
                for pitch in (bytes_,) if reg else ({bytes_ if bytes_ % 4 == 0 else up(bytes_, 128), up(bytes_, 128)}):
                    assert walk.walk_rows(reg, 0, rows, bytes_, 0, 1, pitch, tile) == 0, (bytes_, rows, tile, pitch)


@pytest.mark.parametrize("reg", [0, 1])
def test_rows_across_the_reduction(walk, reg):
    for cols in [n + 7 for n in LENGTHS]:
        for rows in (1, 2, 63, 64, 65, 130):
            for tile in TILES:
                for pitch in (cols * 2,) if reg else ({cols * 2 if cols % 2 == 0 else up(cols * 2, 128), up(cols * 2, 128)}):
                    assert walk.walk_columns(reg, rows, up(cols, 8) if pitch != cols * 2 else cols, pitch, 0, tile) == 0, (
                        cols, rows, tile, pitch)
    # dG and dU as an operand of the weights' gradients: both halves, N from 1
    for N in LENGTHS:
        np_ = up(N, 64)
        for rows in (1, 9, 64, 130):
            for tile in TILES:
                for first in (0, np_ * 2):
                    assert walk.walk_columns(reg, rows, np_, np_ * 4, first, tile) == 0, (N, rows, tile, first)
