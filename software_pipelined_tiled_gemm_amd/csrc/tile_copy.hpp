// Addresses of the feed-forward operators' tile copies: which bytes of an operand a lane
// loads for its 16 bytes of a k-tile.  Plain constexpr C++ (no HIP), so that a CPU test
// compiles these very functions and walks every copy of an operand.
#pragma once

#include <stdint.h>

namespace spg {

constexpr uint32_t kMasked = 0x80000000u;   // buffer offset past any resource: loads 0

// Start and size of a buffer resource.
struct Win {
    uint64_t p;
    uint32_t n;
};

// Rows that lie along the reduction, 128 bytes of each a k-tile.  `lim`: bytes of the k-tile
// that exist; a chunk past them is masked.
// REG (any alignment): the chunk that straddles `lim` is loaded from the 16 bytes that end
// there and shifted, so that nothing past a row is read; they may begin before the k-tile, so
// the resource starts 16 bytes early.  In the row's only k-tile they would begin before the
// row, and in the operand's first row before the operand, if the row were shorter than 16
// bytes: only for rows of at least that.
// WHOLE: rows padded with zeros to whole k-tiles (dG and dU, whose N may be 1): every chunk
// exists, and nothing is masked, moved or shifted.
template <bool REG, bool WHOLE>
struct RowCopy {
    static constexpr uint32_t kBack = REG && !WHOLE ? 16u : 0u;
    // bytes of k-tile k (of seg_kt of a segment, the last `tail` bytes long) that exist
    static constexpr int limit(int k, int seg_kt, int tail) { return !WHOLE && k == seg_kt - 1 ? tail : 128; }
    // the resource of k-tile k: `at` the tile's first row less kBack, `all` the bytes from there
    // to the end of its last row; nothing (reads zero) where the k-tile is not `in` the sum
    static constexpr Win window(uint64_t at, uint32_t all, int k, bool in) {
        return Win{at + (uint32_t)k * 128u, in ? all - (uint32_t)k * 128u : 0u};
    }
    // offset in it for the chunk at byte `pos` of a row's k-tile, `off` (with kBack) unmasked
    static constexpr uint32_t offset(uint32_t off, int pos, int lim) {
        if (kBack) off -= pos + 16 > lim ? (uint32_t)(pos + 16 - lim) : 0u;
        return pos >= lim ? kMasked : off;
    }
    // bits to shift the loaded chunk down by
    static constexpr uint32_t shift(int pos, int lim) {
        return kBack && pos < lim && pos + 16 > lim ? 8u * (uint32_t)(pos + 16 - lim) : 0u;
    }
};

// Rows that lie across the reduction, 64 of them a k-tile.  `over`: columns of a lane's chunk
// (8 of 16 bits from column `col`) past the last.
template <bool REG>
struct ColumnCopy {
    static constexpr int over(int col, int cols) { return col + 8 - cols; }
    // the resource of k-tile k of `rows` rows; nothing where it is not `in` the sum.  Written
    // as selects: a branch here would cut the k-step that carries the copies in two.
    static constexpr Win window(uint64_t p, uint32_t ld, int rows, int k, bool in) {
        const int left = rows - k * 64;
        int r = left < 64 ? left : 64;
        r = in ? r : 0;
        return Win{p + (uint64_t)(uint32_t)(k * 64) * ld, (uint32_t)r * ld};
    }
    // offset in it of row r's chunk.  REG loads the 16 bytes that end at the last column (and
    // shifts them; rows of 8 columns or more); a direct copy takes what follows, the next row's
    // first columns or zeros past the end, which only reach results that are not stored
    static constexpr uint32_t offset(int r, uint32_t ld, int col, int over) {
        const uint32_t off = (uint32_t)r * ld + (uint32_t)col * 2u;
        if (over >= 8) return kMasked;
        return REG && over > 0 ? off - 2u * (uint32_t)over : off;
    }
    static constexpr uint32_t shift(int over) { return over > 0 && over < 8 ? 16u * (uint32_t)over : 0u; }
};

}  // namespace spg
