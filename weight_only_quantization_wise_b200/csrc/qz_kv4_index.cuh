// qz_kv4_index.cuh -- index arithmetic of the paged 4-bit key/value cache and
// of the attention's work split.  Plain C++ for host and device: the kernels
// use it, and the CPU tests compile it with the host compiler and check every
// index and range it gives.
//
// Cache layout.  A page holds `page_size` tokens (a multiple of 16) of every
// key head: [page][kv head][page_size / 16][record].  A record is everything
// attention needs of 16 consecutive tokens of one head, contiguous and a
// multiple of 16 bytes, so that one untiled bulk copy brings it to shared
// memory:
//   K codes   8 D bytes     V codes   8 D bytes
//   K scales  [D/g][16] bf16    V scales  [D/g][16] bf16
//   K zeros   [D/g][16] uint8   V zeros   [D/g][16] uint8
// The codes lie as the lanes of a warp read them for mma.sync m16n8k16 (lane
// = 4 * gid + tid, gid 0..7, tid 0..3): "piece" i holds four 32-bit words of
// each of the 32 lanes, 16 bytes per lane, so every shared-memory load is one
// 16-byte load free of bank conflicts.
//   K (A operand, tokens x d): lane (gid, tid) reads tokens gid and gid + 8;
//     word (hi, j) holds the eight codes d = 32 j + 8 tid + n (nibble n) of
//     token 8 hi + gid.  Word number hi * (D / 32) + j.
//   V (A operand, d x tokens): word (p, hi, w) of lane (gid, tid) holds for
//     tokens 8 p + 2 tid (low half) and 8 p + 2 tid + 1 (high half) the four
//     codes d = 64 w + 16 n + 8 hi + gid (nibble n of the half).  Word number
//     p * (D / 32) + hi * (D / 64) + w.
#pragma once

#include <stdint.h>

#if defined(__CUDACC__)
#define QZ_HD __host__ __device__ __forceinline__
#else
#define QZ_HD inline
#endif

namespace qz {
namespace kv4 {

constexpr int kBlock = 16;     // tokens of a record

// ---- record -------------------------------------------------------------
QZ_HD constexpr int64_t record_bytes(int64_t D, int64_t g) { return 16 * D + 96 * (D / g); }
QZ_HD constexpr int k_codes_off() { return 0; }
QZ_HD constexpr int v_codes_off(int D) { return 8 * D; }
QZ_HD constexpr int k_scales_off(int D) { return 16 * D; }
QZ_HD constexpr int v_scales_off(int D, int ng) { return 16 * D + 32 * ng; }
QZ_HD constexpr int k_zeros_off(int D, int ng) { return 16 * D + 64 * ng; }
QZ_HD constexpr int v_zeros_off(int D, int ng) { return 16 * D + 80 * ng; }

// Byte of word `word` of lane (gid, tid) within a code area.
QZ_HD constexpr int word_byte(int word, int gid, int tid) {
    return ((word >> 2) * 32 + 4 * gid + tid) * 16 + (word & 3) * 4;
}
// K: byte of the 32-bit word holding codes 8 c8 .. 8 c8 + 7 of a token.
QZ_HD constexpr int k_word_byte(int D, int token, int c8) {
    return word_byte((token >> 3) * (D / 32) + (c8 >> 2), token & 7, c8 & 3);
}
// V: byte of the 16-bit unit of a token holding the codes
// d = 64 w + 16 n + 8 hi + gid, n = 0..3 (nibble n).
QZ_HD constexpr int v_unit_byte(int D, int token, int w, int hi, int gid) {
    return word_byte((token >> 3) * (D / 32) + hi * (D / 64) + w, gid, (token & 7) >> 1) +
           2 * (token & 1);
}

// a / b for a >= 0, b > 0; one 32-bit division where both allow it.
QZ_HD int64_t quotient(int64_t a, int64_t b) {
    if (((uint64_t)a | (uint64_t)b) >> 32 == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}

// ---- pages --------------------------------------------------------------
// Record index (in records from the cache's start) of the block of 16 tokens
// that holds position `pos` of head `h`, or -1 when the page table has no
// valid page there.  `row` is the sequence's row of the page table.
QZ_HD int64_t record_index(const int32_t *row, int64_t max_pages, int64_t num_pages,
                           int kv_heads, int h, int page_blocks, int block) {
    if (block < 0) return -1;
    const int pi = (int)((uint32_t)block / (uint32_t)page_blocks);
    if (pi >= max_pages) return -1;
    const int32_t page = row[pi];
    if (page < 0 || page >= num_pages) return -1;
    return ((int64_t)page * kv_heads + h) * page_blocks + (block - pi * page_blocks);
}

// ---- append's and read's work --------------------------------------------
// A sequence's n tokens (rows cu0 .. cu0 + n - 1) stand at positions first ..
// first + n - 1, first = kv_len - n (negative when the length is too small).
// A unit is (block of 16 positions, head), heads fastest; block i of the
// sequence holds positions 16 (block0 + i) ...
struct StoreWork {
    int n, block0, blocks;
    int64_t first, units;
};
QZ_HD StoreWork store_work(int cu0, int cu1, int kv_len, int rows, int kv_heads) {
    StoreWork s;
    s.n = cu0 >= 0 && cu1 > cu0 ? cu1 - cu0 : 0;
    if (s.n > rows) s.n = rows;
    s.first = (int64_t)kv_len - s.n;
    s.block0 = (int)(s.first >> 4);                // rounds down
    s.blocks = s.n > 0 ? (int)(((int64_t)kv_len - 1) >> 4) - s.block0 + 1 : 0;
    s.units = (int64_t)s.blocks * kv_heads;
    return s;
}
// Tokens [lo, hi) of block `block` that are the sequence's.
QZ_HD int block_lo(const StoreWork &s, int block) {
    const int64_t d = s.first - (int64_t)block * kBlock;
    return d > 0 ? (int)d : 0;
}
QZ_HD int block_hi(const StoreWork &s, int block) {
    const int64_t d = s.first + s.n - (int64_t)block * kBlock;
    return d < kBlock ? (int)d : kBlock;
}

// ---- attention's work ---------------------------------------------------
// A sequence with n new tokens (queries) and len cached tokens (the new ones
// included) has n * share query rows per key head (share = query heads per
// key head), in tiles of `tile_rows`.  An item is one (key head, row tile);
// its units are the blocks of 16 keys [block0, block0 + blocks) that any of
// the sequence's rows may see.  Every item has at least one unit, so that
// rows without keys are written too.
struct SeqWork {
    int n, len;           // queries, keys (none behind the page table's end)
    int block0;           // first block of keys
    int blocks;           // units of an item (>= 1)
    int row_tiles;        // row tiles per key head
    int64_t units;        // kv_heads * row_tiles * blocks (0 when n == 0)
};

// Position of the first of a sequence's n queries (len may end before them: at
// the page table's end).
QZ_HD int first_position(int kv_len, int n) { return (kv_len < 0 ? 0 : kv_len) - n; }

// rows: the call's token rows (rows * share < 2^31); capacity < 2^31 - 16.
QZ_HD SeqWork seq_work(int cu0, int cu1, int kv_len, int rows, int capacity, int window, int share,
                       int kv_heads, int tile_rows) {
    SeqWork s;
    s.n = cu0 >= 0 && cu1 > cu0 ? cu1 - cu0 : 0;
    if (s.n > rows) s.n = rows;
    s.len = kv_len < 0 ? 0 : (kv_len > capacity ? capacity : kv_len);
    // (capacity, the multiple of 16 that len ends at, cuts no record)
    const int64_t first = window > 0 ? (int64_t)first_position(kv_len, s.n) - window + 1 : 0;
    const int end = (int)(((int64_t)s.len + kBlock - 1) / kBlock);
    s.block0 = first > 0 ? (int)(first / kBlock) : 0;
    if (s.block0 >= end) s.block0 = end > 0 ? end - 1 : 0;
    s.blocks = end - s.block0 > 1 ? end - s.block0 : 1;
    s.row_tiles = (int)(((int64_t)s.n * share + tile_rows - 1) / tile_rows);
    s.units = (int64_t)s.row_tiles * kv_heads * s.blocks;
    return s;
}

// The units of all items, in (sequence, head, row tile, block) order, are cut
// into contiguous ranges of `quota` units, one per CTA (the last may be
// shorter): as many CTAs as there are, but none with fewer than min_units.  When
// all items are alike (`blocks` units each) and short, a CTA takes whole items
// instead: one more step for its warps costs less than a join through the
// workspace.
QZ_HD int64_t cta_quota(int64_t units, int64_t items, int blocks, int64_t ctas, int min_units,
                        int whole_units) {
    const int64_t q = quotient(units + ctas - 1, ctas);
    if (q <= blocks && blocks <= whole_units && items * blocks == units) return blocks;
    return q > min_units ? q : min_units;
}
QZ_HD int64_t range_begin(int64_t c, int64_t quota, int64_t units) {
    return c * quota < units ? c * quota : units;
}
// Units per warp of a CTA's n units: even (two blocks make a step), so that
// warps * warp_quota >= n.
QZ_HD int warp_quota(int64_t n, int warps) { return (int)((n + 2 * warps - 1) / (2 * warps)) * 2; }
// Partial results in the workspace: a CTA has two slots, 0 for an item that
// is under way where its range begins (or begins there), 1 for one that
// begins inside its range and goes on in the next CTA.
QZ_HD int partial_slot(int64_t item_begin, int64_t cta_begin) { return item_begin > cta_begin; }

}  // namespace kv4
}  // namespace qz
