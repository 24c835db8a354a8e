// Where the new tokens of a sequence go in a paged cache: the arithmetic that
// sas_append_paged's kernels share, in plain C++ (it also compiles for the
// host alone).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SAS_HD __host__ __device__ __forceinline__
#else
#define SAS_HD inline
#endif

namespace sas {

constexpr int kPageRows = 64;

// New tokens of one sequence: `count` token rows from row0 on, at positions
// first .. first + count - 1. `bad`: its lengths break the call's terms (the
// sequence is skipped whole); count 0 without `bad` is nothing to append.
struct SeqNew {
    long long row0;
    int first, count;
    bool bad;
};

// With has_cu the sequence owns the token rows lo .. hi - 1, else row n (none
// when kv_len is 0, a padding entry). kv_len counts the new tokens.
SAS_HD SeqNew seq_new(bool has_cu, int lo, int hi, int n, long long T, int max_new, int kv_len, int max_pages,
                      int max_pos) {
    SeqNew s;
    s.row0 = has_cu ? lo : n;
    s.first = 0;
    s.count = 0;
    s.bad = false;
    long long count = has_cu ? (long long)hi - lo : (kv_len != 0 ? 1 : 0);
    if (count == 0 && (!has_cu || lo >= 0)) return s;
    if ((has_cu && (lo < 0 || hi < lo || hi > T)) || count > max_new || kv_len < count ||
        kv_len > (long long)max_pages * kPageRows || kv_len > max_pos) {
        s.bad = true;
        return s;
    }
    s.count = (int)count;
    s.first = kv_len - s.count;
    return s;
}

// Tile i of a sequence: the rows lo .. hi - 1 of its block `block`, from token
// row `row` on. Empty (hi <= lo) behind the last one.
struct PageTile {
    int block, lo, hi;
    long long row;
};
SAS_HD PageTile page_tile(const SeqNew& s, int i) {
    PageTile t;
    t.block = s.first / kPageRows + i;
    const long long at = (long long)t.block * kPageRows;
    t.lo = at < s.first ? (int)(s.first - at) : 0;
    const long long end = (long long)s.first + s.count - at;
    t.hi = end < kPageRows ? (end > 0 ? (int)end : 0) : kPageRows;
    if (s.count == 0) t.hi = t.lo = 0;
    t.row = s.row0 + (at + t.lo - s.first);
    return t;
}

// Tiles that a sequence of at most max_new new tokens can touch.
SAS_HD int max_tiles(int max_new) { return (max_new - 1 + kPageRows - 1) / kPageRows + 1; }

// First of the tile indices of sequence n, whose rows start at token row lo, when
// the tiles of all sequences are numbered by T / 64 + 2 N indices: it has at least
// len / 64 + 2 of them, and its rows touch at most (len + 62) / 64 + 1 blocks.
SAS_HD uint32_t seq_tile_base(int lo, int n) { return (uint32_t)(lo < 0 ? 0 : lo) / kPageRows + 2u * (uint32_t)n; }

// Exponent of the least power of two s with amax <= 448 s, not under
// kMinScaleExp. amax: finite and not negative, as its fp32 bits. 448 is
// 1.75 * 2^8: a mantissa above 1.75 needs the next power.
constexpr int kMinScaleExp = -64;
SAS_HD int scale_exp(uint32_t amax_bits) {
    const int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < kMinScaleExp ? kMinScaleExp : e;
}

// Scales of 8-bit pages that the kernels accept.
constexpr float kMinScale = 7.888609052210118e-31f;    // 2^-100
constexpr float kMaxScale = 1.329227995784916e36f;     // 2^120
SAS_HD bool scale_ok(float s) { return s >= kMinScale && s <= kMaxScale; }

}  // namespace sas
