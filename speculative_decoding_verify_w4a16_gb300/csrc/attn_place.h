// attn_place.h -- where the last kernel of attention with shared prefixes finds
// a token's results: a word per token and key/value head.  Plain C++, so that
// what every word leads to can be gone through on the host.
#pragma once
#include <cstddef>
#include <cstdint>

#ifdef __CUDACC__
#define W4V_PLACE_FN __host__ __device__ __forceinline__
#else
#define W4V_PLACE_FN inline
#endif

namespace w4v {

constexpr int kPlaceRanges = 256, kPlaceTokens = 128;   // fields of a place: ranges, tokens of a tile

// The first range of the token's row tile, how many ranges hold parts of it (1:
// the whole result is kept; 0: nothing is), its number in the tile, and whether
// it shares a prefix.
struct RowPlace {
    int range, parts, tok;
    bool shares;
};
W4V_PLACE_FN uint32_t place_of(int range, int parts, int tok, bool shares) {
    return uint32_t(range) | uint32_t(parts) << 8 | uint32_t(tok) << 17 | uint32_t(shares) << 24;
}
// Any word at all, for slots of `ranges` ranges with `rows` rows each, `group` a
// token: one that leads outside them (a range that gave up may leave what another
// call kept there) says that nothing is there.
W4V_PLACE_FN RowPlace read_place(uint32_t w, int ranges, int rows, int group) {
    RowPlace x;
    x.range = int(w & 0xFF);
    x.parts = int(w >> 8 & 0x1FF);
    x.tok = int(w >> 17 & 0x7F);
    x.shares = (w >> 24 & 1u) != 0u;
    if (x.parts > 1 && (x.range + x.parts > ranges || x.tok * group >= rows)) x.parts = 0;
    return x;
}
// The slot of part k of several: a range keeps a tile that begins in it in its
// second slot, one that only goes on in its first.
W4V_PLACE_FN size_t part_slot(int range, int k) { return size_t(2 * (range + k) + (k == 0)); }

}  // namespace w4v
