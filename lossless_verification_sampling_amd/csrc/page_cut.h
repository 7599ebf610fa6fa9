// page_cut.h -- where the best of many 64-bit keys end: the narrowing of the keys'
// range, without the counting (internal; for the device and, in the tests, the host).
#pragma once

#include <stdint.h>

namespace sv {

constexpr int kPartBits = 11, kParts = 1 << kPartBits;
// A range of 2^64 keys is one key wide after six levels: parts of 2^53, 2^42, .., 2^9
// keys and of one.
constexpr int kCutLevels = 6;

// The keys above `key` are in, and the first `ties` that equal it.
struct KeyCut {
    uint64_t key;
    uint32_t ties;
};
// The part of a range that holds a cut: its number, the keys in it, and how many of
// those are wanted (1 .. keys).
struct CutPart {
    uint64_t index;
    uint32_t keys, want;
};

// Part of the keys lo .. hi (of kParts, each 2^shift keys) that `key` lies in.
constexpr int part_shift(uint64_t lo, uint64_t hi) {
    const int width = hi == lo ? 0 : 64 - __builtin_clzll(hi - lo);   // of hi - lo, in bits
    return width > kPartBits ? width - kPartBits : 0;
}

// The cut behind the `want` largest of the keys in lo .. hi (which are more, or
// as many, and above 0).  part_of_cut(lo, hi, shift, want) counts the keys lo .. hi by parts and
// gives the one in which the want-th largest lies; it is cut again until it is
// taken whole or is one key.  No end of a range passes 2^64: the distance to the
// end is compared, not the end.
template <typename F>
constexpr KeyCut key_cut(uint64_t lo, uint64_t hi, uint32_t want, F part_of_cut) {
    for (int level = 0; level < kCutLevels; ++level) {
        const int shift = part_shift(lo, hi);
        const CutPart part = part_of_cut(lo, hi, shift, want);
        want = part.want;
        lo += part.index << shift;
        const uint64_t rest = (uint64_t{1} << shift) - 1;
        if (hi - lo > rest) hi = lo + rest;
        if (part.keys == want) return KeyCut{lo - 1, 0};  // every key of the part
        if (shift == 0) break;
    }
    return KeyCut{lo, want};
}

}  // namespace sv
