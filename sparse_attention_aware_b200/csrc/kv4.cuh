// The 4-bit KV record, shared by the kernels that write, read back and attend
// over it.
//
// One record of D + 16 bytes per (page, kv head, token):
//   [0, D/2)      codes of the key: channel 2j in the low nibble of byte j,
//                 channel 2j + 1 in the high one
//   [D/2, D)      codes of the value, likewise
//   [D, D + 16)   8 bf16: {scale, zero} of the key's channels [0, D/2) and
//                 [D/2, D), then of the value's
// A code c of a half row stands for zero + scale * c.
//
// Why this layout: keys and values of a token are one contiguous piece, so a
// token of a list is one 144-byte copy (D = 128) and a page is one copy of
// consecutive bytes; and the row stride of D + 16 bytes (36 or 20 words) puts
// the 16-byte chunks of 8 consecutive rows into 8 distinct bank groups, so the
// 8x8 matrix loads of the decode read shared memory without conflicts and no
// repacking is needed after the copy.
#pragma once

#include "sa_internal.h"

namespace sa {

template <int D>
struct Kv4 {
    static constexpr int REC = D + 16;      // bytes of a record
    static constexpr int V = D / 2;         // offset of the value's codes
    static constexpr int PAR = D;           // offset of the scales and zeros
    static constexpr int HALF = D / 2;      // channels that share a scale and a zero
};

}  // namespace sa
