// The 4-bit cache's layout, shared by the kernels that write and read it (kv4_rows.cu,
// kv4_decode.cu). A page holds page_size tokens (a multiple of 16); per kv head it is a row of
// records, one for every 16 tokens, 18 D bytes each and contiguous:
//   [0, 8 D)      K codes  [token 16][c 4][group NG] u32: dims 32 group + 8 c + e, e = 0 .. 7; dim
//                 e = 2 i in bits 4 i, e = 2 i + 1 in bits 16 + 4 i
//   [8 D, 16 D)   V codes  [half 2][r 8][c 4][group NG] u32: dims 32 group + 4 r + i in bits 4 i of a
//                 16-bit half; token 8 half + 2 c in the low one, 8 half + 2 c + 1 in the high one
//   [16 D, 18 D)  scales   [token 16][K, V][group NG] bf16
// NG = D / 32 groups of 32 dims, each with one scale; a code is stored plus 8 in a nibble and stands
// for (nibble - 8) * scale. The order is the one in which a warp of the decode kernel feeds its matrix
// instructions: lane 4 r + c reads its K words (tokens r and r + 8) and V words (half 0 and 1) as
// vectors, and (word >> 4 i) & 0x000f000f is a pair of neighbours along the product's inner
// dimension (two dims of one key, two keys at one dim). One token's nibbles fill whole bytes, so
// writing a token touches no other token's bytes.
#pragma once

#include <stdint.h>

namespace cb {

constexpr int kKv4Block = 16;  // tokens per record
constexpr int kKv4Group = 32;  // dims per scale

template <int D>
struct Kv4 {
  static constexpr int kGroups = D / kKv4Group;
  static constexpr int kRecord = 18 * D;  // bytes of a record
  static constexpr int kV = 8 * D;        // V codes
  static constexpr int kScales = 16 * D;
  static constexpr int kPlane = 4 * D;    // bytes of 32 lanes' words of all groups
};

}  // namespace cb
