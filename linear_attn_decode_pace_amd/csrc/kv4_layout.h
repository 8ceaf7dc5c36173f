// Layout of the 4-bit paged cache.
//
// A page holds, for each key / value head, page_tokens / 32 tiles of 32
// tokens.  A tile is contiguous: key codes (16 d bytes), value codes (16 d
// bytes), key scales, value scales (each float32 [d / 64][32], one per group
// of 64 channels and token).  Codes are stored in the form that the attention
// kernel unpacks cheapest, keys as c + 8 (1..15) and values in two's
// complement, and in the order in which its matrix products take them, so that
// a lane's operand is one 32-bit word of eight codes and a wavefront's load is
// 1 KiB without gaps:
//   key codes: word (sub, m) of lane 16 q + t, for token 16 sub + t of the
//     tile, holds channels 32 m + 8 q + j, j = 0..7 (a k-slice of 32 channels
//     of the product keys x queries; slices 2 g and 2 g + 1 are group g);
//   value codes: word c of lane 16 q + n, for channel 16 c + n, holds tokens
//     4 q + i (i = 0..3) and 16 + 4 q + i (i = 4..7 after subtracting 4) of the
//     tile: the tokens whose scores that lane holds of the product above.
// Words are grouped by four: word w of lane l is at ((w / 4) * 64 + l) * 16 +
// (w % 4) * 4 (w = sub * d / 32 + m for keys).  Inside a word of keys,
// channel j is nibble (j % 2) * 4 + j / 2; inside a word of values, index i is
// nibble i: shifting a word right by 4 p then leaves the operand's elements 2 p and
// 2 p + 1 in bits 3:0 and 19:16.
#pragma once

#include "pace_layers.h"

namespace pace {

constexpr int KV4_TILE = 32;   // tokens of a tile
constexpr int KV4_GROUP = 64;  // channels that share a scale

__host__ __device__ inline size_t kv4_tile_bytes(int d) { return (size_t)36 * d; }

// byte offset in a tile of the word with channels c .. c + 7 of token t's key
__device__ inline int kv4_key_word(int d, int t, int c) {
    const int w = (t >> 4) * (d >> 5) + (c >> 5), lane = ((c >> 3) & 3) * 16 + (t & 15);
    return ((w >> 2) * 64 + lane) * 16 + (w & 3) * 4;
}
__device__ inline int kv4_key_scales(int d) { return 32 * d; }
__device__ inline int kv4_value_scales(int d) { return 34 * d; }

// column of the page table that holds tile `tile` >= 0
__device__ inline int kv4_column(const Kv4View &c, int tile) {
    return c.per_inv ? (int)__umulhi((uint32_t)tile, c.per_inv) : tile;
}

}  // namespace pace
