// The key/value cache's constants and orders in memory, shared by the kernels that write it and those that read it.
//
// A block is 64 tokens of one request and one kv head.  Complete blocks are E4M3 codes with one fp32 scale for the
// keys and one for the values; the block that a request is still filling (and the blocks that a prompt passes
// through) are bf16 "recent" blocks.  Both are kept in the order in which a wave of the attention kernel reads them
// as operands of v_mfma_f32_16x16x32_bf16 (lane l supplies 8 consecutive contraction slots 8 (l / 16) .. + 7 of row
// l % 16), so that every load of a wave covers 1 KB of consecutive memory.  For key n, channel d of a block:
//   E4M3 keys    byte    ((n/16 * D/64 + d/64) * 64 + d%32/8 * 16 + n%16) * 16 + d%64/32 * 8 + d%8
//   E4M3 values  byte    (d/16 * 64 + n%16/4 * 16 + d%16) * 16 + n/32 * 8 + n%32/16 * 4 + n%4
//   bf16 keys    element ((n/16 * D/32 + d/32) * 64 + d%32/8 * 16 + n%16) * 8 + d%8
//   bf16 values  element ((d/16 * 2 + n/32) * 64 + n%16/4 * 16 + d%16) * 8 + n%32/16 * 4 + n%4
// The values' key order inside 32 keys, (n%16/4, n%32/16, n%4), is the order in which the score product leaves the
// probabilities in a lane: they enter the second product without leaving their registers.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "jetfp8_join.h"

namespace jetfp8 {

constexpr int kKvBlock = 64;       // tokens of a block
constexpr int kUnitWords = 8;      // int32 words of a work unit's record

// One work unit: the new tokens of one request that fall into one block.
struct KvUnit {
    int request;   // -1: no unit
    int block;     // index of the block within the request: the tokens before it are block * 64
    int recent;    // bf16 block that holds the unit's block
    int row;       // row of its first new token in the call's q, k, v
    int rows;      // number of its new tokens, 1 .. 64
    int offset;    // place of its first new token in the block
    int physical;  // cache block to write once the block is complete; -1: not complete after this call
    int zero;
};
static_assert(sizeof(KvUnit) == kUnitWords * 4, "a unit is eight words");

// Whether a record can be used with these buffers.  Every kernel checks, and leaves out a unit that does not fit, so
// that units planned for another call or cache cannot reach beyond the buffers.
__device__ __forceinline__ bool unit_fits(const KvUnit& u, int requests, int tokens, int recent_blocks, int num_blocks) {
    return u.request >= 0 && u.request < requests && u.block >= 0 && u.recent >= 0 && u.recent < recent_blocks &&
           u.row >= 0 && u.rows >= 1 && u.rows <= kKvBlock && u.offset >= 0 && u.offset + u.rows <= kKvBlock &&
           u.row < tokens && u.rows <= tokens - u.row && u.physical >= -1 && u.physical < num_blocks;
}

}  // namespace jetfp8
