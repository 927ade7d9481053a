// Where the choice of blocks keeps bounds in shared memory, plain C++ for host and device (internal; not part
// of the C ABI).
//
// A warp's buffer holds 32 blocks of 16 pieces (16 bytes each).  Blocks of odd number have the halves of every eight
// pieces exchanged, so that the eight lanes of a read, two blocks' pieces, meet different banks.  All of it are offsets from
// the buffer's begin, wherever that lies.
#pragma once

#include "page_index.h"

namespace mikv {

constexpr uint32_t kBoundBytes = 256;   // of a block and key head
// Piece `piece` of block e.
MIKV_HD uint32_t bound_at(uint32_t e, uint32_t piece) { return e * kBoundBytes + ((piece ^ ((e & 1) << 2)) << 4); }
// Piece 4 k + t of block 8 j + g, of `lane` = bound_at(g, t).
MIKV_HD uint32_t bound_of_lane(uint32_t lane, uint32_t j, uint32_t k) { return (lane ^ (k << 6)) + j * 8 * kBoundBytes; }

}  // namespace mikv
