// What the MXFP4 product's kernel shares with checks on the host: how a group's
// rows split into tiles, and the order in which a wave sends off its copies into
// LDS, as numbers that the kernel waits for.  Plain C++.
#pragma once

#include "row_tiles.h"

namespace moe {

// row tiles of a group of n rows, tiles of up to `blocks` blocks of 32 rows
constexpr int row_tiles(int n, int blocks) {
    const int c = row_blocks(n);
    return blocks == 1 ? c : blocks == 2 ? (c + 1) >> 1 : blocks == 3 ? (c + 2) / 3
           : blocks == 4 ? (c + 3) >> 2 : (c + 7) >> 3;
}

// A stage j of a tile of S stages, in a ring of three slots:
//   the second half of the copies of stage j + 2 | turn | the first half of those
//   of stage j + 3, a slab of scales;
// in a ring of two slots (tall tiles):
//   turn | all copies of stage j + 2, a slab of scales.
// Stages behind S are the next tile's.  The turn is a wait and a barrier, behind
// which the next stage's operands are read.  A wave's operations end in order, so
// a wait names how many of the last ones may still be on their way.
constexpr int kSlabCopies = 2;                             // of a slab
constexpr int stage_copies(bool tall) { return tall ? 8 : 6; }
constexpr int half_copies() { return 3; }

struct SlabPlan {
    int per;                               // stages of a slab
    int next_at;                           // the stage that sends the next tile's first one
                                           // (-1: that tile does), once this tile's last has
                                           // been read and the copies are at that tile
    bool late;                             // no turn behind it: waited for when that tile begins
};
// words: scales in whole words, four stages of a slab
constexpr SlabPlan slab_plan(int S, bool words, bool tall) {
    const int per = words ? 4 : 3, ahead = tall ? 2 : 3;
    const int last = (S - 1) / per * per;
    const int at = S < 3 ? -1 : last > S - ahead ? last : S - ahead;
    return {per, at, at == S - 1};
}

// Operations that may be on their way at a turn: those behind the next stage's
// copies.  NO_SLAB: none was sent in the stage before.  SLAB: one was, which has
// other turns to land.  NEXT_SLAB: the next tile's was, and this is the tile's
// last turn, so that only what was sent behind the slab may be on its way.
enum Sent { NO_SLAB, SLAB, NEXT_SLAB };
constexpr int on_their_way(bool tall, Sent sent) {
    if (sent == NEXT_SLAB) return tall ? 0 : stage_copies(false) - half_copies();
    return (tall ? 0 : stage_copies(false)) + (sent == SLAB ? kSlabCopies : 0);
}

}  // namespace moe
