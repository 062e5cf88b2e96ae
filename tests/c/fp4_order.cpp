// Test helper: how a group's rows split into tiles of the MXFP4 product, against
// 64-bit arithmetic up to the largest groups; and a replay of the order in which a
// wave of it sends off its copies into LDS, waits and reads, with the numbers that
// the kernel takes from csrc/fp4_order.h: nothing is read before it has landed
// behind a barrier and nothing is overwritten before a barrier follows its last
// read.  All waves take the same steps, so one stands for all.
#include <cstdio>
#include <vector>

#include "fp4_order.h"

using namespace moe;

namespace {

struct Place {                             // a slot of the ring, or the slab's place
    long long holds = -1;                  // what was sent there last
    int end = 0;                           // its last operation
    int read_at = -1;                      // barriers that had passed when it was read last
};

struct Wave {
    bool ok = true;
    int sent = 0, landed = 0, visible = 0, barriers = 0;
    void wait(int behind) {
        if (behind > 63) behind = 63;      // (what the counter goes to)
        if (sent - behind > landed) landed = sent - behind;
    }
    void barrier() { visible = landed, ++barriers; }
    void send(Place& p, long long what, int n) {
        if (p.read_at >= barriers) ok = false;
        sent += n;
        p.holds = what;
        p.end = sent;
    }
    void read(Place& p, long long what) {
        if (p.holds != what || p.end > visible) ok = false;
        p.read_at = barriers;
    }
};

constexpr int kTiles = 5;

bool replay(int S, bool words, bool tall, int stores) {
    const SlabPlan plan = slab_plan(S, words, tall);
    const int slots = tall ? 2 : 3, copies = stage_copies(tall), half = half_copies();
    Wave w;
    Place ring[3], slab;
    long long feed = 0;                    // the stage that is sent next, over all tiles
    auto stage = [&](int n, bool ends) {
        w.send(ring[feed % slots], feed, n);
        if (ends) ++feed;
    };
    auto slab_id = [&](long long tile, int i) { return tile * 1000 + i; };
    if (S >= 3) w.send(slab, slab_id(0, 0), kSlabCopies);
    stage(copies, true);
    stage(copies, true);
    if (!tall) stage(half, false);
    w.wait(copies + (tall ? 0 : half));
    w.barrier();
    for (int tile = 0, stored = 0; tile < kTiles; ++tile) {
        const long long first = (long long)tile * S;
        auto wait_stores = [&](int n) { w.wait(stored == 64 ? 63 : n + stored); };
        if (S < 3) {
            w.barrier();
            w.send(slab, slab_id(tile, 0), kSlabCopies);
            w.wait(0);
            w.barrier();
        } else if (plan.late && stored) {
            wait_stores(0);
            w.barrier();
        }
        w.read(ring[first % slots], first);
        w.read(slab, slab_id(tile, 0));
        bool sent = false;
        for (int j = 0, at = 0; j < S; ++j) {
            if (!tall) stage(copies - half, true);
            w.read(ring[(first + j) % slots], first + j);
            if (j == 0) wait_stores(on_their_way(tall, NO_SLAB));
            else w.wait(on_their_way(tall, !sent ? NO_SLAB : j + 1 < S ? SLAB : NEXT_SLAB));
            w.barrier();
            w.read(ring[(first + j + 1) % slots], first + j + 1);
            stage(tall ? copies : half, tall);
            const bool inner = at == 0 && j + plan.per < S;
            sent = inner || j == plan.next_at;
            if (sent) {
                // (the copies are at the tile whose slab it is)
                if (!inner && (feed - (tall ? 1 : 0)) / S != tile + 1) w.ok = false;
                w.send(slab, inner ? slab_id(tile, j / plan.per + 1) : slab_id(tile + 1, 0),
                       kSlabCopies);
            }
            if (++at == plan.per) {
                at = 0;
                if (j + 1 < S) w.read(slab, slab_id(tile, (j + 1) / plan.per));
                else slab.read_at = w.barriers;      // (read, and not used)
            }
        }
        stored = stores;
        w.sent += stores;
    }
    return w.ok;
}

bool tiles_right(int n, int blocks) {
    const long long c = ((long long)n + 31) / 32, mt = (c + blocks - 1) / blocks;
    if (row_tiles(n, blocks) != mt) return false;
    if (n == 0) return true;
    const long long per = (((long long)n + mt - 1) / mt + 31) / 32 * 32;
    return tile_rows(n, (int)mt) == per && per <= 32 * blocks && (mt - 1) * per < n &&
           mt * per >= n;
}

}  // namespace

int main() {
    int bad = 0;
    for (int blocks : {1, 2, 3, 4, 8}) {
        auto check = [&](int n) {
            if (tiles_right(n, blocks)) return;
            printf("n=%d blocks=%d\n", n, blocks);
            ++bad;
        };
        for (int n = 0; n < 70000; ++n) check(n);
        for (int n = 0; n < 70000; ++n) check(0x7fffffff - n), check(0x7fffffff - 331 * n);
    }
    for (int tall = 0; tall < 2; ++tall)
        for (int words = 0; words < 2; ++words)
            for (int S = 1; S <= 200; ++S)
                for (int stores = 16; stores <= 64; stores += 16)
                    if (!replay(S, words, tall, stores)) {
                        printf("S=%d words=%d tall=%d stores=%d\n", S, words, tall, stores);
                        ++bad;
                    }
    printf("%d bad\n", bad);
    return bad != 0;
}
