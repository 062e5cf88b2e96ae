// Grouped matrix product of MXFP4 rows and weights on row-major codes: for the
// rows r of group g,
//   out[r, n] = sum_b 2^(Xa[r, b] + Xw[g, n, b]) sum_{k in block b} a[r, k] w[g, n, k],
// b the blocks of 32 of K, codes E2M1, scale bytes X + 127 (255: NaN).
//
// The scaled matrix instructions (32 x 32 outputs, 64 of K) take both operands
// as they are: lane l holds of row (column) l % 32 the 16 bytes of one block of
// 32 and that block's scale byte, one of the four of a register.  Of a stage's
// eight blocks the lower half of the lanes takes 0 to 3 in the stage's four
// steps, the upper half 4 to 7, so that a half's four scales are one word.
//
// Tile: up to 128 rows x 256 weight rows, 8 waves of 64 x 64 or (rows of the
// tile) x 32 outputs, 256 of K (128 bytes a row) a stage, four steps.  The
// codes of both operands go to a ring of three LDS slots by copies that pass
// no register, two and a half stages ahead (a wave's copy covers 8 rows x 128
// bytes; LDS row r holds its 16-byte chunk c at c ^ ((r >> 1) & 7), so that the
// lanes of an operand read spread over the banks).  Where it saves enough
// rounds the tiles have up to 256 rows, 8 waves of up to 128 x 64, in a ring of
// two slots, each refilled as soon as its last step has been read.
//
// Scales: a row's 8 bytes of a stage, but fetched 32 at a time: the 16 bytes of
// one stage for each of 384 rows are 384 lines touched, as many as its codes
// (384 groups x 128 rows x 4096 x 2048 with an earlier order of the stores: 560
// us fetched so, 448 without any scales, 492 now).  A slab of 32 bytes a row
// from the word that holds the first one is four stages (K / 32 and the scales'
// address multiples of 4) or three (any others, the bytes shifted out of the
// words).  Its place in LDS is read into registers at the slab's first stage and
// takes the next slab from then on.
//
// Bound and measured (us):
//   64 groups, 192 rows in all, 2048 x 1024, bf16 out        15  the weights' 70 MB (10 at
//     6.8 TB/s) and the start of the reads: one round, 8 stages
//   384 uneven groups, 49152 rows, 4096 x 2048, fp32 out    455  HBM: weights, rows and
//     outputs are 2.2 GB, what tiles fetch again from memory 0.3 GB: 5.5 TB/s (under the
//     profiler 480 on the average, 440 at least)
//   8191 x 4064 x 2032, bf16 out                          47-51  waits: the matrix cores are
//     busy 29% of the time, the LDS with reads 16% (2.8 PFLOP/s of the 8 that the
//     instructions reach from registers): all waves of a CU meet at each stage's
//     barrier, and a step's products stand behind its reads
//   8192 x 4096 x 2048, bf16 out                             47  the same, 2.9 PFLOP/s
//   one matrix, 1 to 16 rows x 4096 x 2048                   15  one tile's 16 stages, on 8 CUs
#include "fp4.h"
#include "fp4_order.h"
#include "lds_ring.h"

namespace moe {
namespace {

constexpr int BN = 256;                    // weight rows a tile
constexpr int BK = 128;                    // bytes of a row a stage: 256 of K
constexpr int kThreads = 512;
constexpr int kSlotW = BN * BK;
// tiles of up to 128 rows and three slots, or of up to 256 and two
template <bool TALL>
struct Ring {
    static constexpr int BM = TALL ? 256 : 128;
    static constexpr int kSlot = kSlotW + BM * BK, kSlots = TALL ? 2 : 3;
    static constexpr int kSlabs = kSlots * kSlot;  // scales: 32 bytes a row, W's first
    static constexpr int kBytes = kSlabs + 32 * (BN + BM);
    static_assert(kSlot % 128 == 0, "the chunks' places within a row");
};
constexpr int kLds = Ring<false>::kBytes;
static_assert(kLds <= 160 * 1024 && Ring<true>::kBytes <= kLds, "the LDS of a CU");

struct Tile {
    int g, row0, valid, n0;                // n0: first weight row
};

// Waves of a tile of MB blocks of 32 rows (tall tiles: 4, 6 or 8): along the rows
// x along the weight rows, each MI x NJ blocks of 32 x 32.  With NJ = 2 the two
// blocks of weight rows hold every other one of 64, so that a lane has
// neighbouring columns of the output.
template <int MB, bool TALL>
struct Waves {
    static constexpr int WM = TALL || MB == 4 || MB == 2 ? 2 : 1, WN = 8 / WM, MI = MB / WM;
    static constexpr int NJ = 8 / WN;
    static constexpr int kStores = 16 * MI;   // of a wave, whatever the output's type
};
template <bool TALL>
__device__ __forceinline__ bool in_pairs(int valid) {
    return TALL || ((valid - 1) >> 5) & 1;
}

// Items are (group, band of kBand m-tiles, n-tile, m-tile), the 8 XCDs take
// contiguous ranges, so that the m-tiles of a weight tile and the n-tiles of a
// group's rows meet in one XCD's L2.  A group's rows split evenly over its
// m-tiles.  The group of an item comes from a two-level sum that every wave
// keeps in registers: lane l holds the items before run l of ceil(G / 64)
// groups, and looks into the run that holds the item.
constexpr int kBand = 8;
constexpr int kUsual = 4, kTall = 8;
static_assert(MOE_MAX_GROUPS <= 64 * 64, "one lane a run, one lane a group of a run");

struct Schedule {
    const int32_t* offsets;
    int G, rows, NT, run, blocks;
    int mine, upto;                        // of this lane's run
    bool tall;

    __device__ __forceinline__ int clamped(int v) const { return min(max(v, 0), rows); }
    __device__ __forceinline__ void set(const Fp4GemmArgs& p, int lane) {
        offsets = p.offsets;
        G = p.G;
        rows = p.rows;
        NT = (p.N + BN - 1) / BN;
        run = (G + 63) / 64;
        // the row tiles of this lane's run, of up to 1 .. 4 and 8 blocks
        int tiles[kUsual + 1] = {}, talls = 0;
        for (int i = 0; i < run; ++i) {
            const int g = lane * run + i;
            if (g < G) {
                const int n = max(clamped(offsets[g + 1]) - clamped(offsets[g]), 0);
#pragma unroll
                for (int b = 1; b <= kUsual; ++b) tiles[b] += row_tiles(n, b);
                talls += row_tiles(n, kTall);
            }
        }
        blocks = kUsual;
        mine = NT * tiles[kUsual];
        upto = wave_scan(mine, lane);
        const int cus = (int)gridDim.x, usual = items();
        // Tall tiles where their rounds on the CUs, of up to twice the products
        // and 3/4 of the bytes into LDS for each, are fewer than 2/3: 8191 x 4064
        // x 2032 then takes 49 us instead of 57, 8192 x 4096 x 2048 47 instead of
        // 50; 384 uneven groups of 128 rows on the average x 4096 x 2048, all in
        // tall tiles, 505 instead of 465
        tall = false;
        if (usual > cus) {
            const int sum = wave_scan(NT * talls, lane);
            const int rounds = (usual + cus - 1) / cus;
            if (3 * ((__builtin_amdgcn_readlane(sum, 63) + cus - 1) / cus) < 2 * rounds) {
                tall = true;
                blocks = kTall;
                mine = NT * talls;
                upto = sum;
            }
        }
        // few tiles: the lowest of which every one still has a CU of its own
        if ((long long)rows * NT <= 96ll * cus && usual < cus) {
#pragma unroll
            for (int b = 1; b < kUsual; ++b) {
                const int sum = wave_scan(NT * tiles[b], lane);
                if (__builtin_amdgcn_readlane(sum, 63) > cus) continue;
                blocks = b;
                mine = NT * tiles[b];
                upto = sum;
                break;
            }
        }
    }
    __device__ __forceinline__ int items() const { return __builtin_amdgcn_readlane(upto, 63); }
    __device__ __forceinline__ void find(int q, Tile& t) const {
        // the first lane whose sum passes q, then the groups of its run in
        // turn (scalar loads: a vector load would wait for the copies that are
        // on their way)
        const int r = __builtin_ctzll(__builtin_amdgcn_ballot_w64(upto > q));
        int local = q - __builtin_amdgcn_readlane(upto - mine, r);
        t.g = r * run;
        int r0 = clamped(scalar_load(offsets + t.g)), n, mt;
        for (;; ++t.g) {                             // (ends: the run holds item q)
            const int r1 = clamped(scalar_load(offsets + t.g + 1));
            n = max(r1 - r0, 0);
            mt = row_tiles(n, blocks);
            if (local < NT * mt || t.g + 1 >= G) break;
            local -= NT * mt;
            r0 = r1;
        }
        const int per = tile_rows(n, mt);
        const int band = local / (kBand * NT) * kBand, high = min(kBand, mt - band);
        local -= band * NT;
        t.n0 = local / high * BN;
        t.row0 = r0 + (band + local % high) * per;
        t.valid = min(per, r0 + n - t.row0);
    }
};

// What goes into LDS, stage after stage and tile after tile: the copies run two
// and a half stages ahead of the products (two slots: one and a quarter), across
// the ends of tiles.  Buffer
// resources over a tile's rows (wave-uniform base, 32-bit offsets; rows past the
// tile's or the matrix's end lie past them and fetch nothing).
template <bool TALL>
struct Feed {
    using R = Ring<TALL>;
    const Schedule& sched;
    Tile t;                                // the tile that is fetched
    int q, step, end;                      // its item, the next one's distance, their end
    int j, S;                              // its next stage, and its stages
    u32x4 wsrc, asrc, wscale, ascale;
    int wo, ao, rows64, sw, sa;

    __device__ __forceinline__ void set(const Fp4GemmArgs& p) {
        const int tid = threadIdx.x, Kb = p.K / 2;
        const int lr = tid >> 3, c = (tid & 7) ^ swz(lr);   // chunk c of row lr + 64 q
        const size_t wfirst = (size_t)t.g * p.N + t.n0;
        const int wrows = min(p.N - t.n0, BN);
        wsrc = uniform_rsrc(p.w + wfirst * Kb, (size_t)wrows * Kb);
        asrc = uniform_rsrc(p.a + (size_t)t.row0 * Kb, (size_t)t.valid * Kb);
        wo = (in_pairs<TALL>(t.valid) ? 2 * (lr & 31) + (lr >> 5) : lr) * Kb + 16 * c;
        ao = lr * Kb + 16 * c;
        rows64 = 64 * Kb;
        set_scales(p, t);
        j = 0;
    }
    __device__ __forceinline__ void set_scales(const Fp4GemmArgs& p, const Tile& t) {
        const int lane = threadIdx.x & 63, nb = p.K / 32;
        const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        const size_t wfirst = (size_t)t.g * p.N + t.n0;
        const int wrows = min(p.N - t.n0, BN);
        // scales: wave w the slab's weight rows 32 w + (0 .. 31) and rows 32 w +
        // (0 .. 31) (of 128 rows modulo 4, half of them twice, so that every wave
        // issues the same number of copies), 16 bytes a lane; whole words from
        // the one that holds the first byte on
        auto scales = [&](const uint8_t* first, int rows, u32x4& src) {
            const int mis = (int)((uintptr_t)first & 3);
            src = uniform_rsrc(first - mis, ((size_t)rows * nb + mis + 3) & ~size_t(3));
            return mis;
        };
        const int r = lane >> 1, piece = 16 * (lane & 1);
        sw = (((32 * wave + r) * nb + scales(p.ws + wfirst * nb, wrows, wscale)) & ~3) + piece;
        sa = (((32 * (TALL ? wave : wave & 3) + r) * nb +
               scales(p.as + (size_t)t.row0 * nb, t.valid, ascale)) & ~3) + piece;
    }

    // The next stage's copies into the slot at LDS byte `at`, in parts 0 and 1
    // (three copies each; tall tiles have a part 2 of two more); part 0 goes on
    // to the next tile where one ends (past the last with empty resources: every
    // stage issues its copies).  What a tile's last stage holds past K is left
    // out when it is multiplied.
    static constexpr int kCopies = stage_copies(TALL);
    template <int PART>
    __device__ __forceinline__ void copy(const Fp4GemmArgs& p, int at) {
        const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        at += wave * 1024;
        if constexpr (PART == 0) {
            if (j == S) {
                q += step;
                j = 0;
                if (q < end) {
                    sched.find(q, t);
                    set(p);
                } else {
                    q = end;
                    wsrc[2] = asrc[2] = 0;
                }
            }
            copies16<3>(wsrc, wo, wsrc, wo + rows64, wsrc, wo + 2 * rows64, j * BK, at);
        } else if constexpr (PART == 1) {
            copies16<3>(wsrc, wo + 3 * rows64, asrc, ao, asrc, ao + rows64, j * BK,
                        at + 3 * 64 * BK);
            if (!TALL) ++j;
        } else {
            copies16<2>(asrc, ao + 2 * rows64, asrc, ao + 3 * rows64, asrc, 0, j * BK,
                        at + 6 * 64 * BK);
            ++j;
        }
    }
    __device__ __forceinline__ void stage(const Fp4GemmArgs& p, int at) {
        copy<0>(p, at);
        copy<1>(p, at);
        if constexpr (TALL) copy<2>(p, at);
    }
    // the slab whose first stage is j: two copies
    __device__ __forceinline__ void slab(int j) const {
        const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        copy16(wscale, sw, j * 8, R::kSlabs + wave * 1024);
        copy16(ascale, sa, j * 8, R::kSlabs + 32 * BN + (TALL ? wave : wave & 3) * 1024);
    }
};

// at most N and `stores` (0, 16, 32, 48 or 64) of this wave's memory operations
// outstanding (the counter goes to 63)
template <int N>
__device__ __forceinline__ void wait_vm_stores(int stores) {
    switch (stores) {
        case 0: wait_vm<N>(); break;
        case 16: wait_vm<N + 16>(); break;
        case 32: wait_vm<N + 32>(); break;
        case 48: wait_vm<N + 48>(); break;
        default: wait_vm<63>(); break;
    }
}

// Of a tile's last stage, what this thread copied from past K (its blocks from
// `tail` on) becomes zeros, in W alone: the products are then zero, as no code
// is an infinity or NaN.
__device__ __forceinline__ void zeros(unsigned char* ring, int slot, int tail) {
    const int tid = threadIdx.x;
    if (((tid & 7) ^ swz(tid >> 3)) >= tail)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *(u32x4*)(ring + slot + q * 64 * BK + tid * 16) = u32x4{0u, 0u, 0u, 0u};
}

// What a workgroup's tiles have in common
struct Run {
    int S, tail;                           // stages, blocks of a short last one (0: none)
    SlabPlan slabs;
};

// One tile, whose first stage has landed in the ring at `slot` and whose next
// two (one) are on their way (and its first slab; with fewer than three stages it is
// fetched here).  `stored`: stores of the tile before, which were issued behind
// those and need not have ended when they have landed.  All stores are issued,
// those past the rows or columns with offsets past the resource, so that their
// number is known.  Returns the stores of this tile.
template <bool F32, bool PAST, int MB, bool TALL>
__device__ __forceinline__ int run_tile(const Fp4GemmArgs& p, const Tile& t, Feed<TALL>& f,
                                        const Run& c, int& slot, int stored,
                                        unsigned char* ring) {
    // (the thread's place as a value of this variant's own: address terms
    // shared by the variants would be kept, or spilled, for all of them)
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, half = lane >> 5, l32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    using W = Waves<MB, TALL>;
    constexpr int WN = W::WN, MI = W::MI, NJ = W::NJ, NT = MI * NJ;
    constexpr int kSlot = Ring<TALL>::kSlot, kSlabs = Ring<TALL>::kSlabs;
    const int wm = wave / WN, wn = wave % WN;
    const int N = p.N, nb = p.K / 32;
    const int S = c.S, tail = c.tail, per = c.slabs.per;

    // LDS rows 32 apart share their swizzle, so the rest of an operand's
    // address is an immediate; the chunk index enters it by exclusive or
    const int rd0 = l32 * BK + ((4 * half ^ swz(l32)) << 4);
    const int rdw = wn * NJ * 32 * BK + rd0;
    const int rda = kSlotW + wm * MI * 32 * BK + rd0;
    auto wrow = [&](int n) { return wn * NJ * 32 + (NJ == 2 ? 2 * l32 + n : l32); };
    const int rsw = kSlabs + wrow(0) * 32;
    const int rsa = kSlabs + (BN + wm * MI * 32 + l32) * 32;
    // bytes of a row's copied words before its first scale
    const uint32_t wbase = (uint32_t)((uintptr_t)p.ws + ((size_t)t.g * N + t.n0) * nb);
    const uint32_t abase = (uint32_t)((uintptr_t)p.as + (size_t)t.row0 * nb);
    // this half's words of the slab's stages, the next stage's first
    u32x4 cw[NJ], ca[MI];
    auto read_slab = [&]() {
        auto words = [&](int at, uint32_t mis, u32x4& c) {
            u32x4 x = *(const u32x4*)(ring + at), y = *(const u32x4*)(ring + at + 16);
            if (per == 3) {
                x = u32x4{__builtin_amdgcn_alignbyte(x[1], x[0], mis),
                          __builtin_amdgcn_alignbyte(x[2], x[1], mis),
                          __builtin_amdgcn_alignbyte(x[3], x[2], mis),
                          __builtin_amdgcn_alignbyte(y[0], x[3], mis)};
                y = u32x4{__builtin_amdgcn_alignbyte(y[1], y[0], mis),
                          __builtin_amdgcn_alignbyte(y[2], y[1], mis), 0u, 0u};
            }
            c = half ? u32x4{x[1], x[3], y[1], y[3]} : u32x4{x[0], x[2], y[0], y[2]};
        };
#pragma unroll
        for (int n = 0; n < NJ; ++n)
            words(rsw + n * 32, (wbase + (uint32_t)wrow(n) * nb) & 3, cw[n]);
#pragma unroll
        for (int i = 0; i < MI; ++i)
            words(rsa + i * 32 * 32, (abase + (uint32_t)((wm * MI + i) * 32 + l32) * nb) & 3,
                  ca[i]);
    };
    auto next_scales = [&]() {
#pragma unroll
        for (int n = 0; n < NJ; ++n) cw[n] = u32x4{cw[n][1], cw[n][2], cw[n][3], 0u};
#pragma unroll
        for (int i = 0; i < MI; ++i) ca[i] = u32x4{ca[i][1], ca[i][2], ca[i][3], 0u};
    };
    // the last stage's blocks past K: any finite scale
    auto finite = [&]() {
        uint32_t keep = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (4 * half + q < tail) keep |= 0xffu << (8 * q);
#pragma unroll
        for (int n = 0; n < NJ; ++n) cw[n][0] = (cw[n][0] & keep) | (0x7f7f7f7fu & ~keep);
#pragma unroll
        for (int i = 0; i < MI; ++i) ca[i][0] = (ca[i][0] & keep) | (0x7f7f7f7fu & ~keep);
    };

    f32x16 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int n = 0; n < NJ; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][n][e] = 0.0f;

    if (S < 3) {
        // (the feed is past the next tile: this one's slab is not sent ahead)
        __syncthreads();                            // (the last tile's has been read)
        f.set_scales(p, t);
        f.slab(0);
        wait_vm<0>();
        __syncthreads();
    } else if (c.slabs.late && stored) {
        wait_vm_stores<0>(stored);
        __syncthreads();
    }
    // The middle of stage j: the next stage has landed (behind its copies are, of
    // three slots, those of the one after it, a slab between their halves, and the
    // last tile's stores) and every wave has read stage j's operands, whose slot is
    // free, and the slab if stage j is its first.  The next tile's first slab, if it
    // was sent before this tile's last stage, has landed at this tile's last turn.
    bool sent = false;
    auto turn = [&](int j, int next) {
        if (j == 0) wait_vm_stores<on_their_way(TALL, NO_SLAB)>(stored);
        else if (!sent) wait_vm<on_their_way(TALL, NO_SLAB)>();
        else if (j + 1 < S) wait_vm<on_their_way(TALL, SLAB)>();
        else wait_vm<on_their_way(TALL, NEXT_SLAB)>();
        if (tail && (j == S - 2 || S == 1)) zeros(ring, next, tail);
        __syncthreads();
    };

    u32x4 rw[2][NJ], ra[2][MI];
    auto read = [&](int slot, auto step) {
        constexpr int q = decltype(step)::value, B = q & 1;
#pragma unroll
        for (int n = 0; n < NJ; ++n)
            rw[B][n] = *(const u32x4*)(ring + ((rdw ^ (q << 4)) + slot) + n * 32 * BK);
#pragma unroll
        for (int i = 0; i < MI; ++i)
            ra[B][i] = *(const u32x4*)(ring + ((rda ^ (q << 4)) + slot) + i * 32 * BK);
    };
    auto wide = [](const u32x4& v) {
        return v8i{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
    };
    // the products of a step, copies behind the first ones
    auto multiply = [&](auto step, auto copy) {
        constexpr int q = decltype(step)::value, B = q & 1;
        static_for<0, NT < 4 ? 4 : NT>([&](auto index) {
            constexpr int x = decltype(index)::value, i = x / NJ, n = x % NJ;
            if constexpr (x < NT)
                acc[i][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    wide(ra[B][i]), wide(rw[B][n]), acc[i][n], 4, 4, q, (int)ca[i][0], q,
                    (int)cw[n][0]);
            copy(index);
        });
        // (the products stay here: the compiler would take them all to the end of
        // the stage, behind its branches)
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int n = 0; n < NJ; ++n) asm volatile("" : "+v"(acc[i][n]));
        __builtin_amdgcn_sched_barrier(0);
    };
    using Q0 = std::integral_constant<int, 0>;
    using Q1 = std::integral_constant<int, 1>;
    using Q2 = std::integral_constant<int, 2>;
    using Q3 = std::integral_constant<int, 3>;
    read(slot, Q0());
    read_slab();
    if (tail && S == 1) finite();
    int at = 0;                                     // the stage's place in its slab
    for (int j = 0; j < S; ++j) {
        const int next = slot == (Ring<TALL>::kSlots - 1) * kSlot ? 0 : slot + kSlot;
        const int last = next == 2 * kSlot ? 0 : next + kSlot;
        read(slot, Q1());
        multiply(Q0(), [&](auto x) {
            if constexpr (!TALL && x == 0) f.template copy<1>(p, last);
        });
        read(slot, Q2());
        multiply(Q1(), [](auto) {});
        read(slot, Q3());
        multiply(Q2(), [](auto) {});
        turn(j, next);
        read(next, Q0());                           // (of the next tile: read again)
        multiply(Q3(), [&](auto x) {
            if constexpr (x == 0 || (TALL && x < 3)) f.template copy<decltype(x)::value>(p, slot);
        });
        const bool inner = at == 0 && j + per < S;
        sent = inner || j == c.slabs.next_at;
        if (sent) f.slab(inner ? j + per : 0);
        if (++at == per) {
            at = 0;
            read_slab();
        } else {
            next_scales();
        }
        if (tail && j == S - 2) finite();
        slot = next;
    }

    // Lane l holds, of column l % 32 of its block (of columns 2 (l % 32) and the
    // next of two blocks), rows 8 q + 4 (l / 32) + (0 .. 3), q < 4.  A store
    // fills whole lines of two rows, or halves of them (bf16 of one block): with
    // a lane along the rows its 32 bytes of each of 32 lines were what the L2
    // took four times as long for.
    constexpr int ES = F32 ? 4 : 2;
    const uint64_t base = (uint64_t)(uintptr_t)p.out + ((size_t)t.row0 * N + t.n0) * ES;
    const uint64_t first =
        (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)base) |
        (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32)) << 32;
    // (to the tile's last column: below 2^32 for any N)
    const uint32_t bytes = (uint32_t)(((size_t)(t.valid - 1) * N + min(N - t.n0, BN)) * ES);
    const auto out = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(uintptr_t)first, 0, __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
    const int col = wrow(0);
    constexpr int kAux = PAST ? 2 : 0;              // (2: nontemporal)
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int r = (wm * MI + i) * 32 + 8 * (e >> 2) + 4 * half + (e & 3);
            const uint32_t in = ((uint32_t)r * (uint32_t)N + (uint32_t)col) * ES;
            const int at = (int)(r < t.valid && t.n0 + col < N ? in : 0xfffffff0u);
            const float x = acc[i][0][e], y = acc[i][NJ - 1][e];
            if constexpr (F32 && NJ == 2)
                __builtin_amdgcn_raw_buffer_store_b64(
                    u32x2{__float_as_uint(x), __float_as_uint(y)}, out, at, 0, kAux);
            else if constexpr (F32)
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), out, at, 0, kAux);
            else if constexpr (NJ == 2)
                __builtin_amdgcn_raw_buffer_store_b32(bf16_pack2(x, y), out, at, 0, kAux);
            else
                __builtin_amdgcn_raw_buffer_store_b16((uint16_t)bf16_pack2(x, x), out, at, 0, kAux);
        }
    }
    return W::kStores;
}

template <bool F32, bool PAST, bool TALL>
__device__ __forceinline__ void run_tiles(const Fp4GemmArgs& p, const Schedule& sched,
                                          unsigned char* smem) {
    constexpr int kSlot = Ring<TALL>::kSlot;
    const int nb = p.K / 32;
    Run c;
    c.S = (nb + 7) / 8;
    c.tail = nb & 7;
    c.slabs = slab_plan(c.S, !(nb & 3) && !(((uintptr_t)p.as | (uintptr_t)p.ws) & 3), TALL);
    const long long Q = sched.items();
    const int xcd = blockIdx.x & 7, step = gridDim.x >> 3, end = (int)(Q * (xcd + 1) / 8);
    int q = (int)(Q * xcd / 8) + (int)(blockIdx.x >> 3);
    if (q >= end) return;
    Feed<TALL> f{sched};
    f.step = step;
    f.end = end;
    f.S = c.S;
    f.q = q;
    sched.find(q, f.t);
    f.set(p);
    Tile t = f.t;
    if (c.S >= 3) f.slab(0);
    f.stage(p, 0);
    f.stage(p, kSlot);
    if constexpr (TALL) {
        wait_vm<Feed<TALL>::kCopies>();
    } else {
        f.template copy<0>(p, 2 * kSlot);
        wait_vm<Feed<TALL>::kCopies + half_copies()>();
    }
    if (c.tail && c.S == 1) zeros(smem, 0, c.tail);
    __syncthreads();
    for (int slot = 0, stored = 0;;) {
        const int blocks = (t.valid + 31) >> 5;
        auto tile = [&](auto mb) {
            stored = run_tile<F32, PAST, decltype(mb)::value, TALL>(p, t, f, c, slot, stored, smem);
        };
        if constexpr (TALL) {
            if (blocks <= 4) tile(std::integral_constant<int, 4>());
            else if (blocks <= 6) tile(std::integral_constant<int, 6>());
            else tile(std::integral_constant<int, 8>());
        } else {
            switch (blocks) {
                case 1: tile(std::integral_constant<int, 1>()); break;
                case 2: tile(std::integral_constant<int, 2>()); break;
                case 3: tile(std::integral_constant<int, 3>()); break;
                default: tile(std::integral_constant<int, 4>()); break;
            }
        }
        q += step;
        if (q >= end) break;
        if (c.S >= 3) t = f.t;
        else sched.find(q, t);
    }
}

// Persistent grid, one workgroup a CU
template <bool F32, bool PAST>
__global__ __launch_bounds__(kThreads) void gemm_mxfp4_kernel(Fp4GemmArgs p) {
    extern __shared__ __align__(16) unsigned char smem[];
    Schedule sched;
    sched.set(p, threadIdx.x & 63);
    if (sched.tall) run_tiles<F32, PAST, true>(p, sched, smem);
    else run_tiles<F32, PAST, false>(p, sched, smem);
}

// Outputs above this are stored past the caches (nontemporal), which the operands
// then have for themselves: with a kernel behind that reads them (quantise) 384
// groups x 128 rows x 4096 x 2048 490 -> 484 us with bf16 outputs (201 MB), 548
// -> 532 fp32 (403), 32768 x 1024 x 4096 fp32 (537) 285 -> 260; but 65.1 -> 72.6
// for 8192 x 1024 x 4096 (134), 63.8 -> 65.2 for 64 groups of 24576 rows x 2048 x
// 1024 bf16 (50), where it finds them in the 256 MB of cache otherwise, though
// the product alone took 60 -> 46 us in 64 groups of 16384 rows x 1024 x 2048.
constexpr size_t kKept = size_t(160) << 20;

template <bool F32, bool PAST>
hipError_t launch(const Fp4GemmArgs& g, hipStream_t stream) {
    static DeviceSetup setup;
    long long grid = 0, unused = 0;
    const hipError_t err =
        device_setup(setup, grid, unused, [](int, long long& gr, long long&) {
            gr = (device_cu_count() + 7) & ~7;
            return hipFuncSetAttribute((const void*)gemm_mxfp4_kernel<F32, PAST>,
                                       hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
        });
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL((gemm_mxfp4_kernel<F32, PAST>), dim3((unsigned)grid), dim3(kThreads), kLds,
                       stream, g);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_gemm_mxfp4(bool f32, const Fp4GemmArgs& g, hipStream_t stream) {
    if (g.K < 32 || g.K % 32 || g.N < 16 || g.N % 16 || g.G < 1) return hipErrorInvalidValue;
    const bool past = (size_t)g.rows * g.N * (f32 ? 4 : 2) > kKept;
    return f32 ? past ? launch<true, true>(g, stream) : launch<true, false>(g, stream)
               : past ? launch<false, true>(g, stream) : launch<false, false>(g, stream);
}

}  // namespace moe
