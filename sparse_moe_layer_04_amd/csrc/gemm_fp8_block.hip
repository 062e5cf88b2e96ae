// Grouped matrix product of 8-bit rows and weights with a scale for each
// block of 128: for the rows r of group g,
//   out[r, n] = sum_b a_scale[r, b] w_scale[g, n / 128, b]
//                     sum_{k in block b} a[r, k] w[g, n, k],
// codes E4M3, scales fp32, weights as checkpoints hold them ([G, N, K]
// row-major codes, [G, N / 128, K / 128] scales).  K and N are multiples of
// 16; the last block of either may be short.
//
// The sum over a block of 128 is one accumulation on the matrix cores from
// zero; it is then multiplied by the product of the two scales and added to
// the running fp32 sum on the vector units (one fma an output and block),
// beside the next block's matrix products.  Where that product is no normal
// number the sum is scaled in two steps instead (its test costs 1 to 1.5%
// with bf16 output).
//
// Which matrix cores.  The 8-bit ones truncate the products of eight
// neighbouring k to 13 binary places below the largest of the eight before
// they add them (measured: beside +-2^16 in the eight 2^3 stays, 2^2 goes, in
// other eights and beside the sum so far values down to 2^-7 stay), so at most
// 7 2^-13 of sum |products| is lost.  Measured in 2-norms over 4096 terms
// against 64-bit sums: 1.5e-5 of the result for normal codes, 2.1e-5, 3.7e-5
// and 6.8e-5 where magnitudes vary by 2^+-1, 2 and 4, against 7e-8 to 1.2e-7
// for the bf16 ones, on which a product of two E4M3 values is exact.  An
// output rounded to bf16 (half a step: 2^-9 to 2^-8 of it) takes the 8-bit
// ones; an fp32 output and the SwiGLU's quantised h take the bf16 ones at half
// the rate, their codes decoded in registers: the first would show the loss,
// and of the second the codes of small values would move by several steps
// (E4M3 goes down to 2^-18 of a block's largest value).
//
// Tile: up to 160 rows x 256 weight rows (SwiGLU: 128 features, gate and up
// rows interleaved by 16 so that a wave holds both of a feature), 8 waves of
// 64 x 64 or (rows of the tile) x 32 outputs in registers, one 128-wide block
// of K a stage.  256 weight rows, since each CU moves the codes of both
// operands once a tile: at 128 x 256 that is 85 products a byte.  160 rows,
// since the weights of a group of 129 to 160 rows are otherwise fetched twice
// (384 groups of 128 rows on average x 4096 x 2048, tiles of up to 128 rows
// against 160: 1193 and 1036 us with fp32, 839 and 736 with bf16 output).
//
// Both operands go to LDS as codes, by copies that pass no register, through
// a ring of 3 slots of 52.75 KB: a block's copies are issued two stages before
// they are multiplied, so that operand reads run ahead of the matrix products
// across the end of a stage; one barrier a stage.  (Through registers, a block
// less in flight: 384 groups x 128 rows x 4096 x 2048 with bf16 output took
// 1117 us, with the copies 853.)  A wave's copy covers 8 rows x 128 bytes
// (whole lines of the row-major operands); LDS row r holds its 16-byte chunk c
// at c ^ ((r >> 1) & 7), so that the lanes of an operand read (32 rows, one
// chunk index) spread over the banks.
//
// Bound and measured, 1 group x 8192 rows x 4096 x 2048: the matrix cores, at
// 1025 to 1136 TFLOP/s with fp32 output (bf16 cores) and 1740 to 1870 with
// bf16 output (8-bit cores), by the inputs' values and the card's clock (where
// a large library product of the same types reaches 1395 and 2684).  With neither decoding nor scaling the same loop
// reaches 1379 (100 us; decoding adds 16, scaling 5 to 10) and, without the
// scaling, 2160 (64 us; scaling adds 9): the vector units run beside the
// matrix cores, and the clock drops under both.  384 groups x 128 rows x 4096
// x 2048: 3.2 GB of weights, 720 to 736 us with bf16 output (memory, 5 TB/s),
// 0.98 to 1.04 ms with fp32 (cores and memory in turn).  Ten rows a group:
// memory, 5.5 TB/s.  One row of each of few groups: the chain of K's blocks on
// few CUs (12 groups x 4096 x 544: 36 tiles, 16 us with bf16, 25 with fp32).
#include "lds_ring.h"
#include "row_tiles.h"

namespace moe {
namespace {

constexpr int BM = 160;                    // rows a tile, at most
constexpr int BN = 256;                    // weight rows a tile
constexpr int BK = 128;                    // K a stage: one block
constexpr int kThreads = 512;
constexpr int kSlotW = BN * BK;
constexpr int kSlotS = kSlotW + BM * BK;   // the stage's scales: BM rows', then two
constexpr int kSlot = kSlotS + 768;        // of the weights
constexpr int kRing = 3 * kSlot;
constexpr int kMaxX = 8 * BM;              // SwiGLU: the waves' row exponents, a byte each
constexpr int kLds = kRing + kMaxX;
static_assert(kLds <= 160 * 1024 && kSlot % 128 == 0, "three slots of LDS");

struct Tile {
    int g, row0, valid, n0;                // n0: first weight row (SwiGLU: feature)
};

// The copies of a tile's operands into LDS, set up once per tile: buffer
// resources over the tile's rows (wave-uniform base, 32-bit offsets; rows past
// the tile's or the matrix's end lie past them and fetch nothing).  A wave's
// copy fills 8 LDS rows of 128 bytes; the place of a chunk in its row is
// swizzled, so the lanes fetch swizzled chunks.
// copies a wave and stage: 4 of W, one for each 64 rows of A, the scales
constexpr int row_copies(int blocks) { return (blocks + 1) / 2; }
constexpr int kEarly = 3;                  // of them, issued in the stage before
template <int EPI>
struct Fetch {
    u32x4 wsrc, asrc;
    int wo[4], ao[3];
    const float* sp;

    __device__ __forceinline__ void set(const Fp8GemmArgs& p, const Tile& t) {
        constexpr bool SW = EPI == FP8_SWIGLU;
        const int tid = threadIdx.x, lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int K = p.K, N = p.N, S = (K + BK - 1) / BK, nbn = (N + 127) / 128;
        const int lr = tid >> 3, c = (tid & 7) ^ swz(lr);   // chunk c of row lr + 64 q
        // SwiGLU: LDS row R is row R & 15 of 16 features' gate (R & 16 == 0)
        // or up rows; R & 16 is the same for a wave and all q
        const bool up = SW && (wave & 2);
        const size_t wfirst = ((size_t)t.g * N + t.n0) * K;
        wsrc = uniform_rsrc((up ? p.w2 : p.w1) + wfirst, (size_t)min(N - t.n0, BN) * K);
        asrc = uniform_rsrc(p.a + (size_t)t.row0 * K, (size_t)t.valid * K);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int R = lr + 64 * q;
            wo[q] = (SW ? 16 * (R >> 5) + (R & 15) : R) * K + 16 * c;
        }
        // (the last 32 rows twice, the same bytes to the same place, so that
        // every wave issues the same number of copies)
#pragma unroll
        for (int q = 0; q < 3; ++q) ao[q] = ((q == 2 ? lr & 31 : lr) + 64 * q) * K + 16 * c;
        // scales, words of the slot: the rows', at BM those of the tile's two
        // 128-blocks of weight rows, or of gate and up (waves 2 to 7 the same)
        const int word = 64 * min(wave, 2) + lane, nb0 = t.n0 / 128;
        if (word < BM)
            sp = p.as + (size_t)(t.row0 + min(word, t.valid - 1)) * S;
        else if constexpr (SW)
            sp = (word & 1 ? p.s2 : p.s1) + ((size_t)t.g * nbn + nb0) * S;
        else
            sp = p.s1 + ((size_t)t.g * nbn + min(nb0 + (word & 1), nbn - 1)) * S;
    }

    // Copy q (of 4 + NA + 1) of stage j into the slot at LDS byte `at`.  Stage 0
    // takes K's last block, the short one if any, stage j block j - 1.  (Every
    // stage issues its copies: past the last stage with offsets past the
    // resources.)  `past`: the bytes that this thread's chunk reaches past K in
    // the last block; it fetches the row's last chunk instead, which is
    // overwritten by zeros when it has landed.
    template <int NA>
    __device__ __forceinline__ void copy(int q, int j, int S, int past, int at) const {
        const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        const int b = j == 0 ? S - 1 : min(j, S) - 1;
        const int back = j == 0 ? past : 0, out = j < S ? 0 : (int)0x80000000;
        if (q < 4)
            copy16(wsrc, (wo[q] - back) | out, b * BK, at + q * 64 * BK + wave * 1024);
        else if (q < 4 + NA)
            copy16(asrc, (ao[q - 4] - back) | out, b * BK,
                   at + kSlotW + (q - 4) * 64 * BK + (q == 6 ? wave & 3 : wave) * 1024);
        else
            copy4(sp + b, at + kSlotS + min(wave, 2) * 256);
    }
    template <int NA, int Q0, int Q1>
    __device__ __forceinline__ void copies(int j, int S, int past, int at) const {
#pragma unroll
        for (int q = Q0; q < Q1 && q < 4 + NA + 1; ++q) copy<NA>(q, j, S, past, at);
    }
    // what is on its way when a tile (of NA row copies) begins
    template <int NA>
    __device__ __forceinline__ void first(int S, int past) const {
        copies<NA, 0, 8>(0, S, past, 0);
        copies<NA, 0, 8>(1, S, past, kSlot);
        copies<NA, 0, kEarly>(2, S, past, 2 * kSlot);
    }
    __device__ __forceinline__ void first_stages(int valid, int S, int past) const {
        if (valid <= 64) first<1>(S, past);
        else if (valid <= 128) first<2>(S, past);
        else first<3>(S, past);
    }
};

// The stages of a tile of five blocks of rows (its registers do not hold two
// sets of operands): the same steps, taken a product at a time, the operands
// of a product made ready during the one before, those of W once a step.
template <int EPI, class Turn, class Scales, class ReadS, class Add>
__device__ __forceinline__ void run_five(const Fetch<EPI>& f, unsigned char* ring, int rdw, int rda,
                                         int S, int past, const Turn& turn, const Scales& scales,
                                         const ReadS& read_s, const Add& add_part,
                                         f32x16 (&part)[5][1]) {
    constexpr int MI = 5;
    f32x16 zero;
#pragma unroll
    for (int e = 0; e < 16; ++e) zero[e] = 0.0f;
    int slot = 0;
    auto read = [&](int at, int q, int i) {
        return *(const u32x4*)(ring + (at ^ (q << 5)) + i * 32 * BK);
    };
    if constexpr (EPI != FP8_OUT_BF16) {
        // product L = 5 h + i: step h (16 of K), block i.  ra[i] holds 32 of K,
        // read again as soon as its second half is decoded
        u32x4 rw[2], ra[MI];
        bf16x8 w[2], a[2];
        auto half = [](const u32x4& v, int h) {
            return h ? fp8x8_to_bf16x8(u32x2{v[2], v[3]}, 1.0f)
                     : fp8x8_to_bf16x8(u32x2{v[0], v[1]}, 1.0f);
        };
        rw[0] = read(rdw, 0, 0);
#pragma unroll
        for (int i = 0; i < MI; ++i) ra[i] = read(rda, 0, i);
        w[0] = half(rw[0], 0);
        a[0] = half(ra[0], 0);
        for (int j = 0; j < S; ++j) {
            const int next = slot == 2 * kSlot ? 0 : slot + kSlot;
            const int last = next == 2 * kSlot ? 0 : next + kSlot;
            scales();                               // of block j - 1
            read_s(slot);
            static_for<0, 8 * MI>([&](auto index) {
                constexpr int L = decltype(index)::value, h = L / MI, i = L % MI;
                constexpr int L2 = (L + 1) % (8 * MI), h2 = L2 / MI, i2 = L2 % MI;
                if constexpr (L == 6 * MI - 1) turn();
                if constexpr (i == 0 && h < 5)
                    f.template copies<3, kEarly + h, kEarly + h + 1>(j + 2, S, past, last);
                if constexpr (i == 1 && h >= 6)
                    f.template copies<3, h - 6, h == 7 ? kEarly : 1>(j + 3, S, past, slot);
                // W of the next 32 of K
                if constexpr (i == 0 && h % 2 == 0)
                    rw[h / 2 + 1 & 1] = h == 6 ? read(rdw + next, 0, 0) : read(rdw + slot, h / 2 + 1, 0);
                // the next product's operands
                a[L2 & 1] = half(ra[i2], h2 & 1);
                if constexpr (i2 == 0) w[h2 & 1] = half(rw[h2 / 2 & 1], h2 & 1);
                if constexpr (h2 & 1)
                    ra[i2] = h2 == 7 ? read(rda + next, 0, i2) : read(rda + slot, h2 / 2 + 1, i2);
                if constexpr (h == 0) add_part(i, 0);
                part[i][0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    w[h & 1], a[L & 1], h == 0 ? zero : part[i][0], 0, 0, 0);
                if constexpr (i == MI - 1) __builtin_amdgcn_sched_barrier(0);
            });
            slot = next;
        }
    } else {
        // product L = 5 s + i: half s of the block, rows' operands two ahead;
        // beside product TURN the last of them, then the barrier that gives the
        // block's slot away
        constexpr int TURN = 2 * MI - 3;
        u32x4 rw[2][2], ra[2][2];
        auto read2 = [&](u32x4 (&r)[2], int at, int s, int i) {
            r[0] = read(at, 2 * s, i);
            r[1] = read(at, 2 * s + 1, i);
        };
        auto cat = [](const u32x4 (&r)[2]) {
            return v8i{(int)r[0][0], (int)r[0][1], (int)r[0][2], (int)r[0][3],
                       (int)r[1][0], (int)r[1][1], (int)r[1][2], (int)r[1][3]};
        };
        read2(rw[0], rdw, 0, 0);
        read2(ra[0], rda, 0, 0);
        read2(ra[1], rda, 0, 1);
        for (int j = 0; j < S; ++j) {
            const int next = slot == 2 * kSlot ? 0 : slot + kSlot;
            const int last = next == 2 * kSlot ? 0 : next + kSlot;
            scales();                               // of block j - 1
            read_s(slot);
            read2(rw[1], rdw + slot, 1, 0);
            static_for<0, 2 * MI>([&](auto index) {
                constexpr int L = decltype(index)::value, s = L / MI, i = L % MI;
                constexpr int L2 = (L + 2) % (2 * MI);
                if constexpr (s == 0) add_part(i, 0);
                part[i][0] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    cat(rw[s]), cat(ra[L & 1]), s == 0 ? zero : part[i][0], 0, 0, 0, 127, 0, 127);
                if constexpr (kEarly + L < 8)
                    f.template copies<3, kEarly + L, kEarly + L + 1>(j + 2, S, past, last);
                static_assert(L2 < 2 ? L >= TURN : L <= TURN,
                              "the block's reads before the barrier, the next one's after it");
                if constexpr (L2 >= 2) read2(ra[L & 1], rda + slot, L2 / MI, L2 % MI);
                if constexpr (L == TURN) {
                    turn();
                    read2(rw[0], rdw + next, 0, 0);
                }
                if constexpr (L2 < 2) read2(ra[L & 1], rda + next, L2 / MI, L2 % MI);
                if constexpr (L >= TURN)
                    f.template copies<3, L - TURN, L - TURN + 1>(j + 3, S, past, slot);
                __builtin_amdgcn_sched_barrier(0);
            });
            slot = next;
        }
    }
}

// One tile, whose first three stages are on their way into the ring; sends the
// next tile's (if there are more) off before this one's results are written.
template <int EPI, int MB>
__device__ __forceinline__ void run_tile(const Fp8GemmArgs& p, const Tile& t, const Tile& next_t,
                                         bool more, int past, unsigned char* ring) {
    // (the thread's place as a value of this variant's own: address terms
    // shared by the variants would be kept, or spilled, for all of them)
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, half = lane >> 5, l32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    Fetch<EPI> f;
    f.set(p, t);
    // waves: WM along the rows x WN along the weight rows, each MI x NJ
    // blocks of 32 x 32
    constexpr int WM = MB == 4 ? 2 : 1, WN = 8 / WM, MI = MB / WM, NJ = 8 / WN;
    constexpr bool SW = EPI == FP8_SWIGLU;
    constexpr bool EXACT = EPI != FP8_OUT_BF16;
    constexpr int NA = row_copies(MB), kCopies = 4 + NA + 1;
    const int wm = wave / WN, wn = wave % WN;
    const int K = p.K, N = p.N;
    const int S = (K + BK - 1) / BK;

    // LDS rows 32 apart share their swizzle, so the rest of an operand's
    // address is an immediate; the chunk index enters it by exclusive or
    const int rd0 = l32 * BK + ((half ^ swz(l32)) << 4);
    const int rdw = wn * NJ * 32 * BK + rd0;
    const int rda = kSlotW + wm * MI * 32 * BK + rd0;
    const int rds = kSlotS + (wm * MI * 32 + l32) * 4;
    const int rdsw = kSlotS + BM * 4 + (SW ? 0 : wn * NJ * 32 / 128) * 4;
    float sa[MI], sw1 = 1.0f, sw2 = 1.0f;
#pragma unroll
    for (int i = 0; i < MI; ++i) sa[i] = 1.0f;
    auto read_s = [&](int slot) {
#pragma unroll
        for (int i = 0; i < MI; ++i) sa[i] = *(const float*)(ring + rds + slot + i * 128);
        sw1 = *(const float*)(ring + rdsw + slot);
        sw2 = SW ? *(const float*)(ring + rdsw + slot + 4) : sw1;
    };

    f32x16 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int n = 0; n < NJ; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][n][e] = 0.0f;

    // The stage's pipeline, in steps of 16 (bf16) or 64 (8-bit) of K.  In a
    // step the matrix cores take the operands made ready in the step before,
    // the vector units decode the next step's and, in the stage's first one,
    // scale and add the sums of the block before (tile by tile, ahead of the
    // product that starts the tile's new block), and LDS reads run two (one)
    // steps ahead.  The barrier stands where the last reads of block j have
    // been issued and the first of block j + 1 are next.
    f32x16 part[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int n = 0; n < NJ; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) part[i][n][e] = 0.0f;
    float s1[MI], s2[MI];
    // The sums of the last block read are due: the factors that add_part
    // multiplies them by.  A product of two scales that is no normal number
    // (subnormal, with bits lost; infinite; zero) is not taken: the sums are
    // added here, by the scales' mantissas and exponents, which rounds once
    // and overflows or vanishes where the result does.
    auto scales = [&]() {
        constexpr int kNotNormal = 0x2f7;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            s1[i] = sa[i] * sw1;
            s2[i] = sa[i] * sw2;
            odd |= __builtin_amdgcn_classf(s1[i], kNotNormal);
            if constexpr (SW) odd |= __builtin_amdgcn_classf(s2[i], kNotNormal);
        }
        if (__builtin_expect(__builtin_amdgcn_ballot_w64(odd) != 0u, 0)) {
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const float m = __builtin_amdgcn_frexp_mantf(sa[i]);
                const float m1 = m * __builtin_amdgcn_frexp_mantf(sw1);
                const float m2 = m * __builtin_amdgcn_frexp_mantf(sw2);
                const int x = __builtin_amdgcn_frexp_expf(sa[i]);
                const int x1 = x + __builtin_amdgcn_frexp_expf(sw1);
                const int x2 = x + __builtin_amdgcn_frexp_expf(sw2);
#pragma unroll
                for (int n = 0; n < NJ; ++n)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        acc[i][n][e] += __builtin_ldexpf(
                            part[i][n][e] * (SW && e >= 8 ? m2 : m1), SW && e >= 8 ? x2 : x1);
                s1[i] = s2[i] = 0.0f;
            }
        }
    };
    auto add_part = [&](int i, int n) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            acc[i][n][e] =
                __builtin_fmaf(part[i][n][e], SW && e >= 8 ? s2[i] : s1[i], acc[i][n][e]);
    };
    f32x16 zero;
#pragma unroll
    for (int e = 0; e < 16; ++e) zero[e] = 0.0f;
    constexpr int NT = MI * NJ;

    // stage 0 has landed; zeros over this thread's own copies past K
    wait_vm<kCopies + kEarly>();
    if (past) {
        const u32x4 z = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int q = 0; q < (BN + BM + 63) / 64; ++q)
            *(u32x4*)(ring + q * 64 * BK + (q == (BN + BM) / 64 ? tid & 255 : tid) * 16) = z;
    }
    __syncthreads();
    // The middle of stage j: stage j + 1's block has landed and every wave has
    // read stage j's, whose slot takes stage j + 3's.  The copies are spread
    // over the steps, one at a time (all at once hold every wave until the
    // memory pipeline has taken 48 KB): the first after this barrier, the rest in the
    // next stage's steps before its own.
    auto turn = [&]() {
        wait_vm<kCopies>();
        __syncthreads();
    };

    using std::integral_constant;
    if constexpr (MB == 5) {
        run_five<EPI>(f, ring, rdw, rda, S, past, turn, scales, read_s, add_part, part);
    } else if constexpr (EXACT) {
        u32x4 rw[2][NJ], ra[2][MI];        // 32 of K: the codes of two steps
        bf16x8 w[2][NJ], a[2][MI];         // operands of a step
        auto read = [&](int slot, int q, auto set) {
            constexpr int B = decltype(set)::value;
#pragma unroll
            for (int n = 0; n < NJ; ++n)
                rw[B][n] = *(const u32x4*)(ring + ((rdw + slot) ^ (q << 5)) + n * 32 * BK);
#pragma unroll
            for (int i = 0; i < MI; ++i)
                ra[B][i] = *(const u32x4*)(ring + ((rda + slot) ^ (q << 5)) + i * 32 * BK);
        };
        // step h of the block from raw set h / 2 % 2 into operand set h % 2
        auto decode = [&](auto step) {
            constexpr int h = decltype(step)::value, B = (h >> 1) & 1, o = 2 * (h & 1);
#pragma unroll
            for (int n = 0; n < NJ; ++n)
                w[h & 1][n] = fp8x8_to_bf16x8(u32x2{rw[B][n][o], rw[B][n][o + 1]}, 1.0f);
#pragma unroll
            for (int i = 0; i < MI; ++i)
                a[h & 1][i] = fp8x8_to_bf16x8(u32x2{ra[B][i][o], ra[B][i][o + 1]}, 1.0f);
        };
        auto multiply = [&](auto step) {
            constexpr int h = decltype(step)::value;
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int n = 0; n < NJ; ++n) {
                    if constexpr (h == 0) add_part(i, n);
                    part[i][n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        w[h & 1][n], a[h & 1][i], h == 0 ? zero : part[i][n], 0, 0, 0);
                }
        };
        auto step = [&](auto st) {
            constexpr int h = decltype(st)::value;
            decode(integral_constant<int, (h + 1) & 7>());
            multiply(st);
            // one product, then its share of the vector instructions (one or two
            // products a step do not cover a step's: what is left open there
            // saves 5%, 12 groups x 1 row x 4096 x 544 25.3 us to 24.0)
            if constexpr (NT >= 3) {
                constexpr int V = 4 * (MI + NJ) / NT + (h == 0 ? 16 : 0);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x002, h == 0 ? V : 0, 0);
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x002, h == 0 ? 0 : V, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        using H0 = integral_constant<int, 0>;
        using H1 = integral_constant<int, 1>;
        read(0, 0, H0());
        read(0, 1, H1());
        decode(H0());
        int slot = 0;
        for (int j = 0; j < S; ++j) {
            const int next = slot == 2 * kSlot ? 0 : slot + kSlot;
            const int last = next == 2 * kSlot ? 0 : next + kSlot;
            scales();                               // of block j - 1
            read_s(slot);
            f.template copies<NA, 3, 4>(j + 2, S, past, last);
            step(H0());
            read(slot, 2, H0());
            f.template copies<NA, 4, 5>(j + 2, S, past, last);
            step(H1());
            f.template copies<NA, 5, 6>(j + 2, S, past, last);
            step(integral_constant<int, 2>());
            read(slot, 3, H1());
            f.template copies<NA, 6, 7>(j + 2, S, past, last);
            step(integral_constant<int, 3>());
            f.template copies<NA, 7, 8>(j + 2, S, past, last);
            step(integral_constant<int, 4>());
            turn();
            read(next, 0, H0());                    // (past the end: not used)
            f.template copies<NA, 0, 1>(j + 3, S, past, slot);
            step(integral_constant<int, 5>());
            f.template copies<NA, 1, 2>(j + 3, S, past, slot);
            step(integral_constant<int, 6>());
            read(next, 1, H1());
            f.template copies<NA, 2, 3>(j + 3, S, past, slot);
            step(integral_constant<int, 7>());
            slot = next;
        }
    } else {
        // (any order of K within the block will do, the same for both)
        u32x4 rw[2][NJ][2], ra[2][MI][2];
        auto read = [&](int slot, auto set) {
            constexpr int B = decltype(set)::value;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int n = 0; n < NJ; ++n)
                    rw[B][n][r] =
                        *(const u32x4*)(ring + ((rdw + slot) ^ ((2 * B + r) << 5)) + n * 32 * BK);
#pragma unroll
                for (int i = 0; i < MI; ++i)
                    ra[B][i][r] =
                        *(const u32x4*)(ring + ((rda + slot) ^ ((2 * B + r) << 5)) + i * 32 * BK);
            }
        };
        auto cat = [](const u32x4 (&r)[2]) {
            return v8i{(int)r[0][0], (int)r[0][1], (int)r[0][2], (int)r[0][3],
                       (int)r[1][0], (int)r[1][1], (int)r[1][2], (int)r[1][3]};
        };
        // the products of a step, a copy (of up to four) ahead of each
        auto multiply = [&](auto set, auto copy) {
            constexpr int B = decltype(set)::value;
            auto tile = [&](auto index) {
                constexpr int x = decltype(index)::value, i = x / NJ, n = x % NJ;
                if constexpr (x < NT) {
                    if constexpr (B == 0) add_part(i, n);
                    part[i][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        cat(rw[B][n]), cat(ra[B][i]), B == 0 ? zero : part[i][n], 0, 0, 0, 127, 0,
                        127);
                }
                copy(index);
                __builtin_amdgcn_sched_barrier(0);
            };
            tile(std::integral_constant<int, 0>());
            tile(std::integral_constant<int, 1>());
            tile(std::integral_constant<int, 2>());
            tile(std::integral_constant<int, 3>());
        };
        using B0 = std::integral_constant<int, 0>;
        using B1 = std::integral_constant<int, 1>;
        read(0, B0());
        int slot = 0;
        for (int j = 0; j < S; ++j) {
            const int next = slot == 2 * kSlot ? 0 : slot + kSlot;
            const int last = next == 2 * kSlot ? 0 : next + kSlot;
            scales();                               // of block j - 1
            read_s(slot);
            read(slot, B1());
            multiply(B0(), [&](auto q) {
                constexpr int c = kEarly + decltype(q)::value;
                f.template copies<NA, c, c == 6 ? kCopies : c + 1>(j + 2, S, past, last);
            });
            turn();
            read(next, B0());                       // (past the end: not used)
            multiply(B1(), [&](auto q) {
                constexpr int c = decltype(q)::value;
                if constexpr (c < kEarly) f.template copies<NA, c, c + 1>(j + 3, S, past, slot);
            });
            slot = next;
        }
    }
    // (every wave has read the last stage; what the ring still holds is unused)
    if (more) {
        Fetch<EPI> nf;
        nf.set(p, next_t);
        nf.first_stages(next_t.valid, S, past);
    }
    scales();
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int n = 0; n < NJ; ++n) add_part(i, n);

    // Epilogues, from the registers: lane l holds, of row l % 32 of its block,
    // weight rows 8 q + 4 (l / 32) + (0 .. 3), q < 4.  The stores of a wave
    // fill 32 to 64 bytes of a row each; the L2 joins them to lines.
    if constexpr (EPI == FP8_OUT_F32) {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int r = (wm * MI + i) * 32 + l32;
            float* o = (float*)p.out + (size_t)(t.row0 + r) * N + t.n0;
#pragma unroll
            for (int n = 0; n < NJ; ++n)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int col = (wn * NJ + n) * 32 + 8 * q + 4 * half;
                    if (r < t.valid && t.n0 + col < N)
                        *(f32x4*)(o + col) = f32x4{acc[i][n][4 * q], acc[i][n][4 * q + 1],
                                                   acc[i][n][4 * q + 2], acc[i][n][4 * q + 3]};
                }
        }
    } else if constexpr (EPI == FP8_OUT_BF16) {
        // (the half-waves exchange, so that a lane holds 8 columns in a row)
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int r = (wm * MI + i) * 32 + l32;
            uint16_t* o = (uint16_t*)p.out + (size_t)(t.row0 + r) * N + t.n0;
#pragma unroll
            for (int n = 0; n < NJ; ++n)
#pragma unroll
                for (int q = 0; q < 4; q += 2) {
                    const f32x16& v = acc[i][n];
                    const u32x2 x = swap_halves(bf16_pack2(v[4 * q], v[4 * q + 1]),
                                                bf16_pack2(v[4 * q + 4], v[4 * q + 5]));
                    const u32x2 y = swap_halves(bf16_pack2(v[4 * q + 2], v[4 * q + 3]),
                                                bf16_pack2(v[4 * q + 6], v[4 * q + 7]));
                    const int col = (wn * NJ + n) * 32 + 8 * (q + half);
                    if (r < t.valid && t.n0 + col < N)
                        *(u32x4*)(o + col) = u32x4{x[0], y[0], x[1], y[1]};
                }
        }
    } else {
        // h = SwiGLU in fp32, quantised along the tile's 128 features.  The
        // exponent of a row's scale is the largest of its parts' exponents:
        // this lane's and its half-wave partner's features, the other waves'
        // (a byte each; the lowest where a part is all zeros)
        int8_t* xs = (int8_t*)(ring + kRing);         // [WN][BM]
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            float m = 0.0f;
#pragma unroll
            for (int n = 0; n < NJ; ++n) {
                const bool in = t.n0 + 16 * (wn * NJ + n) < N;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = clamped_swiglu(acc[i][n][e], acc[i][n][e + 8], p.clamp_limit,
                                                   p.clamp_mode);
                    acc[i][n][e] = in ? v : 0.0f;
                    m = fmaxf(m, finite_abs(acc[i][n][e]));
                }
            }
            m = fmaxf(m, __shfl_xor(m, 32, 64));
            if (half == 0)
                xs[wn * BM + (wm * MI + i) * 32 + l32] = m > 0.0f ? block_exponent(m) : -128;
        }
        __syncthreads();
        const int nbf = (N + 127) / 128;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int r = (wm * MI + i) * 32 + l32;
            int X = -128;
#pragma unroll
            for (int w = 0; w < WN; ++w) X = max(X, (int)xs[w * BM + r]);
            X = X == -128 ? 0 : X;
            const float inv = pow2(-X);
            uint8_t* o = (uint8_t*)p.out + (size_t)(t.row0 + r) * N + t.n0;
#pragma unroll
            for (int n = 0; n < NJ; ++n) {
                const f32x16& v = acc[i][n];
                const u32x2 w = swap_halves(e4m3_pack4(v[0], v[1], v[2], v[3], inv),
                                            e4m3_pack4(v[4], v[5], v[6], v[7], inv));
                const int f0 = 16 * (wn * NJ + n);
                if (r < t.valid && t.n0 + f0 < N) *(u32x2*)(o + f0 + 8 * half) = w;
            }
            if (wn == 0 && half == 0 && r < t.valid)
                p.out_scale[(size_t)(t.row0 + r) * nbf + t.n0 / 128] = pow2(X);
        }
    }
}

// Row tiles of a group of n rows, tiles of up to `blocks` blocks of 32 rows.
// 4 and 5 are the usual ones: a group of up to 160 rows is one tile (a second
// one would fetch the group's weights again), a larger one has tiles of up to
// 128 or 160 rows.  1 to 3 are for few tiles, where CUs would have none: lower
// ones use more CUs, and the weights they share come from the L2.
// 16 groups x 160 rows x 4096 x 256: 64 us with one tile a group, 27 with five
// (fp32 output; bf16 35 and 18).
constexpr int kTallest = BM / 32;
__device__ __forceinline__ int row_tiles(int n, int blocks) {
    const int c = row_blocks(n);
    if (blocks >= 4) return c <= kTallest ? c > 0 : blocks == 4 ? (c + 3) >> 2 : (c + 4) / 5;
    return blocks == 1 ? c : blocks == 2 ? (c + 1) >> 1 : (c + 2) / 3;
}

// Persistent grid, one workgroup a CU.  Items are (group, band of kBand
// m-tiles, n-tile, m-tile), the 8 XCDs take contiguous ranges, so that the
// m-tiles of a weight tile and the n-tiles of a group's rows meet in one XCD's
// L2: the 32 items that its CUs work on are 8 m-tiles x 4 n-tiles, the shape
// that needs the fewest rows of both.  (1 group x 8192 rows x 4096 x 2048 with
// a column of all m-tiles an XCD: 78 us with bf16, 130 with fp32 output; in
// bands of 8 72 and 121, of 16 73 and 126.)  A group's rows split evenly over
// its m-tiles.  The group of an item comes from a two-level sum that
// every wave keeps in registers: lane l holds the items before run l of
// ceil(G / 64) groups, and looks into the run that holds the item.
constexpr int kBand = 8;
static_assert(MOE_MAX_GROUPS <= 64 * 64, "one lane a run, one lane a group of a run");

template <int EPI>
__global__ __launch_bounds__(kThreads) void gemm_fp8_block_kernel(Fp8GemmArgs p) {
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int TN = EPI == FP8_SWIGLU ? BN / 2 : BN;
    const int tid = threadIdx.x, lane = tid & 63;
    const int G = p.G, rows = p.rows, S = (p.K + BK - 1) / BK;
    const int NT = (p.N + TN - 1) / TN;
    auto clamped = [&](int v) { return min(max(v, 0), rows); };
    const int run = (G + 63) / 64;
    // the row tiles of this lane's run, of up to 1 .. 5 blocks
    int tiles[kTallest + 1] = {};
    for (int i = 0; i < run; ++i) {
        const int g = lane * run + i;
        if (g < G) {
            const int n = max(clamped(p.offsets[g + 1]) - clamped(p.offsets[g]), 0);
#pragma unroll
            for (int b = 1; b <= kTallest; ++b) tiles[b] += row_tiles(n, b);
        }
    }
    int blocks = 4, mine = NT * tiles[4], upto = wave_scan(mine, lane);
    // Tiles of 160 rows where they save CUs a fifth of their rounds and more
    // (such a tile takes 1.18 to 1.26 times one of 128 with bf16, 1.24 to 1.30
    // with fp32 output).  64 groups of 126 to 3500 rows x 2048 x 1024, three
    // rounds for four: 91 us to 80 with bf16, 136 to 127 with fp32 output; 1
    // group x 20480 rows x 4096 x 4096, eight for ten: 360 to 364 us (not
    // taken).
    auto rounds = [&](int tiles) {
        const int cus = (int)gridDim.x;
        return (int)(((long long)tiles + cus - 1) / cus);
    };
    const int first = rounds(__builtin_amdgcn_readlane(upto, 63));
    if (first > 1 && __builtin_amdgcn_ballot_w64(tiles[4] != tiles[kTallest])) {
        const int sum = wave_scan(NT * tiles[kTallest], lane);
        if (rounds(__builtin_amdgcn_readlane(sum, 63)) * 5ll < first * 4ll) {
            blocks = kTallest;
            mine = NT * tiles[kTallest];
            upto = sum;
        }
    }
    // few tiles: the lowest of which every one still has a CU of its own
    if ((long long)rows * NT <= 96ll * gridDim.x &&
        __builtin_amdgcn_readlane(upto, 63) < (int)gridDim.x) {
#pragma unroll
        for (int b = 1; b <= 3; ++b) {
            const int sum = wave_scan(NT * tiles[b], lane);
            if (__builtin_amdgcn_readlane(sum, 63) > (int)gridDim.x) continue;
            blocks = b;
            mine = NT * tiles[b];
            upto = sum;
            break;
        }
    }
    const long long Q = __builtin_amdgcn_readlane(upto, 63);
    const int xcd = blockIdx.x & 7, step = gridDim.x >> 3;
    const int end = (int)(Q * (xcd + 1) / 8);
    auto find = [&](int q, Tile& t) {
        // the first lane whose sum passes q, then the groups of its run in
        // turn (scalar loads: a vector load would wait for the copies that are
        // on their way)
        const int r = __builtin_ctzll(__builtin_amdgcn_ballot_w64(upto > q));
        int local = q - __builtin_amdgcn_readlane(upto - mine, r);
        t.g = r * run;
        int r0 = clamped(scalar_load(p.offsets + t.g)), n, mt;
        for (;; ++t.g) {                             // (ends: the run holds item q)
            const int r1 = clamped(scalar_load(p.offsets + t.g + 1));
            n = max(r1 - r0, 0);
            mt = row_tiles(n, blocks);
            if (local < NT * mt || t.g + 1 >= G) break;
            local -= NT * mt;
            r0 = r1;
        }
        const int per = tile_rows(n, mt);
        const int band = local / (kBand * NT) * kBand, high = min(kBand, mt - band);
        local -= band * NT;
        t.n0 = local / high * TN;
        t.row0 = r0 + (band + local % high) * per;
        t.valid = min(per, r0 + n - t.row0);
    };
    // bytes that this thread's chunk of K's last block reaches past K
    const int past = max(0, (S - 1) * BK + 16 * ((tid & 7) ^ swz(tid >> 3)) + 16 - p.K);
    int q = (int)(Q * xcd / 8) + (int)(blockIdx.x >> 3);
    if (q >= end) return;
    Tile t;
    find(q, t);
    {
        Fetch<EPI> f;
        f.set(p, t);
        f.first_stages(t.valid, S, past);
    }
    for (;;) {
        const bool more = q + step < end;
        Tile next = t;
        if (more) find(q + step, next);
        switch ((t.valid + 31) >> 5) {
            case 1: run_tile<EPI, 1>(p, t, next, more, past, smem); break;
            case 2: run_tile<EPI, 2>(p, t, next, more, past, smem); break;
            case 3: run_tile<EPI, 3>(p, t, next, more, past, smem); break;
            case 4: run_tile<EPI, 4>(p, t, next, more, past, smem); break;
            default: run_tile<EPI, 5>(p, t, next, more, past, smem); break;
        }
        if (!more) break;
        t = next;
        q += step;
    }
}

template <int EPI>
hipError_t launch(const Fp8GemmArgs& g, hipStream_t stream) {
    static DeviceSetup setup;
    long long grid = 0, unused = 0;
    const hipError_t err =
        device_setup(setup, grid, unused, [](int, long long& gr, long long&) {
            gr = (device_cu_count() + 7) & ~7;
            return hipFuncSetAttribute((const void*)gemm_fp8_block_kernel<EPI>,
                                       hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
        });
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL((gemm_fp8_block_kernel<EPI>), dim3((unsigned)grid), dim3(kThreads),
                       kLds, stream, g);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_gemm_fp8_block(int epilogue, const Fp8GemmArgs& g, hipStream_t stream) {
    if (g.K < 16 || g.K % 16 || g.N < 16 || g.N % 16 || g.G < 1) return hipErrorInvalidValue;
    switch (epilogue) {
        case FP8_OUT_BF16: return launch<FP8_OUT_BF16>(g, stream);
        case FP8_OUT_F32: return launch<FP8_OUT_F32>(g, stream);
        case FP8_SWIGLU: return launch<FP8_SWIGLU>(g, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace moe
