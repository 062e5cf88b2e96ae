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
// beside the next block's matrix products.
//
// Which matrix cores.  The 8-bit ones align the products of a step before
// they add them and drop what falls below: 1.5e-5 of the result for normal
// codes (4e-5 where magnitudes vary by 2^+-2), against 7e-8 for the bf16
// ones, on which a product of two E4M3 values is exact (measured over 4096
// terms against 64-bit sums).  An output rounded to bf16 (2^-9) takes the
// 8-bit ones; an fp32 output and the SwiGLU's quantised h take the bf16 ones
// at half the rate, their codes decoded in registers: the first would show
// the loss, and of the second the codes of small values would move by
// several steps (E4M3 goes down to 2^-18 of a block's largest value).
//
// Tile: up to 128 rows x 256 weight rows (SwiGLU: 128 features, gate and up
// rows interleaved by 16 so that a wave holds both of a feature), 8 waves,
// one 128-wide block of K a stage.  Both operands go through a 3-slot LDS
// ring as codes (48 KB a stage): a wave's 64 lanes load 8 rows x 128 bytes
// (whole lines of the row-major operands) into registers a stage before they
// go to LDS, which is two stages before they are multiplied, so that the
// operand reads can run one step ahead of the matrix products all the way
// through; one barrier a stage.
// LDS row r holds its 16-byte chunk c at c ^ ((r >> 1) & 7), so that the
// lanes of an operand read (32 rows, one chunk index) spread over the banks.
#include <type_traits>

#include "fp8_block.h"

namespace moe {
namespace {

constexpr int BM = 128;                    // rows a tile, at most
constexpr int kSplitM = 128;               // rows a tile of a larger group
constexpr int BN = 256;                    // weight rows a tile
constexpr int BK = 128;                    // K a stage: one block
constexpr int kThreads = 512;
constexpr int kSlotW = BN * BK;
constexpr int kSlotS = kSlotW + BM * BK;   // the stage's scales: the rows' (3 x 64
constexpr int kSlot = kSlotS + 1024;       // words), then two of the weights
constexpr int kSlots = 3;
constexpr int kLds = kSlots * kSlot;
static_assert(kLds <= 160 * 1024 && kSlot % 128 == 0, "three slots of LDS");
constexpr int kRowF32 = BN * 4 + 16;       // epilogue staging rows, padded
constexpr int kRowBf16 = BN * 2 + 16;
constexpr int kRowH = 128 + 16;
static_assert(64 * kRowF32 <= kLds && BM * kRowBf16 <= kLds, "epilogue staging fits");

// Copies from memory into LDS that pass no register: lane l's 16 (4) bytes go
// to LDS byte lds + 16 l (4 l), lds wave-uniform.  M0 carries the LDS address
// when the copy issues (one wait state after the write); the compiler may
// keep a value of its own there, so each block leaves M0 as it found it.  The
// compiler does not count these copies: wait_vm does.
__device__ __forceinline__ void copy16(u32x4 rsrc, int voffset, int soffset, int lds) {
    const int at = __builtin_amdgcn_readfirstlane(lds);
    int saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %2, %3, %4 offen lds\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "s"(at), "v"(voffset), "s"(rsrc), "s"(soffset)
        : "memory");
}
__device__ __forceinline__ void copy4(const void* from, int lds) {
    const int at = __builtin_amdgcn_readfirstlane(lds);
    int saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %1\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dword %2, off\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "s"(at), "v"(from)
        : "memory");
}
// at most N of this wave's memory operations outstanding
template <int N>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }

// Buffer resource over [base, base + bytes), wave-uniform (read from the
// first lane, so that it lives in scalar registers)
__device__ __forceinline__ u32x4 uniform_rsrc(const void* base, size_t bytes) {
    const uint64_t p = (uint64_t)(uintptr_t)base;
    u32x4 r;
    r[0] = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p);
    r[1] = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(p >> 32)) & 0xffffu;
    r[2] = (uint32_t)__builtin_amdgcn_readfirstlane((int)min(bytes, (size_t)0x7fffffff));
    r[3] = 0x00020000u;
    return r;
}

struct Tile {
    int tid, lane, wave, half, l32;
    int g, row0, valid, n0;                // n0: first weight row (SwiGLU: feature)
};

template <int EPI, int MB>
__device__ __forceinline__ void run_tile(const Fp8GemmArgs& p, Tile t, unsigned char* ring) {
    // (the thread's place as a value of this variant's own: address terms
    // shared by the variants would be kept, or spilled, for all of them)
    asm volatile("" : "+v"(t.tid));
    t.lane = t.tid & 63;
    t.half = t.lane >> 5;
    t.l32 = t.lane & 31;
    // waves: WM along the rows x WN along the weight rows, each MI x NJ
    // blocks of 32 x 32
    constexpr int WM = MB == 4 ? 2 : 1, WN = 8 / WM, MI = MB / WM, NJ = 8 / WN;
    constexpr int NA = (MB + 1) / 2;       // row loads a thread and stage
    constexpr bool SW = EPI == FP8_SWIGLU;
    constexpr bool EXACT = EPI != FP8_OUT_BF16;
    const int wm = t.wave / WN, wn = t.wave % WN;
    const int K = p.K, N = p.N;
    const int S = (K + BK - 1) / BK;
    const int nbn = (N + 127) / 128;

    // Addresses.  Copies go through buffer resources over the tile's rows
    // (wave-uniform base, 32-bit offsets), rows past the tile's or the
    // matrix's end clamped to the last.  A wave's copy fills 8 LDS rows of 128
    // bytes; the place of a chunk in its row is swizzled, so the lanes fetch
    // swizzled chunks.  LDS rows 32 apart share their swizzle, so the rest of
    // an operand's address is an immediate; the chunk index enters it by
    // exclusive or.
    const int lr = t.tid >> 3, c = (t.tid & 7) ^ swz(lr);   // chunk c of row lr + 64 q
    // SwiGLU: LDS row R is row R & 15 of 16 features' gate (R & 16 == 0) or up
    // rows; R & 16 is the same for a wave and all q
    const bool up = SW && (t.wave & 2);
    const size_t wfirst = ((size_t)t.g * N + t.n0) * K;
    const int wrows = N - t.n0;                     // (>= 1)
    const u32x4 wsrc = uniform_rsrc((up ? p.w2 : p.w1) + wfirst, (size_t)min(wrows, BN) * K);
    const u32x4 asrc = uniform_rsrc(p.a + (size_t)t.row0 * K, (size_t)t.valid * K);
    // (a chunk past the end of K in the last block: the row's last chunk,
    // overwritten by zeros before it is read)
    const int past = max(0, (S - 1) * BK + 16 * c + 16 - K);
    int wo[4], ao[NA];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int R = lr + 64 * q;
        wo[q] = min(SW ? 16 * (R >> 5) + (R & 15) : R, wrows - 1) * K + 16 * c;
    }
    // (an odd number of blocks: the last 32 rows twice, the same bytes to the
    // same place, so that every wave issues the same number of copies)
    constexpr int kLastMask = MB % 2 ? 31 : 63;
#pragma unroll
    for (int q = 0; q < NA; ++q) {
        const int R = (q == NA - 1 ? lr & kLastMask : lr) + 64 * q;
        ao[q] = min(R, t.valid - 1) * K + 16 * c;
    }
    const int last_wave = t.wave & (kLastMask >> 3);
    // scales: waves 0 to 2 fetch the rows', the others (the same ones) the
    // weights' of the tile's two 128-blocks of rows, or of gate and up
    const int nb0 = t.n0 / 128;
    const float* sp;
    if (t.wave < 3) {
        sp = p.as + (size_t)(t.row0 + min(64 * t.wave + t.lane, t.valid - 1)) * S;
    } else if constexpr (SW) {
        sp = (t.lane & 1 ? p.s2 : p.s1) + ((size_t)t.g * nbn + nb0) * S;
    } else {
        sp = p.s1 + ((size_t)t.g * nbn + min(nb0 + (t.lane & 1), nbn - 1)) * S;
    }
    constexpr int NI = 4 + NA + 1;                  // copies a wave and stage
    // Stage 0 takes K's last block, the short one if any, stage j block j - 1.
    // (Every stage issues its copies: past the last stage with offsets past
    // the resources, which fetch nothing.)
    auto fetch = [&](int j, int at) {
        const int b = j == 0 ? S - 1 : min(j, S) - 1;
        const int back = j == 0 ? past : 0, out = j < S ? 0 : (int)0x80000000;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            copy16(wsrc, (wo[q] - back) | out, b * BK, at + q * 64 * BK + t.wave * 1024);
#pragma unroll
        for (int q = 0; q < NA; ++q)
            copy16(asrc, (ao[q] - back) | out, b * BK,
                   at + kSlotW + q * 64 * BK + (q == NA - 1 ? last_wave : t.wave) * 1024);
        copy4(sp + b, at + kSlotS + min(t.wave, 3) * 256);
    };
    // zeros over this thread's own copies past the end of K, once they landed
    auto zero_past = [&]() {
        if (!past) return;
        const u32x4 z = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int q = 0; q < 4; ++q) *(u32x4*)(ring + q * 64 * BK + t.tid * 16) = z;
#pragma unroll
        for (int q = 0; q < NA; ++q)
            *(u32x4*)(ring + kSlotW + q * 64 * BK +
                      (q == NA - 1 ? last_wave * 1024 + t.lane * 16 : t.tid * 16)) = z;
    };
    const int rd0 = t.l32 * BK + ((t.half ^ swz(t.l32)) << 4);
    const int rdw = wn * NJ * 32 * BK + rd0;
    const int rda = kSlotW + wm * MI * 32 * BK + rd0;
    const int rds = kSlotS + (wm * MI * 32 + t.l32) * 4;
    const int rdsw = kSlotS + 768 + (SW ? 0 : (t.n0 + wn * NJ * 32) / 128 - nb0) * 4;
    float sa[MI] = {}, sw1 = 0.0f, sw2 = 0.0f;
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
    auto scales = [&]() {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            s1[i] = sa[i] * sw1;
            s2[i] = sa[i] * sw2;
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

    // stages 0 to 2 on their way; stage 0 landed
    fetch(0, 0);
    fetch(1, kSlot);
    fetch(2, 2 * kSlot);
    wait_vm<2 * NI>();
    zero_past();
    __syncthreads();
    // The middle of stage j: stage j + 1's block has landed and every wave has
    // read stage j's, whose slot takes stage j + 3's.
    auto turn = [&](int j, int slot) {
        wait_vm<NI>();
        __syncthreads();
        fetch(j + 3, slot);
    };

    if constexpr (EXACT) {
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
        using std::integral_constant;
        auto step = [&](auto st) {
            constexpr int h = decltype(st)::value;
            decode(integral_constant<int, (h + 1) & 7>());
            multiply(st);
            // one product, then its share of the vector instructions
            constexpr int V = 4 * (MI + NJ) / NT + (h == 0 ? 16 : 0);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x002, h == 0 ? V : 0, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, h == 0 ? 0 : V, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        using H0 = integral_constant<int, 0>;
        using H1 = integral_constant<int, 1>;
        read(0, 0, H0());
        read(0, 1, H1());
        decode(H0());
        int slot = 0;
        for (int j = 0; j < S; ++j) {
            const int next = slot == 2 * kSlot ? 0 : slot + kSlot;
            scales();                               // of block j - 1
            read_s(slot);
            step(H0());
            read(slot, 2, H0());
            step(H1());
            step(integral_constant<int, 2>());
            read(slot, 3, H1());
            step(integral_constant<int, 3>());
            step(integral_constant<int, 4>());
            turn(j, slot);
            read(next, 0, H0());                    // (past the end: not used)
            step(integral_constant<int, 5>());
            step(integral_constant<int, 6>());
            read(next, 1, H1());
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
        auto multiply = [&](auto set) {
            constexpr int B = decltype(set)::value;
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int n = 0; n < NJ; ++n) {
                    if constexpr (B == 0) add_part(i, n);
                    part[i][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        cat(rw[B][n]), cat(ra[B][i]), B == 0 ? zero : part[i][n], 0, 0, 0, 127, 0,
                        127);
                }
            if constexpr (B == 0) {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x002, 16, 0);
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        using B0 = std::integral_constant<int, 0>;
        using B1 = std::integral_constant<int, 1>;
        read(0, B0());
        int slot = 0;
        for (int j = 0; j < S; ++j) {
            const int next = slot == 2 * kSlot ? 0 : slot + kSlot;
            scales();                               // of block j - 1
            read_s(slot);
            read(slot, B1());
            multiply(B0());
            turn(j, slot);
            read(next, B0());                       // (past the end: not used)
            multiply(B1());
            slot = next;
        }
    }
    scales();
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int n = 0; n < NJ; ++n) add_part(i, n);

    // Epilogues: lane l holds, of row l % 32 of its block, weight rows
    // 8 (e / 4) + 4 (l / 32) + e % 4; through LDS into whole-line stores.
    wait_vm<0>();
    __syncthreads();
    if constexpr (EPI == FP8_OUT_F32) {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            if (i) __syncthreads();
#pragma unroll
            for (int n = 0; n < NJ; ++n)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int col = (wn * NJ + n) * 32 + 8 * q + 4 * t.half;
                    *(f32x4*)(ring + (wm * 32 + t.l32) * kRowF32 + col * 4) =
                        f32x4{acc[i][n][4 * q], acc[i][n][4 * q + 1], acc[i][n][4 * q + 2],
                              acc[i][n][4 * q + 3]};
                }
            __syncthreads();
            const int col = 4 * t.lane;
            for (int sr = t.wave; sr < WM * 32; sr += 8) {
                const int r = ((sr >> 5) * MI + i) * 32 + (sr & 31);
                if (r < t.valid && t.n0 + col < N)
                    *(f32x4*)((float*)p.out + (size_t)(t.row0 + r) * N + t.n0 + col) =
                        *(const f32x4*)(ring + sr * kRowF32 + col * 4);
            }
        }
    } else if constexpr (EPI == FP8_OUT_BF16) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int n = 0; n < NJ; ++n)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int col = (wn * NJ + n) * 32 + 8 * q + 4 * t.half;
                    *(u32x2*)(ring + ((wm * MI + i) * 32 + t.l32) * kRowBf16 + col * 2) =
                        u32x2{bf16_pack2(acc[i][n][4 * q], acc[i][n][4 * q + 1]),
                              bf16_pack2(acc[i][n][4 * q + 2], acc[i][n][4 * q + 3])};
                }
        __syncthreads();
        const int col = 8 * t.l32;
        for (int r = 2 * t.wave + t.half; r < t.valid; r += 16)
            if (t.n0 + col < N)
                *(u32x4*)((uint16_t*)p.out + (size_t)(t.row0 + r) * N + t.n0 + col) =
                    *(const u32x4*)(ring + r * kRowBf16 + col * 2);
    } else {
        // h = SwiGLU in fp32, quantised along the tile's 128 features: the
        // row maximum over this lane's features, its half-wave partner's and
        // the other waves'
        float* rm = (float*)ring;                     // [WN][BM]
        unsigned char* stg = ring + 8 * BM * 4;       // [BM][kRowH] codes
        float h[MI][NJ][8];
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
                    h[i][n][e] = in ? v : 0.0f;
                    m = fmaxf(m, finite_abs(h[i][n][e]));
                }
            }
            m = fmaxf(m, __shfl_xor(m, 32, 64));
            if (t.half == 0) rm[wn * BM + (wm * MI + i) * 32 + t.l32] = m;
        }
        __syncthreads();
        const int nbf = (N + 127) / 128;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int r = (wm * MI + i) * 32 + t.l32;
            float m = 0.0f;
#pragma unroll
            for (int w = 0; w < WN; ++w) m = fmaxf(m, rm[w * BM + r]);
            const int X = block_exponent(m);
            const float inv = pow2(-X);
#pragma unroll
            for (int n = 0; n < NJ; ++n)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int f = 16 * (wn * NJ + n) + 8 * q + 4 * t.half;
                    *(uint32_t*)(stg + r * kRowH + f) =
                        e4m3_pack4(h[i][n][4 * q], h[i][n][4 * q + 1], h[i][n][4 * q + 2],
                                   h[i][n][4 * q + 3], inv);
                }
            if (wn == 0 && t.half == 0 && r < t.valid)
                p.out_scale[(size_t)(t.row0 + r) * nbf + t.n0 / 128] = pow2(X);
        }
        __syncthreads();
        for (int r = lr; r < t.valid; r += 64)
            if (t.n0 + 16 * c < N)
                *(u32x4*)((uint8_t*)p.out + (size_t)(t.row0 + r) * N + t.n0 + 16 * c) =
                    *(const u32x4*)(stg + r * kRowH + 16 * c);
    }
}

// Inclusive sum over the wave's lanes
__device__ __forceinline__ int wave_scan(int x, int lane) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int y = __shfl_up(x, off, 64);
        if (lane >= off) x += y;
    }
    return x;
}

// Row tiles of a group of n rows: one up to BM rows (a second one would fetch
// the group's weights again), else of up to kSplitM rows each.
__device__ __forceinline__ int row_tiles(int n) {
    return n <= BM ? n > 0 : (n + kSplitM - 1) / kSplitM;
}

// Persistent grid, one workgroup a CU.  Items are (group, n-tile, m-tile), the
// 8 XCDs take contiguous ranges, so that the m-tiles of a weight tile and the
// n-tiles of a group's rows meet in one XCD's L2; a group's rows split evenly
// over its m-tiles.  The group of an item comes from a two-level sum that
// every wave keeps in registers: lane l holds the items before run l of
// ceil(G / 64) groups, and looks into the run that holds the item.
static_assert(MOE_MAX_GROUPS <= 64 * 64, "one lane a run, one lane a group of a run");

template <int EPI>
__global__ __launch_bounds__(kThreads) void gemm_fp8_block_kernel(Fp8GemmArgs p) {
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int TN = EPI == FP8_SWIGLU ? BN / 2 : BN;
    Tile t;
    t.tid = threadIdx.x;
    t.lane = t.tid & 63;
    t.wave = __builtin_amdgcn_readfirstlane(t.tid >> 6);
    t.half = t.lane >> 5;
    t.l32 = t.lane & 31;
    const int G = p.G, rows = p.rows;
    const int NT = (p.N + TN - 1) / TN;
    auto group_rows = [&](int g, int& lo, int& hi) {
        lo = min(max(p.offsets[g], 0), rows);
        hi = max(lo, min(max(p.offsets[g + 1], 0), rows));
    };
    auto group_items = [&](int g) {
        int lo = 0, hi = 0;
        if (g < G) group_rows(g, lo, hi);
        return NT * row_tiles(hi - lo);
    };
    const int run = (G + 63) / 64;
    int mine = 0;
    for (int i = 0; i < run; ++i) mine += group_items(t.lane * run + i);
    const int upto = wave_scan(mine, t.lane);
    const long long Q = __builtin_amdgcn_readlane(upto, 63);
    const int xcd = blockIdx.x & 7;
    const int hi_item = (int)(Q * (xcd + 1) / 8);
    for (int q = (int)(Q * xcd / 8) + (int)(blockIdx.x >> 3); q < hi_item; q += gridDim.x >> 3) {
        // the first lane whose sum passes q, then the same within its run
        const int r = __builtin_ctzll(__builtin_amdgcn_ballot_w64(upto > q));
        int local = q - __builtin_amdgcn_readlane(upto - mine, r);
        const int items = t.lane < run ? group_items(r * run + t.lane) : 0;
        const int in_run = wave_scan(items, t.lane);
        const int l = __builtin_ctzll(__builtin_amdgcn_ballot_w64(in_run > local));
        local -= __builtin_amdgcn_readlane(in_run - items, l);
        t.g = r * run + l;
        int r0, r1;
        group_rows(t.g, r0, r1);
        const int n = r1 - r0, mt = row_tiles(n);
        const int per = ((n + mt - 1) / mt + 31) & ~31;
        t.n0 = local / mt * TN;
        t.row0 = r0 + local % mt * per;
        t.valid = min(per, r1 - t.row0);
        switch ((t.valid + 31) >> 5) {
            case 1: run_tile<EPI, 1>(p, t, smem); break;
            case 2: run_tile<EPI, 2>(p, t, smem); break;
            case 3: run_tile<EPI, 3>(p, t, smem); break;
            default: run_tile<EPI, 4>(p, t, smem); break;
        }
        __syncthreads();                             // the ring is free again
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
