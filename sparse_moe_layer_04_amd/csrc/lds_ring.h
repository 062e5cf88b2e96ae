// Pieces of the grouped products whose operands go to a ring of LDS slots by
// copies that pass no register.
#pragma once

#include <type_traits>

#include "fp8_block.h"

namespace moe {
namespace {

// Copies from memory into LDS that pass no register: lane l's 16 (4) bytes go
// to LDS byte lds + 16 l (4 l), lds wave-uniform.  M0 carries the LDS address
// when the copy issues (one wait state after the write); the compiler may
// keep a value of its own there, so each block leaves M0 as it found it.  The
// compiler does not count these copies: wait_vm does.
__device__ __forceinline__ void copy16(u32x4 rsrc, int voffset, int soffset, int lds) {
    const int at = __builtin_amdgcn_readfirstlane(lds);
    soffset = __builtin_amdgcn_readfirstlane(soffset);
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
// Three such copies (N = 2: two) to places 8 KB apart, M0 saved once
template <int N>
__device__ __forceinline__ void copies16(u32x4 r0, int v0, u32x4 r1, int v1, u32x4 r2, int v2,
                                         int soffset, int lds) {
    const int at = __builtin_amdgcn_readfirstlane(lds);
    soffset = __builtin_amdgcn_readfirstlane(soffset);
    int saved;
    if constexpr (N == 3)
        asm volatile(
            "s_mov_b32 %0, m0\n\t"
            "s_mov_b32 m0, %1\n\t"
            "s_nop 0\n\t"
            "buffer_load_dwordx4 %2, %5, %8 offen lds\n\t"
            "s_add_u32 m0, m0, 0x2000\n\t"
            "s_nop 0\n\t"
            "buffer_load_dwordx4 %3, %6, %8 offen lds\n\t"
            "s_add_u32 m0, m0, 0x2000\n\t"
            "s_nop 0\n\t"
            "buffer_load_dwordx4 %4, %7, %8 offen lds\n\t"
            "s_mov_b32 m0, %0"
            : "=&s"(saved)
            : "s"(at), "v"(v0), "v"(v1), "v"(v2), "s"(r0), "s"(r1), "s"(r2), "s"(soffset)
            : "memory", "scc");
    else
        asm volatile(
            "s_mov_b32 %0, m0\n\t"
            "s_mov_b32 m0, %1\n\t"
            "s_nop 0\n\t"
            "buffer_load_dwordx4 %2, %4, %6 offen lds\n\t"
            "s_add_u32 m0, m0, 0x2000\n\t"
            "s_nop 0\n\t"
            "buffer_load_dwordx4 %3, %5, %6 offen lds\n\t"
            "s_mov_b32 m0, %0"
            : "=&s"(saved)
            : "s"(at), "v"(v0), "v"(v1), "s"(r0), "s"(r1), "s"(soffset)
            : "memory", "scc");
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

// f(integral_constant<int, I>()) for I in [I0, I1)
template <int I0, int I1, class F>
__device__ __forceinline__ void static_for(const F& f) {
    if constexpr (I0 < I1) {
        f(std::integral_constant<int, I0>());
        static_for<I0 + 1, I1>(f);
    }
}

// *p for a wave-uniform p
__device__ __forceinline__ int scalar_load(const int32_t* p) {
    const uint64_t a = (uint64_t)(uintptr_t)p;
    const uint64_t u = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a) |
                       (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32))
                           << 32;
    int v;
    asm volatile("s_load_dword %0, %1, 0x0\n\ts_waitcnt lgkmcnt(0)" : "=s"(v) : "s"(u));
    return v;
}

}  // namespace
}  // namespace moe
