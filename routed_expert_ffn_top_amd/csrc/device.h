// Device helpers that the grouped products of quantised operands share.
#pragma once

#include "common.h"

namespace moe {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ int wave_incl_scan(int v, int lane)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int t = __shfl_up(v, o, 64);
        if (lane >= o) v += t;
    }
    return v;
}

// Of a grouped product's arguments: slot s holds the records [lo, hi), brought into [0, M), and
// record rec takes row row_of of A.
template <class Args>
__device__ __forceinline__ void slot_range(const Args &a, int s, int *lo, int *hi)
{
    *lo = a.slot_offset ? min(max(a.slot_offset[s], 0), a.M) : 0;
    *hi = a.slot_offset ? min(max(a.slot_offset[s + 1], *lo), a.M) : a.M;
}
template <class Args>
__device__ __forceinline__ int row_of(const Args &a, int rec)
{
    return min(max(a.row_index ? a.row_index[rec] : rec, 0), a.A_rows - 1);
}

// Two floats rounded to bf16 (nearest even), lo in bits 15:0.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{lo, hi}), bf16x2_t));
}

#define LDS_AS __attribute__((address_space(3)))

// s_waitcnt with only the vector-memory counter constrained (gfx9 encoding:
// vmcnt[3:0] | expcnt[6:4] | lgkmcnt[11:8] | vmcnt[5:4] at bits 15:14).
template <int N>
__device__ __forceinline__ void wait_vmcnt()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}
// At most n * STEP vector memory operations of this wave outstanding, n in [0, MAXN].
template <int STEP, int MAXN>
__device__ __forceinline__ void wait_vmcnt_stages(int n)
{
    if constexpr (MAXN > 0) {
        if (n >= MAXN) {
            wait_vmcnt<MAXN * STEP>();
            return;
        }
        wait_vmcnt_stages<STEP, MAXN - 1>(n);
    } else {
        wait_vmcnt<0>();
    }
}

// Workgroup barrier that waits for this wave's LDS traffic only (see wait_vmcnt).
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// BYTES (4 or 16) a lane from src to LDS, lane after lane from address dst (the
// same in every lane). Written out: of the builtin the compiler does not know
// which bytes it writes, and may let LDS reads of other stages wait for it (gate/up
// with MXFP4 H, 32768 x 2048 x 2048 over 64 slots: 151 -> 116 us). No register is written and the address is read
// at issue, so wait_vmcnt is all that has to know of it. s_nop: a scalar register
// that a vector instruction wrote is not to be read by the next five.
template <int BYTES>
__device__ __forceinline__ void copy_to_lds(const void *src, uint32_t dst)
{
    if constexpr (BYTES == 16)
        asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %1, off" ::"{m0}"(dst), "v"(src) : "memory");
    else
        asm volatile("s_nop 4\n\tglobal_load_lds_dword %1, off" ::"{m0}"(dst), "v"(src) : "memory");
}
// The same, 16 bytes, from base (the same in every lane) + off.
__device__ __forceinline__ void copy_to_lds(const void *base, uint32_t off, uint32_t dst)
{
    asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(dst), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void *p) { return (uint32_t)(uintptr_t)(LDS_AS const void *)p; }

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ float silu_mul(float g, float u)
{
    // hardware exp2 and reciprocal: off by (|g| + 4) 2^-23 at most for g >= kSiluTail,
    // before 4 or 8 bits are kept; below about -88.7 exp2 leaves the range, and this is 0
    const float e = __builtin_amdgcn_exp2f(-g * 1.4426950408889634f);
    return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}
constexpr float kSiluTail = -87.0f;
// Below it 1 + exp(-g) is exp(-g): SiLU(g) u = g exp(g) u, exp(g) in two halves that stay
// normal numbers (down to g = -174, below which it is 0), u between them; within the same bound.
__device__ __forceinline__ float silu_tail_mul(float g, float u)
{
    const float e = __builtin_amdgcn_exp2f(g * 0.72134752044448170f);
    return g * e * u * e;
}
}  // namespace
}  // namespace moe
