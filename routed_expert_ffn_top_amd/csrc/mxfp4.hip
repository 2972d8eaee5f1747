// MXFP4: rows to blocks of 32 values (E2M1 codes and one E8M0 scale each),
// blocks back to values, and the product of two matrices held that way.
//
// Quantisation of a block: with e the biased exponent field of its largest
// magnitude, the scale byte is max(e - 2, 0), the power of two that brings
// that magnitude into [4, 8); each value times 2^(127 - byte) is rounded to the
// nearest E2M1 value, ties to the even code, at most 6. A block that holds an
// infinity or a NaN gets the byte 255 (NaN) and codes 0. A zero has no sign.
#include <algorithm>
#include <type_traits>
#include <utility>

#include "mxfp4.h"

namespace moe {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

// Scale byte of a block from the bits of its largest magnitude, and the factor
// 2^(127 - byte) that its values are quantised with (1 for a NaN block).
__device__ __forceinline__ uint32_t block_scale(uint32_t top)
{
    const int e = (int)(top >> 23);
    return e == 255 ? 255u : (uint32_t)max(e - 2, 0);
}
__device__ __forceinline__ float block_unit(uint32_t byte)
{
    // byte <= 252, so the exponent field is at least 2
    return byte == 255 ? 1.0f : __uint_as_float((254u - byte) << 23);
}
// Eight codes without the signs of those of magnitude 0.
__device__ __forceinline__ uint32_t unsigned_zeros(uint32_t q)
{
    const uint32_t m = q & 0x77777777u, nz = (m | m >> 1 | m >> 2) & 0x11111111u;
    return m | (q & nz << 3);
}

// Element offset of group i of 8 values (i < 2^31), rows of K8 groups ld elements apart.
__device__ __forceinline__ int64_t place(int64_t i, int K8, int64_t ld)
{
    if (ld == (int64_t)K8 * 8) return i * 8;
    const uint32_t row = (uint32_t)i / (uint32_t)K8;
    return row * ld + (int64_t)((uint32_t)i - row * (uint32_t)K8) * 8;
}

// 8 values per lane, 4 lanes per block. Bound by HBM: 4 or 2 bytes read and
// 17/32 written a value.
template <bool BF16>
__global__ __launch_bounds__(256) void k_quantize(const void *__restrict__ src, int64_t n8, int K8, int64_t ld,
                                                  uint32_t *__restrict__ codes, uint8_t *__restrict__ scales)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n8) return;   // whole blocks of 4 lanes: n8 % 4 == 0
    const int64_t at = place(i, K8, ld);
    uint32_t v[8];
    if constexpr (BF16) {
        const u32x4_t w = *(const u32x4_t *)((const uint16_t *)src + at);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            v[2 * c] = w[c] << 16;
            v[2 * c + 1] = w[c] & 0xffff0000u;
        }
    } else {
        const u32x4_t w0 = *(const u32x4_t *)((const float *)src + at);
        const u32x4_t w1 = *(const u32x4_t *)((const float *)src + at + 4);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            v[c] = w0[c];
            v[c + 4] = w1[c];
        }
    }
    // magnitudes order as their bits do (infinities and NaN above all numbers)
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) top = max(top, v[c] & 0x7fffffffu);
    top = max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
    const uint32_t byte = block_scale(top);
    const float up = block_unit(byte);
    uint32_t q = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float a = __uint_as_float(v[2 * c]) * up, b = __uint_as_float(v[2 * c + 1]) * up;
        switch (c) {   // the byte is chosen by an immediate
        case 0: q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, a, b, 1.0f, 0); break;
        case 1: q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, a, b, 1.0f, 1); break;
        case 2: q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, a, b, 1.0f, 2); break;
        default: q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, a, b, 1.0f, 3); break;
        }
    }
    codes[i] = byte == 255 ? 0u : unsigned_zeros(q);
    if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)byte;
}

__device__ __forceinline__ float e8m0(uint32_t b)
{
    return __uint_as_float(b == 0 ? 0x00400000u : (b == 255 ? 0x7fc00000u : b << 23));
}

// 8 values per lane; code value times 2^(byte - 127) in fp32, which is exact
// (in bf16 as well: one significant bit after the first) where it does not
// leave the range.
template <bool BF16>
__global__ __launch_bounds__(256) void k_dequantize(const uint32_t *__restrict__ codes,
                                                    const uint8_t *__restrict__ scales, int64_t n8, int K8,
                                                    void *__restrict__ dst, int64_t ld)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n8) return;
    const int64_t at = place(i, K8, ld);
    const uint32_t q = codes[i];
    const float s = e8m0(scales[i >> 2]);
    const f32x2_t p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3)};
    uint32_t v[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = __float_as_uint(p[c >> 1][c & 1] * s);
    if constexpr (BF16) {
        u32x4_t o;
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = v[2 * c] >> 16 | (v[2 * c + 1] & 0xffff0000u);
        *(u32x4_t *)((uint16_t *)dst + at) = o;
    } else {
        *(u32x4_t *)((float *)dst + at) = u32x4_t{v[0], v[1], v[2], v[3]};
        *(u32x4_t *)((float *)dst + at + 4) = u32x4_t{v[4], v[5], v[6], v[7]};
    }
}

__device__ __forceinline__ int wave_incl_scan(int v, int lane)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int t = __shfl_up(v, o, 64);
        if (lane >= o) v += t;
    }
    return v;
}

__device__ __forceinline__ uint32_t bf16_bits(float x)
{
    uint32_t u = __float_as_uint(x);
    if ((u & 0x7fffffffu) > 0x7f800000u) return (u >> 16) | 0x40u;
    u += 0x7fffu + ((u >> 16) & 1u);
    return u >> 16;
}

// ---------------------------------------------------------------------------
// Product of MXFP4 operands on the scaled matrix instructions
// (v_mfma_scale_f32_32x32x64_f8f6f4: lane l supplies row l % 32 and the 32
// consecutive k values 32 (l / 32) .. +31 of each operand, 16 bytes of codes,
// with that block's scale byte): products and scales are exact, sums in fp32.
// Every element of C is one chain of these instructions in ascending k, in
// both kernels below, so a record's bits hang neither on the size of its group
// nor on which kernel runs.

// Two floats rounded to bf16 (nearest even), lo in bits 15:0.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{lo, hi}), bf16x2_t));
}

// Slot s holds the records [lo, hi), brought into [0, M).
__device__ __forceinline__ void slot_range(const MxArgs &a, int s, int *lo, int *hi)
{
    *lo = a.slot_offset ? min(max(a.slot_offset[s], 0), a.M) : 0;
    *hi = a.slot_offset ? min(max(a.slot_offset[s + 1], *lo), a.M) : a.M;
}
__device__ __forceinline__ int row_of(const MxArgs &a, int rec)
{
    return min(max(a.row_index ? a.row_index[rec] : rec, 0), a.A_rows - 1);
}

// Few records a slot: 64 records x 64 columns per workgroup, 32 x 32 per wave,
// operands straight from global memory, 8 steps of 64 k requested at a time.
// Bound by latency and, with many slots, by reading the weights.
__global__ __launch_bounds__(256) void k_matmul_small(MxArgs a)
{
    __shared__ int32_t s_tile[4];   // slot, first record, records
    const int ntn = a.N / 64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int bid = blockIdx.x / ntn, n0 = (blockIdx.x % ntn) * 64;
    if (threadIdx.x < 64) {
        if (lane == 0) s_tile[0] = -1;
        int run = 0;
        for (int s0 = 0; s0 < a.P; s0 += 64) {
            const int s = s0 + lane;
            int lo = 0, hi = 0;
            if (s < a.P) slot_range(a, s, &lo, &hi);
            const int mt = (hi - lo + 63) / 64;
            const int inc = run + wave_incl_scan(mt, lane);
            if (bid < inc && bid >= inc - mt) {
                s_tile[0] = s;
                s_tile[1] = lo + (bid - (inc - mt)) * 64;
                s_tile[2] = min(64, hi - s_tile[1]);
            }
            run = __shfl(inc, 63, 64);
        }
    }
    __syncthreads();
    const int slot = s_tile[0], row0 = s_tile[1], cnt = s_tile[2];
    if (slot < 0) return;
    const int K = a.K, N = a.N;
    const int m0 = (wave >> 1) * 32, c0 = n0 + (wave & 1) * 32;
    if (m0 >= cnt) return;
    const int half = lane >> 5;
    const int rec = row_of(a, row0 + min(m0 + (lane & 31), cnt - 1));
    const uint8_t *ap = a.A + (int64_t)rec * (K / 2) + half * 16;
    const uint8_t *as = a.As + (int64_t)rec * (K / 32) + half;
    const int n = c0 + (lane & 31), nb = n / kWRows, rows = min(kWRows, N - nb * kWRows);
    const int64_t pb = fp4_piece_bytes(rows);
    const int rb = n - nb * kWRows;
    const uint8_t *bp = a.B + (int64_t)slot * a.B_stride + (int64_t)nb * (K / kWK) * fp4_piece_bytes(kWRows) + half * pb +
                        rb * 16;
    const uint8_t *bs = bp - rb * 16 + rows * 16 + rb;
    f32x16_t acc;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
    constexpr int U = 8;
    const int nk = K / 64;
    for (int k = 0; k < nk; k += U) {
        u32x4_t av[U], bv[U];
        int sa[U], sb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t kk = min(k + u, nk - 1);
            bv[u] = *(const u32x4_t *)(bp + 2 * kk * pb);
            sb[u] = bs[2 * kk * pb];
            av[u] = *(const u32x4_t *)(ap + kk * 32);
            sa[u] = as[2 * kk];
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (k + u >= nk) continue;
            const i32x8_t A = {(int)av[u][0], (int)av[u][1], (int)av[u][2], (int)av[u][3], 0, 0, 0, 0};
            const i32x8_t Bv = {(int)bv[u][0], (int)bv[u][1], (int)bv[u][2], (int)bv[u][3], 0, 0, 0, 0};
            acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, Bv, acc, 4, 4, 0, sa[u], 0, sb[u]);
        }
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int m = m0 + 8 * (r / 4) + 4 * half + (r & 3);
        if (m >= cnt) continue;
        const int64_t at = (int64_t)(row0 + m) * a.ldc + n;
        if (a.c_bf16)
            ((uint16_t *)a.C)[at] = (uint16_t)bf16_bits(acc[r]);
        else
            ((float *)a.C)[at] = acc[r];
    }
}

#define LDS_AS __attribute__((address_space(3)))
#define GLOBAL_AS __attribute__((address_space(1)))

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

constexpr int kXcd = 8;
constexpr int kStream = 2;   // buffer stores of C, which is not read here: non-temporal (fp32 C 141 -> 132 us)

// Many records a slot: a persistent ring kernel. Tile BM records x 256 columns,
// one stage = 128 k: BM rows of 64 code bytes, 4 K pieces of the packed slice
// (256 rows of 16 code bytes each, one contiguous run) and both sides' scale
// bytes, copied straight into LDS (16 bytes a lane), NS stages deep; 8 waves as
// 2 x 4, MI x NI 32 x 32 blocks each, so that the B fragments, whose scales are
// read byte by byte, are the fewer. A rows are stored with their 16-byte chunk
// c at c ^ ((row >> 2) & 3), which keeps the fragment reads free of bank
// conflicts; the pieces of B are so as they stand. A row's scale bytes of a
// stage are one 32-bit word, aligned or not: with SHIFT the lanes cut it out of
// the two aligned words that hold it; without it (K % 128 == 0 and aligned
// scales) it is a word. The words of four stages, a panel, are copied together, a
// quarter of the rows a stage: a word at a time each is a request of its own to
// the L2, 256 of a stage's 650 (copies alone 95 -> 74 us). The tiles of an XCD (workgroup id mod 8) are one
// contiguous range, column block major, walked in step, so that tiles which
// share weights or rows share that XCD's L2.
//
// EPI: what becomes of a tile. STORE: C, rounded to its type. GATE_UP: the
// slice's rows alternate 32 gate, 32 up, so a wave's two column blocks are gate
// and up of the same 32 units, one unit a lane: H = SiLU(g) u is one MXFP4 block
// for each row of a wave, quantised in registers (block maximum over the 32
// lanes, codes of 8 rows gathered in a word and transposed over 8 lanes) and
// written as codes and scale bytes; the fp32 and bf16 H never exist. DOWN: C is
// the routes' fp32 rows, alpha times the record's, and the routes are marked.
//
// The epilogue of gate/up is as long as its products unless its instructions are
// few: the 16 rows' block maxima by halving (24 + 12 + 6 + 3 operations and one
// exchange, not 16 times 10), one scale a lane, brought to the row's 16 lanes as
// an operand of the multiplication (32768 x 2048 x 2048
// over 64 slots 195 -> 151 us, and 116 with the copies written out; the bf16-activation
// kernel takes 290).
__device__ __forceinline__ float silu_mul(float g, float u)
{
    // hardware exp2 and reciprocal: off by (|g| + 4) 2^-23 at most for g >= kSiluTail,
    // before 4 bits are kept; below about -88.7 exp2 leaves the range, and this is 0
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
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
// One halving: of 2n values the lane keeps n, those of its side, each joined with
// the partner's (which CTRL names and which is on the other side).
template <int CTRL, int n>
__device__ __forceinline__ void halve(uint32_t *t, bool upper)
{
#pragma unroll
    for (int r = 0; r < n; ++r) {
        const uint32_t keep = upper ? t[r + n] : t[r], give = upper ? t[r] : t[r + n];
        t[r] = max(keep, dpp<CTRL>(give));
    }
}
// Bits of the largest magnitude (infinities and NaN above all) over the 32 lanes
// of a half of h[lane % 16].
__device__ __forceinline__ uint32_t block_tops(const float *h, int lane)
{
    uint32_t t[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) t[r] = __float_as_uint(h[r]) & 0x7fffffffu;
    halve<0x128, 8>(t, lane & 8);   // lane ^ 8: a rotation by 8 of 16
    halve<0x141, 4>(t, lane & 4);   // 7 - lane of 8
    halve<0x4E, 2>(t, lane & 2);    // lane ^ 2
    halve<0xB1, 1>(t, lane & 1);    // lane ^ 1
    return max(t[0], (uint32_t)__builtin_amdgcn_ds_swizzle((int)t[0], (16 << 10) | 0x1f));   // lane ^ 16
}
// h[r] times the unit that lane r of each 16 holds.
template <int... R>
__device__ __forceinline__ void scale_rows(float *h, float unit, std::integer_sequence<int, R...>)
{
    ((h[R] *= __uint_as_float(dpp<0x150 + R>(__float_as_uint(unit)))), ...);
}
// h[r] with the bits that lane r of each 16 keeps.
template <int... R>
__device__ __forceinline__ void zero_rows(float *h, int keep, std::integer_sequence<int, R...>)
{
    ((h[R] = __uint_as_float(__float_as_uint(h[R]) & dpp<0x150 + R>((uint32_t)keep))), ...);
}
// 8 x 8 nibbles over 8 lanes: lane l's nibble j becomes lane j's nibble l.
__device__ __forceinline__ uint32_t transpose8(uint32_t q, int lane)
{
    uint32_t o = (uint32_t)__builtin_amdgcn_ds_swizzle((int)q, (4 << 10) | 0x1f);
    q = (lane & 4) ? (o >> 16) | (q & 0xffff0000u) : (q & 0xffffu) | (o << 16);
    o = dpp<0x4E>(q);
    q = (lane & 2) ? ((o >> 8) & 0x00ff00ffu) | (q & 0xff00ff00u) : (q & 0x00ff00ffu) | ((o & 0x00ff00ffu) << 8);
    o = dpp<0xB1>(q);
    return (lane & 1) ? ((o >> 4) & 0x0f0f0f0fu) | (q & 0xf0f0f0f0u) : (q & 0x0f0f0f0fu) | ((o & 0x0f0f0f0fu) << 4);
}

enum { EPI_STORE = 0, EPI_GATE_UP = 1, EPI_DOWN = 2 };

template <int BM, int NS, bool SHIFT, int EPI>
__global__ __launch_bounds__(512) void k_matmul_ring(MxArgs a)
{
    constexpr int BN = 256, WM = 2, WN = 4, TM = BM / WM, TN = BN / WN, MI = TM / 32, NI = TN / 32;
    constexpr int ACODE = BM * 64, BCODE = BN * 64, BSC = BN * 4;
    constexpr int STAGE = ACODE + BCODE + BSC;
    constexpr int AI = BM / 128, BI = 2;           // code copies per wave and stage
    constexpr int LOADS = AI + BI + 1;             // and one of scales
    constexpr int APANEL = BM * 16, NP = 3;        // A's scales of 4 stages, [row][4 words]; panels there at a time
    static_assert(BM == 256 && NS == 4, "the copies of the scales are laid out for 256 rows and panels of 4 stages");
    __shared__ __attribute__((aligned(1024))) char lds[NS * STAGE + NP * APANEL];
    char *const apanel = lds + NS * STAGE;
    __shared__ int32_t s_tpref[kMaxExp + 1], s_lo[kMaxExp], s_cnt[kMaxExp];
    __shared__ int32_t s_shift[SHIFT ? BM : 1];   // bytes from the aligned word to a row's scales
    // of three tiles, this one, the next and the one after it: the rows of A of
    // its records, or (down, where record p is row p) their routes
    __shared__ int32_t s_rows[3][BM];
    __shared__ float s_alpha[2][EPI == EPI_DOWN ? BM : 1];
    const uint32_t lds_at = lds_address(lds), rows_at = lds_address(s_rows), alpha_at = lds_address(s_alpha);

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN, half = lane >> 5;
    const int K = a.K, N = a.N, P = a.P;
    const int ntn = (N + BN - 1) / BN;
    if (tid < 64) {
        int run = 0;
        for (int s0 = 0; s0 < P; s0 += 64) {
            const int s = s0 + lane;
            int lo = 0, hi = 0;
            if (s < P) slot_range(a, s, &lo, &hi);
            const int w = (hi - lo + BM - 1) / BM * ntn;
            const int inc = run + wave_incl_scan(w, lane);
            if (s < P) {
                s_tpref[s] = inc - w;
                s_lo[s] = lo;
                s_cnt[s] = hi - lo;
            }
            run = __shfl(inc, 63, 64);
        }
        if (lane == 0) s_tpref[P] = run;
    }
    __syncthreads();
    const int total = s_tpref[P];
    const int xcd = blockIdx.x % kXcd, li = blockIdx.x / kXcd;
    const int nwg = ((int)gridDim.x - xcd + kXcd - 1) / kXcd;
    const int qx = total / kXcd, rx = total % kXcd;
    const int cnt_x = qx + (xcd < rx ? 1 : 0), start_x = xcd * qx + min(xcd, rx);
    if (li >= cnt_x) return;

    struct Tile {
        int slot, row0, rows, n0;
    };
    auto decode = [&](int L) -> Tile {
        int lo = 0, hi = P - 1;   // last slot whose first tile is <= L (skips empty slots)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_tpref[mid] <= L) lo = mid; else hi = mid - 1;
        }
        const int mt = (s_cnt[lo] + BM - 1) / BM, local = L - s_tpref[lo], ml = local % mt;
        Tile t;   // the same in every lane
        t.slot = __builtin_amdgcn_readfirstlane(lo);
        t.row0 = __builtin_amdgcn_readfirstlane(s_lo[lo] + ml * BM);
        t.rows = __builtin_amdgcn_readfirstlane(min(BM, s_cnt[lo] - ml * BM));
        t.n0 = __builtin_amdgcn_readfirstlane((local / mt) * BN);
        return t;
    };

    // Copies of this wave: A codes rows 16 (wave AI + j) .. +15 (lane: row + l/4,
    // chunk position l % 4), B codes 64 rows 64 ((2 wave + j) % 4) .. of piece
    // (2 wave + j) / 4, and scales: waves 0-3 those of A rows 64 wave + 16 q .. +15
    // (lane: row + l/4, word l % 4), q = stage % 4, of the next panel, waves 4-7
    // the 256 of B's piece wave - 4.
    const char *asrc[AI], *bsrc;   // bsrc: the same in every lane
    uint32_t boff[BI], soff;
    int srow[4];
    int bstep = 0;
    // A tile's rows or routes to LDS. No register waits for them: a load into one
    // would be waited for with everything requested after it.
    auto fetch_rows = [&](const Tile &t, int buf) {
        const int32_t *src = EPI == EPI_DOWN ? a.rec_route : a.row_index;
        if (src && wave < BM / 64)
            copy_to_lds<4>(src + t.row0 + min(wave * 64 + lane, t.rows - 1), rows_at + (buf * BM + wave * 64) * 4);
    };
    auto row_in = [&](const Tile &t, int buf, int i) {
        const int r = min(i, t.rows - 1);
        return EPI != EPI_DOWN && a.row_index ? min(max(s_rows[buf][r], 0), a.A_rows - 1) : t.row0 + r;
    };
    auto scales_at = [&](int row) { return (uintptr_t)a.As + (uintptr_t)((int64_t)row * (K / 32)); };
    // the last aligned word that holds scale bytes
    const uintptr_t last_word = (scales_at(a.A_rows) - 1) & ~(uintptr_t)3;
    auto set_sources = [&](const Tile &t, int buf) {
#pragma unroll
        for (int j = 0; j < AI; ++j) {
            const int r = (wave * AI + j) * 16 + (lane >> 2);
            asrc[j] = (const char *)a.A + (int64_t)row_in(t, buf, r) * (K / 2) + ((lane & 3) ^ ((r >> 2) & 3)) * 16;
        }
        const int nb = t.n0 / kWRows, rows_nb = min(kWRows, N - nb * kWRows);
        const int64_t pb = fp4_piece_bytes(rows_nb);
        const char *Bblk = (const char *)a.B + (int64_t)t.slot * a.B_stride + (int64_t)nb * (K / kWK) * fp4_piece_bytes(kWRows);
        bstep = (int)(4 * pb);
#pragma unroll
        for (int j = 0; j < BI; ++j) {
            const int c = wave * BI + j;
            boff[j] = (uint32_t)((c >> 2) * pb) + min((c & 3) * 64 + lane, rows_nb - 1) * 16;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            srow[q] = row_in(t, buf, (wave & 3) * 64 + q * 16 + (lane >> 2));
            if (SHIFT && wave < 4)   // read after the tile's first barrier
                s_shift[wave * 64 + q * 16 + (lane >> 2)] = (int)(scales_at(srow[q]) & 3);
        }
        soff = (uint32_t)((wave & 3) * pb) + rows_nb * 16 + ((lane & 15) * 16 < rows_nb ? (lane & 15) * 16 : 0);
        bsrc = Bblk;
    };
    const int nk = (K + 127) / 128;
    const bool odd = SHIFT && (K & 64) != 0;   // the last stage has 64 k
    // the 16 rows q of this wave's 64, words of panel pn; past the last row's, the last
    auto issue_ascales = [&](int pn, int q, int row) {
        const uintptr_t p = (scales_at(row) & ~(uintptr_t)3) + (uintptr_t)(pn * 16 + (lane & 3) * 4);
        copy_to_lds<4>((const void *)(p < last_word ? p : last_word), lds_at + NS * STAGE + pn % NP * APANEL + (wave * 4 + q) * 256);
    };
    auto issue = [&](int kt) {
        const uint32_t st = lds_at + (kt % NS) * STAGE;
        // the pieces past K of a last half stage are those of its first half again, and not used
        const bool tail = odd && kt == nk - 1;
#pragma unroll
        for (int j = 0; j < AI; ++j) {
            const int c = (lane & 3) ^ ((((wave * AI + j) * 16 + (lane >> 2)) >> 2) & 3);
            copy_to_lds<16>(asrc[j] + (int64_t)kt * 64 - (tail && c >= 2 ? 32 : 0), st + (wave * AI + j) * 1024);
        }
#pragma unroll
        for (int j = 0; j < BI; ++j) {
            const int c = wave * BI + j;
            copy_to_lds(bsrc + (int64_t)kt * bstep - (tail && (c >> 2) >= 2 ? bstep / 2 : 0), boff[j], st + ACODE + c * 1024);
        }
        if (wave < 4) {
            const int q = kt & 3;
            issue_ascales(kt / 4 + 1, q, q & 2 ? (q & 1 ? srow[3] : srow[2]) : (q & 1 ? srow[1] : srow[0]));
        } else if (lane < 16) {
            copy_to_lds(bsrc + (int64_t)kt * bstep - (tail && wave >= 6 ? bstep / 2 : 0), soff, st + ACODE + BCODE + (wave - 4) * 256);
        }
    };

    const int sw = ((lane & 31) >> 2) & 3;
    const int foff[2] = {(lane & 31) * 64 + ((0 + half) ^ sw) * 16, (lane & 31) * 64 + ((2 + half) ^ sw) * 16};
    f32x16_t acc[MI][NI];
    u32x4_t af[2][MI], bf[2][NI];
    int as[MI], bs[2][NI];   // A: this lane's scale bytes at bytes 0 (step 0) and 2 (step 1)
    int asn[MI];
    auto read_frags = [&](int kt, int ks, int set) {
        const char *st = lds + (kt % NS) * STAGE;
        const char *As = st + wm * TM * 64 + foff[ks];
#pragma unroll
        for (int i = 0; i < MI; ++i) af[set][i] = *(const u32x4_t *)(As + i * 32 * 64);
        const char *Bs = st + ACODE + (2 * ks + half) * (BN * 16) + (wn * TN + (lane & 31)) * 16;
#pragma unroll
        for (int j = 0; j < NI; ++j) bf[set][j] = *(const u32x4_t *)(Bs + j * 32 * 16);
        const char *Bc = st + ACODE + BCODE + (2 * ks + half) * BN + wn * TN + (lane & 31);
#pragma unroll
        for (int j = 0; j < NI; ++j) bs[set][j] = *(const uint8_t *)(Bc + j * 32);
        if (ks == 0) {
            const char *Ac = apanel + (wm * TM + (lane & 31)) * 16;
            const int w0 = (kt >> 2) % NP * APANEL + (kt & 3) * 4, w1 = ((kt + 1) >> 2) % NP * APANEL + ((kt + 1) & 3) * 4;
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                uint32_t w = *(const uint32_t *)(Ac + w0 + i * 512);
                if constexpr (SHIFT) w = __builtin_amdgcn_alignbyte(*(const uint32_t *)(Ac + w1 + i * 512), w,
                                                                  s_shift[wm * TM + i * 32 + (lane & 31)]);
                asn[i] = (int)(w >> (8 * half));
            }
        }
    };
    auto mfmas = [&](auto ks_t) {
        constexpr int ks = decltype(ks_t)::value;
        if (ks == 0)
#pragma unroll
            for (int i = 0; i < MI; ++i) as[i] = asn[i];
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const i32x8_t A = {(int)af[ks][i][0], (int)af[ks][i][1], (int)af[ks][i][2], (int)af[ks][i][3], 0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const i32x8_t Bv = {(int)bf[ks][j][0], (int)bf[ks][j][1], (int)bf[ks][j][2], (int)bf[ks][j][3], 0, 0, 0, 0};
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, Bv, acc[i][j], 4, 4, 2 * ks, as[i], 0,
                                                                            bs[ks][j]);
            }
        }
    };

    // the next step's LDS reads are spread over this step's multiplies
    auto interleave = [&]() {
#pragma unroll
        for (int q = 0; q < MI * NI; ++q) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one MFMA
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);   // two LDS reads
        }
    };

    // A tile's first requests: rows of the tile after it, the weights of its
    // routes, the first panel of A's scales, the first stages. They are the oldest
    // of what the wait for its first stage waits for.
    auto begin = [&](const Tile &t, int buf, int par, const Tile &after, int after_buf) {
        fetch_rows(after, after_buf);
        if (EPI == EPI_DOWN && wave < BM / 64)
            copy_to_lds<4>(a.topk_w + s_rows[buf][wave * 64 + lane], alpha_at + (par * BM + wave * 64) * 4);
        if (wave < 4)
#pragma unroll
            for (int q = 0; q < 4; ++q) issue_ascales(0, q, srow[q]);
#pragma unroll
        for (int p = 0; p < NS - 1; ++p)
            if (p < nk) issue(p);
    };

    int tl = li, par = 0, buf = 0;
    Tile cur = decode(start_x + tl), nxt = tl + nwg < cnt_x ? decode(start_x + tl + nwg) : cur;
    fetch_rows(cur, 0);
    wait_vmcnt<0>();
    __syncthreads();
    set_sources(cur, 0);
    begin(cur, 0, 0, nxt, 1);
    for (;;) {
        const bool wave_active = wm * TM < cur.rows;
        const int tn = tl + nwg;
        const bool has_next = tn < cnt_x;
        const Tile after = tn + nwg < cnt_x ? decode(start_x + tn + nwg) : nxt;
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
        // The first stages, and the last tile's stores (leaving these under way
        // gains nothing).
        wait_vmcnt<0>();
        lds_barrier();
        if (wave_active) read_frags(0, 0, 0);
        // At the top of step kt stage kt is visible to every wave, and this wave
        // holds its step-0 fragments. Stage kt + 1 is made visible (own copies
        // waited for, unless it is one of the first, then a barrier) and stage
        // kt + NS - 1 requested into the slot of stage kt - 1, which every wave
        // finished before that barrier. Loads return in order: stage kt + 1 is there
        // once no more than the copies of the next one are outstanding.
        for (int kt = 0; kt < nk; ++kt) {
            const bool more = kt + 1 < nk;
            if (more) {
                if (kt + 1 >= NS - 1) wait_vmcnt_stages<LOADS, NS - 3>(min(NS - 3, nk - 2 - kt));
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");   // for the compiler: reads stay behind
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            }
            if (more && kt + NS - 1 < nk) issue(kt + NS - 1);
            if (wave_active) {
                read_frags(kt, 1, 1);
                mfmas(std::integral_constant<int, 0>());
                interleave();
                // on the last step this reads a resident stage again; the values are not used
                read_frags(kt + 1, 0, 0);
                if (!(odd && !more)) mfmas(std::integral_constant<int, 1>());
                interleave();
            }
        }
        const Tile done = cur;
        if (has_next) {
            lds_barrier();   // nothing reads the ring any more
            const int nb = buf == 2 ? 0 : buf + 1;
            set_sources(nxt, nb);
            begin(nxt, nb, par ^ 1, after, nb == 2 ? 0 : nb + 1);
        }
        // Register r of lane l holds row 8 (r / 4) + 4 (l / 32) + r % 4 and column
        // l % 32 of its block. bf16: adjacent lanes swap a value of rows R, R + 1,
        // so that each stores two columns of one row. The tile's rows of C are a
        // buffer: stores to rows past its last one are dropped by its bounds
        // check, so no store has a branch. A wave's 64 columns are all in N or
        // all past it.
        if constexpr (EPI == EPI_GATE_UP) {
            if (wave_active && done.n0 + wn * TN < N) {
                // opaque, as ld below: the rows' offsets are not held through the tile loop
                int f = N / 2;
                asm volatile("" : "+s"(f));
                const int blk = (done.n0 + wn * TN) / 64;   // block of 32 units
                uint8_t *hc = (uint8_t *)a.C + (int64_t)done.row0 * (f / 2) + blk * 16;
                uint8_t *hs = a.Hs + (int64_t)done.row0 * (f / 32) + blk;
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    float h[16];
#pragma unroll
                    for (int r = 0; r < 16; ++r) h[r] = silu_mul(acc[i][0][r], acc[i][1][r]);
                    // of negative numbers the least has the largest bits (a layer of 4096 tokens
                    // on 64 experts of 2048 x 1024: 325 us with this and without; with fminf 327)
                    uint32_t least = __float_as_uint(acc[i][0][0]);
#pragma unroll
                    for (int r = 1; r < 16; ++r) least = max(least, __float_as_uint(acc[i][0][r]));
                    if (__any(least > __builtin_bit_cast(uint32_t, kSiluTail))) {
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (acc[i][0][r] < kSiluTail) h[r] = silu_tail_mul(acc[i][0][r], acc[i][1][r]);
                    }
                    const uint32_t byte = block_scale(block_tops(h, lane));   // of register lane % 16's row
                    const float unit = block_unit(byte);
                    scale_rows(h, unit, std::make_integer_sequence<int, 16>());
                    if (__any(byte == 255)) zero_rows(h, byte == 255 ? 0 : -1, std::make_integer_sequence<int, 16>());
#pragma unroll
                    for (int r8 = 0; r8 < 16; r8 += 8) {
                        uint32_t q = 0;   // nibble r: this lane's unit in row r8 + r
                        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, h[r8 + 0], h[r8 + 1], 1.0f, 0);
                        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, h[r8 + 2], h[r8 + 3], 1.0f, 1);
                        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, h[r8 + 4], h[r8 + 5], 1.0f, 2);
                        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, h[r8 + 6], h[r8 + 7], 1.0f, 3);
                        q = transpose8(unsigned_zeros(q), lane);   // row r8 + lane % 8, units 8 (lane / 8) .. +7
                        const int rr = r8 + (lane & 7);
                        const int m = wm * TM + i * 32 + 8 * (rr / 4) + 4 * half + (rr & 3);
                        if (m < done.rows) *(uint32_t *)(hc + (int64_t)m * (f / 2) + ((lane & 31) >> 3) * 4) = q;
                    }
                    const int rr = lane & 15, m = wm * TM + i * 32 + 8 * (rr / 4) + 4 * half + (rr & 3);
                    if ((lane & 16) == 0 && m < done.rows) hs[(int64_t)m * (f / 32)] = (uint8_t)byte;
                }
            }
        } else if constexpr (EPI == EPI_DOWN) {
            if (wave_active && done.n0 + wn * TN < N) {
                float *C = (float *)a.C + done.n0 + wn * TN + (lane & 31);
#pragma unroll
                for (int i = 0; i < MI; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int m = wm * TM + i * 32 + 8 * (r / 4) + 4 * half + (r & 3);
                        if (m >= done.rows) continue;
                        const float al = s_alpha[par][m];
                        float *y = C + (int64_t)s_rows[buf][m] * a.ldc;
#pragma unroll
                        for (int j = 0; j < NI; ++j) y[j * 32] = al * acc[i][j][r];
                        for (int q = 1; q < a.splits; ++q)
#pragma unroll
                            for (int j = 0; j < NI; ++j) y[q * a.split_stride + j * 32] = 0.0f;
                    }
            }
            if (done.n0 == 0)
                for (int m = tid; m < done.rows; m += 512) a.done[s_rows[buf][m]] = 1;
        } else if (wave_active && done.n0 + wn * TN < N) {
            const int esz = a.c_bf16 ? 2 : 4;
            char *base = (char *)a.C + ((int64_t)done.row0 * a.ldc + done.n0 + wn * TN) * esz;
            // opaque, or the rows' offsets are computed before the tile loop and
            // held through it (211 registers spilled)
            uint32_t ld = (uint32_t)a.ldc * esz;
            asm volatile("" : "+s"(ld));
            const __amdgpu_buffer_rsrc_t buf = __builtin_amdgcn_make_buffer_rsrc(base, 0, (int)(done.rows * ld), 0x00027000);
            const uint32_t row = wm * TM + 4 * half;
            if (a.c_bf16) {
                const bool even = (lane & 1) == 0;
                const uint32_t at = (row + (even ? 0 : 1)) * ld + (lane & 30) * 2;
#pragma unroll
                for (int i = 0; i < MI; ++i)
#pragma unroll
                    for (int r = 0; r < 16; r += 2) {
                        const uint32_t o = at + (uint32_t)(i * 32 + 8 * (r / 4) + (r & 3)) * ld;
#pragma unroll
                        for (int j = 0; j < NI; ++j) {
                            const float s0 = acc[i][j][r], s1 = acc[i][j][r + 1];
                            const float y = __int_as_float(
                                __builtin_amdgcn_mov_dpp(__float_as_int(even ? s1 : s0), 0xB1, 0xF, 0xF, false));
                            __builtin_amdgcn_raw_buffer_store_b32(even ? bf16_pair(s0, y) : bf16_pair(y, s1), buf,
                                                                  (int)(o + j * 64), 0, kStream);
                        }
                    }
            } else {
                const uint32_t at = row * ld + (lane & 31) * 4;
#pragma unroll
                for (int i = 0; i < MI; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const uint32_t o = at + (uint32_t)(i * 32 + 8 * (r / 4) + (r & 3)) * ld;
#pragma unroll
                        for (int j = 0; j < NI; ++j)
                            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[i][j][r]), buf, (int)(o + j * 128), 0, kStream);
                    }
            }
        }
        if (!has_next) break;
        cur = nxt;
        nxt = after;
        tl = tn;
        par ^= 1;
        buf = buf == 2 ? 0 : buf + 1;
    }
}

}  // namespace

hipError_t launch_quantize_mxfp4(const void *src, bool bf16, int64_t rows, int K, int64_t ld, uint8_t *codes,
                                 uint8_t *scales, hipStream_t st)
{
    const int64_t n8 = rows * (K / 8);
    if (n8 == 0) return hipSuccess;
    const dim3 grid((unsigned)((n8 + 255) / 256));
    if (bf16)
        hipLaunchKernelGGL(k_quantize<true>, grid, dim3(256), 0, st, src, n8, K / 8, ld, (uint32_t *)codes, scales);
    else
        hipLaunchKernelGGL(k_quantize<false>, grid, dim3(256), 0, st, src, n8, K / 8, ld, (uint32_t *)codes, scales);
    return hipGetLastError();
}

hipError_t launch_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, int64_t rows, int K, void *dst,
                                   bool bf16, int64_t ld, hipStream_t st)
{
    const int64_t n8 = rows * (K / 8);
    if (n8 == 0) return hipSuccess;
    const dim3 grid((unsigned)((n8 + 255) / 256));
    if (bf16)
        hipLaunchKernelGGL(k_dequantize<true>, grid, dim3(256), 0, st, (const uint32_t *)codes, scales, n8, K / 8, dst,
                           ld);
    else
        hipLaunchKernelGGL(k_dequantize<false>, grid, dim3(256), 0, st, (const uint32_t *)codes, scales, n8, K / 8, dst,
                           ld);
    return hipGetLastError();
}

// The ring kernel's time is that of whole tiles: 15 us for one round of tiles of
// up to 128 rows and 20 us above (K = 2048), whatever they hold. The small
// kernel's grows with its 32 x 64 pieces, 2.5 us for each 64 of them, and with
// less than 16 rows a slot it is ahead at any size (64 slots of N = K = 2048: 1
// row each 18 against 30 us, 16 rows 32 against 32, 64 rows 84 against 32; one
// slot of 512 rows 12 against 20, of 2048 rows 37 against 21). At the borders the
// other one is up to 14 % faster (one slot of 128 rows, N = 8192: 21 against 24). The rule
// goes by the mean, since only the device knows the slots' rows: where one slot of many
// holds most of them it takes the small kernel and loses (N = K = 2048, 4096 rows in one
// of 512 slots 119 us, as one slice 24; with 8192, where the mean is 16, 38 and 32).
static bool ring_pays(const MxArgs &a)
{
    const int64_t slots = std::min(a.P, a.M), rows = a.M / slots;
    const int64_t pieces = slots * ((rows + 31) / 32) * (a.N / 64);
    return rows >= 16 && pieces >= (rows <= 128 ? 512 : 768);
}

template <int EPI>
static hipError_t launch_ring(const MxArgs &a, hipStream_t st)
{
    const int64_t tiles = ((int64_t)(a.M + 255) / 256 + std::min(a.P, a.M) - 1) * ((a.N + 255) / 256);
    const unsigned grid = (unsigned)std::min<int64_t>(tiles, 256);   // one workgroup per compute unit
    if (a.K % 128 == 0 && ((uintptr_t)a.As & 3) == 0)
        hipLaunchKernelGGL((k_matmul_ring<256, 4, false, EPI>), dim3(grid), dim3(512), 0, st, a);
    else
        hipLaunchKernelGGL((k_matmul_ring<256, 4, true, EPI>), dim3(grid), dim3(512), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_gate_up_mxfp4(const MxArgs &a, hipStream_t st)
{
    return a.M == 0 ? hipSuccess : launch_ring<EPI_GATE_UP>(a, st);
}

hipError_t launch_down_mxfp4(const MxArgs &a, hipStream_t st)
{
    return a.M == 0 ? hipSuccess : launch_ring<EPI_DOWN>(a, st);
}

hipError_t launch_matmul_mxfp4(const MxArgs &a, hipStream_t st)
{
    if (a.M == 0) return hipSuccess;
    if (ring_pays(a)) return launch_ring<EPI_STORE>(a, st);
    // at most this many row tiles: one partial tile per slot with records
    const int64_t mt = (int64_t)(a.M + 63) / 64 + std::min(a.P, a.M) - 1;
    hipLaunchKernelGGL(k_matmul_small, dim3((unsigned)(mt * (a.N / 64))), dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace moe
