// MXFP4: rows to blocks of 32 values (E2M1 codes and one E8M0 scale each),
// blocks back to values, and the product of two matrices held that way.
//
// Quantisation of a block: with e the biased exponent field of its largest
// magnitude, the scale byte is max(e - 2, 0), the power of two that brings
// that magnitude into [4, 8); each value times 2^(127 - byte) is rounded to the
// nearest E2M1 value, ties to the even code, at most 6. A block that holds an
// infinity or a NaN gets the byte 255 (NaN) and codes 0. A zero has no sign.
#include <algorithm>

#include "mxfp4.h"

namespace moe {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

// 8 values per lane, 4 lanes per block. Bound by HBM: 4 or 2 bytes read and
// 17/32 written a value.
template <bool BF16>
__global__ __launch_bounds__(256) void k_quantize(const void *__restrict__ src, int64_t n8, int K8, int64_t ld,
                                                  uint32_t *__restrict__ codes, uint8_t *__restrict__ scales)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n8) return;   // whole blocks of 4 lanes: n8 % 4 == 0
    const int64_t row = i / K8;
    const int64_t at = row * ld + (i - row * K8) * 8;
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
    const int e = (int)(top >> 23);
    const int byte = e == 255 ? 255 : max(e - 2, 0);
    // 2^(127 - byte): byte <= 252, so the exponent field is at least 2
    const float up = __uint_as_float((uint32_t)(254 - min(byte, 252)) << 23);
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
    // drop the sign of codes of magnitude 0
    const uint32_t m = q & 0x77777777u, nz = (m | m >> 1 | m >> 2) & 0x11111111u;
    q = m | (q & nz << 3);
    codes[i] = byte == 255 ? 0u : q;
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
    const int64_t row = i / K8;
    const int64_t at = row * ld + (i - row * K8) * 8;
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

// Product of MXFP4 operands on the scaled matrix instructions
// (v_mfma_scale_f32_32x32x64_f8f6f4: lane l supplies row l % 32 and the 32
// consecutive k values 32 (l / 32) .. +31 of each operand, 16 bytes of codes,
// with that block's scale byte): products and scales are exact, sums in fp32.
// A tile of 64 records x 64 columns per workgroup, 32 x 32 per wave, operands
// straight from global memory.
__global__ __launch_bounds__(256) void k_matmul(MxArgs a)
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
            int off = 0, end = 0;
            if (s < a.P) {
                off = a.slot_offset ? min(max(a.slot_offset[s], 0), a.M) : 0;
                end = a.slot_offset ? min(a.slot_offset[s + 1], a.M) : a.M;
            }
            const int mt = max(end - off + 63, 0) / 64;
            const int inc = run + wave_incl_scan(mt, lane);
            if (bid < inc && bid >= inc - mt) {
                s_tile[0] = s;
                s_tile[1] = off + (bid - (inc - mt)) * 64;
                s_tile[2] = min(64, end - s_tile[1]);
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
    int rec = row0 + min(m0 + (lane & 31), cnt - 1);
    if (a.row_index) rec = a.row_index[rec];
    rec = min(max(rec, 0), a.A_rows - 1);
    const uint8_t *ap = a.A + (int64_t)rec * (K / 2) + half * 16;
    const uint8_t *as = a.As + (int64_t)rec * (K / 32) + half;
    const int n = c0 + (lane & 31), nb = n / kWRows, rows = min(kWRows, N - nb * kWRows);
    const int64_t pb = fp4_piece_bytes(rows);
    const uint8_t *bp = a.B + (int64_t)slot * a.B_stride + (int64_t)nb * (K / kWK) * fp4_piece_bytes(kWRows) + half * pb;
    const int rb = n - nb * kWRows;
    f32x16_t acc;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
    for (int k = 0; k < K / 64; ++k) {
        const u32x4_t av = *(const u32x4_t *)(ap + k * 32);
        const u32x4_t bv = *(const u32x4_t *)(bp + 2 * k * pb + rb * 16);
        const int sa = as[2 * k], sb = bp[2 * k * pb + rows * 16 + rb];
        const i32x8_t A = {(int)av[0], (int)av[1], (int)av[2], (int)av[3], 0, 0, 0, 0};
        const i32x8_t Bv = {(int)bv[0], (int)bv[1], (int)bv[2], (int)bv[3], 0, 0, 0, 0};
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, Bv, acc, 4, 4, 0, sa, 0, sb);
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

hipError_t launch_matmul_mxfp4(const MxArgs &a, hipStream_t st)
{
    if (a.M == 0) return hipSuccess;
    // at most this many row tiles: one partial tile per slot with records
    const int64_t mt = (int64_t)(a.M + 63) / 64 + std::min(a.P, a.M) - 1;
    hipLaunchKernelGGL(k_matmul, dim3((unsigned)(mt * (a.N / 64))), dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace moe
