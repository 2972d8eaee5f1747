// Rows and weights in 8-bit floating point (e4m3: sign, 4 exponent bits with
// bias 7, 3 mantissa bits, no infinities) with a scale for each block of 128,
// and the products of the two.
//
// Rows: a block is 128 consecutive values of a row, its scale one byte b,
// 2^(b - 127). Weights: a block is 128 rows x 128 values, its scale an fp32
// number. Both are quantised with the least power of two that brings the
// block's largest magnitude to 448, the format's largest value, or below: a
// power of two costs no precision (e4m3 is a floating point format), the values
// are scaled exactly and rounded once, and the scaled matrix instructions
// take the rows' scales for nothing. b lies in [1, 247], so that every scale
// is a normal fp32 number. A block that holds an infinity or a NaN gets the
// scale NaN (byte 255) and codes 0.
#include <algorithm>

#include "device.h"
#include "fp8.h"

namespace moe {
namespace {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// Scale byte of a block from the bits of its largest magnitude: 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t block_byte(uint32_t top)
{
    const int e = (int)(top >> 23);
    return e == 255 ? 255u : (uint32_t)max(e - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0), 1);
}
// The factor 2^(127 - byte) that a block's values are quantised with (1 for a NaN block).
__device__ __forceinline__ float block_unit(uint32_t byte)
{
    return byte == 255 ? 1.0f : __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ float block_value(uint32_t byte)
{
    return __uint_as_float(byte == 255 ? 0x7fc00000u : byte << 23);
}

// 8 consecutive values as fp32.
template <bool BF16>
__device__ __forceinline__ void load8(const void *src, int64_t at, uint32_t *v)
{
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
}
// Codes of 8 values times unit.
__device__ __forceinline__ u32x2_t codes8(const uint32_t *v, float unit, bool bad)
{
    u32x2_t q;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = __uint_as_float(v[4 * c + i]) * unit;
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(s[2], s[3], w, true);
        q[c] = bad ? 0u : (uint32_t)w;
    }
    return q;
}
__device__ __forceinline__ uint32_t largest(const uint32_t *v)
{
    uint32_t top = 0;   // magnitudes order as their bits do (infinities and NaN above all numbers)
#pragma unroll
    for (int c = 0; c < 8; ++c) top = max(top, v[c] & 0x7fffffffu);
    return top;
}
template <int N>
__device__ __forceinline__ uint32_t max_over(uint32_t v)
{
#pragma unroll
    for (int o = 1; o < N; o <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
    return v;
}

// Rows: 16 lanes a block, 8 values a lane; a row's last block may be 64 wide.
// Bound by HBM: 4 or 2 bytes read and 1 written a value.
template <bool BF16>
__global__ __launch_bounds__(256) void k_quantize_rows(const void *__restrict__ src, int64_t blocks, int KB, int K,
                                                       int64_t ld, int64_t lds, uint8_t *__restrict__ codes,
                                                       uint8_t *__restrict__ scales)
{
    const int64_t b = (int64_t)blockIdx.x * 16 + threadIdx.x / 16;
    const uint32_t row = (uint32_t)min(b, blocks - 1) / (uint32_t)KB;
    const int kb = (int)((uint32_t)min(b, blocks - 1) - row * (uint32_t)KB), k = kb * kFp8Block + (threadIdx.x & 15) * 8;
    uint32_t v[8] = {};
    const bool in = b < blocks && k < K;
    if (in) load8<BF16>(src, row * ld + k, v);
    const uint32_t byte = block_byte(max_over<16>(largest(v)));
    if (in) *(u32x2_t *)(codes + (int64_t)row * K + k) = codes8(v, block_unit(byte), byte == 255);
    if (in && (threadIdx.x & 15) == 0) scales[row * lds + kb] = (uint8_t)byte;
}

// Weights: a workgroup a block, which it holds in registers, 8 rows of 8 values
// a thread. Bound by HBM.
template <bool BF16>
__global__ __launch_bounds__(256) void k_quantize_blocks(const void *__restrict__ src, int64_t rows, int KB, int K,
                                                         int64_t ld, uint8_t *__restrict__ codes,
                                                         float *__restrict__ scales)
{
    __shared__ uint32_t s_top[4];
    const uint32_t nb = blockIdx.x / (uint32_t)KB;
    const int kb = (int)(blockIdx.x - nb * (uint32_t)KB), k = kb * kFp8Block + (threadIdx.x & 15) * 8;
    const int64_t r0 = (int64_t)nb * kFp8Block + threadIdx.x / 16;
    uint32_t v[8][8] = {}, top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k < K && r0 + 16 * i < rows) load8<BF16>(src, (r0 + 16 * i) * ld + k, v[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, largest(v[i]));
    top = max_over<64>(top);
    if ((threadIdx.x & 63) == 0) s_top[threadIdx.x / 64] = top;
    __syncthreads();
    const uint32_t byte = block_byte(max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3])));
    const float unit = block_unit(byte);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (k < K && r0 + 16 * i < rows) *(u32x2_t *)(codes + (r0 + 16 * i) * K + k) = codes8(v[i], unit, byte == 255);
    if (threadIdx.x == 0) scales[blockIdx.x] = block_value(byte);
}

// 8 values a lane: code value times scale in fp32, rounded once more to bf16
// (exact in both for scales that are powers of two, unless the result leaves the
// normal numbers).
template <bool BF16, bool ROWS>
__global__ __launch_bounds__(256) void k_dequantize(const uint8_t *__restrict__ codes, const void *__restrict__ scales,
                                                    int64_t n8, int K8, int64_t lds, void *__restrict__ dst, int64_t ld)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n8) return;
    const uint32_t row = (uint32_t)i / (uint32_t)K8;
    const int k = (int)((uint32_t)i - row * (uint32_t)K8) * 8;
    const u32x2_t q = *(const u32x2_t *)(codes + i * 8);
    const float s = ROWS ? block_value(((const uint8_t *)scales)[row * lds + k / kFp8Block])
                         : ((const float *)scales)[(row / kFp8Block) * lds + k / kFp8Block];
    float v[8];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[c], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[c], true);
        v[4 * c] = lo[0] * s;
        v[4 * c + 1] = lo[1] * s;
        v[4 * c + 2] = hi[0] * s;
        v[4 * c + 3] = hi[1] * s;
    }
    const int64_t at = row * ld + k;
    if constexpr (BF16) {
        u32x4_t o;
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = bf16_pair(v[2 * c], v[2 * c + 1]);
        *(u32x4_t *)((uint16_t *)dst + at) = o;
    } else {
        *(f32x4_t *)((float *)dst + at) = f32x4_t{v[0], v[1], v[2], v[3]};
        *(f32x4_t *)((float *)dst + at + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
    }
}

// ---------------------------------------------------------------------------
// Products. Two ways to multiply codes:
//  - the fp8 matrix instructions, at twice the rate of bf16. They align the
//    products of 8 neighbouring k and cut what lies more than 13 bits below the
//    largest one's exponent (measured with one large and one small product at
//    every distance; across the groups of 8 sums keep 24 bits): 1.1e-5 of the
//    norm of C for normally distributed operands, whatever K. That is a 350th of a
//    rounding to bf16 and less yet of one to 8 bits, so C in bf16 and H of many
//    records go this way.
//  - codes decoded to bf16, which is exact, on the bf16 instructions, whose sums
//    keep 24 bits (2e-8): fp32 C, and few records a slot, where the time goes into
//    reading the weights and the decoding is free.
// Which of a block's 128 k values a lane supplies in which place is free, as
// long as it is the same for both operands: they have one scale.

// Slot s holds the records [lo, hi), brought into [0, M).
__device__ __forceinline__ void slot_range(const Fp8Args &a, int s, int *lo, int *hi)
{
    *lo = a.slot_offset ? min(max(a.slot_offset[s], 0), a.M) : 0;
    *hi = a.slot_offset ? min(max(a.slot_offset[s + 1], *lo), a.M) : a.M;
}
__device__ __forceinline__ int row_of(const Fp8Args &a, int rec)
{
    return min(max(a.row_index ? a.row_index[rec] : rec, 0), a.A_rows - 1);
}
// Row tile `tile` of R records: its slot (-1: there is none), first record and
// records. Every wave finds it for itself.
template <int R>
__device__ __forceinline__ int find_tile(const Fp8Args &a, int tile, int lane, int *row0, int *cnt)
{
    int run = 0, slot = -1;
    for (int s0 = 0; s0 < a.P && slot < 0; s0 += 64) {
        const int s = s0 + lane;
        int lo = 0, hi = 0;
        if (s < a.P) slot_range(a, s, &lo, &hi);
        const int mt = (hi - lo + R - 1) / R, inc = run + wave_incl_scan(mt, lane);
        const uint64_t mine = __ballot(tile < inc && tile >= inc - mt);
        if (mine) {
            const int l = __builtin_ctzll(mine);
            slot = s0 + l;
            *row0 = __builtin_amdgcn_readlane(lo, l) + (tile - (__builtin_amdgcn_readlane(inc, l) - __builtin_amdgcn_readlane(mt, l))) * R;
            *cnt = min(R, __builtin_amdgcn_readlane(hi, l) - *row0);
        }
        run = __builtin_amdgcn_readlane(inc, 63);
    }
    return slot;
}

// 32 of a row's 128 codes for this lane: 16 at 16 (lane / 16) and 16 at 64 + the
// same, so that an instruction reads 64 contiguous bytes of a row. With only 64
// left (half), the first ones again.
__device__ __forceinline__ i32x8_t codes32(const uint8_t *p, bool half)
{
    const u32x4_t a = *(const u32x4_t *)p, b = *(const u32x4_t *)(p + (half ? 0 : 64));
    return i32x8_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// 32 codes times scale (a power of two) as four operands of 8 bf16.
__device__ __forceinline__ void decode32(const i32x8_t &q, float scale, bf16x8_t (&v)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bf16x2_t p[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * i], scale, false),
                               __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * i], scale, true),
                               __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * i + 1], scale, false),
                               __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * i + 1], scale, true)};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            v[i][2 * c] = p[c][0];
            v[i][2 * c + 1] = p[c][1];
        }
    }
}
// acc += sb times the product of 128 k (16 x 16).
__device__ __forceinline__ void step128(f32x4_t &acc, const bf16x8_t (&A)[4], const i32x8_t &q, float sb)
{
    bf16x8_t Bv[4];
    decode32(q, 1.0f, Bv);
    f32x4_t part = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[i], Bv[i], part, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = fmaf(part[r], sb, acc[r]);
}

// Few records a slot: 16 records x 16 NT columns a workgroup, its W waves taking
// steps of 128 k in turn, their sums joined in LDS in the order of the waves.
template <int NT, int W>
__global__ __launch_bounds__(64 * W) void k_matmul_few(Fp8Args a)
{
    __shared__ f32x4_t s_sum[W][NT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int ntn = (a.N + 16 * NT - 1) / (16 * NT), n0 = blockIdx.x % ntn * (16 * NT);
    int row0 = 0, cnt = 0;
    const int slot = find_tile<16>(a, blockIdx.x / ntn, lane, &row0, &cnt);
    if (slot < 0) return;
    const int K = a.K, KB = (K + kFp8Block - 1) / kFp8Block;
    const int rec = row_of(a, row0 + min(lane & 15, cnt - 1));
    const uint8_t *ap = a.A + (int64_t)rec * K + (lane >> 4) * 16;
    const uint8_t *as = a.As + rec * fp8_scale_bytes(K);
    const uint8_t *bp[NT];
    const float *bs[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int n = min(n0 + 16 * j + (lane & 15), a.N - 1);
        bp[j] = a.B[0] + slot * a.B_stride + (int64_t)n * K + (lane >> 4) * 16;
        bs[j] = a.Bs[0] + slot * a.Bs_stride + (int64_t)(n / kFp8Block) * KB;
    }
    f32x4_t acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int kb = wave; kb < KB; kb += W) {
        const bool half = (kb + 1) * kFp8Block > K;
        i32x8_t A = codes32(ap + (int64_t)kb * kFp8Block, half);
        if (half)
#pragma unroll
            for (int i = 4; i < 8; ++i) A[i] = 0;
        bf16x8_t Av[4];
        decode32(A, block_value(as[kb]), Av);
#pragma unroll
        for (int j = 0; j < NT; ++j) step128(acc[j], Av, codes32(bp[j] + (int64_t)kb * kFp8Block, half), bs[j][kb]);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) s_sum[wave][j][lane] = acc[j];
    __syncthreads();
    for (int j = wave; j < NT; j += W) {
        f32x4_t s = s_sum[0][j][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) s += s_sum[w][j][lane];
        const int n = n0 + 16 * j + (lane & 15);
        if (n >= a.N) continue;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int m = 4 * (lane >> 4) + r;
            if (m >= cnt) continue;
            const int64_t at = (int64_t)(row0 + m) * a.ldc + n;
            if (a.c_bf16)
                ((uint16_t *)a.C)[at] = (uint16_t)bf16_pair(s[r], 0.0f);
            else
                ((float *)a.C)[at] = s[r];
        }
    }
}

__device__ __forceinline__ float swiglu(float g, float u) { return g < kSiluTail ? silu_tail_mul(g, u) : silu_mul(g, u); }

// SiLU(g) u for few records a slot: 16 records x 128 units a workgroup, so that
// the blocks of H are whole; wave w takes gate and up of units 16 (w % 8) .. +15
// and every second step of 128 k. H passes through LDS to a wave a record.
__global__ __launch_bounds__(1024) void k_gate_up_few(Fp8Args a)
{
    __shared__ f32x4_t s_sum[8][2][64];
    __shared__ float s_h[16][kFp8Block + 4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, cg = wave & 7;
    const int fb = (a.N + kFp8Block - 1) / kFp8Block, f0 = blockIdx.x % fb * kFp8Block;
    int row0 = 0, cnt = 0;
    const int slot = find_tile<16>(a, blockIdx.x / fb, lane, &row0, &cnt);
    if (slot < 0) return;   // the same in every wave
    const int K = a.K, KB = (K + kFp8Block - 1) / kFp8Block;
    const int rec = row_of(a, row0 + min(lane & 15, cnt - 1));
    const uint8_t *ap = a.A + (int64_t)rec * K + (lane >> 4) * 16;
    const uint8_t *as = a.As + rec * fp8_scale_bytes(K);
    const int n = min(f0 + 16 * cg + (lane & 15), a.N - 1);
    const int64_t at = slot * a.B_stride + (int64_t)n * K + (lane >> 4) * 16;
    const int64_t sat = slot * a.Bs_stride + (int64_t)(f0 / kFp8Block) * KB;
    f32x4_t acc[2] = {f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}};
    for (int kb = wave >> 3; kb < KB; kb += 2) {
        const bool half = (kb + 1) * kFp8Block > K;
        i32x8_t A = codes32(ap + (int64_t)kb * kFp8Block, half);
        if (half)
#pragma unroll
            for (int i = 4; i < 8; ++i) A[i] = 0;
        bf16x8_t Av[4];
        decode32(A, block_value(as[kb]), Av);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            step128(acc[j], Av, codes32(a.B[j] + at + (int64_t)kb * kFp8Block, half), a.Bs[j][sat + kb]);
    }
    if (wave >= 8) {
        s_sum[cg][0][lane] = acc[0];
        s_sum[cg][1][lane] = acc[1];
    }
    __syncthreads();
    if (wave < 8) {
        const f32x4_t g = acc[0] + s_sum[cg][0][lane], u = acc[1] + s_sum[cg][1][lane];
        const bool in = f0 + 16 * cg + (lane & 15) < a.N;
#pragma unroll
        for (int r = 0; r < 4; ++r) s_h[4 * (lane >> 4) + r][16 * cg + (lane & 15)] = in ? swiglu(g[r], u[r]) : 0.0f;
    }
    __syncthreads();
    if (wave >= cnt) return;
    const float h0 = s_h[wave][2 * lane], h1 = s_h[wave][2 * lane + 1];
    const uint32_t byte = block_byte(max_over<64>(max(__float_as_uint(h0) & 0x7fffffffu, __float_as_uint(h1) & 0x7fffffffu)));
    const float unit = block_unit(byte);
    const int q = __builtin_amdgcn_cvt_pk_fp8_f32(h0 * unit, h1 * unit, 0, false);
    const int64_t p = row0 + wave;
    if (f0 + 2 * lane < a.N) *(uint16_t *)((uint8_t *)a.C + p * a.N + f0 + 2 * lane) = byte == 255 ? 0 : (uint16_t)q;
    if (lane == 0) a.Hs[p * fp8_scale_bytes(a.N) + f0 / kFp8Block] = (uint8_t)byte;
}

}  // namespace

hipError_t launch_quantize_fp8(const void *src, bool bf16, int64_t rows, int K, int64_t ld, int block_rows,
                               uint8_t *codes, void *scales, hipStream_t st)
{
    if (rows == 0) return hipSuccess;
    const int KB = (int)fp8_blocks(K);
    if (block_rows == 1) {
        const int64_t blocks = rows * KB, lds = fp8_scale_bytes(K);
        const dim3 grid((unsigned)((blocks + 15) / 16));
        if (bf16)
            hipLaunchKernelGGL(k_quantize_rows<true>, grid, dim3(256), 0, st, src, blocks, KB, K, ld, lds, codes, (uint8_t *)scales);
        else
            hipLaunchKernelGGL(k_quantize_rows<false>, grid, dim3(256), 0, st, src, blocks, KB, K, ld, lds, codes, (uint8_t *)scales);
    } else {
        const dim3 grid((unsigned)(fp8_blocks(rows) * KB));
        if (bf16)
            hipLaunchKernelGGL(k_quantize_blocks<true>, grid, dim3(256), 0, st, src, rows, KB, K, ld, codes, (float *)scales);
        else
            hipLaunchKernelGGL(k_quantize_blocks<false>, grid, dim3(256), 0, st, src, rows, KB, K, ld, codes, (float *)scales);
    }
    return hipGetLastError();
}

hipError_t launch_dequantize_fp8(const uint8_t *codes, const void *scales, int64_t rows, int K, int block_rows,
                                 void *dst, bool bf16, int64_t ld, hipStream_t st)
{
    const int64_t n8 = rows * (K / 8);
    if (n8 == 0) return hipSuccess;
    const dim3 grid((unsigned)((n8 + 255) / 256));
    auto go = [&](auto kernel, int64_t lds) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, codes, scales, n8, K / 8, lds, dst, ld);
    };
    if (block_rows == 1)
        bf16 ? go(k_dequantize<true, true>, fp8_scale_bytes(K)) : go(k_dequantize<false, true>, fp8_scale_bytes(K));
    else
        bf16 ? go(k_dequantize<true, false>, fp8_blocks(K)) : go(k_dequantize<false, false>, fp8_blocks(K));
    return hipGetLastError();
}

// at most this many row tiles of R records: one partial tile per slot with records
static int64_t row_tiles(const Fp8Args &a, int R) { return (int64_t)(a.M + R - 1) / R + std::min(a.P, a.M) - 1; }

hipError_t launch_matmul_fp8(const Fp8Args &a, hipStream_t st)
{
    if (a.M == 0) return hipSuccess;
    const int64_t grid = row_tiles(a, 16) * (a.N / 64);
    hipLaunchKernelGGL((k_matmul_few<4, 4>), dim3((unsigned)grid), dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_gate_up_fp8(const Fp8Args &a, hipStream_t st)
{
    if (a.M == 0) return hipSuccess;
    const int64_t grid = row_tiles(a, 16) * fp8_blocks(a.N);
    hipLaunchKernelGGL(k_gate_up_few, dim3((unsigned)grid), dim3(1024), 0, st, a);
    return hipGetLastError();
}

}  // namespace moe
