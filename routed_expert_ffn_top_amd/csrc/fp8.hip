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
#include <type_traits>

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

// 2^(e - 127) of an exponent field; 0: 2^-127, 255: NaN.
__device__ __forceinline__ float exponent_value(int e)
{
    return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7fc00000u : (uint32_t)e << 23);
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
// One pass: the maximum goes over 16 lanes while the values stay in registers. 8 values a
// lane make whole 16-byte loads of bf16 and let one row of 2048 fill 4 waves (1.7 us, all of
// it latency). Bound by HBM: 4 or 2 bytes read and 1 written a value; 32768 x 1408 bf16 26.6
// us, 5.2 TB/s, a large copy 5.0 to 5.2.
template <bool BF16>
__global__ __launch_bounds__(256) void k_quantize_rows(const void *__restrict__ src, int64_t blocks, int KB, int K,
                                                       int64_t ld, int64_t lds, uint8_t *__restrict__ codes,
                                                       uint8_t *__restrict__ scales,
                                                       const int32_t *__restrict__ first, const int32_t *__restrict__ last)
{
    const int64_t b = (int64_t)blockIdx.x * 16 + threadIdx.x / 16;
    const uint32_t row = (uint32_t)min(b, blocks - 1) / (uint32_t)KB;
    const int kb = (int)((uint32_t)min(b, blocks - 1) - row * (uint32_t)KB), k = kb * kFp8Block + (threadIdx.x & 15) * 8;
    uint32_t v[8] = {};
    const bool in = b < blocks && k < K && (!first || ((int)row >= *first && (int)row < *last));
    if (in) load8<BF16>(src, row * ld + k, v);
    const uint32_t byte = block_byte(max_over<16>(largest(v)));
    if (in) *(u32x2_t *)(codes + (int64_t)row * K + k) = codes8(v, block_unit(byte), byte == 255);
    if (in && (threadIdx.x & 15) == 0) scales[row * lds + kb] = (uint8_t)byte;
}

// Weights: a workgroup a block, which it holds in registers, 8 rows of 8 values
// a thread: 16 lanes read a row's 128 values, so that the loads are whole lines and all 8 (of
// bf16; 16 of fp32) are in flight before the maximum is taken. Bound by HBM: 65536 x 2048
// fp32 118 us, 5.7 TB/s; a large copy reaches 5.0 to 5.2.
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
// normal numbers). Bound by HBM: 65536 x 2048 to bf16 behind the quantisation, whose 134 MB of codes the
// last-level cache still holds in part, 69 us; over and over on the same codes 59.5, and 75.5 with stores that
// go through the caches, where nothing reads the values again before they leave them.
template <bool BF16, bool ROWS>
__global__ __launch_bounds__(256) void k_dequantize(const uint8_t *__restrict__ codes, const void *__restrict__ scales,
                                                    int64_t n8, int K8, int64_t lds, void *__restrict__ dst, int64_t ld)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n8) return;
    const uint32_t row = (uint32_t)i / (uint32_t)K8;
    const int k = (int)((uint32_t)i - row * (uint32_t)K8) * 8;
    const u32x2_t q = *(const u32x2_t *)(codes + i * 8);
    const float s = ROWS ? exponent_value(((const uint8_t *)scales)[row * lds + k / kFp8Block])
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
        __builtin_nontemporal_store(o, (u32x4_t *)((uint16_t *)dst + at));
    } else {
        __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, (f32x4_t *)((float *)dst + at));
        __builtin_nontemporal_store(f32x4_t{v[4], v[5], v[6], v[7]}, (f32x4_t *)((float *)dst + at + 4));
    }
}

// ---------------------------------------------------------------------------
// Products. Two ways to multiply codes:
//  - the fp8 matrix instructions, at twice the rate of bf16. They align the
//    products of 8 neighbouring k and cut what lies more than 13 bits below the
//    largest one's exponent (measured with one large and one small product at
//    every distance, the same in all of their shapes; across the groups of 8 sums keep 24 bits): 1.1e-5
//    of the norm of C for normally distributed operands, whatever K, and at most 2^-10 of sum |a b|. C in bf16
//    and H of many records go this way. bf16 C: 1.655e-3 from the 64-bit result with the cut and without (32768 x
//    2048 x 1408). H: 0.16 % of its codes come out a step away, where h lies that near the middle
//    between two codes; either is as far from h (2.65e-2 of H's norm as before), but they differ from what
//    sums of 24 bits give: an expert FFN of 4096 tokens on 64 experts is 1.99e-3 from the 64-bit
//    one, with 24 bits 1.68e-3. On decoded codes gate/up of that FFN takes 309 us instead of 187.
//  - codes decoded to bf16, which is exact, on the bf16 instructions, whose sums
//    keep 24 bits (2e-8): fp32 C, and few records a slot, where the time goes into
//    reading the weights and the decoding is free.
// Which of a block's 128 k values a lane supplies in which place is free, as
// long as it is the same for both operands: they have one scale.

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

// 32 codes times scale (a power of two) as four operands of 8 bf16; exact with scale 1.
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
// acc += the product of 128 k (16 weight rows x 16 records) times the row's scale, a power of two, and
// the block's. The codes are multiplied as they are, so that nothing leaves fp32 before the scales are there:
// of the two, one at or above 1 and one below are joined first, others follow each other, and each
// time what lies between is no further from 1 than the result or one of them.
struct Factors {
    float p, q;
};
__device__ __forceinline__ Factors factors(float row, float block)
{
    const bool join = (row >= 1.0f) != (fabsf(block) >= 1.0f);
    return {join ? 1.0f : row, join ? row * block : block};
}
__device__ __forceinline__ void step128(f32x4_t &acc, const i32x8_t &w, const bf16x8_t (&A)[4], Factors s)
{
    bf16x8_t W[4];
    decode32(w, 1.0f, W);
    f32x4_t part = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(W[i], A[i], part, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = fmaf(part[r] * s.p, s.q, acc[r]);
}

__device__ __forceinline__ float swiglu(float g, float u) { return g < kSiluTail ? silu_tail_mul(g, u) : silu_mul(g, u); }

// Few records a slot: 16 records x 16 NT weight rows a workgroup, its W waves taking
// steps of 128 k in turn, U of them requested at a time, their sums joined in LDS in
// the order of the waves. Bound by reading the weights, and for a record or
// two by the chain slot - record - row. GATE_UP: half of the rows are gate, half up of the
// same units; h goes to `hw` in fp32, and is quantised by the next launch: a
// workgroup that held whole blocks of 128 units would leave most compute units idle,
// and one alone reads 50 GB/s at most (one record of 2048 x 2048: 20 us).
// Weights pass through registers, each read once and by one wave: nothing would be shared in
// LDS. 16 rows of an instruction are the least the matrix units take, so that up to 16 records
// of a slot cost what one does. 64 records of 8 slices of 4096 x 14336: 94 us, 5.0 TB/s of
// weights; one token's 8 slices of 2048 x 1024: 6.2 us, 2.7 TB/s, five trips to memory in a row
// (offsets, row index, codes, and the join) with a launch.
enum { EPI_STORE = 0, EPI_GATE_UP = 1 };
template <int EPI, int NT, int W>
__global__ __launch_bounds__(64 * W, NT == 4 ? 2 : NT == 2 ? 3 : 4) void k_few(Fp8Args a, float *__restrict__ hw)
{
    constexpr int U = 4, G = EPI == EPI_GATE_UP ? 2 : 1, COLS = 16 * NT / G;
    __shared__ f32x4_t s_sum[W][NT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int ntn = (a.N + COLS - 1) / COLS, n0 = blockIdx.x % ntn * COLS;
    int row0 = 0, cnt = 0;
    const int slot = find_tile<16>(a, blockIdx.x / ntn, lane, &row0, &cnt);
    if (slot < 0) return;
    const int K = a.K, KB = (K + kFp8Block - 1) / kFp8Block;
    const int rec = row_of(a, row0 + min(lane & 15, cnt - 1));
    const uint8_t *ap = a.A + (int64_t)rec * K + (lane >> 4) * 16;
    const uint8_t *as = a.As + rec * fp8_scale_bytes(K);
    const uint8_t *bp[NT];
    const float *bs[G];   // the workgroup's columns lie within a block
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int n = min(n0 + 16 * (j / G) + (lane & 15), a.N - 1);
        bp[j] = a.B[j % G] + slot * a.B_stride + (int64_t)n * K + (lane >> 4) * 16;
    }
#pragma unroll
    for (int g = 0; g < G; ++g) bs[g] = a.Bs[g] + slot * a.Bs_stride + (int64_t)(n0 / kFp8Block) * KB;
    f32x4_t acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    auto batch = [&](auto u_t, int k0) __attribute__((always_inline)) {
        constexpr int n = decltype(u_t)::value;
        i32x8_t A[n], Bv[n][NT];
        int sa[n];
        float sb[n][G];
#pragma unroll
        for (int u = 0; u < n; ++u) {
            const int kb = k0 + u * W;
            const bool half = (kb + 1) * kFp8Block > K;
#pragma unroll
            for (int j = 0; j < NT; ++j) Bv[u][j] = codes32(bp[j] + (int64_t)kb * kFp8Block, half);
#pragma unroll
            for (int g = 0; g < G; ++g) sb[u][g] = bs[g][kb];
            A[u] = codes32(ap + (int64_t)kb * kFp8Block, half);
            sa[u] = as[kb];
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < n; ++u) {
            if ((k0 + u * W + 1) * kFp8Block > K)
#pragma unroll
                for (int i = 4; i < 8; ++i) A[u][i] = 0;
            bf16x8_t Av[4];
            decode32(A[u], 1.0f, Av);
            Factors s[G];
#pragma unroll
            for (int g = 0; g < G; ++g) s[g] = factors(exponent_value(sa[u]), sb[u][g]);
#pragma unroll
            for (int j = 0; j < NT; ++j) step128(acc[j], Bv[u][j], Av, s[j % G]);
        }
    };
    int k0 = wave;
    for (; k0 + (U - 1) * W < KB; k0 += W * U) batch(std::integral_constant<int, U>(), k0);
    for (; k0 < KB; k0 += W) batch(std::integral_constant<int, 1>(), k0);
    if constexpr (W > 1) {
#pragma unroll
        for (int j = 0; j < NT; ++j) s_sum[wave][j][lane] = acc[j];
        __syncthreads();
    }
    for (int q = wave; q < NT / G; q += W) {
        f32x4_t s[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if constexpr (W > 1) {
                s[g] = s_sum[0][q * G + g][lane];
#pragma unroll
                for (int w = 1; w < W; ++w) s[g] += s_sum[w][q * G + g][lane];
            } else {
#pragma unroll
                for (int c = 0; c < NT / G; ++c)   // a register's index has to be known
                    if (c == q) s[g] = acc[c * G + g];
            }
        }
        // register r: column 4 (lane / 16) + r of record lane % 16
        const int n = n0 + 16 * q + 4 * (lane >> 4), m = lane & 15;
        if (n >= a.N || m >= cnt) continue;
        if constexpr (EPI == EPI_GATE_UP) {
            f32x4_t h;
#pragma unroll
            for (int r = 0; r < 4; ++r) h[r] = swiglu(s[0][r], s[G - 1][r]);
            *(f32x4_t *)(hw + (int64_t)(row0 + m) * a.N + n) = h;
        } else {
            const int64_t at = (int64_t)(row0 + m) * a.ldc + n;
            if (a.c_bf16)
                *(u32x2_t *)((uint16_t *)a.C + at) = u32x2_t{bf16_pair(s[0][0], s[0][1]), bf16_pair(s[0][2], s[0][3])};
            else
                *(f32x4_t *)((float *)a.C + at) = s[0];
        }
    }
}

// ---------------------------------------------------------------------------
// Many records a slot: a persistent kernel. Tile 256 records x 256 weight rows,
// one stage = 128 k: 256 rows of 128 code bytes, a whole line, of each side, copied
// straight into LDS (16 bytes a lane), one stage in use and one on its way; 8 waves as
// 2 x 4. Wave row wm takes the 32-record blocks wm, wm + 2, ..., so that a tile with
// fewer records takes less time (2 or 4 blocks a wave). Rows are stored with their
// 16-byte chunk c at c ^ ((row >> 1) & 7), which spreads the 16 rows that a fragment read takes
// at a time over all banks. The scales come in panels of 2048 k: 16 bytes a record, 16 numbers for
// each of the tile's two blocks of 128 weight rows.
//
// The records' scales, powers of two, are operands of the matrix instruction. So
// are the powers of two of the weights' scales m 2^e; the m are
// brought in by holding the sums in units of the current one: before the first
// multiply of a block of k the sums are multiplied by m_last / m, and at the end by the last m. |m| >= 1,
// so that sums in units of it are no larger than the sums, and nothing overflows on the way. Where
// the weights' scales are powers of two there is nothing to multiply.
//
// Bound by how little of it overlaps. Multiplied from registers alone a stage of 128 k takes 1.1 us; it takes
// 1.7 to 1.9. Counted (gate/up and down of 4096 tokens on 64 experts, one slice of 8192 x 8192 x 8192): the matrix
// units are busy 39, 33 and 50 % of the time, LDS 22, 18 and 25 % (of which bank conflicts are a fifth),
// waves sit at a wait or barrier 38, 41 and 35 %; with a multiply of 64 cycles come about 18, 19 and 14 vector
// instructions of 4, 8 of them for the change of units: a SIMD issues these for as long as it multiplies, and only its
// two waves can do the one beside the other.
// 8192 x 8192 x 8192 in bf16: 533 us, 2.1 PFLOP/s, with scales that are powers of two 471, 2.3. Gate/up of
// 4096 tokens on 64 slices of 2 x 1024 x 2048 182 to 190 us, down 110, 32768 records of 66 slices of 2048 x 1408
// 139, in fp32, decoded, at half of the instruction rate, 226. Two stages of 128 k and not four of 64: half of the barriers, whole lines
// of memory. Without gain: lines of later stages requested into the L2 ahead, other wave
// priorities, copies left out where a tile has no rows (gate/up -2 %, down +3 %), tiles of more than
// 128 records before the others (gate/up -2 %, down +7 %: small tiles, bound by their copies, all
// at the same time).
//
// EPI: STORE: C, rounded to its type. With DEC (fp32 C) the codes are decoded to
// bf16 when they leave LDS. GATE_UP: the tile's weight rows are 128 of gate and
// the 128 of up; the operands change places, so that a lane holds 16 units of one
// record, H's blocks are the tile's 128 units, their maxima joined over the four
// waves through LDS.
constexpr int kXcd = 8;
constexpr int kStream = 2;   // buffer stores of C, which is not read here: non-temporal

// A weight scale as m 2^e, e in -126 .. 118, m of magnitude 1 up to 2, from 2^119 on up to 2^10; NaN and
// infinity as NaN. What is below 2^-126 in magnitude, which e cannot hold, counts as 0: its block's
// codes do, those of NaN aside.
constexpr int kMaxField = 118 + 127;
__device__ __forceinline__ float scale_m(float s)
{
    const uint32_t u = __float_as_uint(s);
    const int e = (int)((u >> 23) & 255u);
    return __uint_as_float(e == 0 || e == 255 ? (u & 0x80000000u) | 0x3f800000u
                                              : (u & 0x807fffffu) | (uint32_t)(127 + max(e - kMaxField, 0)) << 23);
}
__device__ __forceinline__ int scale_e(float s)
{
    const int e = (int)((__float_as_uint(s) >> 23) & 255u);
    return e == 255 ? 255 : min(e, kMaxField);
}
// Codes decoded to bf16 (DEC) carry their scales: a record's halved, the weights' 2^e doubled, so that
// neither side's largest code, 448, leaves bf16 (2^119 448 < 2^128), for row bytes up to 247. A row's byte 1 to 3
// takes small codes below bf16's smallest number, 2^-133.
__device__ __forceinline__ float decoded_row(int byte) { return exponent_value(byte == 255 ? 255 : max(byte - 1, 0)); }
__device__ __forceinline__ float decoded_weight(int e) { return exponent_value(e == 255 ? 255 : e + 1); }

__device__ __forceinline__ void opaque(f32x16_t &v) { asm volatile("" : "+v"(v)); }

template <int EPI, bool DEC>
__global__ __launch_bounds__(512) void k_ring(Fp8Args a)
{
    constexpr int BM = 256, NS = 2, WN = 4, NI = 2, MI = 4;
    constexpr int CODES = 256 * kFp8Block, STAGE = 2 * CODES;   // bytes: one side, both
    constexpr int APANEL = BM * 16, BPANEL = 2 * 64, PANEL = APANEL + BPANEL;
    __shared__ __attribute__((aligned(1024))) char lds[NS * STAGE + 2 * PANEL];
    __shared__ int32_t s_tpref[kMaxExp + 1], s_lo[kMaxExp], s_cnt[kMaxExp];
    __shared__ u32x4_t s_tiles[2][64];
    __shared__ int32_t s_rows[3][BM];   // the rows of A of three tiles' records, this one, the next and the one after it
    __shared__ u32x4_t s_top[EPI == EPI_GATE_UP ? BM : 1];
    char *const panels = lds + NS * STAGE;
    const uint32_t lds_at = lds_address(lds), panels_at = lds_at + NS * STAGE, rows_at = lds_address(s_rows);

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN, half = lane >> 5;
    const int K = a.K, N = a.N, P = a.P, KB = (K + kFp8Block - 1) / kFp8Block;
    constexpr int BN = EPI == EPI_GATE_UP ? 128 : 256;
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
        int slot, row0, rows, n0;   // the same in every lane
    };
    // Tiles 64 b .. + 63 of this workgroup, a lane each, to LDS. Groups of 8 row tiles, columns
    // in turn within: what runs at the same time shares both sides' rows.
    const int tiles = (cnt_x - li + nwg - 1) / nwg;
    auto list = [&](int b) __attribute__((always_inline)) {
        const int L = start_x + li + min(64 * b + lane, tiles - 1) * nwg;
        int lo = 0, hi = P - 1;   // last slot whose first tile is <= L (skips empty slots)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_tpref[mid] <= L) lo = mid; else hi = mid - 1;
        }
        const int cnt = s_cnt[lo], mt = (cnt + BM - 1) / BM, group = (L - s_tpref[lo]) / (8 * ntn);
        const int local = (L - s_tpref[lo]) % (8 * ntn), high = min(8, mt - 8 * group), ml = 8 * group + local % high;
        s_tiles[b & 1][lane] = u32x4_t{(uint32_t)lo, (uint32_t)(s_lo[lo] + ml * BM), (uint32_t)min(BM, cnt - ml * BM),
                                       (uint32_t)(local / high * BN)};
    };
    auto tile = [&](int i) __attribute__((always_inline)) {   // past the last one: that one
        const u32x4_t t = s_tiles[min(i, tiles - 1) >> 6 & 1][min(i, tiles - 1) & 63];
        return Tile{__builtin_amdgcn_readfirstlane((int)t[0]), __builtin_amdgcn_readfirstlane((int)t[1]),
                    __builtin_amdgcn_readfirstlane((int)t[2]), __builtin_amdgcn_readfirstlane((int)t[3])};
    };
    if (wave == 0) list(0);
    __syncthreads();

    // Copies of this wave: rows 32 wave + 8 j .. +7 of both sides (lane: row + l/8,
    // chunk position l % 8); of a panel, waves 0-3 the records 64 wave .. +63, wave 4
    // the weights' scales.
    const char *bbase;   // the same in every lane
    uint32_t aoff[4], boff[4];   // aoff in 16 bytes
    // A tile's rows to LDS. No register waits for them: a load into one
    // would be waited for with everything requested after it.
    auto fetch_rows = [&](const Tile &t, int buf) __attribute__((always_inline)) {
        if (a.row_index && wave < BM / 64)
            copy_to_lds<4>(a.row_index + t.row0 + min(wave * 64 + lane, t.rows - 1), rows_at + (buf * BM + wave * 64) * 4);
    };
    auto row_in = [&](const Tile &t, int buf, int i) __attribute__((always_inline)) {
        const int r = min(i, t.rows - 1);
        return a.row_index ? min(max(s_rows[buf][r], 0), a.A_rows - 1) : t.row0 + r;
    };
    auto set_sources = [&](const Tile &t, int buf) __attribute__((always_inline)) {
        const int side = EPI == EPI_GATE_UP ? wave >> 2 : 0;
        const int64_t first = EPI == EPI_GATE_UP ? t.n0 + (wave & 3) * 32 : t.n0 + wave * 32;
        bbase = (const char *)a.B[side] + t.slot * a.B_stride;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = j * 8 + (lane >> 3), sw = ((lane & 7) ^ ((r >> 1) & 7)) * 16;
            aoff[j] = (uint32_t)row_in(t, buf, wave * 32 + r) * (uint32_t)(K / 16) + sw / 16;
            boff[j] = (uint32_t)(min((int)first + r, N - 1) - t.n0) * (uint32_t)K + sw;
        }
        bbase += (int64_t)t.n0 * K;
    };
    // Where stages and panels of the current tile are: they go on from the last one's.
    int par = 0, ppar = 0;
    auto at_stage = [&](int kb) __attribute__((always_inline)) { return ((kb + par) & 1) * STAGE; };
    auto at_panel = [&](int pn) __attribute__((always_inline)) { return ((pn + ppar) & 1) * PANEL; };
    auto issue_panel = [&](const Tile &t, int buf, int pn, int place) __attribute__((always_inline)) {
        const uint32_t at = panels_at + place;
        if (wave < 4) {
            copy_to_lds<16>(a.As + row_in(t, buf, wave * 64 + lane) * fp8_scale_bytes(K) + pn * 16, at + wave * 1024);
        } else if (wave == 4 && lane < 32) {
            const int b = lane >> 4, nbs = (N + kFp8Block - 1) / kFp8Block;
            const int nb = min(t.n0 / kFp8Block + (EPI == EPI_GATE_UP ? 0 : b), nbs - 1);
            copy_to_lds<4>(a.Bs[EPI == EPI_GATE_UP ? b : 0] + t.slot * a.Bs_stride + (int64_t)nb * KB + min(pn * 16 + (lane & 15), KB - 1),
                           at + APANEL);
        }
    };
    const bool odd = (K & 64) != 0;   // the last stage has 64 k: chunks 4-7 are not copied, and not read
    const bool first64 = (((lane & 7) ^ (lane >> 4)) & 4) == 0;   // this lane's chunk is below 4, of rows 8 j .. with even j; odd ones: is not
    auto issue = [&](int kb, int side, int place) __attribute__((always_inline)) {
        const uint32_t st = lds_at + place + side * CODES + wave * 4096;
        const char *base = (side == 0 ? (const char *)a.A : bbase) + kb * kFp8Block;
        auto copy = [&](int j) __attribute__((always_inline)) {
            if (side == 0)
                copy_to_lds<16>(base + (uint64_t)aoff[j] * 16, st + j * 1024);
            else
                copy_to_lds(base, boff[j], st + j * 1024);
        };
        if (!(odd && kb == KB - 1)) {
#pragma unroll
            for (int j = 0; j < 4; ++j) copy(j);
        } else if (first64) {
            copy(0);
            copy(2);
        } else {
            copy(1);
            copy(3);
        }
    };

    const int sw = (lane >> 1) & 7, frow = (lane & 31) * kFp8Block;
    auto cblock = [&](int j) __attribute__((always_inline)) { return EPI == EPI_GATE_UP ? wn + 4 * j : 2 * wn + j; };
    f32x16_t acc[MI][NI];
    i32x8_t af[2], bf[2][NI];   // records' blocks in turn, weights of this half stage and the next
    int sa[MI];                 // scale bytes of this lane's records
    // of the weights' scales of a panel, lane l: block l % 16 of k, (l / 16) % 2 of the tile's
    // two blocks of rows: the bits of 2^e, the last m over this one
    int se_panel;
    float ratio_panel;
    int se[NI];
    float ratio[NI];
    auto frag = [&](const char *p, int h) __attribute__((always_inline)) {
        const u32x4_t lo = *(const u32x4_t *)(p + frow + ((4 * h + 2 * half) ^ sw) * 16);
        const u32x4_t hi = *(const u32x4_t *)(p + frow + ((4 * h + 2 * half + 1) ^ sw) * 16);
        return i32x8_t{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
    };
    auto a_frag = [&](int kb, int h, int i) __attribute__((always_inline)) { return frag(lds + at_stage(kb) + (2 * i + wm) * 4096, h); };
    auto b_frag = [&](int kb, int h, int j) __attribute__((always_inline)) { return frag(lds + at_stage(kb) + CODES + cblock(j) * 4096, h); };
    // scale of block kb of k in the tile's row block r, and of the one before
    auto weight_scale = [&](int kb, int r) __attribute__((always_inline)) { return *(const float *)(panels + at_panel(kb / 16) + APANEL + r * 64 + (kb & 15) * 4); };
    auto row_block = [&](int j) __attribute__((always_inline)) { return EPI == EPI_GATE_UP ? j : wn >> 1; };
    auto read_panel = [&](int pn) __attribute__((always_inline)) {
        const int kb = pn * 16 + (lane & 15), r = EPI == EPI_GATE_UP ? (lane >> 4) & 1 : wn >> 1;
        const float s = weight_scale(min(kb, KB - 1), r), last = weight_scale(max(min(kb, KB) - 1, 0), r);
        ratio_panel = scale_m(last) / scale_m(s);   // behind the last block: 1
        se_panel = scale_e(s);
    };
    // scale byte of this lane's record of block i (behind the last block of k: anything)
    auto row_scale = [&](int kb, int i) __attribute__((always_inline)) {
        return *(const uint8_t *)(panels + at_panel(kb / 16) + ((2 * i + wm) * 32 + (lane & 31)) * 16 + (kb & 15));
    };
    bool scaled = false;   // whether one of them is not 1
    auto take_ratios = [&](int kb) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NI; ++j)
            ratio[j] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ratio_panel), (EPI == EPI_GATE_UP ? j * 16 : 0) + (kb & 15)));
        scaled = ratio[0] != 1.0f || ratio[1] != 1.0f;
    };
    auto take_powers = [&](int kb) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NI; ++j) se[j] = __builtin_amdgcn_readlane(se_panel, (EPI == EPI_GATE_UP ? j * 16 : 0) + (kb & 15));
    };
    auto multiply = [&](int i, int j, int set, int cur) __attribute__((always_inline)) {
        acc[i][j] = EPI == EPI_GATE_UP
                        ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(bf[set][j], af[cur], acc[i][j], 0, 0, 0, se[j], 0, sa[i])
                        : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(af[cur], bf[set][j], acc[i][j], 0, 0, 0, sa[i], 0, se[j]);
    };
    auto rescale = [&](int i, int j) __attribute__((always_inline)) {
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] *= ratio[j];
    };
    // The stores of a tile are requested behind the first two stages' copies of the
    // next one, and are not waited for with them: loads and stores return in order.
    int stores = 0;   // of this wave, a multiple of 16
    auto wait_behind = [&](int n) __attribute__((always_inline)) {
        if (n >= 64) wait_vmcnt<63>();
        else if (n == 48) wait_vmcnt<48>();
        else if (n == 32) wait_vmcnt<32>();
        else if (n == 16) wait_vmcnt<16>();
        else wait_vmcnt<0>();
    };
    // Scales that count as 0: a bit for each of a panel's 16 blocks of k and the tile's two row
    // blocks. Such a block's codes are blanked in LDS, NaN left, before any wave reads them.
    uint32_t zeros = 0;
    auto read_zeros = [&](int pn) __attribute__((always_inline)) {
        const float s = weight_scale(min(pn * 16 + (lane & 15), KB - 1), (lane >> 4) & 1);
        zeros = (uint32_t)__ballot(fabsf(s) < 0x1p-126f);
    };
    auto blank = [&](int kb) __attribute__((always_inline)) {
        const uint32_t here = zeros >> (kb & 15) & 0x10001u;
        if (__builtin_expect(here == 0, 1)) return;
        if (here >> (16 * (tid >> 8)) & 1)
            for (int q = 0; q < 4; ++q) {
                u32x4_t *p = (u32x4_t *)(lds + at_stage(kb) + CODES + tid * 64 + q * 16);
                u32x4_t v = *p;
                for (int c = 0; c < 4; ++c) {
                    const uint32_t nan = ((v[c] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                    v[c] = nan - (nan >> 7);
                }
                *p = v;
            }
        lds_barrier();
    };
    // The stage behind kb, the next tile's first one behind the last, is made visible: this
    // wave's reads of stage kb are done, its copies have landed, and behind the barrier so
    // have all waves'. Then stage kb's place is free, and `follow` requests the stage after that one
    // into it, of this tile or the next.
    Tile cur;
    int o = 0;   // which of this workgroup's tiles it is
    int buf = 0, buf1 = 1, buf2 = 2;   // of their rows
    bool has_next, cross;
    auto next_stage = [&](int kb) __attribute__((always_inline)) {
        if (kb + 1 < KB || cross) {
            if (kb == 0) wait_behind(stores); else wait_vmcnt<0>();
            __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));   // lgkmcnt(0)
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");   // for the compiler: reads stay behind
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        }
        if (kb + 1 < KB) {
            if ((kb & 15) == 15) read_zeros(kb / 16 + 1);
            blank(kb + 1);
        }
    };
    auto follow = [&](int kb, int side) __attribute__((always_inline)) {
        const int place = at_stage(kb);
        if (kb + 2 < KB) {
            issue(kb + 2, side, place);
            if (side == 1 && (kb & 15) == 6 && kb + 10 < KB) issue_panel(cur, buf, kb / 16 + 1, at_panel(kb / 16 + 1));
        } else if (cross) {
            if (side == 0 && kb + 2 == KB) {
                const Tile nxt = tile(o + 1);
                set_sources(nxt, buf1);
                fetch_rows(tile(o + 2), buf2);
                issue_panel(nxt, buf1, 0, at_panel((KB + 15) / 16));
            }
            issue(kb + 2 - KB, side, place);
        }
    };
    // Half h of stage kb. While block i is multiplied, the next block's codes are read,
    // and its sums brought into the current units (first half; block 0's at the end of
    // the half before): what the scheduler is held from moving runs in the
    // shadow of the matrix instructions. The next stage begins before the last block
    // is multiplied, whose codes are in registers by then. The sums are opaque
    // where there are branches: the compiler would move a stage's multiplies behind
    // them, with all of its codes in registers until then.
    int mine = 0;   // blocks of records of this wave, 0, 2 or 4 of them multiplied
    bf16x8_t Bv[DEC ? NI : 1][4];   // the weights of a half stage, decoded
    auto step = [&](auto half_t, auto block_t, int kb, bool last) __attribute__((always_inline)) {
        constexpr int h = decltype(half_t)::value, i = decltype(block_t)::value, cur = i & 1;
        const bool end = h == 1 && last;
        if (end) next_stage(kb);
        if (!last) {
            af[cur ^ 1] = a_frag(kb, h, i + 1);
        } else {   // past the last stage: a resident one, not used
            af[cur ^ 1] = a_frag(kb + h, h ^ 1, 0);
#pragma unroll
            for (int j = 0; j < NI; ++j) bf[h ^ 1][j] = b_frag(kb + h, h ^ 1, j);
        }
        if (h == 1 && i == 0 && (kb & 15) == 15) read_panel(kb / 16 + 1);
        if (end) take_ratios(kb + 1);
        if constexpr (h == 1 && i > 0) sa[i - 1] = row_scale(kb + 1, i - 1);
        __builtin_amdgcn_sched_barrier(0);
        const int next = last ? 0 : i + 1;
        const bool scales = h == 0 ? !last : last;
        if constexpr (DEC) {
            bf16x8_t Av[4];
            decode32(af[cur], decoded_row(sa[i]), Av);
#pragma unroll
            for (int j = 0; j < NI; ++j) {
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(Av[c], Bv[j][c], acc[i][j], 0, 0, 0);
                opaque(acc[i][j]);
                __builtin_amdgcn_sched_barrier(0);
                if (end) follow(kb, j);
                if (scales && scaled) {
                    rescale(next, j);
                    opaque(acc[next][j]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                multiply(i, j, h, cur);
                opaque(acc[i][j]);
                __builtin_amdgcn_sched_barrier(0);
                if (end) follow(kb, j);
                if (scales && scaled) {
                    rescale(next, j);
                    opaque(acc[next][j]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    auto half_stage = [&](auto mi, auto half_t, int kb) __attribute__((always_inline)) {
        constexpr int n = decltype(mi)::value;
        if constexpr (DEC)
#pragma unroll
            for (int j = 0; j < NI; ++j) decode32(bf[decltype(half_t)::value][j], decoded_weight(se[j]), Bv[j]);
        step(half_t, std::integral_constant<int, 0>(), kb, false);
        step(half_t, std::integral_constant<int, 1>(), kb, n == 2);
        if constexpr (n == 4) {
            step(half_t, std::integral_constant<int, 2>(), kb, false);
            step(half_t, std::integral_constant<int, 3>(), kb, true);
        }
    };

    // The first tile's first requests, and those of a tile behind one of a single stage.
    auto begin = [&]() __attribute__((always_inline)) {
        set_sources(cur, buf);
        fetch_rows(tile(o + 1), buf1);
        issue_panel(cur, buf, 0, at_panel(0));
        issue(0, 0, at_stage(0));
        issue(0, 1, at_stage(0));
        if (KB > 1) {
            issue(1, 0, at_stage(1));
            issue(1, 1, at_stage(1));
        }
    };

    auto tile_loop = [&](auto mi) __attribute__((always_inline)) {
        constexpr int n = decltype(mi)::value;
        if constexpr (n > 0) {
#pragma unroll
            for (int i = 0; i < n; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
            read_panel(0);
            take_powers(0);
            take_ratios(0);   // 1
#pragma unroll
            for (int i = 0; i < n; ++i) sa[i] = row_scale(0, i);
            af[0] = a_frag(0, 0, 0);
#pragma unroll
            for (int j = 0; j < NI; ++j) bf[0][j] = b_frag(0, 0, j);
        }
        const int whole = K / kFp8Block;   // stages, and half a one
        for (int kb = 0; kb < whole; ++kb) {
            if constexpr (n > 0) {
                half_stage(mi, std::integral_constant<int, 0>(), kb);
                half_stage(mi, std::integral_constant<int, 1>(), kb);
                sa[n - 1] = row_scale(kb + 1, n - 1);
                take_powers(kb + 1);
            } else {
                next_stage(kb);
                follow(kb, 0);
                follow(kb, 1);
            }
        }
        if (odd) {
            if constexpr (n > 0) half_stage(mi, std::integral_constant<int, 0>(), whole);
            if (cross) {
                next_stage(whole);
                follow(whole, 0);
                follow(whole, 1);
            }
        }
    };

    cur = tile(0);
    fetch_rows(cur, buf);
    wait_vmcnt<0>();
    __syncthreads();
    begin();
    for (;;) {
        has_next = o + 1 < tiles;
        cross = has_next && KB > 1;
        if (wave == 0 && (o & 63) == 32) list((o >> 6) + 1);   // read half a list later
        mine = __builtin_amdgcn_readfirstlane(((cur.rows + 31) / 32 - wm + 1) >> 1);
        if (o == 0 || KB == 1) {   // else the first stage is visible already
            wait_behind(stores);
            lds_barrier();
        }
        read_zeros(0);
        blank(0);
        if (mine > 2) tile_loop(std::integral_constant<int, 4>());
        else if (mine > 0) tile_loop(std::integral_constant<int, 2>());
        else tile_loop(std::integral_constant<int, 0>());
        const Tile done = cur;
        float sm[NI];   // the units that the sums are in
#pragma unroll
        for (int j = 0; j < NI; ++j) sm[j] = scale_m(weight_scale(KB - 1, row_block(j)));
        stores = 0;
        if constexpr (EPI == EPI_GATE_UP) {
            // register r of lane l: unit 32 wn + 8 (r / 4) + 4 (l / 32) + r % 4 of record l % 32 of the block
            const bool in = done.n0 + wn * 32 < N;
            uint32_t *tops = (uint32_t *)s_top;
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                if (i >= mine) continue;
                f32x16_t &g = acc[i][0], &u = acc[i][1];
                uint32_t least = 0, t = 0;   // of negative numbers the least has the largest bits
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    g[r] *= sm[0];
                    u[r] *= sm[1];
                    least = max(least, __float_as_uint(g[r]));
                }
                float h[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) h[r] = silu_mul(g[r], u[r]);
                if (__any(least > __builtin_bit_cast(uint32_t, kSiluTail))) {
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (g[r] < kSiluTail) h[r] = silu_tail_mul(g[r], u[r]);
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    g[r] = in ? h[r] : 0.0f;
                    t = max(t, __float_as_uint(g[r]) & 0x7fffffffu);
                }
                t = max(t, (uint32_t)__shfl_xor((int)t, 32, 64));
                if (half == 0) tops[((2 * i + wm) * 32 + lane) * 4 + wn] = t;
            }
            lds_barrier();
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                if (i >= mine) continue;
                const int m = (2 * i + wm) * 32 + (lane & 31);
                const u32x4_t t = s_top[m];
                const uint32_t byte = block_byte(max(max(t[0], t[1]), max(t[2], t[3])));
                const float unit = block_unit(byte);
                uint32_t q[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const f32x16_t &h = acc[i][0];
                    int w = __builtin_amdgcn_cvt_pk_fp8_f32(h[4 * c] * unit, h[4 * c + 1] * unit, 0, false);
                    w = __builtin_amdgcn_cvt_pk_fp8_f32(h[4 * c + 2] * unit, h[4 * c + 3] * unit, w, true);
                    q[c] = byte == 255 ? 0u : (uint32_t)w;
                }
                // units 0-15 to the lower half, 16-31 to the upper
                const uint32_t g0 = (uint32_t)__shfl_xor((int)(half ? q[0] : q[2]), 32, 64);
                const uint32_t g1 = (uint32_t)__shfl_xor((int)(half ? q[1] : q[3]), 32, 64);
                const u32x4_t o = half ? u32x4_t{g0, q[2], g1, q[3]} : u32x4_t{q[0], g0, q[1], g1};
                if (in && m < done.rows) {
                    *(u32x4_t *)((uint8_t *)a.C + (int64_t)(done.row0 + m) * N + done.n0 + wn * 32 + half * 16) = o;
                    if (wn == 0 && half == 0) a.Hs[(int64_t)(done.row0 + m) * fp8_scale_bytes(N) + done.n0 / kFp8Block] = (uint8_t)byte;
                }
            }
        } else if (mine > 0 && done.n0 + wn * 64 < N) {
            if (cross) stores = mine * (DEC ? 32 : 16);
            // Register r of lane l holds record 8 (r / 4) + 4 (l / 32) + r % 4 and column
            // l % 32 of its block. bf16: adjacent lanes swap a value of records R, R + 1,
            // so that each stores two columns of one. The tile's rows of C are a
            // buffer: stores to rows past its last one are dropped by its bounds
            // check, so no store has a branch. A wave's 64 columns are all in N or
            // all past it.
            constexpr int esz = DEC ? 4 : 2;
            char *base = (char *)a.C + ((int64_t)done.row0 * a.ldc + done.n0 + wn * 64) * esz;
            // opaque, or the rows' offsets are computed before the tile loop and held through it
            uint32_t ld = (uint32_t)a.ldc * esz;
            asm volatile("" : "+s"(ld));
            const __amdgpu_buffer_rsrc_t out = __builtin_amdgcn_make_buffer_rsrc(base, 0, (int)(done.rows * ld), 0x00027000);
            const uint32_t row = wm * 32 + 4 * half;
            if constexpr (!DEC) {
                const bool even = (lane & 1) == 0;
                const uint32_t at = (row + (even ? 0 : 1)) * ld + (lane & 30) * 2;
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    if (i >= mine) continue;
#pragma unroll
                    for (int r = 0; r < 16; r += 2) {
                        const uint32_t o = at + (uint32_t)(i * 64 + 8 * (r / 4) + (r & 3)) * ld;
#pragma unroll
                        for (int j = 0; j < NI; ++j) {
                            const float s0 = acc[i][j][r] * sm[j], s1 = acc[i][j][r + 1] * sm[j];
                            const float y = __uint_as_float(dpp<0xB1>(__float_as_uint(even ? s1 : s0)));
                            __builtin_amdgcn_raw_buffer_store_b32(even ? bf16_pair(s0, y) : bf16_pair(y, s1), out,
                                                                  (int)(o + j * 64), 0, kStream);
                        }
                    }
                }
            } else {
                const uint32_t at = row * ld + (lane & 31) * 4;
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    if (i >= mine) continue;
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const uint32_t o = at + (uint32_t)(i * 64 + 8 * (r / 4) + (r & 3)) * ld;
#pragma unroll
                        for (int j = 0; j < NI; ++j)
                            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[i][j][r] * sm[j]), out, (int)(o + j * 128), 0,
                                                                  kStream);
                    }
                }
            }
        }
        if (!has_next) break;
        cur = tile(++o);
        const int b = buf;
        buf = buf1;
        buf1 = buf2;
        buf2 = b;
        par ^= KB & 1;
        ppar ^= (KB + 15) / 16 & 1;
        if (KB == 1) {
            lds_barrier();   // nothing reads the stages any more
            begin();
        }
    }
}

}  // namespace

// Rows [*first, *last), or with null pointers all of them.
static void quantize_rows(const void *src, bool bf16, int64_t rows, int K, int64_t ld, uint8_t *codes, uint8_t *scales,
                          const int32_t *first, const int32_t *last, hipStream_t st)
{
    const int KB = (int)fp8_blocks(K);
    const int64_t blocks = rows * KB;
    const auto kernel = bf16 ? k_quantize_rows<true> : k_quantize_rows<false>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((blocks + 15) / 16)), dim3(256), 0, st, src, blocks, KB, K, ld, fp8_scale_bytes(K),
                       codes, scales, first, last);
}

hipError_t launch_quantize_fp8(const void *src, bool bf16, int64_t rows, int K, int64_t ld, int block_rows,
                               uint8_t *codes, void *scales, hipStream_t st)
{
    if (rows == 0) return hipSuccess;
    const int KB = (int)fp8_blocks(K);
    if (block_rows == 1) {
        quantize_rows(src, bf16, rows, K, ld, codes, (uint8_t *)scales, nullptr, nullptr, st);
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

// Whether the persistent kernel is ahead, by what the two take (us; fitted to calls at sizes from 8 records
// of 2048 x 2048 to 16384 of 64 slices): the few-records kernel 4 and 0.16 for each million of weights that a tile of 16
// records meets, the persistent one a round of tiles of 5 and a time for each
// stage, by whether a slot has more than 128 records (1.7, fp32 C 2.9) or not (0.85, 1.4). On
// weights that no cache holds (few, persistent): 64 slices of 2048 x 1024, 8 records each 31 and 36 us, 16 42 and
// 37, 64 97 and 42; one of 8192 x 2048, 64 records 15 and 28, 128 26 and 30 (the rule takes the
// second there), 256 45 and 38; one of 1024 x 4096, where 4 tiles of the persistent kernel are all there are, 1024
// records 46 and 61. Only the device knows the slots' records, the rule goes by the mean.
static bool ring_pays(const Fp8Args &a, int sides, bool f32)
{
    const int64_t slots = std::min(a.P, a.M), rows = a.M / slots, cols = sides == 2 ? 128 : 256;
    const double few = 4.0 + 0.16e-6 * ((double)a.M / 16 + slots / 2.0) * a.N * sides * a.K;
    const int64_t tiles = slots * ((rows + 255) / 256) * ((a.N + cols - 1) / cols);
    const double ring = (tiles + 255) / 256 * (5.0 + (double)fp8_blocks(a.K) * (rows > 128 ? (f32 ? 2.9 : 1.7) : (f32 ? 1.4 : 0.85)));
    return ring < few || row_tiles(a, 16) * (a.N / 8 + 1) >= 1 << 22;   // a launch has fewer than 2^32 threads
}

template <int EPI, bool DEC>
static hipError_t launch_ring(const Fp8Args &a, hipStream_t st)
{
    const int64_t cols = EPI == EPI_GATE_UP ? 128 : 256;
    const unsigned grid = (unsigned)std::min<int64_t>(row_tiles(a, 256) * ((a.N + cols - 1) / cols), 256);   // a workgroup a CU
    hipLaunchKernelGGL((k_ring<EPI, DEC>), dim3(grid), dim3(512), 0, st, a);
    return hipGetLastError();
}

// Weight rows a workgroup, 16 nt: 64 where that leaves 256 workgroups, else 32, for one product only from 192 of
// them on, else 16. Waves: 4; 1 where there is one step of K; 8 from 16 steps on where workgroups are fewer than 512.
// Measured in a graph of calls on 5 to 24 sets of weights in turn, which no cache holds together (us, rows x waves,
// the rule's first): 64 records of 8 slices of 4096 x 14336 64 x 4 93.6, 64 x 8 95.1, 32 x 4 98.5, 16 x 4 108; one record
// of 7168 x 2048 32 x 8 5.9, 32 x 4 6.8, 16 x 8 6.1, 64 x 8 7.5, of 4096 x 4096 16 x 8 7.3, 16 x 4 8.6, 32 x 8 9.2, of 2048 x
// 7168 16 x 8 8.9, 16 x 4 10.3; 64 slices of 2048 x 1024, 8 records 64 x 4 6.2, 64 x 1 8.5, 64 x 8 6.3, 128 64 x 4 27.1, 64 x
// 2 29.7, 64 x 8 32.7; 16 of 2048 x 512 64 x 4 6.2, 64 x 1 7.5. Between 32 and 64 rows there is no clear border: 32 x
// 4 takes 27.2 of the 128 records, 155 where gate/up of 32 records of 8 slices of 14336 x 4096 takes 169 with 64 x 4.
template <int EPI>
static hipError_t launch_few(const Fp8Args &a, float *hw, hipStream_t st)
{
    constexpr int G = EPI == EPI_GATE_UP ? 2 : 1;
    const int64_t tiles = row_tiles(a, 16), KB = fp8_blocks(a.K);
    auto groups = [&](int nt) { return tiles * ((a.N + 16 * nt / G - 1) / (16 * nt / G)); };
    const int nt = groups(4) >= 256 ? 4 : groups(2) >= 192 || G == 2 ? 2 : 1;
    const int w = KB == 1 ? 1 : KB < 16 || groups(nt) >= 512 ? 4 : 8;
    auto go = [&](auto nt_t, auto w_t) {
        constexpr int NT = decltype(nt_t)::value, W = decltype(w_t)::value;
        if constexpr (NT >= G)
            hipLaunchKernelGGL((k_few<EPI, NT, W>), dim3((unsigned)groups(NT)), dim3(64 * W), 0, st, a, hw);
    };
    auto with = [&](auto nt_t) {
        if (w == 1) go(nt_t, std::integral_constant<int, 1>());
        else if (w == 4) go(nt_t, std::integral_constant<int, 4>());
        else go(nt_t, std::integral_constant<int, 8>());
    };
    if (nt == 1) with(std::integral_constant<int, 1>());
    else if (nt == 2) with(std::integral_constant<int, 2>());
    else with(std::integral_constant<int, 4>());
    return hipGetLastError();
}

hipError_t launch_matmul_fp8(const Fp8Args &a, hipStream_t st)
{
    if (a.M == 0) return hipSuccess;
    if (ring_pays(a, 1, !a.c_bf16)) return a.c_bf16 ? launch_ring<EPI_STORE, false>(a, st) : launch_ring<EPI_STORE, true>(a, st);
    return launch_few<EPI_STORE>(a, nullptr, st);
}

size_t gate_up_fp8_workspace(const Fp8Args &a) { return a.M == 0 || ring_pays(a, 2, false) ? 0 : (size_t)a.M * a.N * 4; }

hipError_t launch_gate_up_fp8(const Fp8Args &a, void *ws, hipStream_t st)
{
    if (a.M == 0) return hipSuccess;
    if (ring_pays(a, 2, false)) return launch_ring<EPI_GATE_UP, false>(a, st);
    const hipError_t e = launch_few<EPI_GATE_UP>(a, (float *)ws, st);
    if (e != hipSuccess) return e;
    quantize_rows(ws, false, a.M, a.N, a.N, (uint8_t *)a.C, a.Hs, a.slot_offset, a.slot_offset ? a.slot_offset + a.P : nullptr, st);
    return hipGetLastError();
}

}  // namespace moe
