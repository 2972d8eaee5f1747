// One mixture-of-experts layer for a few tokens (T <= 64): the answering step
// of the layer that expert_gemm.hip runs over a whole prompt.
//
//   H_i = SiLU(W_g x_t) * (W_u x_t),  o_i = alpha_i W_d H_i  for route i = (t, j),
//   Y_t += sum_j o_i in ascending j.
//
// With one to a few rows an expert, the layer's time is that of reading the
// weights of the experts hit, once; every product is a matrix times at most 64
// columns. A workgroup takes 64 rows of one slot's weight slice over all of K
// and all of the slot's routes, so that a weight is read by one workgroup only.
// Its waves cut K among themselves (each its own stretch of the slice, whose
// 64 rows of a K piece are contiguous in the tiled layout) and add their sums
// in a fixed order through LDS.
//
// The weights are the first matrix operand (16 rows of the slice), the tokens
// the second (16 of them), v_mfma_f32_16x16x32_bf16: lane l holds row l % 16
// and 8 values of k. Any assignment of k values to lanes and instructions is
// a valid dot product so long as both operands follow it, so a lane takes 16
// consecutive bytes of its weight row whatever the format (8 bf16, 16 fp8, 32
// MXFP4 or 4 fp32 values: one 16-byte load), and the matching run of the
// token's row.
//
// H is kept to full fp32 between the projections: it is written as three bf16
// terms h = h1 + h2 + h3 of 8 bits each, cut (not rounded) from fp32, which
// is exact, and the down projection multiplies each weight operand by all
// three. Three instructions instead of one cost nothing beside the weights'
// load. fp32 layers keep H as fp32 and use the fp32 matrix instruction.
#include <algorithm>

#include "decode.h"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

enum { W_F32 = 0, W_BF16 = 1, W_FP8 = 2, W_FP4 = 3 };

// One workgroup: the routes sorted by slot. Thread s counts slot s's routes,
// then places them; R <= 1024.
__global__ __launch_bounds__(kMaxExp) void k_dec_lists(const int32_t *__restrict__ idx, int R, int P, PhiArg phi,
                                                       DecLists l)
{
    __shared__ int32_t key[kDecMaxRoutes];
    __shared__ int32_t wsum[2][kMaxExp / 64];
    const int s = threadIdx.x, lane = s & 63, wave = s >> 6;
    for (int i = s; i < R; i += kMaxExp) key[i] = phi.v[idx[i]];
    __syncthreads();
    int cnt = 0;
    if (s < P)
        for (int i = 0; i < R; ++i) cnt += key[i] == s;
    // exclusive prefixes over slots of the route counts and of the slots in use
    int off = cnt, pos = cnt > 0;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(off, o, 64), v = __shfl_up(pos, o, 64);
        if (lane >= o) {
            off += u;
            pos += v;
        }
    }
    if (lane == 63) {
        wsum[0][wave] = off;
        wsum[1][wave] = pos;
    }
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        off += wsum[0][w];
        pos += wsum[1][w];
    }
    if (s == kMaxExp - 1) *l.n_act = pos;
    off -= cnt;
    if (cnt > 0) {
        l.slot[pos - 1] = s;
        l.off[pos - 1] = off;
        l.cnt[pos - 1] = cnt;
        for (int i = 0; i < R; ++i)
            if (key[i] == s) l.rec[off++] = i;
    }
}

// E8M0 scale byte -> fp32 2^(s-127); 255 is NaN
__device__ __forceinline__ float e8m0(uint32_t b)
{
    return __uint_as_float(b == 0 ? 0x00400000u : (b == 255 ? 0x7fc00000u : b << 23));
}

// Values of the 16 bytes of a weight row that one lane holds, as matrix
// operands of 8: fp8 codes 8j .. 8j+7, or MXFP4 codes with their block's scale.
__device__ __forceinline__ bf16x8_t fp8_operand(u32x4_t w, int j)
{
    bf16x8_t r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w[2 * j + h], 1.0f, false);
        const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w[2 * j + h], 1.0f, true);
        r[4 * h] = a[0], r[4 * h + 1] = a[1], r[4 * h + 2] = b[0], r[4 * h + 3] = b[1];
    }
    return r;
}
__device__ __forceinline__ bf16x8_t fp4_operand(uint32_t w, float scale)
{
    const u32x4_t u = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
                       __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
                       __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
                       __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3))};
    return __builtin_bit_cast(bf16x8_t, u);
}

constexpr int kDecRows = 64;    // rows of the slice per workgroup
constexpr int kDecWaves = 8;

// WF: weight format. MT: 16-row groups of routes a slot can have (T <= 16 MT).
template <int WF, int MT, bool GATEUP>
__global__ __launch_bounds__(kDecWaves * 64) void k_dec_proj(DecArgs a)
{
    constexpr int NT = kDecRows / 16;                                  // weight row groups
    constexpr int LK = WF == W_F32 ? 4 : WF == W_BF16 ? 8 : WF == W_FP8 ? 16 : 32;   // k values per lane and step
    constexpr int KS = 4 * LK;                                         // k values per step
    constexpr int NI = LK > 8 ? LK / 8 : 1;                            // bf16 operands of 8 per lane and step
    constexpr int PL = !GATEUP && WF != W_F32 ? 3 : 1;                 // terms of the second operand
    constexpr int U = WF == W_FP4 ? 2 : 4;                             // steps in flight
    __shared__ f32x4_t red[kDecWaves][MT * NT][64];

    const int act = blockIdx.x / a.nchunk, chunk = blockIdx.x % a.nchunk;
    if (act >= *a.l.n_act) return;
    const int slot = a.l.slot[act], off = a.l.off[act], cnt = a.l.cnt[act];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int K = a.K, N = a.N, n0 = chunk * kDecRows;
    const int nmt = MT == 1 ? 1 : (cnt + 15) / 16;

    // second operand rows of this lane: tokens (gate/up) or routes (down)
    int64_t xoff[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int i = a.l.rec[off + min(16 * m + r, cnt - 1)];
        xoff[m] = (int64_t)(GATEUP ? i / a.kp : i) * a.ldx;
    }
    // the chunk's 64 rows lie in one 256-row block of the tiled slice
    const int nb = n0 / kWRows, rows = min(kWRows, N - nb * kWRows);
    const char *W = a.W + (int64_t)slot * a.slot_bytes;
    int rb[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) rb[t] = min(n0 + 16 * t + r, N - 1) - nb * kWRows;

    f32x4_t acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[m][t] = f32x4_t{0, 0, 0, 0};

    const int steps = (K + KS - 1) / KS;
    const int s0 = (int)((int64_t)steps * wave / kDecWaves), s1 = (int)((int64_t)steps * (wave + 1) / kDecWaves);
    for (int s = s0; s < s1; s += U) {
        u32x4_t w[U][NT];
        uint32_t sc[U][NT];
        u32x4_t x[U][MT][PL][NI];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s + u) * KS + q * LK;
            const bool in = s + u < s1 && k < K;
            const int kc = in ? k : 0;
            const int64_t piece = kc / kWK;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const char *p;
                if constexpr (WF == W_F32) {
                    const int wd = min(kWK, K - (int)piece * kWK);
                    p = W + ((int64_t)nb * kWRows * K + piece * rows * kWK + (int64_t)rb[t] * wd + kc % kWK) * 4;
                } else if constexpr (WF == W_BF16) {
                    p = W + ((int64_t)nb * kWRows * K + piece * rows * kWK + rb[t] * kWK + kc % kWK) * 2;
                } else if constexpr (WF == W_FP8) {
                    p = W + (int64_t)nb * kWRows * K + piece * rows * kWK + rb[t] * kWK + kc % kWK;
                } else {
                    p = W + (int64_t)nb * (K / kWK) * fp4_piece_bytes(kWRows) + piece * fp4_piece_bytes(rows);
                    sc[u][t] = *(const uint8_t *)(p + rows * 16 + rb[t]);
                    p += rb[t] * 16;
                }
                w[u][t] = *(const u32x4_t *)p;
                if (!in) w[u][t] = u32x4_t{0, 0, 0, 0};
                if (WF == W_FP4 && !in) sc[u][t] = 127;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s + u) * KS + q * LK;
            const bool in = s + u < s1 && k < K;
            const int kc = in ? k : 0;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (m >= nmt) continue;
#pragma unroll
                for (int pl = 0; pl < PL; ++pl) {
                    const char *p = (const char *)a.X + (xoff[m] + (int64_t)pl * a.R * a.ldx + kc) * (WF == W_F32 ? 4 : 2);
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        x[u][m][pl][i] = *(const u32x4_t *)(p + 16 * i);
                        if (!in) x[u][m][pl][i] = u32x4_t{0, 0, 0, 0};
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    bf16x8_t wv;
                    if constexpr (WF == W_BF16) wv = __builtin_bit_cast(bf16x8_t, w[u][t]);
                    if constexpr (WF == W_FP8) wv = fp8_operand(w[u][t], i);
                    if constexpr (WF == W_FP4) wv = fp4_operand(w[u][t][i], e8m0(sc[u][t]));
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        if (m >= nmt) continue;
                        if constexpr (WF == W_F32) {
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                    __uint_as_float(w[u][t][c]), __uint_as_float(x[u][m][0][0][c]), acc[m][t], 0, 0, 0);
                        } else {
#pragma unroll
                            for (int pl = 0; pl < PL; ++pl)
                                acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                    wv, __builtin_bit_cast(bf16x8_t, x[u][m][pl][i]), acc[m][t], 0, 0, 0);
                        }
                    }
                }
    }

#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) red[wave][m * NT + t][lane] = acc[m][t];
    __syncthreads();

    // Result layout: element c of lane l is weight row 4 (l / 16) + c of its
    // group, route l % 16. Sums of the waves in ascending order.
    auto total = [&](int g, int l) {
        f32x4_t v = red[0][g][l];
#pragma unroll
        for (int w = 1; w < kDecWaves; ++w) v += red[w][g][l];
        return v;
    };
    auto scale = [&](f32x4_t v, int n) {   // fp8: the rows' scales
        if constexpr (WF == W_FP8)
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] *= *(const float *)(W + a.scale_off + (int64_t)(n + c) * 4);
        return v;
    };
    if constexpr (GATEUP) {
        // groups 0, 1 are gate rows, 2, 3 the up rows of the same 32 units
        for (int e = threadIdx.x; e < nmt * 2 * 64; e += kDecWaves * 64) {
            const int l = e & 63, h = (e >> 6) & 1, m = e >> 7;
            const int row = 16 * m + (l & 15), n = 16 * h + 4 * (l >> 4);
            if (row >= cnt) continue;
            const f32x4_t g = scale(total(m * NT + h, l), n0 + n), u = scale(total(m * NT + 2 + h, l), n0 + 32 + n);
            const int64_t at = (int64_t)a.l.rec[off + row] * a.ldo + chunk * 32 + n;
            float v[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = g[c] / (1.0f + expf(-g[c])) * u[c];
            if constexpr (WF == W_F32) {
                *(float4 *)((float *)a.out + at) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
                uint16_t t3[3][4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    // cut 8 bits at a time: each difference is exact, and the
                    // third has at most 8 bits left
                    float rest = v[c];
                    if (rest != rest) rest = __uint_as_float(0x7fc00000u);
                    const bool inf = __builtin_isinf(rest);
#pragma unroll
                    for (int pl = 0; pl < 3; ++pl) {
                        const uint32_t b = __float_as_uint(rest) & 0xffff0000u;
                        t3[pl][c] = (uint16_t)(b >> 16);
                        rest = inf ? 0.0f : rest - __uint_as_float(b);
                    }
                }
#pragma unroll
                for (int pl = 0; pl < 3; ++pl)
                    *(uint2 *)((uint16_t *)a.out + (int64_t)pl * a.R * a.ldo + at) =
                        make_uint2(t3[pl][0] | (uint32_t)t3[pl][1] << 16, t3[pl][2] | (uint32_t)t3[pl][3] << 16);
            }
        }
    } else {
        for (int e = threadIdx.x; e < nmt * NT * 64; e += kDecWaves * 64) {
            const int l = e & 63, t = (e >> 6) % NT, m = (e >> 6) / NT;
            const int row = 16 * m + (l & 15), n = n0 + 16 * t + 4 * (l >> 4);
            if (row >= cnt || n >= N) continue;   // N % 4 == 0
            const int i = a.l.rec[off + row];
            const f32x4_t v = scale(total(m * NT + t, l), n);
            const float al = a.topk_w[i];
            *(float4 *)((float *)a.out + (int64_t)i * a.ldo + n) =
                make_float4(al * v[0], al * v[1], al * v[2], al * v[3]);
        }
    }
}

// Y_t += the token's route rows in ascending j.
__global__ __launch_bounds__(256) void k_dec_combine(float *__restrict__ Y, int64_t ldy, const float *__restrict__ Yr,
                                                     int d, int kp, int cblocks)
{
    const int t = blockIdx.x / cblocks, c = ((int)(blockIdx.x % cblocks) * 256 + threadIdx.x) * 4;
    if (c >= d) return;
    float4 y = *(const float4 *)(Y + (int64_t)t * ldy + c);
    for (int j = 0; j < kp; ++j) {
        const float4 v = *(const float4 *)(Yr + ((int64_t)t * kp + j) * d + c);
        y.x += v.x;
        y.y += v.y;
        y.z += v.z;
        y.w += v.w;
    }
    *(float4 *)(Y + (int64_t)t * ldy + c) = y;
}

template <int WF, bool GATEUP>
hipError_t launch_proj_t(const moe_shape &s, const DecArgs &a, unsigned grid, hipStream_t st)
{
    if (s.T <= 16)
        hipLaunchKernelGGL((k_dec_proj<WF, 1, GATEUP>), dim3(grid), dim3(kDecWaves * 64), 0, st, a);
    else if (s.T <= 32)
        hipLaunchKernelGGL((k_dec_proj<WF, 2, GATEUP>), dim3(grid), dim3(kDecWaves * 64), 0, st, a);
    else
        hipLaunchKernelGGL((k_dec_proj<WF, 4, GATEUP>), dim3(grid), dim3(kDecWaves * 64), 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_dec_lists(const moe_shape &s, const int32_t *idx, const PhiArg &phi, const DecLists &l, hipStream_t st)
{
    hipLaunchKernelGGL(k_dec_lists, dim3(1), dim3(kMaxExp), 0, st, idx, s.T * (s.k + s.n_shared), s.P, phi, l);
    return hipGetLastError();
}

hipError_t launch_dec_proj(const moe_shape &s, const DecArgs &a0, bool gateup, hipStream_t st)
{
    DecArgs a = a0;
    a.nchunk = (a.N + kDecRows - 1) / kDecRows;
    // at most this many slots have routes
    const int64_t slots = std::min<int64_t>(s.E + s.n_shared, a.R);
    const unsigned grid = (unsigned)(slots * a.nchunk);
    if (gateup) {
        if (s.dtype == MOE_DT_F32) return launch_proj_t<W_F32, true>(s, a, grid, st);
        if (w_fp8(s)) return launch_proj_t<W_FP8, true>(s, a, grid, st);
        if (w_fp4(s)) return launch_proj_t<W_FP4, true>(s, a, grid, st);
        return launch_proj_t<W_BF16, true>(s, a, grid, st);
    }
    if (s.dtype == MOE_DT_F32) return launch_proj_t<W_F32, false>(s, a, grid, st);
    if (w_fp8(s)) return launch_proj_t<W_FP8, false>(s, a, grid, st);
    if (w_fp4(s)) return launch_proj_t<W_FP4, false>(s, a, grid, st);
    return launch_proj_t<W_BF16, false>(s, a, grid, st);
}

hipError_t launch_dec_combine(const moe_shape &s, float *Y, const float *Yr, hipStream_t st)
{
    const int cblocks = (s.d / 4 + 255) / 256;
    hipLaunchKernelGGL(k_dec_combine, dim3((unsigned)(s.T * cblocks)), dim3(256), 0, st, Y, s.ldy, Yr, s.d,
                       s.k + s.n_shared, cblocks);
    return hipGetLastError();
}

}  // namespace moe
