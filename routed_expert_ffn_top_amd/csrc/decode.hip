// One mixture-of-experts layer for a few tokens (T <= 64): the answering step
// of the layer that expert_gemm.hip runs over a whole prompt.
//
//   H_i = SiLU(W_g x_t) * (W_u x_t),  o_i = alpha_i W_d H_i  for route i = (t, j),
//   Y_t += sum_j o_i in ascending j.
//
// With one to a few rows an expert, the layer's time is that of reading the
// weights of the experts hit, once; every product is a matrix times at most 64
// columns. A workgroup takes 64 rows of one slot's weight slice over all of K
// and an entry's routes (dec_rpe: most slots' routes are one entry), so that a
// weight is read by one workgroup only. Its waves cut K among themselves (each its
// own stretch of the slice, whose 64 rows of a K piece are contiguous in the tiled
// layout) and add their sums in a fixed order through LDS.
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
// three: 5 routes are 15 of the 16 columns of one operand (column 3 i + j: term
// j of route i), joined at the end. So up to 5 routes of a slot cost what one
// does. fp32 layers keep H as fp32 and use the fp32 matrix instruction.
#include <algorithm>
#include <type_traits>

#include "decode.h"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

enum { W_F32 = 0, W_BF16 = 1, W_FP8 = 2, W_FP4 = 3 };

// ---- values handed from workgroup to workgroup within a launch ----
// The compute dies have an L2 each. A release or acquire at device scope
// writes back or drops a whole L2, which costs every other workgroup there its
// lines (measured: 2048 arrivals made the MXFP4 down projection 87 us instead
// of 35). So what is handed over is stored and loaded past the L2, value by
// value (relaxed atomics at device scope), and an arrival only has to wait for
// its own stores.
template <typename T>
__device__ __forceinline__ void put(T *p, T v)
{
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ T get(const T *p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Every wave's put()s are complete, then one thread adds 1 to the counter.
// True for the workgroup whose arrival is the last of `all`, which may get()
// what the others put; it clears the counter for the next call. Nobody waits.
__device__ __forceinline__ bool last_to_arrive(int32_t *ctr, int all)
{
    __shared__ int32_t s_last;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_waitcnt(0);   // the stores have reached memory
    __syncthreads();
    if (threadIdx.x == 0) {
        const int n = __hip_atomic_fetch_add(ctr, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = n == all - 1;
        if (s_last) put(ctr, 0);
    }
    __syncthreads();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    return s_last != 0;
}

__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    return v;
}
__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// Order-preserving 64-bit key of (logit, expert): larger logit first, equal
// ones by lower id; NaN as -infinity, -0 as +0.
__device__ __forceinline__ uint64_t topk_key(float x, int e)
{
    if (x != x) x = -__builtin_huge_valf();
    if (x == 0.0f) x = 0.0f;
    const uint32_t u = __float_as_uint(x);
    return ((uint64_t)((u & 0x80000000u) ? ~u : (u | 0x80000000u)) << 32) | (uint32_t)~(uint32_t)e;
}

// ---- routing ----
// Router logits of one token for experts e0 .. e0+3, by one wave (16 lanes an
// expert): lane p holds the partial sum p of the router's fixed order (runs of
// 8 hidden indices, run r to partial sum r mod 16, ascending, one fused
// multiply-add a term), so the loads are whole 512-byte stretches of W_r and
// the bits are the prompt router's. U groups of 128 hidden indices are asked
// for at once. part: 64 floats of this wave. out(e, logit) in lanes 0 .. 3.
template <typename TX, int U, typename F>
__device__ __forceinline__ void wave_logits(const DecRouteArgs &a, int t, int e0, float *part, F out)
{
    constexpr int XE = 16 / sizeof(TX), XV = 8 / XE;   // x values per 16 bytes, 16-byte pieces per run
    const int lane = threadIdx.x & 63, p = lane & 15, d = a.d, ng = (d + 127) / 128;
    const float *w = a.Wr + (int64_t)min(e0 + (lane >> 4), a.E - 1) * d + p * 8;
    const TX *x = (const TX *)a.X + (int64_t)t * a.ldx + p * 8;
    float acc = 0.0f;
    for (int g = 0; g < ng; g += U) {
        u32x4_t wv[U][2], xv[U][XV];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // pieces at or past d are read from the row start and not used
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int i = (g + u) * 128 + 4 * h;
                wv[u][h] = *(const u32x4_t *)(w + (i + p * 8 < d ? i : -p * 8));
            }
#pragma unroll
            for (int h = 0; h < XV; ++h) {
                const int i = (g + u) * 128 + XE * h;
                xv[u][h] = *(const u32x4_t *)(x + (i + p * 8 < d ? i : -p * 8));
            }
        }
        __builtin_amdgcn_sched_barrier(0);   // all requested before the first is used
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float wc = __uint_as_float(wv[u][c >> 2][c & 3]);
                float xc;
                if constexpr (sizeof(TX) == 2) {
                    const uint32_t w2 = xv[u][0][c >> 1];
                    xc = __uint_as_float((c & 1) ? (w2 & 0xffff0000u) : (w2 << 16));
                } else {
                    xc = __uint_as_float(xv[u][c >> 2][c & 3]);
                }
                const float s = __builtin_fmaf(xc, wc, acc);
                acc = (g + u) * 128 + p * 8 + c < d ? s : acc;
            }
    }
    __builtin_amdgcn_wave_barrier();   // this wave's own writes and reads, in order
    part[lane] = acc;
    __builtin_amdgcn_wave_barrier();
    if (lane < 4 && e0 + lane < a.E) {   // the 16 partial sums of an expert in ascending order
        float v[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) v[c] = part[lane * 16 + c];
        float s = v[0];
#pragma unroll
        for (int c = 1; c < 16; ++c) s = s + v[c];
        out(e0 + lane, a.bias ? s + a.bias[e0 + lane] : s);
    }
}

// Top-k of one token by one wave, in the prompt kernel's arithmetic (lane l
// holds experts l, l + 64, ..). logit(e); keys: 64 C + 2 words of this wave;
// out(rank, expert, weight), shared experts included.
template <int C, typename V, typename F>
__device__ __forceinline__ void wave_topk(const DecRouteArgs &a, uint64_t *keys, V logit, F out)
{
    const int lane = threadIdx.x & 63;
    const float NEG_INF = -__builtin_huge_valf();
    float v[C];
    uint64_t key[C];
    int rank[C];
    __builtin_amdgcn_wave_barrier();   // this wave's own writes and reads, in order
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = lane + 64 * c;
        v[c] = e < a.E ? logit(e) : NEG_INF;
        if (v[c] != v[c]) v[c] = NEG_INF;
        key[c] = topk_key(v[c], e);
        keys[e] = e < a.E ? key[c] : 0ull;
        rank[c] = 0;
    }
    if (lane < 2) keys[64 * C + lane] = 0ull;
    __builtin_amdgcn_wave_barrier();
#pragma unroll 8
    for (int e2 = 0; e2 < ((a.E + 1) & ~1); e2 += 2) {
        const uint64_t k0 = keys[e2], k1 = keys[e2 + 1];
#pragma unroll
        for (int c = 0; c < C; ++c) rank[c] += (int)(k0 > key[c]) + (int)(k1 > key[c]);
    }
    float m = NEG_INF;
#pragma unroll
    for (int c = 0; c < C; ++c) m = fmaxf(m, v[c]);
    m = wave_max(m);
    if (m == NEG_INF) m = 0.0f;
    float z[C], s = 0.0f, ssel = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = lane + 64 * c;
        z[c] = e < a.E ? expf(v[c] - m) : 0.0f;
        s += z[c];
        if (e < a.E && rank[c] < a.k) ssel += z[c];
    }
    s = wave_sum(s);
    ssel = wave_sum(ssel);
    const float den = a.renorm ? ssel : s;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = lane + 64 * c;
        if (e < a.E && rank[c] < a.k) out(rank[c], e, den > 0.0f ? z[c] / den : 0.0f);
    }
    if (lane < a.n_shared) out(a.k + lane, a.E + lane, 1.0f);
}

// The routes by slot, by a workgroup of 256: counts, offsets, places; at most
// rpe routes to an entry. slot_of(i) of route i < R; put_entry(n, slot, off, cnt),
// put_rec(place, i); returns the number of entries. The routes of a slot stand in
// ascending order, whichever workgroup does this: where gate/up routes for itself
// every workgroup does, and the entries it takes a part of have to be the same in
// all. So 64 routes at a time take their places, not whichever wave comes first.
template <int RT, typename S, typename PE, typename PR>
__device__ __forceinline__ int build_lists(int R, int rpe, int32_t *cnt, int32_t *off, int32_t *wsum, S slot_of,
                                           PE put_entry, PR put_rec)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    static_assert(kMaxExp == 512, "two slots a thread, 9 bits a slot");
    cnt[tid] = cnt[tid + 256] = 0;
    __syncthreads();
    int slot[RT], pos[RT];
#pragma unroll
    for (int q = 0; q < RT; ++q) {
        if (256 * q >= R) continue;
        const bool is = tid + 256 * q < R;
        slot[q] = is ? slot_of(tid + 256 * q) : 0;
        // the wave's routes of the same slot
        uint64_t same = __ballot(is);
#pragma unroll
        for (int b = 0; b < 9; ++b) {
            const uint64_t one = __ballot((slot[q] >> b) & 1);
            same &= (slot[q] >> b) & 1 ? one : ~one;
        }
        const int before = __popcll(same & ((1ull << lane) - 1));
        for (int w = 0; w < 4 && 256 * q + 64 * w < R; ++w) {
            if (wave == w && is) {
                const int base = cnt[slot[q]];
                pos[q] = base + before;
                if (before == 0) cnt[slot[q]] = base + __popcll(same);
            }
            __syncthreads();
        }
    }
    // thread tid: slots 2 tid and 2 tid + 1
    const int c0 = cnt[2 * tid], c1 = cnt[2 * tid + 1];
    const int e0 = (c0 + rpe - 1) / rpe, e1 = (c1 + rpe - 1) / rpe;
    int so = c0 + c1, sn = e0 + e1;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(so, o, 64), n = __shfl_up(sn, o, 64);
        if (lane >= o) {
            so += u;
            sn += n;
        }
    }
    if (lane == 63) {
        wsum[wave] = so;
        wsum[4 + wave] = sn;
    }
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        so += wsum[w];
        sn += wsum[4 + w];
    }
    const int all = wsum[4] + wsum[5] + wsum[6] + wsum[7];
    so -= c0 + c1;
    sn -= e0 + e1;
    off[2 * tid] = so;
    off[2 * tid + 1] = so + c0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int c = h ? c1 : c0, o = h ? so + c0 : so;
        for (int q = 0; q < c; q += rpe) put_entry(sn++, 2 * tid + h, o + q, min(rpe, c - q));
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < RT; ++q)
        if (tid + 256 * q < R) put_rec(off[slot[q]] + pos[q], tid + 256 * q);
    return all;
}

// Router, top-k and (`sort`) the routes by slot, in one launch. A workgroup takes 4
// experts for 4 tokens, a wave a token; the last workgroup of a token block
// does its top-k, and the last block of all sorts the routes by slot. Bound by
// latency: a wave has 32 KB of W_r to read for d = 2048, asked for at once (16
// experts a workgroup, a wave 4 of them for 4 tokens: 15 us for one token
// instead of 7.7).
template <typename TX, int C>
__global__ __launch_bounds__(256) void k_dec_route(DecRouteArgs a, PhiArg phi)
{
    constexpr int TB = kDecTokBlock;
    __shared__ float part[TB][64];
    __shared__ uint64_t keys[4][64 * C + 2];
    __shared__ int32_t cnt[kMaxExp], off[kMaxExp], wsum[8], sphi[kMaxExp], s_idx[TB * 64];
    const int tid = threadIdx.x, wave = tid >> 6;
    const int t0 = blockIdx.x * TB, nt = min(TB, a.T - t0);
    const int kp = a.k + a.n_shared;
    // asked for before anything waits: kernel arguments come from far away
    const int32_t phi0 = phi.v[tid], phi1 = phi.v[tid + 256];
    if (a.Wr) {
        if (wave < nt)
            wave_logits<TX, sizeof(TX) == 2 ? 16 : 8>(a, t0 + wave, blockIdx.y * 4, part[wave], [&](int e, float l) {
                put(a.logits + (int64_t)(t0 + wave) * a.E + e, l);
            });
        if (gridDim.y > 1) {
            if (!last_to_arrive(a.ctr + 1 + blockIdx.x, gridDim.y)) return;
        } else {
            __builtin_amdgcn_s_waitcnt(0);   // this wave's logits, read below past the caches
        }
    }
    if (wave < nt) {
        const float *L = (a.Wr ? a.logits : a.given) + (int64_t)(t0 + wave) * a.E;
        const int64_t r0 = (int64_t)(t0 + wave) * kp;
        wave_topk<C>(a, keys[wave], [&](int e) { return get(L + e); }, [&](int rank, int e, float w) {
            put(a.idx + r0 + rank, e);
            s_idx[wave * kp + rank] = e;
            a.w[r0 + rank] = w;
        });
    }
    if (!a.sort) return;
    const bool alone = gridDim.x == 1;   // every token's ids are this workgroup's own
    if (!alone && !last_to_arrive(a.ctr, gridDim.x)) return;
    sphi[tid] = phi0;
    sphi[tid + 256] = phi1;
    const int n = build_lists<kDecMaxRoutes / 256>(
        a.T * kp, a.rpe, cnt, off, wsum, [&](int i) { return sphi[alone ? s_idx[i] : get(a.idx + i)]; },
        [&](int n, int slot, int o, int c) {
            a.l.slot[n] = slot;
            a.l.off[n] = o;
            a.l.cnt[n] = c;
        },
        [&](int place, int i) { a.l.rec[place] = i; });
    if (tid == 0) *a.l.n_act = n;
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

// SiLU(g) u. Below -88, where exp(-g) leaves the range: 1 + exp(-g) is exp(-g) there, and
// exp(g) is taken in two halves, u between them, that stay normal numbers (down to g = -174).
__device__ __forceinline__ float silu_mul(float g, float u)
{
    if (g < -88.0f) {
        const float e = expf(0.5f * g);
        return g * e * u * e;
    }
    return g / (1.0f + expf(-g)) * u;
}

constexpr uint32_t kNowhere = 0x80000000u;   // a buffer offset past every slice: such a load gives zeros and reads nothing

// Workgroup barrier that waits for this wave's LDS traffic only: loads in
// flight stay so (gfx9 s_waitcnt encoding: vmcnt[3:0] | expcnt[6:4] |
// lgkmcnt[11:8] | vmcnt[5:4] at bits 15:14).
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (0 << 8) | (3 << 14));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// WF: weight format. RPE: an entry of the lists has at most this many routes.
// NT: 16-row groups of the slice per tile.
//
// The workgroups are persistent: each walks its tiles (slot, 16 NT rows) and
// requests the next stretch of weights, of the same tile or of the next,
// before it multiplies the present one, so that loads are under way during the
// products and a tile's joining of sums and its stores. (Taking the next stretch
// over waits for it. Two stretches in turn, without that wait, measured the same
// with up to 5 routes an entry, and 5 - 10 % slower above, for their registers:
// the other waves fill it.) The operand of the tokens is
// requested before that next stretch: loads return in order, and the wait for
// it then leaves the weights in flight. Weights come through buffer loads, whose
// bounds check makes a stretch that is not there zeros without a branch, so
// that the number of loads in flight is the same on every path.
template <int WF, int RPE, int NT, int NW>
struct ProjShared {
    f32x4_t red[NW][(RPE + 15) / 16 * NT][64];
    int32_t slot[kDecMaxEntries], off[kDecMaxEntries], cnt[kDecMaxEntries], rec[kDecMaxRoutes];
};

template <int WF, int RPE, int NT, int NW, bool GATEUP>
__device__ __forceinline__ void proj_tiles(const DecArgs &a, const int n_act, ProjShared<WF, RPE, NT, NW> &sh)
{
    constexpr int LK = WF == W_F32 ? 4 : WF == W_BF16 ? 8 : WF == W_FP8 ? 16 : 32;   // k values per lane and step
    constexpr int KS = 4 * LK;                                         // k values per step
    constexpr int NI = LK > 8 ? LK / 8 : 1;                            // bf16 operands of 8 per lane and step
    constexpr int PL = !GATEUP && WF != W_F32 ? 3 : 1;                 // terms (columns) per route
    constexpr int RG = 16 / PL, G = (RPE + RG - 1) / RG;               // routes per operand, operands
    constexpr int MT = (RPE + 15) / 16;                                // 16-route groups of the joined sums
    // Steps per stretch: 4 KB of weights a wave and step in bf16, as much with two
    // of MXFP4 or fp8; more do not gain and cost registers (16 tokens of 8 routes
    // on 64 experts, MXFP4: 66 us with one, 72 with two).
    constexpr int U = (WF == W_BF16 || WF == W_F32) && (RPE <= 16 || (RPE == 32 && PL == 1)) ? 2 : 1;
    constexpr int XR = U * NI * 4;                                     // registers of one operand's stretch
    constexpr int GP = G * XR <= 48 ? G : (48 / XR > 1 ? 48 / XR : 1); // operands requested ahead of the weights
    constexpr int ROWB = WF == W_F32 ? 0 : WF == W_BF16 ? 64 : WF == W_FP8 ? 32 : 16;   // bytes of a row in a K piece
    auto &red = sh.red;
    const int32_t *s_slot = sh.slot, *s_off = sh.off, *s_cnt = sh.cnt, *s_rec = sh.rec;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int K = a.K, N = a.N, nchunk = a.nchunk;

    // Tiles of this workgroup. Gate/up: every gridDim-th of all. Down: one
    // column chunk (every gridDim-th, where there are more chunks than
    // workgroups) and every `groups`-th slot, so that it arrives at each of
    // its chunks once.
    const int groups = GATEUP ? 1 : max(1, (int)gridDim.x / nchunk);
    int chunk = blockIdx.x % nchunk, act = blockIdx.x / nchunk;
    const int act0 = act;
    auto advance = [&](int &ac, int &ch) {
        if (GATEUP) {
            const int g = ac * nchunk + ch + (int)gridDim.x;
            ac = g / nchunk;
            ch = g % nchunk;
        } else {
            ac += groups;
            if (ac >= n_act && groups == 1) {
                ac = 0;
                ch += gridDim.x;
                if (ch >= nchunk) ac = n_act;
            }
        }
    };
    if (!GATEUP && act0 >= groups) return;
    if (act >= n_act) return;   // down: fewer slots than groups; the others arrive alone

    const int steps = (K + KS - 1) / KS;
    const int s0 = (int)((int64_t)steps * wave / NW), s1 = (int)((int64_t)steps * (wave + 1) / NW);

    // Where a tile's weights are: the slot's slice as a buffer, this lane's
    // offset of step 0, and bytes from step to step.
    struct Src {
        __amdgpu_buffer_rsrc_t buf;
        uint32_t at, sc_at, stride;
        int rows, nb;
    };
    auto source = [&](int ac, int ch) {
        Src p;
        const int slot = __builtin_amdgcn_readfirstlane(s_slot[ac]);
        p.buf = __builtin_amdgcn_make_buffer_rsrc((void *)(a.W + (int64_t)slot * a.slot_bytes), 0, (int)a.slice_bytes,
                                                  0x00027000);
        const int n0 = ch * (16 * NT);
        p.nb = n0 / kWRows;
        p.rows = min(kWRows, N - p.nb * kWRows);
        const uint32_t rb = n0 - p.nb * kWRows + r;
        if constexpr (WF == W_FP4) {
            const uint32_t pb = (uint32_t)fp4_piece_bytes(p.rows);
            p.at = (uint32_t)p.nb * (K / kWK) * (uint32_t)fp4_piece_bytes(kWRows) + q * pb;
            p.sc_at = p.at + p.rows * 16 + rb;
            p.at += rb * 16;
            p.stride = 4 * pb;
        } else {
            p.at = (uint32_t)p.nb * kWRows * K * (ROWB / kWK) + rb * ROWB;
            if constexpr (WF == W_FP8) p.at += (q & 1) * 16 + (q >> 1) * p.rows * ROWB;
            if constexpr (WF == W_BF16) p.at += q * 16;
            p.sc_at = 0;
            p.stride = (WF == W_FP8 ? 2 : 1) * p.rows * ROWB;
        }
        return p;
    };
    struct Stretch {
        u32x4_t w[U][NT];
        uint32_t sc[U][WF == W_FP4 ? NT : 1];
    };
    auto request = [&](Stretch &d, const Src &p, int s, bool any) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s + u) * KS + q * LK;
            const bool in = any && s + u < s1 && k < K;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                uint32_t at;
                if constexpr (WF == W_F32) {
                    // K pieces of the last columns are narrower, and N may end inside the tile
                    const int piece = k / kWK, wd = min(kWK, K - piece * kWK);
                    const int rb = min((int)p.at + 16 * t, p.rows - 1);
                    at = (uint32_t)(p.nb * kWRows * K + piece * p.rows * kWK + rb * wd + k % kWK) * 4;
                } else {
                    at = p.at + (uint32_t)(s + u) * p.stride + t * 16 * ROWB;
                }
                d.w[u][t] = __builtin_amdgcn_raw_buffer_load_b128(p.buf, (int)(in ? at : kNowhere), 0, 0);
                if constexpr (WF == W_FP4)
                    d.sc[u][t] = __builtin_amdgcn_raw_buffer_load_b8(
                        p.buf, (int)(in ? p.sc_at + (uint32_t)(s + u) * p.stride + t * 16 : kNowhere), 0, 0);
            }
        }
    };

    Src src = source(act, chunk);
    if constexpr (WF == W_F32) src.at = chunk * (16 * NT) - src.nb * kWRows + r;
    Stretch cur, nxt;
    request(cur, src, s0, true);
    for (;;) {
        const int off = __builtin_amdgcn_readfirstlane(s_off[act]), cnt = __builtin_amdgcn_readfirstlane(s_cnt[act]);
        const int n0 = chunk * (16 * NT);
        int nact = act, nch = chunk;
        advance(nact, nch);
        const bool more = nact < n_act;
        Src nsrc = source(more ? nact : act, more ? nch : chunk);
        if constexpr (WF == W_F32) nsrc.at = (more ? nch : chunk) * (16 * NT) - nsrc.nb * kWRows + r;

        // second operands of this lane: tokens (gate/up) or terms of routes (down)
        const int ng = G == 1 ? 1 : (cnt + RG - 1) / RG;
        const char *xp[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int i = s_rec[off + min(g * RG + min(r / PL, RG - 1), cnt - 1)];
            xp[g] = (const char *)a.X + ((int64_t)(GATEUP ? i / a.kp : i) * a.ldx +
                                         (PL == 3 ? (int64_t)(r % 3) * a.R * a.ldx : 0)) * (WF == W_F32 ? 4 : 2);
        }
        // what this thread needs for its result (one of 4 rows x 1 route), asked
        // for now: at the end of the tile it would wait behind the weights
        const int rl = tid & 63, rg = tid >> 6;
        const int rm = GATEUP ? rg >> 1 : rg / NT, rt = GATEUP ? rg & 1 : rg % NT;
        const int rrow = 16 * rm + (rl & 15), rn = 16 * rt + 4 * (rl >> 4);
        const bool mine = rrow < cnt && (GATEUP || n0 + rn < N);   // N % 4 == 0
        const int route = s_rec[off + min(rrow, cnt - 1)];
        const float alpha = GATEUP ? 1.0f : a.topk_w[route];
        f32x4_t rs0 = {1, 1, 1, 1}, rs1 = {1, 1, 1, 1};
        if constexpr (WF == W_FP8) {
            const char *S = a.W + (int64_t)__builtin_amdgcn_readfirstlane(s_slot[act]) * a.slot_bytes + a.scale_off;
            rs0 = *(const f32x4_t *)(S + (int64_t)(n0 + min(rn, 16 * NT - 4)) * 4);
            if (GATEUP) rs1 = *(const f32x4_t *)(S + (int64_t)(n0 + 32 + rn) * 4);
        }
        f32x4_t acc[G][NT];
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[g][t] = f32x4_t{0, 0, 0, 0};

        int s = s0;
        do {
            u32x4_t x[GP][U][NI];
            auto load_x = [&](u32x4_t &d, int g, int u, int i) {
                const int k = (s + u) * KS + q * LK;
                const bool in = s + u < s1 && k < K;
                d = *(const u32x4_t *)(xp[g] + ((in ? k : 0) + 8 * i) * (WF == W_F32 ? 4 : 2));
                // a weight of zero times whatever stands there is to add nothing
                if (WF == W_FP4 || WF == W_F32)
                    if (!in) d = u32x4_t{0, 0, 0, 0};
            };
#pragma unroll
            for (int g = 0; g < GP; ++g) {
                if (g > 0 && g >= ng) continue;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < NI; ++i) load_x(x[g][u][i], g, u, i);
            }
            __builtin_amdgcn_sched_barrier(0);
            const bool last = s + U >= s1;
            request(nxt, last ? nsrc : src, last ? s0 : s + U, !last || more);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (s + u >= s1) continue;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    bf16x8_t wv[NT];
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if constexpr (WF == W_BF16) wv[t] = __builtin_bit_cast(bf16x8_t, cur.w[u][t]);
                        if constexpr (WF == W_FP8) wv[t] = fp8_operand(cur.w[u][t], i);
                        if constexpr (WF == W_FP4) wv[t] = fp4_operand(cur.w[u][t][i], e8m0(cur.sc[u][t]));
                    }
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        if (g > 0 && g >= ng) continue;
                        u32x4_t xv;
                        if (g < GP)
                            xv = x[g < GP ? g : 0][u][i];
                        else
                            load_x(xv, g, u, i);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            if constexpr (WF == W_F32) {
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    acc[g][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                        __uint_as_float(cur.w[u][t][c]), __uint_as_float(xv[c]), acc[g][t], 0, 0, 0);
                            } else {
                                acc[g][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                    wv[t], __builtin_bit_cast(bf16x8_t, xv), acc[g][t], 0, 0, 0);
                            }
                        }
                    }
                }
            }
            cur = nxt;
            s += U;
        } while (s < s1);

        // this wave's sums, a route's terms joined in ascending order, to LDS
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (g > 0 && g >= ng) continue;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                f32x4_t v = acc[g][t];
                if constexpr (PL == 3) {
                    f32x4_t v1, v2;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        v1[c] = __shfl_down(v[c], 1, 64);
                        v2[c] = __shfl_down(v[c], 2, 64);
                    }
                    v = (v + v1) + v2;
                    const int row = g * RG + r / 3;
                    if (r % 3 == 0 && r < 15 && row < 16 * MT) red[wave][(row >> 4) * NT + t][(lane & 48) + (row & 15)] = v;
                } else {
                    red[wave][g * NT + t][lane] = v;
                }
            }
        }
        lds_barrier();

        // Result layout: element c of lane l is weight row 4 (l / 16) + c of its
        // group, route l % 16. Sums of the waves in ascending order.
        auto total = [&](int g, int l) {
            f32x4_t v = red[0][g][l];
#pragma unroll
            for (int w = 1; w < NW; ++w) v += red[w][g][l];
            return v;
        };
        static_assert(MT * (GATEUP ? 2 : NT) <= NW, "a thread has one result");
        if constexpr (GATEUP) {
            // groups 0, 1 are gate rows, 2, 3 the up rows of the same 32 units
            static_assert(NT == 4, "a tile is 32 gate and 32 up rows");
            if (mine) {
                f32x4_t g = total(rm * NT + rt, rl), u = total(rm * NT + 2 + rt, rl);
                if constexpr (WF == W_FP8) {
                    g *= rs0;
                    u *= rs1;
                }
                const int64_t at = (int64_t)route * a.ldo + chunk * 32 + rn;
                float v[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = silu_mul(g[c], u[c]);
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
            if (mine) {
                f32x4_t v = total(rm * NT + rt, rl);
                if constexpr (WF == W_FP8) v *= rs0;
#pragma unroll
                for (int c = 0; c < 4; ++c) put((float *)a.out + (int64_t)route * a.ldo + n0 + rn + c, alpha * v[c]);
            }
            if (!more || nch != chunk) {
                // The last workgroup to finish these columns adds the tokens'
                // rows: Y_t += the token's route rows in ascending j.
                if (last_to_arrive(a.ctr + chunk, min(groups, n_act))) {
                    const int n = n0 + 4 * (tid % (4 * NT));
                    for (int t = tid / (4 * NT); t < a.T && n < N; t += NW * 16 / NT) {
                        float4 y = *(const float4 *)(a.Y + (int64_t)t * a.ldy + n);
                        const float *Yr = (const float *)a.out + (int64_t)t * a.kp * a.ldo + n;
#pragma unroll 4
                        for (int j = 0; j < a.kp; ++j) {
                            const float *v = Yr + (int64_t)j * a.ldo;
                            y.x += get(v);
                            y.y += get(v + 1);
                            y.z += get(v + 2);
                            y.w += get(v + 3);
                        }
                        *(float4 *)(a.Y + (int64_t)t * a.ldy + n) = y;
                    }
                }
            }
        }
        if (!more) break;
        lds_barrier();   // the sums are read: the next tile's may be written
        act = nact;
        chunk = nch;
        src = nsrc;
    }
}

template <int WF, int RPE, int NT, int NW, bool GATEUP>
__global__ __launch_bounds__(NW * 64, 2) void k_dec_proj(DecArgs a)
{
    __shared__ ProjShared<WF, RPE, NT, NW> sh;
    const int tid = threadIdx.x;
    // entries past the last are there, and not used
    const int n_act = *a.l.n_act;
    for (int i = tid; i < a.entries; i += NW * 64) {
        sh.slot[i] = a.l.slot[i];
        sh.off[i] = a.l.off[i];
        sh.cnt[i] = a.l.cnt[i];
    }
    for (int i = tid; i < a.R; i += NW * 64) sh.rec[i] = a.l.rec[i];
    __syncthreads();
    proj_tiles<WF, RPE, NT, NW, GATEUP>(a, n_act, sh);
}

// Gate/up that sorts the routes by slot for itself: every workgroup does it, and
// the first writes it down for down. ROUTE: and does all of the routing before,
// for few tokens and experts, where that takes less than a launch of its own
// (dec_self_routes); otherwise the route launch has left the ids.
template <int WF, int RPE, bool ROUTE>
__global__ __launch_bounds__(256, 2) void k_dec_route_proj(DecArgs a, DecRouteArgs q, PhiArg phi)
{
    constexpr int NT = 4, NW = 4;
    using TX = typename std::conditional<WF == W_F32, float, uint16_t>::type;
    struct Scratch {   // in the place of the sums, which come later
        float part[4][64], logit[4][64];
        uint64_t keys[4][66];
        int32_t cnt[kMaxExp], off[kMaxExp], wsum[8], phi[kMaxExp], idx[ROUTE ? kDecSelfRoutes : kDecMaxRoutes];
    };
    __shared__ ProjShared<WF, RPE, NT, NW> sh;
    static_assert(sizeof(Scratch) <= sizeof(sh.red), "scratch");
    Scratch &c = *(Scratch *)&sh.red;
    const int tid = threadIdx.x, wave = tid >> 6, kp = a.kp;
    const bool writes = blockIdx.x == 0;
    // asked for before anything waits: kernel arguments come from far away
    const int32_t phi0 = phi.v[tid], phi1 = phi.v[tid + 256];
    if (!ROUTE)
        for (int i = tid; i < a.R; i += 256) c.idx[i] = q.idx[i];
    for (int t = wave; ROUTE && t < a.T; t += NW) {
        if (q.Wr)
            for (int e0 = 0; e0 < q.E; e0 += 4)
                wave_logits<TX, 8>(q, t, e0, c.part[wave], [&](int e, float l) { c.logit[wave][e] = l; });
        wave_topk<1>(q, c.keys[wave], [&](int e) { return q.Wr ? c.logit[wave][e] : q.given[(int64_t)t * q.E + e]; },
                     [&](int rank, int e, float w) {
                         c.idx[t * kp + rank] = e;
                         if (writes) {
                             q.idx[t * kp + rank] = e;
                             q.w[t * kp + rank] = w;
                         }
                     });
    }
    c.phi[tid] = phi0;
    c.phi[tid + 256] = phi1;
    __syncthreads();
    const int n_lists = build_lists<(ROUTE ? kDecSelfRoutes : kDecMaxRoutes) / 256>(
        a.R, q.rpe, c.cnt, c.off, c.wsum, [&](int i) { return c.phi[c.idx[i]]; },
        [&](int n, int slot, int o, int k) {
            sh.slot[n] = slot;
            sh.off[n] = o;
            sh.cnt[n] = k;
            if (writes) {
                a.l.slot[n] = slot;
                a.l.off[n] = o;
                a.l.cnt[n] = k;
            }
        },
        [&](int place, int i) {
            sh.rec[place] = i;
            if (writes) a.l.rec[place] = i;
        });
    const int n = __builtin_amdgcn_readfirstlane(n_lists);   // the same in every lane, and now known to be
    if (writes && tid == 0) *a.l.n_act = n;
    __syncthreads();
    proj_tiles<WF, RPE, NT, NW, true>(a, n, sh);
}

// Persistent workgroups: two of 8 waves, or four of 4, per compute unit of the 256.
constexpr int kDecGrid = 512;

template <int WF, int RPE, int NT, int NW, bool GATEUP>
hipError_t launch_proj_n(DecArgs a, hipStream_t st)
{
    a.nchunk = (a.N + 16 * NT - 1) / (16 * NT);
    const int64_t most = kDecGrid * 8 / NW, tiles = (int64_t)a.entries * a.nchunk;
    int64_t grid = std::min(most, tiles);
    if (!GATEUP && a.nchunk < grid) grid = grid / a.nchunk * a.nchunk;
    hipLaunchKernelGGL((k_dec_proj<WF, RPE, NT, NW, GATEUP>), dim3((unsigned)grid), dim3(NW * 64), 0, st, a);
    return hipGetLastError();
}

// Gate/up with entries of 16 sorts the routes for itself (dec_gate_up_sorts: more than
// 4 tokens, or the entries were of 5) and is launch_route_proj_t's.
template <int WF, bool GATEUP>
hipError_t launch_proj_t(const DecArgs &a, hipStream_t st)
{
    if (a.rpe == 5) return launch_proj_n<WF, 5, 4, 4, GATEUP>(a, st);
    if constexpr (!GATEUP)
        if (a.rpe == 16) return launch_proj_n<WF, 16, 4, 4, GATEUP>(a, st);
    if (a.rpe == 32) return launch_proj_n<WF, 32, 4, 8, GATEUP>(a, st);
    return hipErrorInvalidValue;
}

}  // namespace

template <typename TX>
static hipError_t launch_route_t(const DecRouteArgs &a, const PhiArg &phi, hipStream_t st)
{
    const dim3 grid((unsigned)((a.T + kDecTokBlock - 1) / kDecTokBlock), a.Wr ? (unsigned)((a.E + 3) / 4) : 1u);
    if (a.E <= 64)
        hipLaunchKernelGGL((k_dec_route<TX, 1>), grid, dim3(256), 0, st, a, phi);
    else if (a.E <= 128)
        hipLaunchKernelGGL((k_dec_route<TX, 2>), grid, dim3(256), 0, st, a, phi);
    else
        hipLaunchKernelGGL((k_dec_route<TX, 4>), grid, dim3(256), 0, st, a, phi);
    return hipGetLastError();
}

// The routing within the gate/up launch: at most 64 experts, 16 tokens and 256
// routes, and each wave has few round trips to memory to make for it.
bool dec_self_routes(const moe_shape &s, bool router)
{
    if (s.E > 64 || s.T > 16 || s.T * (s.k + s.n_shared) > kDecSelfRoutes || dec_rpe(s) > 16) return false;
    return !router || (s.d <= 1024 && ((s.T + 3) / 4) * ((s.E + 3) / 4) <= 2);
}

// Sorting the routes within the gate/up launch, after a route launch of several
// token blocks: that one then has one hand-over less (64 experts of 2048 x 1024, top-8,
// MXFP4, 16 tokens: 65.5 -> 64.3 us; small layers of 8 to 50 tokens 2 - 4 %). With
// one block it sorts its own routes at once.
bool dec_gate_up_sorts(const moe_shape &s, bool router)
{
    return !dec_self_routes(s, router) && s.T > kDecTokBlock && dec_rpe(s) <= 16;
}

template <int WF, bool ROUTE>
static hipError_t launch_route_proj_t(DecArgs a, const DecRouteArgs &q, const PhiArg &phi, hipStream_t st)
{
    a.nchunk = (a.N + 63) / 64;
    const unsigned grid = (unsigned)std::min<int64_t>(kDecGrid * 2, (int64_t)a.entries * a.nchunk);
    if (a.rpe == 5)
        hipLaunchKernelGGL((k_dec_route_proj<WF, 5, ROUTE>), dim3(grid), dim3(256), 0, st, a, q, phi);
    else if (a.rpe == 16)
        hipLaunchKernelGGL((k_dec_route_proj<WF, 16, ROUTE>), dim3(grid), dim3(256), 0, st, a, q, phi);
    else
        return hipErrorInvalidValue;
    return hipGetLastError();
}

template <bool ROUTE>
static hipError_t launch_route_proj_f(const moe_shape &s, const DecArgs &a, const DecRouteArgs &q, const PhiArg &phi,
                                      hipStream_t st)
{
    if (s.dtype == MOE_DT_F32) return launch_route_proj_t<W_F32, ROUTE>(a, q, phi, st);
    if (w_fp8(s)) return launch_route_proj_t<W_FP8, ROUTE>(a, q, phi, st);
    if (w_fp4(s)) return launch_route_proj_t<W_FP4, ROUTE>(a, q, phi, st);
    return launch_route_proj_t<W_BF16, ROUTE>(a, q, phi, st);
}

hipError_t launch_dec_route_proj(const moe_shape &s, const DecArgs &a, const DecRouteArgs &q, const PhiArg &phi, bool route,
                                 hipStream_t st)
{
    return route ? launch_route_proj_f<true>(s, a, q, phi, st) : launch_route_proj_f<false>(s, a, q, phi, st);
}

hipError_t launch_dec_route(const moe_shape &s, const DecRouteArgs &a, const PhiArg &phi, hipStream_t st)
{
    return act_bf16(s) ? launch_route_t<uint16_t>(a, phi, st) : launch_route_t<float>(a, phi, st);
}

// Routes per entry of the lists: what holds most slots' routes whole (7/4 of the
// mean of the experts hit), but more than 16 only for large experts. A slot with
// more has several entries and its weights are read again for each (by then from
// the L2 or the cache behind it); a kernel for more routes has more sums, and
// with them fewer waves a compute unit, and fewer workgroups, each with a longer
// chain of loads. Measured, us a layer with 5 / 16 / 32 / 64 (which none is built
// for): 64 experts of 2048 x 1024, top-8, MXFP4, 16 tokens 65 / 70 / 95 / 109; the same
// in bf16, 64 tokens 210 / 182 / 198 / 218; 8 experts of 4096 x 14336, top-2, bf16, 32
// tokens 888 / 504 / 521 / 573, 64 tokens 1389 / 701 / 584 / 661; 3 + 2 experts of 512 x
// 3392, top-1, fp8, 62 tokens 50 / 46 / 59 / 82; 7 + 1 of 3840 x 1280, top-6, bf16, 53
// tokens 225 / 136 / 143 / 148. The border at 64 MB, with 16 / 32: 8 experts of 4096 x f,
// top-2, bf16, f = 1344 (32 MB) 48 tokens 74 / 81, 64 tokens 87 / 88; 2688 (63 MB) 133 / 143,
// 156 / 152; 4096 (96 MB) 180 / 194, 221 / 202; 5376 225 / 242, 269 / 259; 8192 341 / 338,
// 424 / 367; fp8, f = 4096 (48 MB) 107 / 124, 129 / 134; 8192 (96 MB) 193 / 206, 246 / 228;
// up to 32 tokens there the two agree within 3 %. Against it: 9 + 1 experts of 1408 x 1856
// (15 MB), top-5, bf16, 32 tokens 77 / 62, 48 tokens 78 / 67, 64 tokens 115 / 104; and MXFP4,
// 4096 x 14336 (89 MB), 64 tokens 311 / 320.
int dec_rpe(const moe_shape &s)
{
    double miss = 1.0;   // that a routed expert is hit by none of the tokens
    for (int t = 0; t < s.T; ++t) miss *= 1.0 - (double)s.k / s.E;
    const double mean = (double)s.T * s.k / (s.E * (1.0 - miss));
    const double want = std::min<double>(s.T, 1.75 * mean);
    const bool large = gu_slice_bytes(s) + d_slice_bytes(s) >= (size_t)64 << 20;
    return want <= 5 ? 5 : want <= 16 || !large ? 16 : 32;
}

hipError_t launch_dec_proj(const moe_shape &s, const DecArgs &a, bool gateup, hipStream_t st)
{
    if (gateup) {
        if (s.dtype == MOE_DT_F32) return launch_proj_t<W_F32, true>(a, st);
        if (w_fp8(s)) return launch_proj_t<W_FP8, true>(a, st);
        if (w_fp4(s)) return launch_proj_t<W_FP4, true>(a, st);
        return launch_proj_t<W_BF16, true>(a, st);
    }
    if (s.dtype == MOE_DT_F32) return launch_proj_t<W_F32, false>(a, st);
    if (w_fp8(s)) return launch_proj_t<W_FP8, false>(a, st);
    if (w_fp4(s)) return launch_proj_t<W_FP4, false>(a, st);
    return launch_proj_t<W_BF16, false>(a, st);
}

}  // namespace moe
