// What stands behind an expert's products in record order and what trains the
// router: the records' rows summed into their tokens and the gradients of that
// sum, the load-balancing loss of a routing, and the gradient of the router's
// logits.
#include <initializer_list>

#include "device.h"
#include "train.h"

namespace moe {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Over a wave's 64 lanes, the same result in all of them: exchanges within rows of 16
// as operands of the instructions, the four rows' results through scalar registers (a shuffle
// through LDS takes some 100 cycles, and a token has three of these in a row).
template <class F>
__device__ __forceinline__ float wave_reduce(float v, F op)
{
    v = op(v, __uint_as_float(dpp<0xB1>(__float_as_uint(v))));    // lane ^ 1
    v = op(v, __uint_as_float(dpp<0x4E>(__float_as_uint(v))));    // lane ^ 2
    v = op(v, __uint_as_float(dpp<0x141>(__float_as_uint(v))));   // 7 - lane of 8
    v = op(v, __uint_as_float(dpp<0x140>(__float_as_uint(v))));   // 15 - lane of 16
    auto row = [&](int r) { return __uint_as_float((uint32_t)__builtin_amdgcn_readlane(__float_as_int(v), 16 * r)); };
    return op(op(row(0), row(1)), op(row(2), row(3)));
}
__device__ __forceinline__ float wave_max(float v)
{
    return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float wave_sum(float v)
{
    return wave_reduce(v, [](float a, float b) { return a + b; });
}

// ---------------------------------------------------------------------------
// Combine. V consecutive columns a thread: 8 bf16 or 4 fp32 where the strides
// allow it (16 bytes), else 4.

template <bool BF16, int V>
__device__ __forceinline__ void load_row(const void *C, int64_t at, float *v)
{
    if constexpr (!BF16) {
        const f32x4_t w = *(const f32x4_t *)((const float *)C + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = w[i];
    } else if constexpr (V == 8) {
        const u32x4_t w = *(const u32x4_t *)((const uint16_t *)C + at);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    } else {
        const u32x2_t w = *(const u32x2_t *)((const uint16_t *)C + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
}
template <bool BF16, int V>
__device__ __forceinline__ void store_row(void *C, int64_t at, const float *v)
{
    if constexpr (!BF16) {
        __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, (f32x4_t *)((float *)C + at));
    } else if constexpr (V == 8) {
        __builtin_nontemporal_store(u32x4_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])},
                                    (u32x4_t *)((uint16_t *)C + at));
    } else {
        __builtin_nontemporal_store(u32x2_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])}, (u32x2_t *)((uint16_t *)C + at));
    }
}

constexpr int kRoutes = 8;   // routes whose rows are asked for together

// Y[t] += sum over the token's routes, ascending, of weight times row: one
// fused multiply-add each, in fp32. The rows of 8 routes are requested together, their
// positions before them. Bound by HBM: every row read once; 4096 tokens of 8 routes, 2048
// bf16 columns: 41 us, 4.9 TB/s.
template <bool BF16, int V>
__global__ __launch_bounds__(256) void k_combine_rows(CombineArgs a, int blocks_x)
{
    const int t = blockIdx.x / blocks_x, c = (blockIdx.x % blocks_x * blockDim.x + threadIdx.x) * V;
    if (c >= a.d) return;
    float *y = a.Y + t * a.ldy + c;
    float s[V];
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const f32x4_t w = *(const f32x4_t *)(y + i);
#pragma unroll
        for (int q = 0; q < 4; ++q) s[i + q] = w[q];
    }
    const int64_t i0 = (int64_t)t * a.kp;
    for (int j0 = 0; j0 < a.kp; j0 += kRoutes) {
        int pos[kRoutes];
        float w[kRoutes], v[kRoutes][V];
#pragma unroll
        for (int j = 0; j < kRoutes; ++j) {
            pos[j] = j0 + j < a.kp ? a.route_pos[i0 + j0 + j] : -1;
            w[j] = j0 + j < a.kp ? a.topk_w[i0 + j0 + j] : 0.0f;
            if (pos[j] >= a.M) pos[j] = -1;
        }
#pragma unroll
        for (int j = 0; j < kRoutes; ++j)
            if (pos[j] >= 0) load_row<BF16, V>(a.C, pos[j] * a.ldc + c, v[j]);
#pragma unroll
        for (int j = 0; j < kRoutes; ++j)
            if (pos[j] >= 0)
#pragma unroll
                for (int i = 0; i < V; ++i) s[i] = fmaf(w[j], v[j][i], s[i]);
    }
#pragma unroll
    for (int i = 0; i < V; i += 4) *(f32x4_t *)(y + i) = f32x4_t{s[i], s[i + 1], s[i + 2], s[i + 3]};
}

// A workgroup a token: dC[pos] = w dY[t], dw = <dY[t], C[pos]>, the sums over a
// thread's columns ascending, then over the lanes and the waves in a fixed order. dY is read
// once for 8 routes. Bound by HBM: rows read and written once; the same sizes 63 us behind the forward
// pass on the same rows, 4.8 TB/s, 74 alone. Stores past the caches: 8 us less for both passes, 5 for
// this one alone; loads past them gain 5 forward and cost 12 here, whose rows may still be there.
template <bool BF16, int V>
__global__ __launch_bounds__(256) void k_combine_rows_backward(CombineArgs a)
{
    __shared__ float s_dot[4][kRoutes];
    const int t = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int64_t i0 = (int64_t)t * a.kp;
    for (int j0 = 0; j0 < a.kp; j0 += kRoutes) {
        int pos[kRoutes];
        float w[kRoutes], dot[kRoutes];
#pragma unroll
        for (int j = 0; j < kRoutes; ++j) {
            pos[j] = j0 + j < a.kp ? a.route_pos[i0 + j0 + j] : -1;
            w[j] = j0 + j < a.kp ? a.topk_w[i0 + j0 + j] : 0.0f;
            if (pos[j] >= a.M) pos[j] = -1;
            dot[j] = 0.0f;
        }
        for (int c = threadIdx.x * V; c < a.d; c += blockDim.x * V) {
            float g[V], v[kRoutes][V];
#pragma unroll
            for (int i = 0; i < V; i += 4) load_row<false, 4>(a.dY, t * a.ldy + c + i, g + i);
#pragma unroll
            for (int j = 0; j < kRoutes; ++j)
                if (pos[j] >= 0) load_row<BF16, V>(a.C, pos[j] * a.ldc + c, v[j]);
#pragma unroll
            for (int j = 0; j < kRoutes; ++j) {
                if (pos[j] < 0) continue;
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    dot[j] = fmaf(g[i], v[j][i], dot[j]);
                    o[i] = w[j] * g[i];
                }
                if (a.dC) store_row<BF16, V>(a.dC, pos[j] * a.lddc + c, o);
            }
        }
#pragma unroll
        for (int j = 0; j < kRoutes; ++j) {
            const float s = wave_sum(dot[j]);
            if (lane == 0) s_dot[wave][j] = s;
        }
        __syncthreads();
        if (threadIdx.x < kRoutes && j0 + (int)threadIdx.x < a.kp) {
            float s = s_dot[0][threadIdx.x];
            for (int q = 1; q < waves; ++q) s += s_dot[q][threadIdx.x];
            a.dw[i0 + j0 + threadIdx.x] = s;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Balance loss. Of a sequence s with n counted tokens, c_e routes to expert e
// and mean probability P_e (softmax over all E, as the top-k takes it: NaN as
// -infinity): loss_s = E / (k n) sum_e c_e P_e, 1 where both are uniform;
// loss = the mean of loss_s over the sequences that have tokens. Its gradient
// with respect to p_te is E / (k n^2 S+) c_e; a softmax's backward drops what
// all experts have in common, so what is kept for it is the same with c_e less
// k n / E, its mean if every route counts, which the differences there do not lose in rounding.
//
// Three steps: chunks of w.ch tokens, a workgroup each, which writes an entry for each
// sequence that it meets (sums of at most w.ch / 4 terms a wave in fp32, then 4 waves);
// the entries of a sequence, 32 experts at a time, in fp64; the last of those
// workgroups sums the loss. Every sum is in a fixed order. Entry b + s is chunk b's of
// sequence s: that is in ascending order of both, and every entry is written.
//
// Bound by instructions issued more than by the logits read (67 MB, 13 us): 65536 tokens of 256
// experts in 16 sequences, a fifth of them masked, 17.4 us (134 vector instructions a counted token, two thirds of the
// time) and 10.6 for the second step, trips to memory in a row; of 64 or of 8 experts 12.5 and 8, a token takes a wave
// whatever E; 16 tokens of 8 experts 3.5 and 4.0, all latency. Before the second step's last part took its acquire
// and release, chunks of 16, 64, 256 tokens on 256 experts: 22.6 + 17.9, 20.5 + 9.8, 41.0 + 7.4.

// C experts a lane: with V, C lane + c, read and written together (rows of whole 4 C bytes), else lane + 64 c.
template <int C, bool V>
__device__ __forceinline__ int expert(int lane, int c) { return V ? lane * C + c : lane + 64 * c; }
template <int C, bool V>
__device__ __forceinline__ int lane_of(int e) { return V ? e / C : e & 63; }
template <int C, bool V>
__device__ __forceinline__ int place_of(int e) { return V ? e % C : e >> 6; }
template <int C>
struct Row { typedef float type __attribute__((ext_vector_type(C))); };
// A row's values, `none` past E.
template <int C, bool V>
__device__ __forceinline__ void load_experts(const float *L, int E, int lane, float (&v)[C], float none)
{
    if constexpr (V) {
        const bool in = lane * C < E;
        const typename Row<C>::type w = *(const typename Row<C>::type *)(L + (in ? lane * C : 0));
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = in ? w[c] : none;
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = lane + 64 * c < E ? L[lane + 64 * c] : none;
    }
}
// exp(x) for x <= 0, within 3 2^-24: 2^y by the instruction (1 unit in the last place) with y = x log2(e)
// rounded, and what the rounding left, d, by 1 + d ln(2). Below 2^-126 it is 0. NaN stays. 8
// instructions where expf has 15, and both kernels are bound by how many they issue.
__device__ __forceinline__ float exp_down(float x)
{
    const float log2e = 0x1.715476p+0f, rest = 0x1.4ae0cp-26f;   // log2(e) in two pieces
    x = x < -120.0f ? -120.0f : x;
    const float y = x * log2e, d = fmaf(x, rest, fmaf(x, log2e, -y)), p = __builtin_amdgcn_exp2f(y);
    return fmaf(p, d * 0x1.62e43p-1f, p);
}
// Softmax numerators in place, and their sum.
template <int C>
__device__ __forceinline__ float numerators(float (&z)[C])
{
    const float none = -__builtin_huge_valf();
    float m = none, s = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (z[c] != z[c]) z[c] = none;
        m = fmaxf(m, z[c]);
    }
    m = wave_max(m);
    if (m == none) m = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        z[c] = exp_down(z[c] - m);
        s += z[c];
    }
    return wave_sum(s);
}
// 1 / s, and 0 for a row without a finite logit.
__device__ __forceinline__ float over(float s) { return s > 0.0f || s != s ? 1.0f / s : 0.0f; }

__device__ __forceinline__ void seq_range(const int32_t *off, int T, int s, int *lo, int *hi)
{
    *lo = off ? min(max(off[s], 0), T) : 0;
    *hi = off ? min(max(off[s + 1], *lo), T) : T;
}
// The last of offsets 0 .. S that is at most t, 64 of them at a time; -1 for none. Every lane.
__device__ __forceinline__ int seq_at(const int32_t *off, int S, int64_t t, int lane)
{
    int first = 0, step = 1;
    while (step * 64 < S + 1) step *= 64;
    for (;; step /= 64) {
        const int i = first + lane * step;
        const int n = __popcll(__ballot(i <= S && off[min(i, S)] <= t));
        if (n == 0) return -1;
        first += (n - 1) * step;
        if (step == 1) return min(first, S);
    }
}

template <int C>
__global__ __launch_bounds__(256) void k_balance_chunks(BalanceArgs a, int ch, int32_t *__restrict__ entry,
                                                        int32_t *__restrict__ count, float *__restrict__ prob,
                                                        uint32_t *__restrict__ ticket)
{
    __shared__ float s_p[4][64 * C];
    __shared__ int32_t s_c[64 * C], s_n[4], s_list[kMaxChunk], s_many;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b = blockIdx.x;
    if (threadIdx.x == 0) s_many = 0;
    if (b == 0 && threadIdx.x == 0) *ticket = 0;   // for the next kernel
    const int64_t t0 = (int64_t)b * ch, t1 = t0 + ch;
    // the sequences that this chunk has entries of
    int s0 = 0, s1 = 0;
    if (a.seq_offset) {
        s0 = b == 0 ? 0 : max(seq_at(a.seq_offset, a.S, t0, lane), 0);
        // the last chunk's go on to the end, also where offsets lie behind it: no entry keeps what was there
        s1 = b == (int)gridDim.x - 1 ? a.S : max(seq_at(a.seq_offset, a.S, t1, lane), s0);
    }
    auto range = [&](int s, int *lo, int *hi) {
        *lo = *hi = 0;
        if (s < a.S) seq_range(a.seq_offset, a.T, s, lo, hi);
        *lo = (int)max((int64_t)*lo, t0);
        *hi = (int)min((int64_t)*hi, t1);
    };
    // those with tokens here, each with one of its own
    __syncthreads();
    for (int s = s0 + (int)threadIdx.x; s <= s1; s += 256) {
        int lo, hi;
        range(s, &lo, &hi);
        const int i = lo < hi ? atomicAdd(&s_many, 1) : kMaxChunk;
        if (i < kMaxChunk)
            s_list[i] = s;
        else
            entry[2 * ((int64_t)b + s)] = s, entry[2 * ((int64_t)b + s) + 1] = 0;
    }
    __syncthreads();
    for (int i = 0; i < min(s_many, kMaxChunk); ++i) {
        const int s = s_list[i];
        int lo, hi;
        range(s, &lo, &hi);
        const int64_t at = (int64_t)b + s;
        __syncthreads();   // of the entry before
        for (int e = threadIdx.x; e < 64 * C; e += 256) s_c[e] = 0;
        __syncthreads();
        // this wave's tokens lo + wave + 4 i, those that count
        const int mine = lo + wave + 4 * lane;
        uint64_t live = __ballot(mine < hi && (!a.mask || a.mask[min(mine, hi - 1)] != 0));
        const int n = __popcll(live);
        float p[C], next[C];
        int next_id = -1;
#pragma unroll
        for (int c = 0; c < C; ++c) p[c] = 0.0f;
        auto ask = [&]() {   // the next token's logits and routes
            const int64_t t = lo + wave + 4 * __builtin_ctzll(live);
            load_experts<C, false>(a.logits + t * a.E, a.E, lane, next, -__builtin_huge_valf());
            next_id = lane < a.k ? a.idx[t * a.kp + lane] : -1;
        };
        if (live) ask();
        while (live) {
            float z[C];
#pragma unroll
            for (int c = 0; c < C; ++c) z[c] = next[c];
            const int e = next_id;
            live &= live - 1;
            if (live) ask();
            const float r = over(numerators<C>(z));
#pragma unroll
            for (int c = 0; c < C; ++c) p[c] = fmaf(z[c], r, p[c]);
            if (e >= 0 && e < a.E) atomicAdd(&s_c[e], 1);   // whole numbers: any order
        }
#pragma unroll
        for (int c = 0; c < C; ++c) s_p[wave][lane + 64 * c] = p[c];
        if (lane == 0) s_n[wave] = n;
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += 256) {
            prob[at * a.E + e] = (s_p[0][e] + s_p[1][e]) + (s_p[2][e] + s_p[3][e]);
            count[at * a.E + e] = s_c[e];
        }
        if (threadIdx.x == 0) entry[2 * at] = s, entry[2 * at + 1] = s_n[0] + s_n[1] + s_n[2] + s_n[3];
    }
}

// Workgroup (sequence, y): 32 experts at a time, 32 shares of the entries.
__global__ __launch_bounds__(1024) void k_balance_sequences(BalanceArgs a, int ch, int V, const int32_t *__restrict__ entry,
                                                            const int32_t *__restrict__ count,
                                                            const float *__restrict__ prob, double *part,
                                                            uint32_t *ticket)
{
    __shared__ uint32_t s_full[kMaxSeq / 32];   // sequences with counted tokens
    __shared__ int32_t s_n, s_some, s_last;
    __shared__ double s_p[16][32];
    __shared__ int32_t s_c[16][32];
    const int tid = threadIdx.x, seq = blockIdx.x;
    for (int i = tid; i < kMaxSeq / 32; i += 1024) s_full[i] = 0;
    if (tid == 0) s_n = 0, s_some = 0;
    __syncthreads();
    for (int v = tid; v < V; v += 1024) {
        const int s = entry[2 * v], n = entry[2 * v + 1];
        if (n <= 0 || (uint32_t)s >= (uint32_t)a.S) continue;
        atomicOr(&s_full[s / 32], 1u << (s & 31));
        if (s == seq) atomicAdd(&s_n, n);
    }
    __syncthreads();
    if (tid < kMaxSeq / 32 && s_full[tid]) atomicAdd(&s_some, __popc(s_full[tid]));
    int lo, hi;
    seq_range(a.seq_offset, a.T, seq, &lo, &hi);
    const int b0 = lo / ch, b1 = hi > lo ? (hi - 1) / ch + 1 : b0;   // the chunks that have tokens of it
    const int el = tid & 31, share = tid >> 5;
    double loss = 0.0;
    for (int eb = blockIdx.y; eb * 32 < a.E; eb += gridDim.y) {
        const int e = eb * 32 + el;
        double p = 0.0;
        int c = 0;
        if (e < a.E)
            for (int b = b0 + share; b < b1; b += 32) {
                const int64_t at = ((int64_t)b + seq) * a.E + e;
                p += (double)prob[at];
                c += count[at];
            }
        p += __shfl_xor(p, 32, 64);
        c += __shfl_xor(c, 32, 64);
        __syncthreads();
        if ((tid & 32) == 0) s_p[share / 2][el] = p, s_c[share / 2][el] = c;
        __syncthreads();
        if (tid >= 32) continue;
        p = 0.0;
        c = 0;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            p += s_p[q][el];
            c += s_c[q][el];
        }
        if (e < a.E) {
            const double n = s_n, some = s_some;
            const int64_t at = (int64_t)seq * a.E + e;
            const double per = n > 0.0 ? a.E / (a.k * n) : 0.0, mean = a.k * n / a.E;
            p = n > 0.0 ? p / n : 0.0;
            a.counts[at] = c;
            a.prob[at] = (float)p;
            a.slope[at] = n > 0.0 ? (float)(per / (n * some) * (c - mean)) : 0.0f;
            loss += some > 0.0 ? per / some * c * p : 0.0;
        }
    }
    const int blocks = gridDim.x * gridDim.y;
    if (tid < 32) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) loss += __shfl_xor(loss, o, 64);
        if (tid == 0) {
            part[seq * gridDim.y + blockIdx.y] = loss;
            // release: its part is there before it arrives; acquire: the last one to arrive sees all of them
            s_last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)blocks - 1;
        }
    }
    __syncthreads();
    if (!s_last || tid >= 64) return;
    loss = 0.0;
    for (int i = tid; i < blocks; i += 64) loss += part[i];
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) loss += __shfl_xor(loss, o, 64);
    if (tid == 0) *a.loss = (float)loss;
}

// dL = p (u - sum u p) with u = d_loss slope (counted tokens) and, for route
// weights that are not renormalised, their gradients; renormalised ones, a
// softmax over the chosen, add w (dw - sum w dw). A wave a token; lane j holds route j's
// id and gradient, which pass to the others through scalar registers. Bound by instructions
// issued: 65536 tokens of 256 experts, 8 routes, 35 us (its 136 MB take 27): 317 vector instructions a token, 64
// tokens a SIMD, 4 cycles each, are 34 us at 2.4 GHz. 41 with stores through the
// caches; then two tokens a wave with their loads together 43.6, four 46.6. Of 64 experts 24.5 us (173 a token), of 8
// with 2 routes 20.4 (143): a token takes a wave whatever E.
template <int C, bool V>
__global__ __launch_bounds__(256) void k_router_backward(RouterBackArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= a.T) return;
    float z[C], u[C], x[C];
    load_experts<C, V>(a.logits + t * a.E, a.E, lane, z, -__builtin_huge_valf());
    int id = -1;
    float dw = 0.0f;
    if (a.dw && lane < a.k) {
        id = a.idx[t * a.kp + lane];
        dw = a.dw[t * a.kp + lane];
        if ((uint32_t)id >= (uint32_t)a.E) id = -1, dw = 0.0f;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) u[c] = x[c] = 0.0f;
    if (a.slope) {   // all loads at once, the mask's too, but that of the sequence before its slope's
        const int on = a.mask ? a.mask[t] : 1;
        const float g = a.d_loss ? *a.d_loss : 1.0f;
        const int seq = a.seq_offset ? seq_at(a.seq_offset, a.S, t, lane) : 0;
        load_experts<C, V>(a.slope + (int64_t)min(max(seq, 0), a.S - 1) * a.E, a.E, lane, u, 0.0f);
        const bool counts = on != 0 && seq >= 0 && seq < a.S;
#pragma unroll
        for (int c = 0; c < C; ++c) u[c] = counts ? u[c] * g : 0.0f;
    }
    auto id_of = [&](int j) { return __builtin_amdgcn_readlane(id, j); };
    auto of = [&](float v, int j) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), j)); };
    if (a.dw && !a.renorm) {
        for (int j = 0; j < a.k; ++j) {
            const int e = id_of(j);
            const float v = of(dw, j);
#pragma unroll
            for (int q = 0; q < C; ++q)
                if (e == expert<C, V>(lane, q)) u[q] += v;
        }
    }
    // With nothing to pass on the row is 0 whatever its logits hold: padding may hold anything.
    bool mine = false;
#pragma unroll
    for (int c = 0; c < C; ++c) mine = mine || u[c] != 0.0f;
    const bool some = __any(mine), chosen = a.dw && a.renorm && __any(dw != 0.0f);
    float r = 0.0f, dot = 0.0f;
    if (some || chosen) r = over(numerators<C>(z));
    if (chosen) {
        float zj = 0.0f;   // lane j: the numerator of route j
        for (int j = 0; j < a.k; ++j) {
            const int e = id_of(j);
            if (e < 0) continue;
            float v = z[0];
#pragma unroll
            for (int q = 1; q < C; ++q)
                if (place_of<C, V>(e) == q) v = z[q];
            v = of(v, lane_of<C, V>(e));
            if (lane == j) zj = v;
        }
        const float rd = over(wave_sum(zj)), w = zj * rd;
        const float mean = wave_sum(w * dw), part = w * (dw - mean);
        for (int j = 0; j < a.k; ++j) {
            const int e = id_of(j);
            const float v = of(part, j);
#pragma unroll
            for (int q = 0; q < C; ++q)
                if (e == expert<C, V>(lane, q)) x[q] += v;
        }
    }
    if (some) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            z[c] *= r;
            dot = fmaf(u[c], z[c], dot);
        }
        dot = wave_sum(dot);
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) z[c] = 0.0f;
    }
    float *out = a.dlogits + t * a.E;
    if constexpr (V) {
        typename Row<C>::type w;
#pragma unroll
        for (int c = 0; c < C; ++c) w[c] = fmaf(z[c], u[c] - dot, x[c]);
        if (lane * C < a.E) __builtin_nontemporal_store(w, (typename Row<C>::type *)(out + lane * C));
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (lane + 64 * c < a.E) __builtin_nontemporal_store(fmaf(z[c], u[c] - dot, x[c]), out + lane + 64 * c);
    }
}

}  // namespace

static bool wide(const CombineArgs &a, bool back)
{
    return a.c_bf16 && a.d % 8 == 0 && a.ldc % 8 == 0 && ((uintptr_t)a.C & 15) == 0 &&
           (!back || !a.dC || (a.lddc % 8 == 0 && ((uintptr_t)a.dC & 15) == 0));
}
// threads for n of them: whole waves, 256 at most
static int threads_for(int n) { return n >= 256 ? 256 : (n + 63) / 64 * 64; }

hipError_t launch_combine_rows(const CombineArgs &a, hipStream_t st)
{
    if (a.T == 0) return hipSuccess;
    const int v = wide(a, false) ? 8 : 4, threads = threads_for((a.d + v - 1) / v);
    const int bx = (a.d + threads * v - 1) / (threads * v);
    const dim3 grid((unsigned)((int64_t)a.T * bx));
    if (v == 8)
        hipLaunchKernelGGL((k_combine_rows<true, 8>), grid, dim3(threads), 0, st, a, bx);
    else if (a.c_bf16)
        hipLaunchKernelGGL((k_combine_rows<true, 4>), grid, dim3(threads), 0, st, a, bx);
    else
        hipLaunchKernelGGL((k_combine_rows<false, 4>), grid, dim3(threads), 0, st, a, bx);
    return hipGetLastError();
}

hipError_t launch_combine_rows_backward(const CombineArgs &a, hipStream_t st)
{
    if (a.T == 0) return hipSuccess;
    const int v = wide(a, true) ? 8 : 4, threads = threads_for((a.d + v - 1) / v);
    const dim3 grid((unsigned)a.T);
    if (v == 8)
        hipLaunchKernelGGL((k_combine_rows_backward<true, 8>), grid, dim3(threads), 0, st, a);
    else if (a.c_bf16)
        hipLaunchKernelGGL((k_combine_rows_backward<true, 4>), grid, dim3(threads), 0, st, a);
    else
        hipLaunchKernelGGL((k_combine_rows_backward<false, 4>), grid, dim3(threads), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_balance(const BalanceArgs &a, const BalanceLayout &w, void *ws, hipStream_t st)
{
    char *p = (char *)ws;
    int32_t *entry = (int32_t *)(p + w.entry), *count = (int32_t *)(p + w.count);
    float *prob = (float *)(p + w.prob);
    uint32_t *ticket = (uint32_t *)(p + w.ticket);
    const auto kernel = a.E <= 64 ? k_balance_chunks<1> : a.E <= 128 ? k_balance_chunks<2> : k_balance_chunks<4>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)w.chunks), dim3(256), 0, st, a, w.ch, entry, count, prob, ticket);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // the experts over several workgroups where sequences are few and long
    const unsigned y = a.S >= 256 ? 1 : (unsigned)((a.E + 31) / 32);
    hipLaunchKernelGGL(k_balance_sequences, dim3((unsigned)a.S, y), dim3(1024), 0, st, a, w.ch, a.seq_offset ? w.V : w.chunks,
                       entry, count, prob, (double *)(p + w.part), ticket);
    return hipGetLastError();
}

// Whether every row of E fp32 values of these arrays can be read C values at a time
// (65536 rows of 256 backward: 3 of 44 us; the forward pass gains nothing by it).
static bool together(int E, int C, std::initializer_list<const void *> rows)
{
    bool yes = E % C == 0;
    for (const void *p : rows) yes = yes && ((uintptr_t)p & (4 * C - 1)) == 0;
    return yes;
}

hipError_t launch_router_backward(const RouterBackArgs &a, hipStream_t st)
{
    if (a.T == 0) return hipSuccess;
    const dim3 grid((unsigned)(((int64_t)a.T + 3) / 4));
    const auto kernel =
        a.E <= 64 ? k_router_backward<1, false>
        : a.E <= 128 ? (together(a.E, 2, {a.logits, a.slope, a.dlogits}) ? k_router_backward<2, true> : k_router_backward<2, false>)
                     : (together(a.E, 4, {a.logits, a.slope, a.dlogits}) ? k_router_backward<4, true> : k_router_backward<4, false>);
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace moe
