// What stands behind an expert's products in record order and what trains the
// router: the records' rows summed into their tokens and the gradients of that
// sum, the load-balancing loss of a routing, and the gradient of the router's
// logits.
#include "device.h"
#include "train.h"

namespace moe {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

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
        *(f32x4_t *)((float *)C + at) = f32x4_t{v[0], v[1], v[2], v[3]};
    } else if constexpr (V == 8) {
        *(u32x4_t *)((uint16_t *)C + at) = u32x4_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
    } else {
        *(u32x2_t *)((uint16_t *)C + at) = u32x2_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    }
}

constexpr int kRoutes = 8;   // routes whose rows are asked for together

// Y[t] += sum over the token's routes, ascending, of weight times row: one
// fused multiply-add each, in fp32. Bound by HBM: every row read once.
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
// thread's columns ascending, then over the lanes and the waves in a fixed order.
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
// its mean, which the differences there do not lose in rounding.
//
// Three steps: chunks of up to w.ch tokens of one sequence, a workgroup each
// (sums of at most w.ch / 4 terms a wave in fp32, then 4 waves); the chunks of
// a sequence, 32 experts a workgroup, in fp64; the last of those workgroups
// sums the loss. Every sum is in a fixed order.

// Softmax numerators of a token's logits, C a lane (expert lane + 64 c), and their sum.
template <int C>
__device__ __forceinline__ float numerators(const float *L, int E, int lane, float (&z)[C])
{
    const float none = -__builtin_huge_valf();
    float v[C], m = none, s = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = lane + 64 * c;
        v[c] = e < E ? L[e] : none;
        if (v[c] != v[c]) v[c] = none;
        m = fmaxf(m, v[c]);
    }
    m = wave_max(m);
    if (m == none) m = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        z[c] = expf(v[c] - m);
        s += z[c];
    }
    return wave_sum(s);
}

__device__ __forceinline__ void seq_range(const int32_t *off, int T, int s, int *lo, int *hi)
{
    *lo = off ? min(max(off[s], 0), T) : 0;
    *hi = off ? min(max(off[s + 1], *lo), T) : T;
}

template <int C>
__global__ __launch_bounds__(256) void k_balance_chunks(BalanceArgs a, int ch, int32_t *__restrict__ chunk,
                                                        int32_t *__restrict__ count, float *__restrict__ prob,
                                                        uint32_t *__restrict__ ticket)
{
    __shared__ float s_p[4][64 * C];
    __shared__ int32_t s_c[64 * C], s_n[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, b = blockIdx.x;
    if (b == 0 && threadIdx.x == 0) *ticket = 0;   // for the next kernel
    // the sequence whose chunk this is
    int run = 0, seq = -1, t0 = 0, t1 = 0;
    for (int q = 0; q < a.S && seq < 0; q += 64) {
        int lo = 0, hi = 0;
        if (q + lane < a.S) seq_range(a.seq_offset, a.T, q + lane, &lo, &hi);
        const int n = (hi - lo + ch - 1) / ch, inc = run + wave_incl_scan(n, lane);
        const uint64_t mine = __ballot(b < inc && b >= inc - n);
        if (mine) {
            const int l = __builtin_ctzll(mine);
            seq = q + l;
            t0 = __builtin_amdgcn_readlane(lo, l) + (b - (__builtin_amdgcn_readlane(inc, l) - __builtin_amdgcn_readlane(n, l))) * ch;
            t1 = min(t0 + ch, __builtin_amdgcn_readlane(hi, l));
        }
        run = __builtin_amdgcn_readlane(inc, 63);
    }
    if (seq < 0) {
        if (threadIdx.x == 0) chunk[2 * b] = -1, chunk[2 * b + 1] = 0;
        return;
    }
    for (int e = threadIdx.x; e < 64 * C; e += 256) s_c[e] = 0;
    __syncthreads();
    float p[C];
#pragma unroll
    for (int c = 0; c < C; ++c) p[c] = 0.0f;
    int n = 0;
    for (int t = t0 + wave; t < t1; t += 4) {
        if (a.mask && a.mask[t] == 0) continue;
        ++n;
        float z[C];
        const float s = numerators<C>(a.logits + (int64_t)t * a.E, a.E, lane, z);
        const float r = s > 0.0f || s != s ? 1.0f / s : 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) p[c] = fmaf(z[c], r, p[c]);
        if (lane < a.k) {
            const int e = a.idx[(int64_t)t * a.kp + lane];
            if (e >= 0 && e < a.E) atomicAdd(&s_c[e], 1);   // whole numbers: any order
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) s_p[wave][lane + 64 * c] = p[c];
    if (lane == 0) s_n[wave] = n;
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += 256) {
        prob[(int64_t)b * a.E + e] = (s_p[0][e] + s_p[1][e]) + (s_p[2][e] + s_p[3][e]);
        count[(int64_t)b * a.E + e] = s_c[e];
    }
    if (threadIdx.x == 0) chunk[2 * b] = seq, chunk[2 * b + 1] = s_n[0] + s_n[1] + s_n[2] + s_n[3];
}

// Workgroup (sequence, 32 experts): 32 lanes of experts x 32 shares of the chunks.
__global__ __launch_bounds__(1024) void k_balance_sequences(BalanceArgs a, int V, const int32_t *__restrict__ chunk,
                                                            const int32_t *__restrict__ count,
                                                            const float *__restrict__ prob, double *part,
                                                            uint32_t *ticket)
{
    __shared__ uint32_t s_full[kMaxSeq / 32];   // sequences with counted tokens
    __shared__ int32_t s_lo, s_hi, s_n, s_some, s_last;
    __shared__ double s_p[32][33];
    __shared__ int32_t s_c[32][33];
    const int tid = threadIdx.x, seq = blockIdx.x, eb = blockIdx.y;
    for (int i = tid; i < kMaxSeq / 32; i += 1024) s_full[i] = 0;
    if (tid == 0) s_lo = V, s_hi = 0, s_n = 0, s_some = 0;
    __syncthreads();
    for (int v = tid; v < V; v += 1024) {
        const int s = chunk[2 * v], n = chunk[2 * v + 1];
        if (s < 0) continue;
        if (n > 0) atomicOr(&s_full[s / 32], 1u << (s & 31));
        if (s == seq) {
            atomicMin(&s_lo, v);
            atomicMax(&s_hi, v + 1);
            atomicAdd(&s_n, n);
        }
    }
    __syncthreads();
    if (tid < kMaxSeq / 32 && s_full[tid]) atomicAdd(&s_some, __popc(s_full[tid]));
    const int el = tid & 31, share = tid >> 5, e = eb * 32 + el;
    double p = 0.0;
    int c = 0;
    if (e < a.E)
        for (int v = s_lo + share; v < s_hi; v += 32) {
            p += (double)prob[(int64_t)v * a.E + e];
            c += count[(int64_t)v * a.E + e];
        }
    s_p[share][el] = p;
    s_c[share][el] = c;
    __syncthreads();
    const double n = s_n, some = s_some;
    if (tid < 32) {
        p = 0.0;
        c = 0;
        for (int q = 0; q < 32; ++q) {
            p += s_p[q][el];
            c += s_c[q][el];
        }
        double l = 0.0;
        if (e < a.E) {
            const int64_t at = (int64_t)seq * a.E + e;
            const double per = n > 0.0 ? a.E / (a.k * n) : 0.0, mean = a.k * n / a.E;
            p = n > 0.0 ? p / n : 0.0;
            a.counts[at] = c;
            a.prob[at] = (float)p;
            a.slope[at] = n > 0.0 ? (float)(per / (n * some) * (c - mean)) : 0.0f;
            l = some > 0.0 ? per / some * c * p : 0.0;
        }
        s_p[0][el] = l;   // the same wave's
    }
    __syncthreads();
    const int blocks = gridDim.x * gridDim.y;
    if (tid == 0) {
        double l = 0.0;
        for (int q = 0; q < 32; ++q) l += s_p[0][q];
        __hip_atomic_store(&part[seq * gridDim.y + eb], l, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)blocks - 1;
    }
    __syncthreads();
    if (!s_last) return;
    double l = 0.0;
    for (int i = tid; i < blocks; i += 1024) l += __hip_atomic_load(&part[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    s_p[tid >> 5][tid & 31] = l;
    __syncthreads();
    if (tid == 0) {
        l = 0.0;
        for (int i = 0; i < 1024; ++i) l += s_p[i >> 5][i & 31];
        *a.loss = (float)l;
    }
}

// dL = p (u - sum u p) with u = d_loss slope (counted tokens) and, for route
// weights that are not renormalised, their gradients; renormalised ones, a
// softmax over the chosen, add w (dw - sum w dw). A wave a token.
template <int C>
__global__ __launch_bounds__(256) void k_router_backward(RouterBackArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= a.T) return;
    float z[C], u[C], x[C];
    const float s = numerators<C>(a.logits + t * a.E, a.E, lane, z);
    const float r = s > 0.0f || s != s ? 1.0f / s : 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) u[c] = x[c] = 0.0f;
    if (a.slope && (!a.mask || a.mask[t] != 0)) {
        int seq = 0;
        bool in = true;
        if (a.seq_offset) {   // the last sequence that starts at or before t, 64 offsets at a time
            int first = 0, many = a.S + 1, step = 1;
            while (step * 64 < many) step *= 64;
            for (;; step /= 64) {
                const int i = first + lane * step;
                const bool le = i <= a.S && a.seq_offset[min(i, a.S)] <= t;
                const int n = __popcll(__ballot(le));
                if (n == 0) {
                    in = false;
                    break;
                }
                first += (n - 1) * step;
                if (step == 1) break;
            }
            seq = first;
            in = in && seq < a.S;
        }
        if (in) {
            const float g = a.d_loss ? *a.d_loss : 1.0f;
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (lane + 64 * c < a.E) u[c] = g * a.slope[(int64_t)seq * a.E + lane + 64 * c];
        }
    }
    if (a.dw) {
        const int32_t *id = a.idx + t * a.kp;
        const float *dw = a.dw + t * a.kp;
        if (a.renorm) {
            // sums over the routes: lane j holds route j's
            float zj = 0.0f, den = 0.0f, dot = 0.0f;
            for (int j = 0; j < a.k; ++j) {
                const int e = id[j];
                const int c = e >> 6;
                float v = 0.0f;
#pragma unroll
                for (int q = 0; q < C; ++q)
                    if (q == c) v = z[q];
                v = e >= 0 && e < a.E ? __shfl(v, e & 63, 64) : 0.0f;
                den += v;
                dot = fmaf(v, dw[j], dot);
                if (lane == j) zj = v;
            }
            const float rd = den > 0.0f || den != den ? 1.0f / den : 0.0f;
            const float mine = lane < a.k ? zj * rd * (dw[lane] - dot * rd) : 0.0f;
            for (int j = 0; j < a.k; ++j) {
                const float v = __shfl(mine, j, 64);
                const int e = id[j];
#pragma unroll
                for (int q = 0; q < C; ++q)
                    if (e == lane + 64 * q) x[q] += v;
            }
        } else {
            for (int j = 0; j < a.k; ++j)
#pragma unroll
                for (int q = 0; q < C; ++q)
                    if (id[j] == lane + 64 * q && id[j] < a.E) u[q] += dw[j];
        }
    }
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) dot = fmaf(u[c], z[c] * r, dot);
    dot = wave_sum(dot);
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (lane + 64 * c < a.E) a.dlogits[t * a.E + lane + 64 * c] = fmaf(z[c] * r, u[c] - dot, x[c]);
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
    int32_t *chunk = (int32_t *)(p + w.chunk), *count = (int32_t *)(p + w.count);
    float *prob = (float *)(p + w.prob);
    uint32_t *ticket = (uint32_t *)(p + w.ticket);
    const auto kernel = a.E <= 64 ? k_balance_chunks<1> : a.E <= 128 ? k_balance_chunks<2> : k_balance_chunks<4>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)w.V), dim3(256), 0, st, a, w.ch, chunk, count, prob, ticket);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_balance_sequences, dim3((unsigned)a.S, (unsigned)((a.E + 31) / 32)), dim3(1024), 0, st, a, w.V, chunk,
                       count, prob, (double *)(p + w.part), ticket);
    return hipGetLastError();
}

hipError_t launch_router_backward(const RouterBackArgs &a, hipStream_t st)
{
    if (a.T == 0) return hipSuccess;
    const dim3 grid((unsigned)(((int64_t)a.T + 3) / 4));
    const auto kernel = a.E <= 64 ? k_router_backward<1> : a.E <= 128 ? k_router_backward<2> : k_router_backward<4>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace moe
