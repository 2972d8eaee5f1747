// Internal declarations: the combine of record rows with its gradients, the
// balance loss and the gradient of the router's logits.
#pragma once

#include <algorithm>

#include "common.h"

namespace moe {

struct CombineArgs {
    int T, d, kp, M;
    const void *C;               // rows in record order [M][ldc], bf16 or fp32
    int c_bf16;
    int64_t ldc;
    const int32_t *route_pos;    // [T*kp]: record of a route, or outside [0, M)
    const float *topk_w;         // [T*kp]
    float *Y;                    // forward: [T][ldy], in place
    const float *dY;             // backward
    int64_t ldy;
    void *dC;                    // backward: rows as C's, or null
    int64_t lddc;
    float *dw;                   // backward: [T*kp]
};
hipError_t launch_combine_rows(const CombineArgs &a, hipStream_t st);
hipError_t launch_combine_rows_backward(const CombineArgs &a, hipStream_t st);

constexpr int kMaxSeq = 4096;    // sequences of a balance call
constexpr int kMaxChunk = 256;   // tokens of a chunk of it, 64 a wave

struct BalanceArgs {
    int T, E, k, kp;
    const float *logits;         // [T][E]
    const int32_t *idx;          // [T][kp]
    const int32_t *seq_offset;   // [S+1] or null (S == 1: every token)
    int S;
    const uint8_t *mask;         // [T] or null
    float *loss;                 // [1]
    int32_t *counts;             // [S][E]
    float *prob, *slope;         // [S][E]
};
struct BalanceLayout {
    size_t entry;   // int32[V][2]: sequence, tokens counted
    size_t count;   // int32[V][E]
    size_t prob;    // float[V][E]
    size_t part;    // double[S][ceil(E/32)]
    size_t ticket;  // uint32
    size_t total;
    int ch, chunks, V;
};
// Tokens a chunk: what a workgroup sums, 4 waves of its tokens each, at most 64 a wave.
// Up to 16384 tokens 16, whose chunks are done soonest; then 64, and as many more as keep 1024 chunks, which
// fill the GPU, where more of them lengthen the sums over them. Both steps on 256 experts: 16384 tokens 21.1 us
// with 16, 16385 20.2 with 64 and 21.2 with 20; 65537 30.5 with 68, 41.6 with 256; 131072
// 45.8 with 128, 54.5 with 256. A chunk has an entry for each
// sequence that it meets, one of them the one behind the last: V at most.
inline BalanceLayout balance_layout(int64_t T, int E, int S)
{
    BalanceLayout w{};
    w.ch = T <= 16384 ? 16 : (int)std::min<int64_t>(std::max<int64_t>((T + 4095) / 4096 * 4, 64), kMaxChunk);
    w.chunks = (int)std::max<int64_t>((T + w.ch - 1) / w.ch, 1);
    w.V = w.chunks + S;
    size_t o = 0;
    w.entry = o;  o = align_up(o + (size_t)w.V * 8, 256);
    w.count = o;  o = align_up(o + (size_t)w.V * E * 4, 256);
    w.prob = o;   o = align_up(o + (size_t)w.V * E * 4, 256);
    w.part = o;   o = align_up(o + (size_t)S * ((E + 31) / 32) * 8, 256);
    w.ticket = o; o = align_up(o + 4, 256);
    w.total = o;
    return w;
}
hipError_t launch_balance(const BalanceArgs &a, const BalanceLayout &w, void *ws, hipStream_t st);

struct RouterBackArgs {
    int T, E, k, kp, renorm;
    const float *logits;
    const int32_t *idx;
    const int32_t *seq_offset;
    int S;
    const uint8_t *mask;
    const float *slope;          // [S][E] or null
    const float *d_loss;         // [1] or null (1)
    const float *dw;             // [T][kp] or null
    float *dlogits;              // [T][E]
};
hipError_t launch_router_backward(const RouterBackArgs &a, hipStream_t st);

}  // namespace moe
