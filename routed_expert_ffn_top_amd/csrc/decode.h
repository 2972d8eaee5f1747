// Internal declarations of the few-token layer (moe_layer_decode).
#pragma once

#include "common.h"

namespace moe {

constexpr int kDecMaxT = MOE_DECODE_MAX_T;             // a slot has at most this many rows
constexpr int kDecMaxRoutes = MOE_DECODE_MAX_ROUTES;   // T * K'

constexpr int kDecRows = 64;                           // output columns per workgroup (one counter each)
constexpr int kDecMaxD = MOE_DECODE_MAX_D;
constexpr int kDecTokBlock = 4;                        // tokens per route workgroup
constexpr int kDecSelfRoutes = 256;                    // at most, where gate/up routes for itself

// The routes sorted by slot, at most rpe to an entry: entry a < *n_act is a slot
// and up to rpe of its routes, rec[off .. off + cnt).
constexpr int kDecMaxEntries = kMaxExp + kDecMaxRoutes / 5;
int dec_rpe(const moe_shape &s);   // 5, 16 or 32
inline int dec_entries(const moe_shape &s)   // at most this many
{
    const int R = s.T * (s.k + s.n_shared), ne = s.E + s.n_shared;
    const int e = ne + R / dec_rpe(s);
    return e < R ? e : R;
}

// Byte offsets of the decode workspace's regions. The counters stand first and
// have one size, so that they stay where they are when the shape changes: they
// are zero between calls (cleared once by moe_decode_workspace_init; the last
// workgroup to arrive at a counter clears it).
struct DecLayout {
    size_t ctr;      // int32: [0] token blocks routed, then per token block, then per column chunk of the output
    size_t logits;   // float[T][E]
    size_t list;     // int32: [0] slots with routes, then the DecLists arrays
    size_t H;        // fp32 layers: float[R][f]; bf16 layers: uint16[3][R][f], H as a sum of three bf16 terms
    size_t Yr;       // float[R][d], alpha times each route's output row
    size_t total;
};

inline DecLayout dec_layout(const moe_shape &s)
{
    DecLayout w{};
    const size_t R = (size_t)s.T * (s.k + s.n_shared);
    size_t o = 0;
    w.ctr = o;    o = align_up(o + (size_t)(1 + kDecMaxT + kDecMaxD / kDecRows) * 4, 256);
    w.logits = o; o = align_up(o + (size_t)s.T * s.E * 4, 256);
    w.list = o;   o = align_up(o + (size_t)(1 + 3 * kDecMaxEntries + kDecMaxRoutes) * 4, 256);
    w.H = o;      o = align_up(o + R * s.f * (act_bf16(s) ? 6 : 4), 256);
    w.Yr = o;     o = align_up(o + R * s.d * 4, 256);
    w.total = o;
    return w;
}

struct DecLists {
    int32_t *n_act, *slot, *off, *cnt, *rec;
};

struct DecArgs {
    DecLists l;
    const void *X;        // gate/up: activations; down: H
    int64_t ldx;
    const char *W;        // plane base
    int64_t slot_bytes;   // bytes between slots
    int64_t scale_off;    // fp8: bytes from a slice's start to its row scales
    int64_t slice_bytes;  // of one slice, below 2^31
    int N, K, kp, R, nchunk, entries, rpe;
    void *out;            // gate/up: H; down: Yr
    int64_t ldo;
    const float *topk_w;
    float *Y;             // down: the tokens' rows, their routes' sums added
    int64_t ldy;
    int T;
    int32_t *ctr;         // down: arrivals per chunk
};

struct DecRouteArgs {
    const void *X;
    int64_t ldx;
    const float *Wr, *bias;   // Wr null: logits holds the caller's
    const float *given;
    float *logits;
    int T, d, E, k, n_shared, renorm, rpe;
    int sort;                 // the route launch sorts the routes by slot too
    int32_t *idx;
    float *w;
    int32_t *ctr;
    DecLists l;
};

// Whether gate/up does all of the routing, or its last part, the sorting by slot,
// itself (launch_dec_route_proj, with `route` for the first, instead of
// launch_dec_proj).
bool dec_self_routes(const moe_shape &s, bool router);
bool dec_gate_up_sorts(const moe_shape &s, bool router);
hipError_t launch_dec_route_proj(const moe_shape &s, const DecArgs &a, const DecRouteArgs &q, const PhiArg &phi, bool route,
                                 hipStream_t st);
hipError_t launch_dec_route(const moe_shape &s, const DecRouteArgs &a, const PhiArg &phi, hipStream_t st);
hipError_t launch_dec_proj(const moe_shape &s, const DecArgs &a, bool gateup, hipStream_t st);

}  // namespace moe
