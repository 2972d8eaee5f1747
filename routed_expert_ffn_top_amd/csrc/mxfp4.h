// Internal declarations of the MXFP4 operators (quantise, read back, product).
#pragma once

#include "common.h"

namespace moe {

hipError_t launch_quantize_mxfp4(const void *src, bool bf16, int64_t rows, int K, int64_t ld, uint8_t *codes,
                                 uint8_t *scales, hipStream_t st);
hipError_t launch_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, int64_t rows, int K, void *dst,
                                   bool bf16, int64_t ld, hipStream_t st);

// C[p] = A[row_index ? row_index[p] : p] . B_slot^T for the records p of each
// slot, [slot_offset[s], slot_offset[s+1]) or [0, M) of the one slice.
struct MxArgs {
    const uint8_t *A, *As;       // codes [A_rows][K/2], scale bytes [A_rows][K/32]
    int A_rows;
    const int32_t *row_index;    // or null
    const int32_t *slot_offset;  // [P+1] or null (P == 1)
    int P;
    const uint8_t *B;            // packed slices [N][K]
    int64_t B_stride;            // bytes
    int M, N, K;
    void *C;
    int c_bf16;
    int64_t ldc;
    // the expert FFN's projections only
    uint8_t *Hs;                 // gate/up: scale bytes [M][N/64] of H, whose codes [M][N/4] are C
    const int32_t *rec_route;    // down: route of a record; C is Yr, fp32 [splits][routes][ldc]
    const float *topk_w;
    int32_t *done;
    int splits;                  // partial rows a route has: the first holds the result, the others zeros
    int64_t split_stride;
};
hipError_t launch_matmul_mxfp4(const MxArgs &a, hipStream_t st);
// The expert FFN's projections on MXFP4 activations, over a route build:
// gate/up with SwiGLU and the quantisation of H, and down with the route
// weights, a row of C per route.
hipError_t launch_gate_up_mxfp4(const MxArgs &a, hipStream_t st);
hipError_t launch_down_mxfp4(const MxArgs &a, hipStream_t st);

}  // namespace moe
