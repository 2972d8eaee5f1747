// Internal declarations of the operators on fp8 blocks of 128 (quantise, read
// back, products).
#pragma once

#include "common.h"

namespace moe {

constexpr int kFp8Block = 128;

// Bytes between the scale rows of quantised rows of K values: a byte for each
// block, in whole 16-byte pieces.
__host__ __device__ inline int64_t fp8_scale_bytes(int64_t K) { return (K + 2047) / 2048 * 16; }
inline int64_t fp8_blocks(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }

// block_rows 1: a scale byte for each 128 of a row; 128: an fp32 scale for each 128 x 128.
hipError_t launch_quantize_fp8(const void *src, bool bf16, int64_t rows, int K, int64_t ld, int block_rows,
                               uint8_t *codes, void *scales, hipStream_t st);
hipError_t launch_dequantize_fp8(const uint8_t *codes, const void *scales, int64_t rows, int K, int block_rows,
                                 void *dst, bool bf16, int64_t ld, hipStream_t st);

// C[p] = A[row_index ? row_index[p] : p] . B_slot^T for the records p of each
// slot, [slot_offset[s], slot_offset[s+1]) or [0, M) of the one slice.
struct Fp8Args {
    const uint8_t *A, *As;       // codes [A_rows][K], scale bytes [A_rows][fp8_scale_bytes(K)]
    int A_rows;
    const int32_t *row_index;    // or null
    const int32_t *slot_offset;  // [P+1] or null (P == 1)
    int P;
    const uint8_t *B[2];         // codes [N][K] of a slice; gate and up for the SwiGLU product
    const float *Bs[2];          // scales [ceil(N/128)][ceil(K/128)]
    int64_t B_stride, Bs_stride; // bytes, floats from a slice to the next
    int M, N, K;                 // N: rows of a slice (the SwiGLU product: of each of the two)
    void *C;                     // the SwiGLU product: codes of H [M][N]
    int c_bf16;
    int64_t ldc;
    uint8_t *Hs;                 // the SwiGLU product: scale bytes of H [M][fp8_scale_bytes(N)]
};
hipError_t launch_matmul_fp8(const Fp8Args &a, hipStream_t st);
// Bytes of workspace the SwiGLU product takes (few records a slot: h in fp32).
size_t gate_up_fp8_workspace(const Fp8Args &a);
hipError_t launch_gate_up_fp8(const Fp8Args &a, void *ws, hipStream_t st);

}  // namespace moe
