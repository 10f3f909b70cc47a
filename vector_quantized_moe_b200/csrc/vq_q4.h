// Arguments of the dense 4-bit kernels (vq_q4.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace vq {

struct Q4Args {
    const uint32_t *words[2];    // tile layout; [1]: the up module of a pair
    const uint16_t *scales[2];
    const uint16_t *biases[2];
    const uint16_t *x;           // [T, cols] bf16
    void *y;                     // [T, rows]
    int64_t x_ld, y_ld;
    int rows, cols, T;
    int tiles, nsb;              // 16-row tiles, 128-column tiles
    int pair, y_dtype;
};

cudaError_t launch_q4_gemv(const Q4Args &a, int group, cudaStream_t s);
cudaError_t launch_q4_pack(const uint32_t *codes, const uint16_t *scales, const uint16_t *biases, int rows, int cols,
                           int group, uint32_t *words_out, uint16_t *scales_out, uint16_t *biases_out, cudaStream_t s);

}  // namespace vq
