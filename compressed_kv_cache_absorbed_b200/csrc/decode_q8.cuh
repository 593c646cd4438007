// Absorbed attention over the 8-bit paged latent cache (E4M3 codes, one scale per page).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"

namespace mla {
namespace q8 {

struct Problem {
    int H, B, q_len;            // heads (<= 128), sequences, new tokens per sequence
    const uint8_t* codes;       // [num_pages, 64, 576]
    const float* scales;        // [num_pages]
    long long num_pages;
    const int32_t* block_table; // [B, max_blocks]
    const int32_t* seq_lens;    // [B]
    int max_blocks;
    float scale;                // softmax scale
};

// Split-KV attention on CUDA cores: part_o [ns, B q_len, H, 512] unnormalised, part_ml
// [ns, B q_len, H, 2] (running max of the scaled scores, sum), fp32.
cudaError_t decode_split(const Problem& p, const float* q_lat, const __nv_bfloat16* q_rope, int ns, float* part_o,
                         float* part_ml, DevErr err, cudaStream_t s);

}  // namespace q8
}  // namespace mla
