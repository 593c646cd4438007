// Appending given latents and rotary keys to a paged cache, in the storage type or as 8-bit
// codes with one scale per page.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace mla {

constexpr int kMaxRopePairs = 128;

// theta^(-2i / d_hR) of every pair, computed once on the host (kernel argument)
struct RopeFreqs {
    double f[kMaxRopePairs];
};

struct AppendPaged {
    const void* c;             // rows of d_c values, ld_c elements apart
    const void* k_r;           // rows of d_hR values, ld_kr elements apart (not rotated)
    long long ld_c, ld_kr;
    const int32_t* new_offsets;   // [B + 1]
    const int32_t* seq_lens;      // [B], after the append
    const int32_t* pos;           // [n] rotation positions, or null: the token's place in its sequence
    const int32_t* block_table;   // [B, max_blocks]
    int B, n, max_blocks;
    long long num_pages;
    int d_c, d_hR;
};

// cache [num_pages, 64, d_c + d_hR] in the storage type T (float or bf16)
template <typename T>
cudaError_t append_paged(const AppendPaged& a, float theta, T* cache, DevErr err, cudaStream_t s);

// codes [num_pages, 64, 576] E4M3, scales [num_pages] fp32; d_c = 512, d_hR = 64, bf16 inputs
cudaError_t append_paged_q8(const AppendPaged& a, float theta, uint8_t* codes, float* scales, DevErr err,
                            cudaStream_t s);

}  // namespace mla
