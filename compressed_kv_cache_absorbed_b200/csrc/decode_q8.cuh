// Absorbed attention over the 8-bit paged latent cache (E4M3 codes, one scale per page).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.cuh"

namespace mla {
namespace q8 {

// How the rows (new token t, head h) of a sequence, r = t H + h, are cut into groups of R
// rows, and how many CTAs walk one sequence's tiles side by side.
struct Shape {
    int B, q_len, H;
    int R;        // rows per group: 16 or 32
    int G;        // groups per sequence
    int sib;      // > 1: the G groups of a sequence are walked by G neighbouring CTAs; 1: one after another
    int ctas;     // CTAs of the attention kernel
};

Shape make_shape(int B, int q_len, int H, int num_sms);

struct Ws {
    uint8_t* q_img;     // [B G][2 R rows x 576]: the queries as 8-bit operands
    float* q_scale;     // [B G][R]
    __half* part_o;     // [slots][R][512] partial outputs, each row in units of its own
    float4* part_ml;    // [slots][R] (reference, sum, unit of the output, -)
    int4* start;        // [ctas]: where each range of the work split starts
    int2* pieces;       // [B G]: slots and number of each item's partials
    size_t bytes;
};

Ws carve(char* base, const Shape& s);

struct Problem {
    const __nv_bfloat16 *q_nope, *q_rope;   // [B q_len, H, 128], [B q_len, H, 64]
    const __nv_bfloat16 *W_UKT, *W_UV;      // [H, 512, 128], [H, 128, 512]
    const uint8_t* codes;                   // [num_pages, 64, 576]
    const float* scales;                    // [num_pages]
    long long num_pages;
    const int32_t* block_table;             // [B, max_blocks]
    const int32_t* seq_lens;                // [B]
    int max_blocks;
    float scale;                            // softmax scale
    __nv_bfloat16* out;                     // [B q_len, H, 128]
};

cudaError_t decode(const Problem& p, const Shape& s, const Ws& ws, DevErr err, cudaStream_t st);

cudaError_t set_wait_limit_decode_q8(uint32_t polls);
cudaError_t set_starve_decode_q8(int on);

}  // namespace q8
}  // namespace mla
