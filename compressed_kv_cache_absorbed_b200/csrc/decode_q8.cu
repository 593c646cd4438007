// Absorbed attention over the 8-bit paged latent cache.
//
// For query token v = (b, t), head h, cached token j (value row = code row * scale of its page):
//     s_j = scale ([q_lat | q_rope][v, h] . row_j),   o_lat[v, h] = sum_j softmax(s)_j row_j[0:512]
// over the first seq_lens[b] - q_len + t + 1 tokens of sequence b.
//
// CUDA-core form: a warp owns one head of one query token and walks a range of tokens in
// groups of 32 staged in shared memory, with a running maximum and sum.
#include <cuda_fp16.h>
#include <math.h>

#include "decode_q8.cuh"
#include "paged_plan.h"

namespace mla {
namespace q8 {

namespace {

constexpr int kDc = 512, kRow = 576;
constexpr int kGroup = 32, kWarps = 8;

__global__ void __launch_bounds__(32 * kWarps)
decode_split_kernel(const Problem p, const float* __restrict__ q_lat, const __nv_bfloat16* __restrict__ q_rope, int ns,
                    float* __restrict__ part_o, float* __restrict__ part_ml, DevErr err) {
    extern __shared__ float sm[];
    constexpr int ld = kRow + 1;
    float* tile = sm;                // [kGroup][ld] values
    float* qs = sm + kGroup * ld;    // [kWarps][kRow]
    const int v = blockIdx.x, split = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = v / p.q_len, t = v % p.q_len, h = blockIdx.z * kWarps + warp, NV = p.B * p.q_len;
    int len = p.seq_lens[b];
    if (len < 0 || (long long)len > (long long)p.max_blocks * kPageRows) {
        if (threadIdx.x == 0) latch(err, kErrOutOfRange, b);
        len = 0;
    }
    const int keys = max(0, len - (p.q_len - 1 - t));
    const int chunk = (keys + ns - 1) / ns;
    const int j0 = min(keys, split * chunk), j1 = min(keys, j0 + chunk);
    for (int i = threadIdx.x; i < kWarps * kRow; i += blockDim.x) {
        const int hh = blockIdx.z * kWarps + i / kRow, c = i % kRow;
        const long long r = (long long)v * p.H + hh;
        qs[i] = hh >= p.H ? 0.f : c < kDc ? q_lat[r * kDc + c] : to_f(q_rope[r * (kRow - kDc) + c - kDc]);
    }
    float m = -INFINITY, l = 0.f, acc[kDc / 32];
#pragma unroll
    for (int i = 0; i < kDc / 32; ++i) acc[i] = 0.f;
    for (int jb = j0; jb < j1; jb += kGroup) {
        const int nt = min(kGroup, j1 - jb);
        __syncthreads();
        for (int r = warp; r < nt; r += kWarps) {
            const int j = jb + r;
            const long long page = p.block_table[(long long)b * p.max_blocks + j / kPageRows];
            const bool good = page >= 0 && page < p.num_pages;
            if (!good && lane == 0) latch(err, kErrOutOfRange, b);
            const uint8_t* src = p.codes + ((good ? page : 0) * kPageRows + j % kPageRows) * kRow;
            const float s = good ? p.scales[page] : 0.f;
            for (int c = 2 * lane; c < kRow; c += 64) {
                uint32_t h2;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(*(const unsigned short*)(src + c)));
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
                tile[r * ld + c] = good ? f.x * s : 0.f;
                tile[r * ld + c + 1] = good ? f.y * s : 0.f;
            }
        }
        __syncthreads();
        if (h >= p.H) continue;
        float s = -INFINITY;
        if (lane < nt) {
            float a = 0.f;
            for (int c = 0; c < kRow; ++c) a = fmaf(qs[warp * kRow + c], tile[lane * ld + c], a);
            s = a * p.scale;
        }
        float mn = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mn = fmaxf(m, mn);
        const float alpha = m == -INFINITY ? 0.f : expf(m - mn), w = lane < nt ? expf(s - mn) : 0.f;
        float sum = w;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l = l * alpha + sum;
#pragma unroll
        for (int i = 0; i < kDc / 32; ++i) acc[i] *= alpha;
        for (int r = 0; r < nt; ++r) {
            const float wr = __shfl_sync(0xffffffffu, w, r);
#pragma unroll
            for (int i = 0; i < kDc / 32; ++i) acc[i] = fmaf(wr, tile[r * ld + lane + 32 * i], acc[i]);
        }
        m = mn;
    }
    if (h >= p.H) return;
    const long long at = ((long long)split * NV + v) * p.H + h;
#pragma unroll
    for (int i = 0; i < kDc / 32; ++i) part_o[at * kDc + lane + 32 * i] = acc[i];
    if (lane == 0) {
        // a NaN sum (a NaN in a row that counts) as an infinite one, which the merge keeps: O is NaN
        part_ml[2 * at] = isnan(l) && m == -INFINITY ? 0.f : m;
        part_ml[2 * at + 1] = isnan(l) ? INFINITY : l;
    }
}

}  // namespace

cudaError_t decode_split(const Problem& p, const float* q_lat, const __nv_bfloat16* q_rope, int ns, float* part_o,
                         float* part_ml, DevErr err, cudaStream_t s) {
    constexpr int smem = (kGroup * (kRow + 1) + kWarps * kRow) * 4;
    cudaError_t e = cudaFuncSetAttribute(decode_split_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    decode_split_kernel<<<dim3(p.B * p.q_len, ns, (p.H + kWarps - 1) / kWarps), 32 * kWarps, smem, s>>>(
        p, q_lat, q_rope, ns, part_o, part_ml, err);
    return cudaGetLastError();
}

}  // namespace q8
}  // namespace mla
