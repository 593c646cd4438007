// Paged cache append: rotation of the keys, quantisation, page writes.
//
// For new token i of sequence b at position p (its place in the sequence, or pos[i]):
//     row = [c_i | R(p) k_r,i],   R(p) rotating pair (2j, 2j + 1) by p theta^(-2j / d_hR)
// into row p % 64 of page block_table[b, p / 64].  The work is cut by page (paged_plan.h):
// one block writes all of a page's new rows, so the 8-bit form can give the page its one
// scale without atomics or a second launch, and no two blocks write the same line.
//
// The 8-bit form: value = code * s, E4M3 codes, s a power of two per page: the smallest with
// amax <= 448 s over the page's new values, and not below the page's present scale when
// earlier tokens are on it.  E4M3 is a floating-point code, so a power-of-two scale costs no
// precision against amax / 448 (codes keep their 3 mantissa bits) and makes re-expressing the
// earlier codes under a larger scale exact but for codes that become subnormal.
#include <cuda_fp16.h>
#include <math.h>

#include "paged.cuh"
#include "paged_plan.h"

namespace mla {

namespace {

constexpr int kAppendThreads = 256;

// The block's item: finds its sequence (every thread looks at a share of the offsets) and
// checks all offsets; false (for the whole block) if there is nothing to write.
__device__ __forceinline__ bool find_item(const AppendPaged& a, DevErr err, AppendItem& it, int& b, long long& page) {
    __shared__ int s_b;
    const long long item = blockIdx.x;
    bool ok = true;
    for (int i = threadIdx.x; i < a.B; i += blockDim.x) {
        const int o0 = a.new_offsets[i], o1 = a.new_offsets[i + 1];
        ok = ok && append_offsets_ok(o0, o1, i, a.B, a.n);
        if (append_item_base(o0, i) <= item && item < append_item_base(o1, i + 1)) s_b = i;
    }
    if (!__syncthreads_and(ok)) {
        if (threadIdx.x == 0 && item == 0) latch(err, kErrOutOfRange, -1);
        return false;
    }
    // the offsets are good, so the ranges of items cover [0, gridDim.x) and s_b was written
    b = s_b;
    const int o0 = a.new_offsets[b], o1 = a.new_offsets[b + 1];
    const int r = append_item(o0, o1, a.seq_lens[b], a.max_blocks, item - append_item_base(o0, b), &it);
    if (r <= 0) {
        if (r < 0 && threadIdx.x == 0) latch(err, kErrOutOfRange, b);
        return false;
    }
    page = a.block_table[(long long)b * a.max_blocks + it.block];
    if (page < 0 || page >= a.num_pages) {
        if (threadIdx.x == 0) latch(err, kErrOutOfRange, b);
        return false;
    }
    return true;
}

__device__ __forceinline__ int position(const AppendPaged& a, const AppendItem& it, int row) {
    return a.pos ? a.pos[it.src + row - it.r0] : it.block * kPageRows + row;
}

// One warp per row.
template <typename T>
__global__ void __launch_bounds__(kAppendThreads)
append_paged_kernel(const AppendPaged a, const __grid_constant__ RopeFreqs fr, T* __restrict__ cache, DevErr err) {
    AppendItem it;
    int b;
    long long page;
    if (!find_item(a, err, it, b, page)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int width = a.d_c + a.d_hR;
    for (int row = it.r0 + warp; row < it.r1; row += kAppendThreads / 32) {
        const long long src = it.src + row - it.r0;
        const T* c = (const T*)a.c + src * a.ld_c;
        const T* k = (const T*)a.k_r + src * a.ld_kr;
        T* out = cache + (page * kPageRows + row) * width;
        const int p = position(a, it, row);
        for (int i = lane; i < a.d_c; i += 32) out[i] = c[i];
        for (int i = lane; i < a.d_hR / 2; i += 32) {
            double sn, cs;
            sincos((double)p * fr.f[i], &sn, &cs);
            float x0 = to_f(k[2 * i]), x1 = to_f(k[2 * i + 1]);
            rope_rotate(x0, x1, cs, sn);
            out[a.d_c + 2 * i] = from_f<T>(x0);
            out[a.d_c + 2 * i + 1] = from_f<T>(x1);
        }
    }
}

// ------------------------------------------------------------------- 8-bit pages

constexpr int kQDc = 512, kQRow = 576;

// two fp32 -> two E4M3 codes, `lo` in the low byte (nearest even, saturating to +-448; NaN
// gives the NaN code)
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)code));
    return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu)));
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// |x|, or 0 for an infinity or NaN: those take no part in a page's scale
__device__ __forceinline__ float finite_abs(float x) {
    const float y = fabsf(x);
    return y < INFINITY ? y : 0.f;
}

// The exponent e of the smallest power of two with amax <= 448 * 2^e (0 for amax = 0), not
// below -60: with amax = f 2^E, 1 <= f < 2, and 448 = 1.75 * 2^8, e is E - 8 while f <= 1.75.
__device__ __forceinline__ int scale_exponent(float amax) {
    if (!(amax > 0.f)) return 0;
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return e < -60 ? -60 : e;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

constexpr int kRowsPerWarp = kPageRows / (kAppendThreads / 32);

// Lane l of a warp holds columns 16 l .. 16 l + 15 of the latent (bf16 pairs) and rotary pair l
// of each of its rows, from the load to the store: the inputs are read once, the scale is a
// block maximum, and each row's codes leave as one 16-byte and one 2-byte store a lane.
// kVec: the inputs' rows allow 16-byte (latent) and 4-byte (key) loads.
template <bool kVec>
__global__ void __launch_bounds__(kAppendThreads)
append_paged_q8_kernel(const AppendPaged a, const __grid_constant__ RopeFreqs fr, uint8_t* __restrict__ codes,
                       float* __restrict__ scales, DevErr err) {
    __shared__ float s_max[kAppendThreads / 32];
    AppendItem it;
    int b;
    long long page;
    if (!find_item(a, err, it, b, page)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row0 = warp * kRowsPerWarp;
    uint32_t w[kRowsPerWarp][8], wk[kRowsPerWarp];
#pragma unroll
    for (int j = 0; j < kRowsPerWarp; ++j) {
        const int row = row0 + j;
        if (row < it.r0 || row >= it.r1) continue;
        const long long src = it.src + row - it.r0;
        const __nv_bfloat16* c = (const __nv_bfloat16*)a.c + src * a.ld_c + 16 * lane;
        const __nv_bfloat16* k = (const __nv_bfloat16*)a.k_r + src * a.ld_kr + 2 * lane;
        if (kVec) {
            const uint4 u = ((const uint4*)c)[0], v = ((const uint4*)c)[1];
            w[j][0] = u.x, w[j][1] = u.y, w[j][2] = u.z, w[j][3] = u.w;
            w[j][4] = v.x, w[j][5] = v.y, w[j][6] = v.z, w[j][7] = v.w;
            wk[j] = *(const uint32_t*)k;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[j][i] = __bfloat16_as_ushort(c[2 * i]) | ((uint32_t)__bfloat16_as_ushort(c[2 * i + 1]) << 16);
            wk[j] = __bfloat16_as_ushort(k[0]) | ((uint32_t)__bfloat16_as_ushort(k[1]) << 16);
        }
    }
    float amax = 0.f, kr[kRowsPerWarp][2];
#pragma unroll
    for (int j = 0; j < kRowsPerWarp; ++j) {
        const int row = row0 + j;
        if (row < it.r0 || row >= it.r1) continue;
        double sn, cs;
        sincos((double)position(a, it, row) * fr.f[lane], &sn, &cs);
        kr[j][0] = bf16_lo(wk[j]);
        kr[j][1] = bf16_hi(wk[j]);
        rope_rotate(kr[j][0], kr[j][1], cs, sn);
        amax = fmaxf(amax, fmaxf(finite_abs(kr[j][0]), finite_abs(kr[j][1])));
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(finite_abs(bf16_lo(w[j][i])), finite_abs(bf16_hi(w[j][i]))));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) s_max[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kAppendThreads / 32; ++i) amax = fmaxf(amax, s_max[i]);
    float s = pow2(scale_exponent(amax));
    uint8_t* out = codes + page * (long long)(kPageRows * kQRow);
    if (it.r0 > 0) {   // earlier tokens are on the page
        const float before = scales[page];
        if (before >= s) {
            s = before;
        } else {
            const float ratio = before / s;
            for (int i = threadIdx.x; i < it.r0 * (kQRow / 4); i += kAppendThreads) {
                uint32_t v = ((const uint32_t*)out)[i];
                v = e4m3x2(e4m3_value(v & 0xFFu) * ratio, e4m3_value((v >> 8) & 0xFFu) * ratio) |
                    (e4m3x2(e4m3_value((v >> 16) & 0xFFu) * ratio, e4m3_value(v >> 24) * ratio) << 16);
                ((uint32_t*)out)[i] = v;
            }
        }
        __syncthreads();   // every thread has read the page's old scale
    }
    if (threadIdx.x == 0) scales[page] = s;
    const float inv = 1.f / s;
#pragma unroll
    for (int j = 0; j < kRowsPerWarp; ++j) {
        const int row = row0 + j;
        if (row < it.r0 || row >= it.r1) continue;
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = e4m3x2(bf16_lo(w[j][2 * i]) * inv, bf16_hi(w[j][2 * i]) * inv) |
                   (e4m3x2(bf16_lo(w[j][2 * i + 1]) * inv, bf16_hi(w[j][2 * i + 1]) * inv) << 16);
        ((uint4*)(out + row * kQRow))[lane] = make_uint4(q[0], q[1], q[2], q[3]);
        ((unsigned short*)(out + row * kQRow + kQDc))[lane] =
            (unsigned short)e4m3x2(kr[j][0] * inv, kr[j][1] * inv);
    }
}

RopeFreqs rope_freqs(float theta, int d_hR) {
    RopeFreqs f{};
    for (int i = 0; i < d_hR / 2; ++i) f.f[i] = pow((double)theta, -2.0 * (double)i / (double)d_hR);
    return f;
}

}  // namespace

template <typename T>
cudaError_t append_paged(const AppendPaged& a, float theta, T* cache, DevErr err, cudaStream_t s) {
    append_paged_kernel<T><<<(unsigned)append_items(a.n, a.B), kAppendThreads, 0, s>>>(a, rope_freqs(theta, a.d_hR),
                                                                                       cache, err);
    return cudaGetLastError();
}
template cudaError_t append_paged<float>(const AppendPaged&, float, float*, DevErr, cudaStream_t);
template cudaError_t append_paged<__nv_bfloat16>(const AppendPaged&, float, __nv_bfloat16*, DevErr, cudaStream_t);

cudaError_t append_paged_q8(const AppendPaged& a, float theta, uint8_t* codes, float* scales, DevErr err,
                            cudaStream_t s) {
    const bool vec = ((uintptr_t)a.c & 15) == 0 && a.ld_c % 8 == 0 && ((uintptr_t)a.k_r & 3) == 0 && a.ld_kr % 2 == 0;
    auto kernel = vec ? append_paged_q8_kernel<true> : append_paged_q8_kernel<false>;
    kernel<<<(unsigned)append_items(a.n, a.B), kAppendThreads, 0, s>>>(a, rope_freqs(theta, a.d_hR), codes, scales,
                                                                       err);
    return cudaGetLastError();
}

}  // namespace mla
