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
constexpr int kRowsPerWarp = kPageRows / (kAppendThreads / 32);
constexpr int kVDc = 512, kVDr = 64, kVRow = 576;   // the row shape of the vector forms

// The block's item: every thread looks at a share of the sequences, the one that finds the
// item's leaves the sequence's numbers in shared memory (its length came with the offsets, so
// the page number is one load away), and all offsets are checked; false (for the whole block)
// if there is nothing to write.
__device__ __forceinline__ bool find_item(const AppendPaged& a, DevErr err, AppendItem& it, int& b) {
    __shared__ int s_seq[4];
    const long long item = blockIdx.x;
    bool ok = true;
#pragma unroll 1
    for (int i = threadIdx.x; i < a.B; i += blockDim.x) {
        const int o0 = a.new_offsets[i], o1 = a.new_offsets[i + 1], len = a.seq_lens[i];
        ok = ok && append_offsets_ok(o0, o1, i, a.B, a.n);
        if (append_item_base(o0, i) <= item && item < append_item_base(o1, i + 1)) {
            s_seq[0] = i;
            s_seq[1] = o0;
            s_seq[2] = o1;
            s_seq[3] = len;
        }
    }
    if (!__syncthreads_and(ok)) {
        if (threadIdx.x == 0 && item == 0) latch(err, kErrOutOfRange, -1);
        return false;
    }
    // the offsets are good, so the ranges of items cover [0, gridDim.x) and s_seq was written
    b = s_seq[0];
    const int r = append_item(s_seq[1], s_seq[2], s_seq[3], a.max_blocks, item - append_item_base(s_seq[1], b), &it);
    if (r < 0 && threadIdx.x == 0) latch(err, kErrOutOfRange, b);
    return r > 0;
}
// The item's page; false (for the whole block) if it is outside the cache.
__device__ __forceinline__ bool page_ok(const AppendPaged& a, DevErr err, int b, long long page) {
    const bool ok = page >= 0 && page < a.num_pages;
    if (!ok && threadIdx.x == 0) latch(err, kErrOutOfRange, b);
    return ok;
}

__device__ __forceinline__ int position(const AppendPaged& a, const AppendItem& it, int row) {
    return a.pos ? a.pos[it.src + row - it.r0] : it.block * kPageRows + row;
}

// Any type and width: one warp per row, value by value.
template <typename T>
__global__ void __launch_bounds__(kAppendThreads)
append_paged_kernel(const AppendPaged a, const __grid_constant__ RopeFreqs fr, T* __restrict__ cache, DevErr err) {
    AppendItem it;
    int b;
    if (!find_item(a, err, it, b)) return;
    const long long page = a.block_table[(long long)b * a.max_blocks + it.block];
    if (!page_ok(a, err, b, page)) return;
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

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// theta^(-2i / 64) of the 32 pairs of the vector forms, and its cosine and sine (kernel argument)
struct RopeSteps {
    double f[3 * kVDr / 2];   // frequencies, cosines, sines
};

// The table into shared memory, before the block's first barrier (find_item has one): kernel
// arguments read at an index that differs by lane come one lane at a time, which every warp
// would wait for.
__device__ __forceinline__ void stage_steps(const RopeSteps& st, double* tab) {
    if (threadIdx.x < 3 * kVDr / 2) tab[threadIdx.x] = st.f[threadIdx.x];
}

// The latents of a warp's rows (row0 .. row0 + 7 of the page): 16-byte units lane and 32 + lane
// of each, all requested before any is used.
__device__ __forceinline__ void load_latents(const AppendPaged& a, const AppendItem& it, int row0, int lane,
                                             uint4 (&w)[kRowsPerWarp][2]) {
#pragma unroll
    for (int j = 0; j < kRowsPerWarp; ++j) {
        const int row = row0 + j;
        if (row < it.r0 || row >= it.r1) continue;
        const uint4* c = (const uint4*)((const __nv_bfloat16*)a.c + (it.src + row - it.r0) * a.ld_c);
        w[j][0] = c[lane];
        w[j][1] = c[32 + lane];
    }
}

// The keys of the same rows (pair `lane` of each) into shared memory, for a rolled loop over the
// rotations (eight unrolled sines and cosines in double would be most of the kernel's code) that
// waits for no load.
template <bool kVec>
__device__ __forceinline__ void load_keys(const AppendPaged& a, const AppendItem& it, int row0, int lane,
                                          uint32_t (*keys)[kVDr / 2]) {
    uint32_t u[kRowsPerWarp];
#pragma unroll
    for (int j = 0; j < kRowsPerWarp; ++j) {
        const int row = row0 + j;
        if (row < it.r0 || row >= it.r1) continue;
        const __nv_bfloat16* k = (const __nv_bfloat16*)a.k_r + (it.src + row - it.r0) * a.ld_kr + 2 * lane;
        u[j] = kVec ? *(const uint32_t*)k : __bfloat16_as_ushort(k[0]) | ((uint32_t)__bfloat16_as_ushort(k[1]) << 16);
    }
#pragma unroll
    for (int j = 0; j < kRowsPerWarp; ++j)
        if (row0 + j >= it.r0 && row0 + j < it.r1) keys[row0 + j][lane] = u[j];
}

// Cosine and sine of rotary pair `lane` at the positions of a warp's rows, one after another.  A
// page's rows are consecutive positions: after the first, each is the one before turned by the
// pair's frequency (in double: a few last places after seven turns), where a sine and a cosine in
// double are a long chain of dependent FP64 instructions.  Positions given by the caller may be any
// and are computed one by one; a 16384-token prompt, turned and one by one, repeated on warm
// caches: 7.1 and 8.7 us (8-bit pages: 8.5 and 10.3).
struct Turn {
    double f, c1, s1, cs, sn;
    __device__ Turn(const double* tab, int lane) : f(tab[lane]), c1(tab[32 + lane]), s1(tab[64 + lane]), cs(1.0), sn(0.0) {}
    __device__ __forceinline__ void to(const AppendPaged& a, const AppendItem& it, int row, bool first) {
        if (first || a.pos) {
            sincos((double)position(a, it, row) * f, &sn, &cs);
        } else {
            const double c = cs * c1 - sn * s1;
            sn = sn * c1 + cs * s1;
            cs = c;
        }
    }
};

// bf16 rows of 512 + 64 with 16-byte aligned latents and pages: a warp takes eight rows, lane l
// units l and 32 + l of each latent and rotary pair l.  Latency bounds a step's call (offsets and
// lengths, page number, row: three dependent loads) and the pages' bandwidth a long one; a
// 16384-token prompt takes 7.1 us on warm caches, and 29.9 one value at a time.
__global__ void __launch_bounds__(kAppendThreads)
append_paged_vec_kernel(const AppendPaged a, const __grid_constant__ RopeSteps st, __nv_bfloat16* __restrict__ cache,
                        DevErr err) {
    __shared__ uint32_t s_key[kPageRows][kVDr / 2];   // a lane reads what it wrote
    __shared__ double s_tab[3 * kVDr / 2];
    stage_steps(st, s_tab);
    AppendItem it;
    int b;
    if (!find_item(a, err, it, b)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row0 = warp * kRowsPerWarp;
    const long long page = a.block_table[(long long)b * a.max_blocks + it.block];
    uint4 w[kRowsPerWarp][2];
    load_latents(a, it, row0, lane, w);   // while the page number is on its way
    load_keys<true>(a, it, row0, lane, s_key);
    if (!page_ok(a, err, b, page)) return;
    __nv_bfloat16* out = cache + page * (long long)(kPageRows * kVRow);
    Turn turn(s_tab, lane);
    const int first = max(row0, it.r0);
#pragma unroll 1
    for (int row = first; row < min(row0 + kRowsPerWarp, it.r1); ++row) {
        const uint32_t k = s_key[row][lane];
        turn.to(a, it, row, row == first);
        float x0 = bf16_lo(k), x1 = bf16_hi(k);
        rope_rotate(x0, x1, turn.cs, turn.sn);
        *(__nv_bfloat162*)(out + row * kVRow + kVDc + 2 * lane) = __floats2bfloat162_rn(x0, x1);
    }
#pragma unroll
    for (int j = 0; j < kRowsPerWarp; ++j) {
        const int row = row0 + j;
        if (row < it.r0 || row >= it.r1) continue;
        uint4* to = (uint4*)(out + row * kVRow);
        to[lane] = w[j][0];
        to[32 + lane] = w[j][1];
    }
}

// ------------------------------------------------------------------- 8-bit pages

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

// Each row is read once: a warp keeps its eight rows' latents in registers (units as above) and
// the block its rotated keys in shared memory, from the load to the store; the scale is a block
// maximum, and no second launch or atomic is needed for it.  kVec: the latents allow 16-byte
// loads and the keys 4-byte ones.
template <bool kVec>
__global__ void __launch_bounds__(kAppendThreads)
append_paged_q8_kernel(const AppendPaged a, const __grid_constant__ RopeSteps st, uint8_t* __restrict__ codes,
                       float* __restrict__ scales, DevErr err) {
    __shared__ float s_max[kAppendThreads / 32];
    __shared__ uint32_t s_raw[kPageRows][kVDr / 2];   // a lane reads what it wrote
    __shared__ float2 s_key[kPageRows][kVDr / 2];
    __shared__ double s_tab[3 * kVDr / 2];
    stage_steps(st, s_tab);
    AppendItem it;
    int b;
    if (!find_item(a, err, it, b)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row0 = warp * kRowsPerWarp;
    const long long page = a.block_table[(long long)b * a.max_blocks + it.block];
    uint4 w[kRowsPerWarp][2];
    if (kVec) {
        load_latents(a, it, row0, lane, w);   // while the page number is on its way
    } else {
#pragma unroll
        for (int j = 0; j < kRowsPerWarp; ++j) {
            const int row = row0 + j;
            if (row < it.r0 || row >= it.r1) continue;
            const __nv_bfloat16* c = (const __nv_bfloat16*)a.c + (it.src + row - it.r0) * a.ld_c + 8 * lane;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    u[i] = __bfloat16_as_ushort(c[256 * h + 2 * i]) | ((uint32_t)__bfloat16_as_ushort(c[256 * h + 2 * i + 1]) << 16);
                w[j][h] = make_uint4(u[0], u[1], u[2], u[3]);
            }
        }
    }
    load_keys<kVec>(a, it, row0, lane, s_raw);
    if (!page_ok(a, err, b, page)) return;
    const float before = it.r0 > 0 ? scales[page] : 0.f;   // earlier tokens are on the page
    float amax = 0.f;
    Turn turn(s_tab, lane);
    const int first = max(row0, it.r0);
#pragma unroll 1
    for (int row = first; row < min(row0 + kRowsPerWarp, it.r1); ++row) {
        const uint32_t u = s_raw[row][lane];
        float x0 = bf16_lo(u), x1 = bf16_hi(u);
        turn.to(a, it, row, row == first);
        rope_rotate(x0, x1, turn.cs, turn.sn);
        s_key[row][lane] = make_float2(x0, x1);
        amax = fmaxf(amax, fmaxf(finite_abs(x0), finite_abs(x1)));
    }
#pragma unroll
    for (int j = 0; j < kRowsPerWarp; ++j) {
        const int row = row0 + j;
        if (row < it.r0 || row >= it.r1) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t u[4] = {w[j][h].x, w[j][h].y, w[j][h].z, w[j][h].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fmaxf(finite_abs(bf16_lo(u[i])), finite_abs(bf16_hi(u[i]))));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) s_max[warp] = amax;
    __syncthreads();   // also: every thread has read the page's old scale
#pragma unroll
    for (int i = 0; i < kAppendThreads / 32; ++i) amax = fmaxf(amax, s_max[i]);
    float s = pow2(scale_exponent(amax));
    uint8_t* out = codes + page * (long long)(kPageRows * kVRow);
    if (before >= s) {
        s = before;
    } else if (it.r0 > 0) {
        const float ratio = before / s;
#pragma unroll 1
        for (int i = threadIdx.x; i < it.r0 * (kVRow / 4); i += kAppendThreads) {
            uint32_t v = ((const uint32_t*)out)[i];
            v = e4m3x2(e4m3_value(v & 0xFFu) * ratio, e4m3_value((v >> 8) & 0xFFu) * ratio) |
                (e4m3x2(e4m3_value((v >> 16) & 0xFFu) * ratio, e4m3_value(v >> 24) * ratio) << 16);
            ((uint32_t*)out)[i] = v;
        }
    }
    if (threadIdx.x == 0) scales[page] = s;
    const float inv = 1.f / s;
#pragma unroll
    for (int j = 0; j < kRowsPerWarp; ++j) {
        const int row = row0 + j;
        if (row < it.r0 || row >= it.r1) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t u[4] = {w[j][h].x, w[j][h].y, w[j][h].z, w[j][h].w};
            uint32_t q[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                q[i] = e4m3x2(bf16_lo(u[2 * i]) * inv, bf16_hi(u[2 * i]) * inv) |
                       (e4m3x2(bf16_lo(u[2 * i + 1]) * inv, bf16_hi(u[2 * i + 1]) * inv) << 16);
            ((uint2*)(out + row * kVRow))[32 * h + lane] = make_uint2(q[0], q[1]);
        }
        const float2 k = s_key[row][lane];
        ((unsigned short*)(out + row * kVRow + kVDc))[lane] = (unsigned short)e4m3x2(k.x * inv, k.y * inv);
    }
}

RopeFreqs rope_freqs(float theta, int d_hR) {
    RopeFreqs f{};
    for (int i = 0; i < d_hR / 2; ++i) f.f[i] = pow((double)theta, -2.0 * (double)i / (double)d_hR);
    return f;
}

// kept for the next call of the thread: the pow calls took as long as a launch
const RopeSteps& rope_steps(float theta) {
    thread_local RopeSteps st{};
    thread_local float of = 0.f;
    if (of != theta) {
        const RopeFreqs f = rope_freqs(theta, kVDr);
        for (int i = 0; i < kVDr / 2; ++i) {
            st.f[i] = f.f[i];
            st.f[kVDr / 2 + i] = cos(f.f[i]);
            st.f[kVDr + i] = sin(f.f[i]);
        }
        of = theta;
    }
    return st;
}

bool aligned(const void* p, size_t k) { return ((uintptr_t)p & (k - 1)) == 0; }

// latents by 16 bytes, keys by 4
bool vector_rows(const AppendPaged& a) {
    return aligned(a.c, 16) && a.ld_c % 8 == 0 && aligned(a.k_r, 4) && a.ld_kr % 2 == 0;
}

}  // namespace

template <typename T>
cudaError_t append_paged(const AppendPaged& a, float theta, T* cache, DevErr err, cudaStream_t s) {
    const unsigned items = (unsigned)append_items(a.n, a.B);
    if (Dt<T>::id == 1 && a.d_c == kVDc && a.d_hR == kVDr && vector_rows(a) && aligned(cache, 16))
        append_paged_vec_kernel<<<items, kAppendThreads, 0, s>>>(a, rope_steps(theta), (__nv_bfloat16*)cache, err);
    else
        append_paged_kernel<T><<<items, kAppendThreads, 0, s>>>(a, rope_freqs(theta, a.d_hR), cache, err);
    return cudaGetLastError();
}
template cudaError_t append_paged<float>(const AppendPaged&, float, float*, DevErr, cudaStream_t);
template cudaError_t append_paged<__nv_bfloat16>(const AppendPaged&, float, __nv_bfloat16*, DevErr, cudaStream_t);

cudaError_t append_paged_q8(const AppendPaged& a, float theta, uint8_t* codes, float* scales, DevErr err,
                            cudaStream_t s) {
    auto kernel = vector_rows(a) ? append_paged_q8_kernel<true> : append_paged_q8_kernel<false>;
    kernel<<<(unsigned)append_items(a.n, a.B), kAppendThreads, 0, s>>>(a, rope_steps(theta), codes, scales, err);
    return cudaGetLastError();
}

}  // namespace mla
