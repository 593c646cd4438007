// Absorbed attention over the 8-bit paged latent cache, on the tcgen05 tensor cores.
//
// For query row r = (new token t, head h) of sequence b and cached token j, whose value row is
// its code row times the scale s_j of its page:
//     z_j = scale s_j ([q_lat | q_rope][r] . code_j),    o_lat[r] = sum_j softmax(z)_j s_j code_j[0:512]
// over the first seq_lens[b] - q_len + t + 1 tokens, then out[r] = W_UV[h] o_lat[r].
//
// The codes are MMA operands as they are (kind::f8f6f4, E4M3); nothing is dequantised.  The
// other operand of each product is a sum of 8-bit terms.  A query value is two E4M3 terms against
// its row's largest value: hi = e4m3(x) and lo = e4m3(x - hi) leave 2^-8 |x| (half a step of 4
// bits twice), or 2^-17 of the row's largest value where that is more.  A probability must keep its
// precision however small it is beside its tile's largest: a token that takes most of the weight
// may carry no value (an attention sink), and then the small ones make up the output.  It is three
// E5M2 terms, each of what the ones before it left, times 8 from term to term: p = t0 + t1 / 8 + t2 / 64
// within 2^-9 p (half a step of 3 bits three times) + 2^-11 p (fp16, in which they are made) for
// p >= 2^-14, and 2^-23 below.  The terms are columns of one product, each with its own accumulator.
//
// Tokens are the MMA's M.  A tile is 128 tokens (two pages); a group is R <= 32 query rows:
//     S^T [128 tokens x 2R]  = codes [128 x 576] . [q_hi | q_lo]^T      (both terms in one product)
//     O^T [4 x 128 latents x 3R] += codes^T [512 x 128] . P [128 x 3R]  (all three terms in one)
// so the codes are the A operand of both, K-major for the scores and MN-major for O, from the
// one copy in shared memory; 32 rows' O takes 384 TMEM columns, two score buffers the other
// 128, and a CTA needs no other CTA's scores.  A thread of the softmax holds one token and 8
// rows: P goes to shared memory in the layout the product reads, sums stay per
// thread until the end of a piece, and the only thing the token lanes must agree on is each
// row's reference M (below).
//
// What bounds it.  A tile of 32 rows is 18 score products (N = 64, 48.5 cycles each: the A operand's
// 4 KB from shared memory, not the arithmetic) and 16 O products (N = 96); the tensor pipe is
// busy with them for ~1970 of the ~2500 cycles a tile takes beside start and end.  Two tiles are in flight (two score
// buffers, two P slots), and a tile's loads, scores, softmax and O follow one another.
// Measured, 128 heads, 32 sequences of 4096 tokens: 59.1 us (100.4 k cycles, tensor pipe 54 % of
// them, 81 MB from DRAM); 16 heads, 48 ragged sequences of 4500 tokens on average: 29.2 us, 119
// MB, 62 % of a copy's bandwidth, the rest start and end.
//
// The reference.  p = 2^-6 2^(z' - M) must fit fp16 and E5M2 and must not sink below them, so M
// follows the scores in both directions: it is set so that the tile's largest p is 2^4, and set
// anew (O and the sums rescaled) when a tile's largest p leaves [2^-6, 2^15.5].  The row's largest
// so far is thus at 2^4 or above: what is 2^-18 of it keeps all of P's bits, and the least step
// is 2^-27 of it.  A new reference costs a wait for the O product before and a pass over O, so the
// window is as wide as those bits allow and its set point leaves most of the room above, where new
// maxima come: with scores of 3 nats' spread, 32 sequences of 4096 tokens, 128 heads, 77.8 us a step,
// and 87.5 with the window [2^4, 2^15.5] set at 2^10.
//
// The scales.  They ride on the probabilities: z' = z + log2(s_j / s_ref) with s_ref the piece's first
// page's scale.  A page of large scale need not hold large values (a page of zeros has the scale 1,
// one large value raises its whole page's), so no page's probabilities may cost another's bits: where
// the two pages of a tile are more than 2^4 apart the tile is visited twice, each page's tokens alone,
// and a visit whose scale is as far from the one before sets the references anew.  The output of a
// piece with such pages leaves in fp16 against each row's largest value.  What remains is fp32's range:
// O is rescaled by up to 2^kFarLog2 as the references go down.
#include <math.h>

#include <atomic>

#include "decode_q8.cuh"
#include "paged_plan.h"
#include "tc_common.cuh"

namespace mla {
namespace q8 {

namespace {

constexpr int kDc = 512, kDr = 64, kRow = 576;
constexpr int kT = 128;                       // tokens per tile
constexpr int kChunkBytes = kT * 128;         // 128 latent columns of a tile (128-byte swizzle)
constexpr int kRopeBytes = kT * kDr;          // the rotary columns of a tile (64-byte swizzle)
constexpr int kRoleThreads = 128;             // TMA warp, score issuer, O issuer, the warp that finds the pieces
// Cost units of a piece's query load and epilogue, in tiles: 1.  With 2 the longest ranges are as
// long and the step no faster (graph replays; 128 heads, 32 x 4096 tokens: 71.2 us both; 100-token
// chunks: 151.4 and 151.1; ragged long contexts: 430 and 431).
constexpr int kPieceCost = 1;
// Up to this many groups of a sequence are walked side by side, so that its pages come from HBM
// once and from L2 for the others.  Side by side and one after another: 4 groups 71.2 and 73.3
// us, 64 ragged sequences of up to 32768 tokens 430 and 515; 8 groups 121.3 and 125.9.
constexpr int kMaxSib = 8;
constexpr float kPGain = 1.f / 64;            // p = 2^-6 2^(z' - M)
constexpr float kTopLog2 = 21.5f;             // p <= 2^15.5 (the largest E5M2 value is 1.75 x 2^15)
constexpr float kSetLog2 = 10.f;              // a new reference puts the tile's largest p at 2^4
// How far below its highest value a reference may go: O, at most 2^15.5 x 448 x 2^20 tokens, stays
// below 2^127.  Scales 2^60 apart leave 2^20 of it to the scores.
constexpr float kFarLog2 = 80.f;
constexpr float kApart = 16.f;                // scales further apart than this do not share a visit

// Shared memory: NC chunk slots (as many as fit), NR slots that hold a tile's rotary columns and
// then its P (three terms of R bytes per token), the group's queries.
// Softmax warps: four (one per 32 tokens) for each of CG groups of HC rows.
template <int R> struct Cfg {
    static constexpr int HC = 8, CG = R / HC;
    static constexpr int kSoft = 128 * CG, kThreads = kRoleThreads + kSoft;
    static constexpr int kTerms = 3, NP = kTerms * R;    // N of an O product
    static constexpr int kPRow = R == 32 ? 128 : 64;     // bytes of a token's P, swizzled over as many
    static constexpr int NC = R == 32 ? 9 : 10;
    static constexpr int NR = 2;
    static constexpr int kSlotBytes = kT * kPRow;
    static constexpr int kQBytes = 2 * R * kRow;
    static constexpr uint32_t kColO = 4 * R;
    static constexpr uint32_t kTmemCols = R == 16 ? 256 : 512;
    static constexpr int kMisc = 3 * 1024;
    static constexpr int kSmem = NC * kChunkBytes + NR * kSlotBytes + kQBytes + kMisc;
    static_assert(NP <= kPRow && kRopeBytes <= kSlotBytes, "a tile's P or rotary columns in a slot");
    static_assert(kColO + 4 * NP <= kTmemCols, "TMEM columns");
    static_assert(kSmem <= 232448, "shared memory over the 227 KB limit");
};

// One lane of a converged warp.  Asynchronous instructions (products, commits, bulk and TMA
// copies) are issued under this predicate: it tells the compiler that one lane is active, where
// a test of the lane number makes it loop over the active lanes around each of them (a product
// then took some twenty instructions, which four softmax warps per scheduler stretched to ~90
// cycles).
__device__ __forceinline__ bool elect() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
// tcgen05.mma kind::f8f6f4, both operands in shared memory
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "mov.b64 da, {%1, %2};\n\t"
        "mov.b64 db, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
// A value that is the same in all lanes, as one the compiler knows to be so (loops around the
// products run on it)
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }
__device__ __forceinline__ bool uniform(bool x) { return __any_sync(0xffffffffu, x); }
// Descriptor words: low = address and leading offset (both / 16), high = stride offset / 16,
// version 1, swizzle (2: 128 bytes, 4: 64 bytes)
__device__ constexpr uint32_t desc_hi(uint32_t sbo, uint32_t swizzle) { return (sbo >> 4) | (1u << 14) | (swizzle << 29); }
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }
// E4M3 x E4M3 (b_format 0) or E5M2 (1) -> fp32
constexpr uint32_t idesc_f8(int M, int N, int b_format, int a_mn_major, int b_mn_major) {
    return (1u << 4) | ((uint32_t)b_format << 10) | ((uint32_t)a_mn_major << 15) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Two fp32 values in one 64-bit register pair: one instruction for both
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(uint32_t x, uint32_t y) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
    return r;
}
__device__ __forceinline__ f32x2 pair(float x, float y) { return pair(__float_as_uint(x), __float_as_uint(y)); }
__device__ __forceinline__ void unpair(f32x2 v, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 sub2(f32x2 a, f32x2 b) { return fma2(b, pair(-1.f, -1.f), a); }

__device__ __forceinline__ float ex2(float x) {   // flushes results below 2^-126
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// largest value of a warp's lanes (NaN does not count)
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
// two values -> two E4M3 codes, `lo` in the low byte (nearest even, saturating, NaN kept)
__device__ __forceinline__ uint32_t e4m3x2_f32(float lo, float hi) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// four fp16 values -> four E5M2 codes (nearest even, saturating, NaN kept)
__device__ __forceinline__ uint32_t e5m2x4(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e5m2x2.f16x2 x, %1;\n\tcvt.rn.satfinite.e5m2x2.f16x2 y, %2;\n\t"
        "mov.b32 %0, {x, y};\n\t}"
        : "=r"(r)
        : "r"(a), "r"(b));
    return r;
}
// 8 (x - t), x two fp16 values and t their E5M2 codes, which are fp16's upper bytes (bytes `sel`
// of `codes`); exact unless it is below fp16's normal numbers
__device__ __forceinline__ uint32_t rest_of(uint32_t x, uint32_t codes, uint32_t sel) {
    const uint32_t t = __byte_perm(codes, 0, sel);
    const __half2 r = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&t)),
                              __float2half2_rn(8.f));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint32_t code2) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)code2));
    return h;
}
// ---------------------------------------------------------------- work split
// As in the other decode kernels: the tiles of all sequences, in order, are cut into equal
// ranges; a range may hold pieces of several sequences.  A virtual sequence is a sequence
// whose G groups are walked side by side by G neighbouring CTAs ("siblings": the pages then
// come from HBM once), or, past kMaxSib groups, one (sequence, group) pair.
struct Src {
    const int32_t* seq_lens;
    int max_blocks;
    Shape s;
    __device__ int raw_len(int b) const {
        const int L = seq_lens[b];
        return (L < 0 || (long long)L > (long long)max_blocks * kPageRows) ? -1 : L;
    }
    __device__ int len(int b) const { return max(raw_len(b), 0); }
    __device__ int first_token(int g) const { return g * s.R / s.H; }
    __device__ int last_token(int g) const { return (min((g + 1) * s.R, s.q_len * s.H) - 1) / s.H; }
    // keys of new token t of a sequence with L tokens
    __device__ int keys(int L, int t) const { return L - (s.q_len - 1 - t); }
    __device__ int vseqs() const { return s.sib > 1 ? s.B : s.B * s.G; }
    __device__ int vseq_b(int i) const { return s.sib > 1 ? i : i / s.G; }
    // what virtual sequence i is charged for, its sequence having L tokens
    __device__ int vkeys(int L, int i) const { return s.sib > 1 ? L : max(keys(L, last_token(i % s.G)), 0); }
};

__device__ __forceinline__ int tiles_of(int L) { return L > 0 ? (L + kT - 1) / kT : 0; }
__device__ __forceinline__ long long cost_of(int n) { return n > 0 ? n + kPieceCost : 0; }

// Marks of a visit: the same tile comes again, its first (second) page does not count, its scale is
// far from the visit's before, the piece's scales so far are far apart
constexpr int kAgain = 1, kNotFirst = 2, kNotSecond = 4, kJump = 8, kWide = 16;
__device__ __forceinline__ int marks(const float4& visit) { return __float_as_int(visit.z); }

// tiles [j0, j1) of group g of sequence b (j0 = j1: no more pieces)
struct Seg {
    int b, item, g, j0, j1, len, kmin, kmax, slot, pad[3];
};
static_assert(sizeof(Seg) % 16 == 0, "alignment of what lies behind");
// Walks the pieces of this CTA's range.  Positions are counted from the range's start.
struct SegIter {
    const Src& src;
    int i;
    int cs;     // where virtual sequence i's cost starts (not above 0 at first)
    int span;   // cost units of the range
    int len;    // tokens of sequence i's sequence, or -1: look
    __device__ bool next(Seg& s) {
        const int nv = src.vseqs();
        while (i < nv && cs < span) {
            const int ii = i++;
            s.b = src.s.sib > 1 ? ii : ii / src.s.G;
            s.g = src.s.sib > 1 ? (int)blockIdx.x % src.s.sib : ii - s.b * src.s.G;
            s.len = len >= 0 ? len : src.len(s.b);
            len = -1;
            const int n = tiles_of(src.vkeys(s.len, ii));
            const int f = cs + kPieceCost;
            cs += (int)cost_of(n);
            if (n == 0) continue;
            s.item = s.b * src.s.G + s.g;
            s.kmin = src.keys(s.len, src.first_token(s.g));
            s.kmax = src.keys(s.len, src.last_token(s.g));
            s.j0 = max(-f, 0);
            s.j1 = min(span - f, tiles_of(s.kmax));
            if (s.j0 < s.j1) {
                s.slot = s.j0 == 0 ? s.item : src.s.B * src.s.G + (int)blockIdx.x;
                return true;
            }
        }
        return false;
    }
};

// A bounded wait of a whole warp, in few instructions (there are some thirty of them)
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const volatile int* abort_flag) {
    uint32_t left = ptx::g_wait_limit;
#pragma unroll 1
    do {
        if (__all_sync(0xffffffffu, ptx::mbar_try(bar, parity))) return true;
    } while (--left != 0 && !(__any_sync(0xffffffffu, *abort_flag != 0)));
    return false;
}

// Test hook (mla_test_starve_projection): nonzero = the attention's loader asks for the latents but
// not for the rotary columns, so that the waits behind them run out with copies under way.
__device__ int g_starve_loads = 0;

__device__ __noinline__ void fail(DevErr err, volatile int* abort_flag, int where) {
    latch(err, kErrTimeout, (long long)where * 1000000 + blockIdx.x);
    *abort_flag = 1;
}

// ------------------------------------------------------------------ attention
template <int R>
__global__ void __launch_bounds__(Cfg<R>::kThreads, 1)
attn_kernel(const __grid_constant__ CUtensorMap tm_lat, const __grid_constant__ CUtensorMap tm_rope, const __grid_constant__ Src src,
            const int32_t* __restrict__ block_table, const float* __restrict__ scales, long long num_pages,
            float scale_log2, const __grid_constant__ Ws ws, const DevErr err) {
    using C = Cfg<R>;
    constexpr int HC = C::HC, CG = C::CG, NC = C::NC, NR = C::NR, kThreads = C::kThreads;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (ptx::smem_u32(smem) & 1023) {   // uniform: leave before any barrier
        if (threadIdx.x == 0) latch(err, kErrTimeout, 9000000);
        return;
    }
    uint8_t* chunks = smem;
    uint8_t* ropes = chunks + NC * kChunkBytes;
    uint8_t* qimg = ropes + NR * C::kSlotBytes;
    float* qs = (float*)(qimg + C::kQBytes);            // [R] row scales of the queries
    float4* red = (float4*)(qs + 32);                   // [CG][16] per row, one value per token quarter
    float* nrefs = (float*)(red + 64);                  // [R] each row's reference, negated
    float* row_kt = nrefs + 32;                         // [R] row scale x softmax scale x the piece's first page's scale
    uint64_t* bars = (uint64_t*)(row_kt + 32);
    uint64_t *chunk_full = bars, *chunk_empty = bars + NC, *rope_full = bars + 2 * NC, *rope_empty = rope_full + 2;
    uint64_t *q_full = rope_full + 4, *s_full = rope_full + 5, *s_free = rope_full + 7, *p_ready = rope_full + 9;
    uint64_t *o_done = rope_full + 12, *grp_bar = rope_full + 14, *drain = rope_full + 18;
    uint64_t *seg_full = rope_full + 20, *seg_empty = rope_full + 22;
    Seg* segs = (Seg*)(rope_full + 24);                 // [2] the pieces of this CTA, from the planning warp
    uint32_t* flags = (uint32_t*)(segs + 2);            // [2 tiles][CG][4]
    float4* visit = (float4*)(flags + 32);              // [4 visits] scales of the tile's two pages, marks (kAgain ..), largest scale so far
    uint32_t* tmem_slot = (uint32_t*)(visit + 4);
    volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
    static_assert(32 * 4 + 64 * 16 + 64 * 4 + (2 * NC + 24) * 8 + 2 * sizeof(Seg) + (32 + 16 + 2) * 4 <= C::kMisc, "barrier area");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NC; ++i) {
            ptx::mbar_init(&chunk_full[i], 1);
            ptx::mbar_init(&chunk_empty[i], 1);
        }
        for (int i = 0; i < NR; ++i) {
            ptx::mbar_init(&rope_full[i], 1);
            ptx::mbar_init(&rope_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&s_full[i], 1);
            ptx::mbar_init(&s_free[i], C::kSoft);
            ptx::mbar_init(&p_ready[i], C::kSoft);
            ptx::mbar_init(&o_done[i], 1);
            ptx::mbar_init(&seg_full[i], 1);
            ptx::mbar_init(&seg_empty[i], kThreads / 32 - 1);
        }
        for (int i = 0; i < 4; ++i) ptx::mbar_init(&grp_bar[i], 4);
        ptx::mbar_init(q_full, 1);
        ptx::mbar_init(drain, 2);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::tma_prefetch(&tm_lat);
        ptx::tma_prefetch(&tm_rope);
    }
    if (warp == 1) {
        ptx::tmem_alloc(tmem_slot, C::kTmemCols);
        ptx::tmem_relinquish();
    }
    if (threadIdx.x == 0) pdl_trigger();

    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);

    // The pieces, in order, as every role sees them: warp 3 finds them ahead of time
    Seg sg;
    uint32_t segs_seen = 0;
    auto next_piece = [&]() -> bool {
        const uint32_t k = segs_seen & 1;
        if (!wait_warp(&seg_full[k], (segs_seen >> 1) & 1, abort_flag)) {
            fail(err, abort_flag, 10);
            return false;
        }
        sg = segs[k];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&seg_empty[k]);
        ++segs_seen;
        return uniform(sg.j0 < sg.j1);
    };
    if (warp == 3) {
        pdl_wait();   // the previous kernel of this call planned, and all before it is done
        const int4 start = ws.start[blockIdx.x / src.s.sib];
        SegIter it{src, start.x, start.y, start.z, start.w};
        bool more = true;
#pragma unroll 1
        for (uint32_t n = 0; more; ++n) {
            more = it.next(sg);
            if (n >= 2 && !wait_warp(&seg_empty[n & 1], ((n >> 1) - 1) & 1, abort_flag)) {
                fail(err, abort_flag, 15);
                break;
            }
            if (!more) sg.j0 = sg.j1 = 0;
            if (lane == 0) {
                segs[n & 1] = sg;
                ptx::mbar_arrive(&seg_full[n & 1]);
            }
            __syncwarp();
        }
    } else if (warp == 0) {
        // ---------------------------------------------------------- TMA producer
        // lane l holds the page (and its scale) of block base + l of the sequence
        const uint64_t policy = src.s.G > 1 ? ptx::policy_evict_normal() : ptx::policy_evict_first();
        const long long none = num_pages * kPageRows;   // a box past the last row reads zeros
        uint32_t g = 0, cn = 0, slot = 0, use = 0;      // visits and chunks requested, next slot and its uses
        const bool starve = g_starve_loads;
        bool ok = true;
        while (ok && next_piece()) {
            const int blocks = (sg.len + kPageRows - 1) / kPageRows;
            long long row = none;
            float sc = 0.f;
            int mark = 0;
            float s_ref = 0.f, s_last = 0.f, s_hi = 0.f, s_lo = INFINITY;   // scales: the first visit's (0: none yet), the one's before, extremes
#pragma unroll 1
            for (int j = sg.j0; ok && j < sg.j1; j += !(mark & kAgain)) {
                const int at = (j - sg.j0) & 15;
                if (at == 0 && !(mark & kAgain)) {
                    const int blk = 2 * j + lane;
                    const long long page = blk < blocks ? block_table[(long long)sg.b * src.max_blocks + blk] : -1;
                    const bool good = page >= 0 && page < num_pages;
                    row = good ? page * kPageRows : none;
                    sc = good ? scales[page] : 0.f;
                    // only the pages this piece reads are its to report
                    if (!good && blk < blocks && blk < 2 * sg.j1) latch(err, kErrOutOfRange, sg.b);
                }
                const int r0 = (int)__shfl_sync(0xffffffffu, row, 2 * at), r1 = (int)__shfl_sync(0xffffffffu, row, 2 * at + 1);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (ok && use > 0 && !wait_warp(&chunk_empty[slot], (use - 1) & 1, abort_flag)) ok = false;
                    if (ok) if (elect()) {
                        uint8_t* dst = chunks + slot * kChunkBytes;
                        ptx::mbar_expect_tx(&chunk_full[slot], kChunkBytes);
                        ptx::tma_load_2d_hint(dst, &tm_lat, &chunk_full[slot], 128 * c, r0, policy);
                        ptx::tma_load_2d_hint(dst + kChunkBytes / 2, &tm_lat, &chunk_full[slot], 128 * c, r1, policy);
                    }
                    cn += ok;
                    if (++slot == NC) slot = 0, ++use;
                }
                // the scales may still be on their way here, which must not hold up the loads above
                float s0 = __shfl_sync(0xffffffffu, sc, 2 * at), s1 = __shfl_sync(0xffffffffu, sc, 2 * at + 1);
                if (ok && g >= NR && !wait_warp(&rope_empty[g % NR], (g / NR - 1) & 1, abort_flag)) ok = false;
                if (mark & kAgain)
                    mark = kNotFirst;
                else
                    mark = s0 > 0.f && s1 > 0.f && (s0 > kApart * s1 || s1 > kApart * s0) ? kAgain | kNotSecond : 0;
                // the visit's scale (0: neither page is in the cache)
                const float s_now = mark & kNotFirst ? s1 : mark & kNotSecond ? s0 : fmaxf(s0, s1);
                if (j == sg.j0 && !(mark & kNotFirst)) s_ref = s_last = s_now > 0.f ? s_now : 1.f;
                if (s_now > 0.f) {
                    if (s_now > kApart * s_last || s_last > kApart * s_now) mark |= kJump;
                    s_last = s_now;
                }
                s_hi = fmaxf(s_hi, s_last);
                s_lo = fminf(s_lo, s_last);
                if (s_hi > kApart * s_lo) mark |= kWide;
                // no page: zero rows; the softmax need not look at the scale of what does not count
                if (s0 == 0.f || (mark & kNotFirst)) s0 = s_ref;
                if (s1 == 0.f || (mark & kNotSecond)) s1 = s_ref;
                if (ok && !starve && elect()) {
                    visit[g & 3] = make_float4(s0, s1, __int_as_float(mark), s_hi);
                    uint8_t* dst = ropes + (g % NR) * C::kSlotBytes;
                    ptx::mbar_expect_tx(&rope_full[g % NR], kRopeBytes);
                    ptx::tma_load_2d_hint(dst, &tm_rope, &rope_full[g % NR], kDc, r0, policy);
                    ptx::tma_load_2d_hint(dst + kRopeBytes / 2, &tm_rope, &rope_full[g % NR], kDc, r1, policy);
                }
                g += ok && !starve;
            }
        }
        if (!ok) fail(err, abort_flag, 11);
        if (lane == 0) {
            // loads still in flight (after an abort) land before the CTA leaves
#pragma unroll 1
            for (uint32_t k = 0; k < (uint32_t)NC && k < cn; ++k)
                ptx::mbar_wait(&chunk_full[(cn - 1 - k) % NC], ((cn - 1 - k) / NC) & 1, nullptr);
#pragma unroll 1
            for (uint32_t k = 0; k < (uint32_t)NR && k < g; ++k)
                ptx::mbar_wait(&rope_full[(g - 1 - k) % NR], ((g - 1 - k) / NR) & 1, nullptr);
        }
    } else if (warp == 1) {
        // ---------------------------------------------- queries and score products
        constexpr uint32_t idesc = idesc_f8(128, 2 * R, 0, 0, 0);
        constexpr uint32_t h128 = desc_hi(1024, 2), h64 = desc_hi(512, 4);
        const uint32_t chunk0 = desc_lo(ptx::smem_u32(chunks), 16), rope0 = desc_lo(ptx::smem_u32(ropes), 16),
                       q0 = desc_lo(ptx::smem_u32(qimg), 16);
        auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_warp(bar, parity, abort_flag); };
        pdl_wait();   // the queries come from the previous kernel of this call
        uint32_t g = 0, piece = 0, slot = 0, use = 0;   // tile, piece, chunk slot and how often the slots were gone through
        bool ok = true;
        while (ok && next_piece()) {
            // Every softmax thread has read the last scores: their products are done with the
            // queries, and it is done with the row scales.
            if (g > 0 && !wait(&s_free[(g - 1) & 1], ((g - 1) >> 1) & 1)) { ok = false; break; }
            if (elect()) {
                ptx::mbar_expect_tx(q_full, C::kQBytes + R * 4);
                const uint8_t* from = ws.q_img + (size_t)sg.item * C::kQBytes;
                for (int o = 0; o < C::kQBytes; o += C::kQBytes / 4)
                    ptx::bulk_load(qimg + o, from + o, C::kQBytes / 4, q_full);
                ptx::bulk_load(qs, ws.q_scale + (size_t)sg.item * R, R * 4, q_full);
            }
            __syncwarp();
            // in flight after an abort: waited for without a look at the flag
            if (!__all_sync(0xffffffffu, ptx::mbar_wait(q_full, piece & 1, nullptr))) { ok = false; break; }
            ++piece;
#pragma unroll 1
            for (int left = uniform(sg.j1 - sg.j0); left > 0; ++g) {
                if (g >= 2 && !wait(&s_free[g & 1], ((g >> 1) - 1) & 1)) { ok = false; break; }
                const uint32_t d = tmem + (g & 1) * (2 * R);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (!wait(&chunk_full[slot], use & 1)) { ok = false; break; }
                    ptx::tc_fence_after();
                    const uint32_t a = chunk0 + slot * (kChunkBytes >> 4), b = q0 + c * (2 * R * 128 >> 4);
                    if (elect()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma_f8(d, a + 2 * k, h128, b + 2 * k, h128, idesc, (c | k) != 0);
                    }
                    if (++slot == NC) slot = 0, ++use;
                }
                if (!ok || !wait(&rope_full[g % NR], (g / NR) & 1)) { ok = false; break; }
                ptx::tc_fence_after();
                const uint32_t a = rope0 + (g % NR) * (C::kSlotBytes >> 4), b = q0 + 4 * (2 * R * 128 >> 4);
                if (elect()) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) mma_f8(d, a + 2 * k, h64, b + 2 * k, h64, idesc, 1);
                    ptx::mma_commit(&s_full[g & 1]);
                }
                left -= uniform(!(marks(visit[g & 3]) & kAgain));
            }
        }
        if (!ok) fail(err, abort_flag, 12);
        if (elect()) ptx::mma_commit(drain);
        if (!ptx::mbar_wait(drain, 0, nullptr)) fail(err, abort_flag, 14);
    } else if (warp == 2) {
        // ---------------------------------------------------------- O products
        constexpr uint32_t idesc = idesc_f8(128, C::NP, 1, 1, 1);
        constexpr uint32_t h128 = desc_hi(1024, 2), hp = C::kPRow == 128 ? h128 : desc_hi(512, 4);
        const uint32_t chunk0 = desc_lo(ptx::smem_u32(chunks), kChunkBytes),
                       p0 = desc_lo(ptx::smem_u32(ropes), C::kSlotBytes);
        uint32_t g = 0, slot0 = 0;
        bool ok = true;
        while (ok && next_piece()) {
            uint32_t acc0 = 0;
#pragma unroll 1
            for (int left = uniform(sg.j1 - sg.j0); left > 0; ++g) {
                if (!wait_warp(&p_ready[g & 1], (g >> 1) & 1, abort_flag)) { ok = false; break; }
                ptx::tc_fence_after();
                const uint32_t p = p0 + (g % NR) * (C::kSlotBytes >> 4);
                // chunk by chunk, so that the first slots are free for the next loads early
                if (elect()) {
                    uint32_t slot = slot0;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t a = chunk0 + slot * (kChunkBytes >> 4), d = tmem + C::kColO + c * C::NP;
#pragma unroll
                        for (int k = 0; k < kT / 32; ++k)
                            mma_f8(d, a + 256 * k, h128, p + (32 * C::kPRow >> 4) * k, hp, idesc, acc0 | (k > 0));
                        ptx::mma_commit(&chunk_empty[slot]);
                        slot = slot + 1 == NC ? 0 : slot + 1;
                    }
                    ptx::mma_commit(&o_done[g & 1]);
                    ptx::mma_commit(&rope_empty[g % NR]);
                }
                slot0 = (slot0 + 4) % NC;
                acc0 = 1;
                left -= uniform(!(marks(visit[g & 3]) & kAgain));
            }
        }
        if (!ok) fail(err, abort_flag, 16);
        if (elect()) ptx::mma_commit(drain);
        if (!ptx::mbar_wait(drain, 0, nullptr)) fail(err, abort_flag, 17);
    } else if (warp >= kRoleThreads / 32) {
        // ------------------------------------------------- softmax and epilogue
        const int quad = warp & 3, grp = (warp - kRoleThreads / 32) >> 2;
        const int tok = 32 * quad + lane;                       // token of the tile = TMEM lane
        const int c0 = grp * HC;                                // first row of this thread
        const uint32_t lane_addr = tmem + ((uint32_t)(32 * quad) << 16);
        bool ok = true;
        auto uwait = [&](uint64_t* bar, uint32_t parity) { return wait_warp(bar, parity, abort_flag); };
        uint32_t meets = 0;
        auto meet = [&]() {   // the four warps that share these rows
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&grp_bar[grp]);
            if (!uwait(&grp_bar[grp], meets & 1)) ok = false;
            ++meets;
        };
        uint32_t piece = 0, g = 0;
        f32x2 l[HC / 2];           // this thread's share of each row's sum
        float m_row = 0.f, m_top = 0.f;   // lane i: reference of row c0 + i, and the highest it has had
        while (ok && next_piece()) {
            float s_ref = 1.f, s_hi = 1.f;   // the first visit's scale and the largest so far
            bool first = true;
            int mark = 0;
#pragma unroll 1
            for (int j = sg.j0; j < sg.j1; j += !(mark & kAgain), ++g, first = false) {
                if (first && !uwait(q_full, piece & 1)) { ok = false; break; }   // row scales
                if (!uwait(&rope_full[g % NR], (g / NR) & 1)) { ok = false; break; }   // page scales
                // O of tile g - 2 is done, whose P lay where this tile's goes.  Every phase of a
                // barrier is waited for, so that a later wait cannot take an older one for its own.
                if (g >= 2 && !uwait(&o_done[g & 1], ((g >> 1) - 1) & 1)) { ok = false; break; }
                const float4 vi = visit[g & 3];
                mark = marks(vi);
                s_hi = vi.w;
                const float s = quad < 2 ? vi.x : vi.y;
                if (first) {
                    s_ref = vi.w;
#pragma unroll
                    for (int i = 0; i < HC / 2; ++i) l[i] = 0;
                    m_row = 0.f;
                    if (lane < HC) {   // the four warps write the same; read by a warp that wrote
                        nrefs[c0 + lane] = 0.f;
                        row_kt[c0 + lane] = qs[c0 + lane] * (scale_log2 * s_ref);
                    }
                    __syncwarp();
                }
                const bool same = s == s_ref;
                const float back = same ? 1.f : s_ref / s;
                if (!uwait(&s_full[g & 1], (g >> 1) & 1)) { ok = false; break; }
                ptx::tc_fence_after();
                f32x2 arg[HC / 2];   // two rows each
                {
                    uint32_t a[HC], b[HC];
                    tmem_ld(lane_addr + (g & 1) * (2 * R) + c0, a);
                    tmem_ld(lane_addr + (g & 1) * (2 * R) + R + c0, b);
                    ptx::tmem_wait_ld();
                    ptx::tc_fence_before();
#pragma unroll
                    for (int i = 0; i < HC / 2; ++i) arg[i] = add2(pair(a[2 * i], a[2 * i + 1]), pair(b[2 * i], b[2 * i + 1]));
                }
                if (same) {
#pragma unroll
                    for (int i = 0; i < HC / 2; i += 2) {
                        const ulonglong2 f = *(const ulonglong2*)(row_kt + c0 + 2 * i), m = *(const ulonglong2*)(nrefs + c0 + 2 * i);
                        arg[i] = fma2(arg[i], f.x, m.x);
                        arg[i + 1] = fma2(arg[i + 1], f.y, m.y);
                    }
                } else {   // a page of another scale than the piece's first
                    const float kt = scale_log2 * s, shift = log2f(s) - log2f(s_ref);
#pragma unroll
                    for (int i = 0; i < HC / 2; i += 2) {
                        const ulonglong2 f = *(const ulonglong2*)(qs + c0 + 2 * i), m = *(const ulonglong2*)(nrefs + c0 + 2 * i);
                        arg[i] = fma2(arg[i], mul2(f.x, pair(kt, kt)), add2(m.x, pair(shift, shift)));
                        arg[i + 1] = fma2(arg[i + 1], mul2(f.y, pair(kt, kt)), add2(m.y, pair(shift, shift)));
                    }
                }
                ptx::mbar_arrive(&s_free[g & 1]);   // also done with the row scales
                // some row does not see the whole tile, or a page does not count
                const bool edge = (j + 1) * kT > sg.kmin || (mark & (kNotFirst | kNotSecond));
                if (edge) {
                    const int at = mark & (quad < 2 ? kNotFirst : kNotSecond) ? 0x7fffffff : j * kT + tok;
                    if (sg.kmin == sg.kmax) {
                        if (at >= sg.kmax) {
#pragma unroll
                            for (int i = 0; i < HC / 2; ++i) arg[i] = pair(-INFINITY, -INFINITY);
                        }
                    } else {
                        const int row = sg.g * R + c0;
                        int t = row / src.s.H, h = row - t * src.s.H;   // of the thread's first row
                        int keys = src.keys(sg.len, t);
#pragma unroll
                        for (int i = 0; i < HC / 2; ++i) {
                            float x, y;
                            unpair(arg[i], x, y);
                            if (at >= keys) x = -INFINITY;
                            if (++h == src.s.H) h = 0, ++keys;
                            if (at >= keys) y = -INFINITY;
                            if (++h == src.s.H) h = 0, ++keys;
                            arg[i] = pair(x, y);
                        }
                    }
                }
                // Does every row keep its reference?  Sign bits of the arguments, anded over the
                // tile's tokens, name the rows whose largest p is below 2^-6; any argument past the
                // top sends the warp's word to "all".
                {
                    uint32_t low = 0;
                    float top = -INFINITY;
#pragma unroll
                    for (int i = 0; i < HC / 2; ++i) {
                        float x, y;
                        unpair(arg[i], x, y);
                        low = __funnelshift_l(__float_as_uint(x), low, 1);
                        low = __funnelshift_l(__float_as_uint(y), low, 1);
                        top = fmaxf(fmaxf(top, x), y);
                    }
                    low = __reduce_and_sync(0xffffffffu, low);
                    if (__any_sync(0xffffffffu, top > kTopLog2)) low = 0xffffffffu;
                    if (lane == 0) flags[((g & 1) * CG + grp) * 4 + quad] = low;
                }
                meet();
                if (!ok) break;
                const uint4 fl = *(const uint4*)(flags + ((g & 1) * CG + grp) * 4);
                const bool over = fl.x == 0xffffffffu || fl.y == 0xffffffffu || fl.z == 0xffffffffu || fl.w == 0xffffffffu;
                if (first || (mark & kJump) || over || (fl.x & fl.y & fl.z & fl.w) != 0) {
                    // this warp's largest argument of each row, then the tile's, row i in lane i
                    float keep = -INFINITY;
#pragma unroll
                    for (int i = 0; i < HC / 2; ++i) {
                        float x, y;
                        unpair(arg[i], x, y);
                        x = warp_max(x);
                        y = warp_max(y);
                        if (lane == 2 * i) keep = x;
                        if (lane == 2 * i + 1) keep = y;
                    }
                    if (lane < HC) ((float*)(red + grp * 16 + lane))[quad] = keep;
                    meet();
                    if (!ok) break;
                    float step = 0.f;   // new reference - old one
                    if (lane < HC) {
                        const float4 v = red[grp * 16 + lane];
                        const float mx = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
                        if (mx > -INFINITY && (first || (mark & kJump) || mx > kTopLog2 || mx < 0.f)) {
                            step = mx - kSetLog2;
                            if (!first) step = fmaxf(step, m_top - kFarLog2 - m_row);
                        }
                        m_row += step;
                        m_top = first ? m_row : fmaxf(m_top, m_row);
                        nrefs[c0 + lane] = -m_row;   // the four warps write the same
                    }
                    const float alpha = ex2(-step);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < HC / 2; ++i)
                        arg[i] = sub2(arg[i], pair(__shfl_sync(0xffffffffu, step, 2 * i), __shfl_sync(0xffffffffu, step, 2 * i + 1)));
                    if (!first && __any_sync(0xffffffffu, step != 0.f)) {   // the same in the four warps
                        if (!uwait(&o_done[(g - 1) & 1], ((g - 1) >> 1) & 1)) { ok = false; break; }
                        ptx::tc_fence_after();
#pragma unroll
                        for (int i = 0; i < HC / 2; ++i)
                            l[i] = mul2(l[i], pair(__shfl_sync(0xffffffffu, alpha, 2 * i), __shfl_sync(0xffffffffu, alpha, 2 * i + 1)));
                        float al[HC];
#pragma unroll
                        for (int i = 0; i < HC; ++i) al[i] = __shfl_sync(0xffffffffu, alpha, i);
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t r[C::kTerms][HC];
                            const uint32_t ad = lane_addr + C::kColO + c * C::NP + c0;
#pragma unroll
                            for (int t = 0; t < C::kTerms; ++t) tmem_ld(ad + t * R, r[t]);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int t = 0; t < C::kTerms; ++t) {
#pragma unroll
                                for (int i = 0; i < HC; ++i) r[t][i] = __float_as_uint(__uint_as_float(r[t][i]) * al[i]);
                                tmem_st(ad + t * R, r[t]);
                            }
                        }
                        ptx::tmem_wait_st();
                    }
                }
                // P in three E5M2 terms; the sums take 2^(z - M), not rounded
                uint32_t p8[C::kTerms][HC / 4];
                const f32x2 back2 = pair(back, back);
#pragma unroll
                for (int i = 0; i < HC / 4; ++i) {
                    float x[4];
                    unpair(arg[2 * i], x[0], x[1]);
                    unpair(arg[2 * i + 1], x[2], x[3]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) x[q] = ex2(x[q]);
                    l[2 * i] = fma2(pair(x[0], x[1]), back2, l[2 * i]);
                    l[2 * i + 1] = fma2(pair(x[2], x[3]), back2, l[2 * i + 1]);
                    uint32_t v0 = ptx::pack_f16(x[0] * kPGain, x[1] * kPGain), v1 = ptx::pack_f16(x[2] * kPGain, x[3] * kPGain);
#pragma unroll
                    for (int t = 0; t < C::kTerms; ++t) {
                        p8[t][i] = e5m2x4(v0, v1);
                        if (t + 1 < C::kTerms) {
                            v0 = rest_of(v0, p8[t][i], 0x1404);
                            v1 = rest_of(v1, p8[t][i], 0x3424);
                        }
                    }
                }
                // row tok of P: columns t R + c0 .. + 7, 16-byte unit u at u ^ (tok mod 8) in 128-byte
                // rows, u ^ (tok / 2 mod 4) in 64-byte ones
                uint8_t* prow = ropes + (g % NR) * C::kSlotBytes + tok * C::kPRow;
                const int sw = C::kPRow == 128 ? tok & 7 : (tok >> 1) & 3;
#pragma unroll
                for (int t = 0; t < C::kTerms; ++t) {
                    const int at = t * R + c0;
                    *(uint2*)(prow + (((at >> 4) ^ sw) << 4) + (at & 8)) = make_uint2(p8[t][0], p8[t][1]);
                }
                if (edge) {
                    // Rows that some row of the group must not see may hold NaN codes (what lies
                    // behind the sequence's end, a later token's row), and 0 x NaN is NaN: those
                    // codes become 0.  A row that does see them has NaN scores already.
                    const int n0 = max(sg.kmin - j * kT, 0);
#pragma unroll 1
                    for (int e = threadIdx.x - kRoleThreads; e < (kT - n0) * 32; e += C::kSoft) {
                        const int r = n0 + (e >> 5), c = (e >> 3) & 3, u = e & 7;
                        uint4* at = (uint4*)(chunks + ((4 * g + c) % NC) * kChunkBytes + r * 128) + u;
                        uint4 v = *at;
                        v.x &= ~__vcmpeq4(v.x & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        v.y &= ~__vcmpeq4(v.y & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        v.z &= ~__vcmpeq4(v.z & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        v.w &= ~__vcmpeq4(v.w & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        *at = v;
                    }
                }
                ptx::fence_proxy_async_smem();   // read by the tensor cores
                ptx::tc_fence_before();
                ptx::mbar_arrive(&p_ready[g & 1]);
            }
            if (!ok) break;
            // ---- the piece's sums over all tokens, then its normalised output
            // after step o, a lane holds the sums over 32 / o lanes of the rows whose bits match its own
            float ls[HC];
#pragma unroll
            for (int i = 0; i < HC / 2; ++i) unpair(l[i], ls[2 * i], ls[2 * i + 1]);
#pragma unroll
            for (int w = HC / 2, o = 16; o > 0; o >>= 1, w = w > 0 ? w / 2 : 0) {
                if (w > 0) {
                    const bool up = (lane & o) != 0;
#pragma unroll
                    for (int i = 0; i < HC / 2; ++i)
                        if (i < w) {
                            const float mine = up ? ls[i + w] : ls[i], give = up ? ls[i] : ls[i + w];
                            ls[i] = mine + __shfl_xor_sync(0xffffffffu, give, o);
                        }
                } else {
                    ls[0] += __shfl_xor_sync(0xffffffffu, ls[0], o);
                }
            }
            auto o_ready = [&]() {
                if (!uwait(&o_done[(g - 1) & 1], ((g - 1) >> 1) & 1)) ok = false;
                ptx::tc_fence_after();
            };
            // latents 128 c + tok of O
            auto load_o = [&](int c, float (&y)[HC]) {
                uint32_t r[C::kTerms][HC];
#pragma unroll
                for (int t = 0; t < C::kTerms; ++t) tmem_ld(lane_addr + C::kColO + c * C::NP + t * R + c0, r[t]);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < HC; ++i)
                    y[i] = fmaf(0.125f, fmaf(0.125f, __uint_as_float(r[2][i]), __uint_as_float(r[1][i])), __uint_as_float(r[0][i]));
            };
            // Lane i: row c0 + i leaves as fp16 values f O, with a unit of its own.  Pages of about one scale:
            // 64 x the mean code (at most 448 each, so <= 28672, and down to 2^-20 with all bits), in
            // units of the largest scale.  Pages of very different scales: against the row's largest
            // |O|, which takes another pass over it (a row under 2^-100 counts as zero).
            const bool wide = mark & kWide;
            float keep = 0.f;                         // lane i: the largest |O| of row c0 + i this warp has
            if (wide) {
                o_ready();
                if (!ok) break;
                float most[HC];
#pragma unroll
                for (int i = 0; i < HC; ++i) most[i] = 0.f;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    float y[HC];
                    load_o(c, y);
#pragma unroll
                    for (int i = 0; i < HC; ++i) most[i] = fmaxf(most[i], fabsf(y[i]));
                }
#pragma unroll
                for (int i = 0; i < HC; ++i) {
                    const float m = warp_max(most[i]);
                    if (lane == i) keep = m;
                }
            }
            // row held by this lane: the lane bits from 16 down, as many as HC has
            const int my_row = lane >> 2;
            float* sums = (float*)(red + grp * 16);   // [4 quarters][8 sums, 8 largest |O|]
            meet();   // red is read
            if (!ok) break;
            sums[quad * 16 + my_row] = ls[0];
            if (lane < HC) sums[quad * 16 + 8 + lane] = keep;
            meet();
            o_ready();
            if (!ok) break;
            float f = 0.f;
            if (lane < HC) {
                const float t = (sums[lane] + sums[16 + lane]) + (sums[32 + lane] + sums[48 + lane]);
                const float mean = t != 0.f ? s_ref / (kPGain * t) : 0.f;   // times O: the row's values
                float unit;
                if (wide) {
                    const float top = fmaxf(fmaxf(sums[8 + lane], sums[24 + lane]), fmaxf(sums[40 + lane], sums[56 + lane]));
                    f = top >= 0x1p-100f ? 0x1p14f / top : 0.f;
                    unit = mean * (top * 0x1p-14f);
                } else {
                    unit = s_hi * 0x1p-6f;
                    f = mean / unit;
                }
                if (quad == 0) ws.part_ml[(size_t)sg.slot * R + c0 + lane] = make_float4(m_row, t, unit, 0.f);
            }
            // (a warp's store is 64 contiguous bytes; turning the tile around with shuffles for
            // 16-byte stores took longer)
            __half* po = ws.part_o + ((size_t)sg.slot * R + c0) * kDc + tok;
            float fr[HC];
#pragma unroll
            for (int i = 0; i < HC; ++i) fr[i] = __shfl_sync(0xffffffffu, f, i);
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                float y[HC];
                load_o(c, y);
#pragma unroll
                for (int i = 0; i < HC; ++i) po[i * kDc + 128 * c] = __float2half_rn(y[i] * fr[i]);
            }
            ptx::tc_fence_before();
            meet();   // the sums are read
            ++piece;
        }
        if (!ok) fail(err, abort_flag, 13);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) ptx::tmem_dealloc(tmem, C::kTmemCols);
}

// ------------------------------------------------------------------ the queries
// q_lat[v, h, :] = W_UK[h]^T q_nope[v, h, :] for 128 queries v = (b, t) of one head.  A cluster
// of two CTAs shares a (head, 128 queries): CTA r makes latent columns 256 r ..., as
// D [128 queries x 256] = Q_h [128 x 128] . W_UK^T[h][256 r ..]^T, and takes rotary columns 32 r ...
// A query is a TMEM lane; its largest value is agreed on through distributed shared memory,
// and the row [q_lat | q_rope] gets one power-of-two scale that puts that value in (224, 448].
// It leaves as two E4M3 terms in the shared-memory image the attention kernel loads whole.
// Latency bounds it.  One CTA per head took 6.1 us of a one-sequence step; a cluster of four
// is as quick as this one, but 128 heads' 512 CTAs need a second wave, and the attention
// kernel may start only when the last of them has.
constexpr int kAbsorbThreads = 512, kAbsorbCluster = 2;
constexpr int kAbsorbA = 2 * 128 * 128, kAbsorbB = 2 * 256 * 128;
constexpr int kAbsorbSmem = kAbsorbA + kAbsorbB + 5 * 128 * 4 + 64 + 1024;

// smallest e with amax <= 448 * 2^e (0 for 0), not below -100
__device__ __forceinline__ int query_exponent(float amax) {
    if (!(amax > 0.f)) return 0;
    const uint32_t u = __float_as_uint(amax);
    return max((int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0), -100);
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// 2 n values times inv -> n words' worth of hi and lo codes (two codes per 16 bits)
template <int N>
__device__ __forceinline__ void split_e4m3(const float (&x)[2 * N], float inv, uint32_t (&hi)[N / 2], uint32_t (&lo)[N / 2]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float a = x[2 * i] * inv, b = x[2 * i + 1] * inv;
        const uint32_t h = e4m3x2_f32(a, b), f = f16x2_of_e4m3(h);
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f));
        const uint32_t t = e4m3x2_f32(a - v.x, b - v.y);
        hi[i / 2] = i % 2 ? hi[i / 2] | h << 16 : h;
        lo[i / 2] = i % 2 ? lo[i / 2] | t << 16 : t;
    }
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster(const float* p, uint32_t rank) {   // the same place in CTA `rank`
    float v;
    asm volatile(
        "{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %1, %2;\n\tld.shared::cluster.f32 %0, [ra];\n\t}"
        : "=f"(v)
        : "r"(ptx::smem_u32(p)), "r"(rank)
        : "memory");
    return v;
}

// The work split, by one CTA beside those that make the queries: for every range the virtual
// sequence that holds its first unit (ws.start), for every item where its pieces' partials
// lie (ws.pieces).
__device__ void plan(const Src& src, const Ws& ws, DevErr err) {
    __shared__ long long wsum[kAbsorbThreads / 32];
    constexpr int kWarps = kAbsorbThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Shape& s = src.s;
    const int nv = src.vseqs(), ranges = s.ctas / s.sib;
    // lengths of the first 512 virtual sequences stay in registers
    const int len0 = (int)threadIdx.x < nv ? src.len(src.vseq_b(threadIdx.x)) : 0;
    auto length = [&](int i) { return i < kAbsorbThreads ? len0 : src.len(src.vseq_b(i)); };
    long long mine = 0;
#pragma unroll 1
    for (int i = threadIdx.x; i < nv; i += kAbsorbThreads) mine += cost_of(tiles_of(src.vkeys(length(i), i)));
#pragma unroll 1
    for (int b = threadIdx.x; b < s.B; b += kAbsorbThreads)
        if (src.raw_len(b) < 0) latch(err, kErrOutOfRange, b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) wsum[warp] = mine;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) total += wsum[i];
    const long long per = total > 0 ? (total + ranges - 1) / ranges : 1;
    // ranges without work
    for (int r = threadIdx.x; r < s.ctas; r += kAbsorbThreads)
        if (r >= ranges || r * per >= total) ws.start[r] = make_int4(nv, 0, 0, -1);
    long long carry = 0;
#pragma unroll 1
    for (int c0 = 0; c0 < nv; c0 += kAbsorbThreads) {
        const int i = c0 + (int)threadIdx.x, L = i < nv ? length(i) : 0;
        const int n = i < nv ? tiles_of(src.vkeys(L, i)) : 0;
        const long long cb = cost_of(n);
        long long incl = cb;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        __syncthreads();
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        long long before = carry;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            const long long v = wsum[k];
            before += k < warp ? v : 0;
            carry += v;
        }
        const long long cs = before + incl - cb;
        if (i < nv) {
            // the ranges that start in [cs, cs + cb)
#pragma unroll 1
            for (long long r = (cs + per - 1) / per; r * per < cs + cb && r < ranges; ++r)
                ws.start[r] = make_int4(i, (int)(cs - r * per), (int)min(per, total - r * per), L);
            const long long f = cs + kPieceCost, r0 = f / per;
            const int at = (int)(f - r0 * per);   // place of the first tile in its range
#pragma unroll 1
            for (int k = 0; k < (s.sib > 1 ? s.G : 1); ++k) {
                const int item = s.sib > 1 ? i * s.G + k : i, g = s.sib > 1 ? k : i % s.G;
                const int nt = n > 0 ? tiles_of(src.keys(L, src.last_token(g))) : 0;
                const int np = nt > 0 ? (int)((at + nt - 1) / per) + 1 : 0;
                // slot of piece p > 0: .x + (p - 1) sib
                ws.pieces[item] = make_int2((int)(s.B * s.G + (r0 + 1) * s.sib + (s.sib > 1 ? k : 0)), np);
            }
        }
    }
}

__global__ void __cluster_dims__(kAbsorbCluster, 1, 1) __launch_bounds__(kAbsorbThreads, 2)
absorb_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_w,
              const __nv_bfloat16* __restrict__ q_rope, const Src src, const Ws ws, const DevErr err) {
    const Shape& s = src.s;
    if (blockIdx.x >= kAbsorbCluster * s.H) {   // a cluster apart: uniform
        pdl_wait();
        if (threadIdx.x == 0) pdl_trigger();
        if (blockIdx.x == kAbsorbCluster * s.H && blockIdx.y == 0) plan(src, ws, err);
        return;
    }
    extern __shared__ uint8_t absorb_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)absorb_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *sA = smem, *sB = smem + kAbsorbA;
    float* s_max = (float*)(sB + kAbsorbB);   // [512] each thread's
    float* s_row = s_max + 512;               // [128] this CTA's largest value of each query
    uint64_t* full = (uint64_t*)(s_row + 128);
    uint64_t* d_full = full + 1;
    uint32_t* tmem_slot = (uint32_t*)(d_full + 1);
    const int h = blockIdx.x / kAbsorbCluster, rank = blockIdx.x % kAbsorbCluster;
    const int v0 = blockIdx.y * 128, NV = s.B * s.q_len;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = warp & 3, cg = warp >> 2;
    // With 64 queries or fewer, the lane quarters hold them twice or four times over, and each
    // copy's warps convert a share of the columns: 16 warps at work instead of 4 on a step of 32.
    const int blocks = NV - v0 <= 32 ? 1 : NV - v0 <= 64 ? 2 : 4, share = quad / blocks, width = 16 * blocks;
    if (threadIdx.x == 0) {
        ptx::mbar_init(full, 1);
        ptx::mbar_init(d_full, 1);
        ptx::fence_mbar_init();
        ptx::mbar_expect_tx(full, kAbsorbA + kAbsorbB);
        // the weights first: the call that packed them ended with a kernel of its own (launch_order)
#pragma unroll
        for (int kc = 0; kc < 2; ++kc) ptx::tma_load_2d(sB + kc * 32768, &tm_w, full, 64 * kc, h * kDc + 256 * rank);
        pdl_wait();      // all earlier work is done
        pdl_trigger();   // only now may the next kernel launch
#pragma unroll
        for (int kc = 0; kc < 2; ++kc)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ptx::tma_load_3d(sA + kc * 16384 + i * 4096, &tm_q, full, 64 * kc, v0 + 32 * (i % blocks), h);
    }
    if (warp == 1) {
        ptx::tmem_alloc(tmem_slot, 256);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
    if (warp == 1) {
        const bool landed = ptx::mbar_wait(full, 0, nullptr);
        if (!landed) latch(err, kErrTimeout, 9200000 + h);
        ptx::tc_fence_after();
        if (elect()) {
            constexpr uint32_t idesc = ptx::idesc_bf16_f32(128, 256, 0, 0);
            if (landed) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    ptx::mma_ss(tmem, ptx::desc_kmajor_sw128(ptx::smem_u32(sA) + (k >> 2) * 16384 + 32 * (k & 3)),
                                ptx::desc_kmajor_sw128(ptx::smem_u32(sB) + (k >> 2) * 32768 + 32 * (k & 3)), idesc, k != 0);
                }
            }
            ptx::mma_commit(d_full);   // after a timeout nothing was issued and this completes at once
        }
        __syncwarp();
    }
    const int v = v0 + 32 * (quad % blocks) + lane;
    const bool warp_on = v0 + 32 * (quad % blocks) < NV, on = v < NV;
    const int c0 = 64 * cg + width * share;   // this warp's columns: width from c0
    const uint32_t src_col = tmem + ((uint32_t)(32 * quad) << 16) + c0;
    // this warp's 8 rotary columns; they may come from the previous kernel
    pdl_wait();
    float rope[8] = {};
    if (on) {
        const uint4 a = *(const uint4*)(q_rope + ((size_t)v * s.H + h) * kDr + 32 * rank + 8 * cg);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rope[2 * i] = __uint_as_float(w[i] << 16);
            rope[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    // where the row goes (divisions off the critical path)
    const int R = s.R, b = v / s.q_len, t = v - b * s.q_len, row = t * s.H + h, g = row / R, rh = row - g * R, rl = R + rh;
    const size_t img = (size_t)2 * R * kRow, item = (size_t)b * s.G + g;
    uint8_t* chunk = ws.q_img + item * img + (size_t)(2 * rank + (cg >> 1)) * (2 * R * 128);
    uint8_t* rp = ws.q_img + item * img + (size_t)4 * (2 * R * 128);
    const bool done = __all_sync(0xffffffffu, ptx::mbar_wait(d_full, 0, nullptr));
    if (!done && lane == 0) latch(err, kErrTimeout, 9300000 + h);
    ptx::tc_fence_after();
    float amax = 0.f;
    if (warp_on) {
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(rope[i]));
#pragma unroll 1
        for (int c = 0; c < width; c += 16) {
            uint32_t r[16];
            tmem_ld(src_col + c, r);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(__uint_as_float(r[i])));
        }
    }
    s_max[threadIdx.x] = amax;
    __syncthreads();
    if (threadIdx.x < 128) {   // query threadIdx.x of the CTA: the warps that hold a part of it
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if ((i & 3) % blocks == (int)(threadIdx.x >> 5) % blocks) m = fmaxf(m, s_max[32 * i + lane]);
        s_row[threadIdx.x] = m;
    }
    cluster_sync();
    if (warp_on) {
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < kAbsorbCluster; ++i) amax = fmaxf(amax, ld_cluster(s_row + 32 * (quad % blocks) + lane, i));
        const int e = query_exponent(amax);
        // an infinite query value must not saturate: times 0 it is NaN, as its scores are
        const float inv = amax < INFINITY ? pow2i(-e) : 0.f;
#pragma unroll 1
        for (int c = 0; c < width; c += 16) {
            uint32_t r[16];
            tmem_ld(src_col + c, r);
            ptx::tmem_wait_ld();
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
            uint32_t hi[4], lo[4];
            split_e4m3<8>(x, inv, hi, lo);
            const int u = (c0 + c) / 16 & 7;   // 16-byte unit of the row's chunk
            if (on) {
                *(uint4*)(chunk + rh * 128 + ((u ^ (rh & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *(uint4*)(chunk + rl * 128 + ((u ^ (rl & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        }
        if (on && share == 0) {
            uint32_t hi[2], lo[2];
            split_e4m3<4>(rope, inv, hi, lo);
            const int ru = 2 * rank + (cg >> 1);   // 16-byte unit of the rotary part
            *(uint2*)(rp + rh * 64 + ((ru ^ ((rh >> 1) & 3)) << 4) + 8 * (cg & 1)) = make_uint2(hi[0], hi[1]);
            *(uint2*)(rp + rl * 64 + ((ru ^ ((rl >> 1) & 3)) << 4) + 8 * (cg & 1)) = make_uint2(lo[0], lo[1]);
            if (rank == 0 && cg == 0) ws.q_scale[item * R + rh] = pow2i(e);
            // rows that pad a sequence's last group are zero: head h writes the h-th, (h + H)-th, ...
            if (t == s.q_len - 1) {
#pragma unroll 1
                for (int p = s.q_len * s.H + h; p < s.G * R; p += s.H) {
                    const int ph = p % R, pl = R + ph;
                    uint8_t* pb = ws.q_img + ((size_t)b * s.G + p / R) * img;
                    uint8_t* pc = pb + (size_t)(2 * rank + (cg >> 1)) * (2 * R * 128);
                    const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        *(uint4*)(pc + ph * 128 + 64 * (cg & 1) + 16 * u) = z;
                        *(uint4*)(pc + pl * 128 + 64 * (cg & 1) + 16 * u) = z;
                    }
                    *(uint2*)(pb + (size_t)4 * (2 * R * 128) + ph * 64 + 32 * rank + 8 * cg) = make_uint2(0, 0);
                    *(uint2*)(pb + (size_t)4 * (2 * R * 128) + pl * 64 + 32 * rank + 8 * cg) = make_uint2(0, 0);
                    if (rank == 0 && cg == 0) ws.q_scale[((size_t)b * s.G + p / R) * R + ph] = 1.f;
                }
            }
        }
    }
    ptx::tc_fence_before();
    cluster_sync();   // no CTA leaves while another reads its shared memory
    if (warp == 1) ptx::tmem_dealloc(tmem, 256);
}

// ------------------------------------------------------------- merge and W_UV
// out[v, h, :] = W_UV[h] o_lat[v, h, :],
// o_lat = sum_p 2^(m_p - m) l_p u_p y_p / sum_p 2^(m_p - m) l_p over the row's pieces, y_p the
// piece's output in units of u_p.  One CTA per (head, `per` queries), per = 32, or 16
// or 8 where that still is one wave of CTAs (48 sequences, 16 heads, cold caches: 50.2 -> 47.1 us).  W_UV[h]
// comes by TMA before the wait for the attention kernel; sixteen warps merge the rows into the B
// operand as two bf16 terms (together 16 bits, so o_lat is not rounded to 8), rows r and 32 + r,
// and the two halves of D [128 x 64] = W_UV[h] . o_lat^T are added as they are read: W_UV leaves
// shared memory once.  Latency bounds it: the list of pieces, their statistics and outputs.
constexpr int kMergeThreads = 512, kMergeN = 32;
constexpr int kMergeA = 8 * 128 * 128, kMergeRows = 2 * kMergeN * 128, kMergeB = 8 * kMergeRows;
constexpr int kMergeSmem = kMergeA + kMergeB + 64 + 1024;

__global__ void __launch_bounds__(kMergeThreads, 1)
merge_kernel(const __grid_constant__ CUtensorMap tm_w, const Src src, const Ws ws, __nv_bfloat16* __restrict__ out,
             int per, const DevErr err) {
    extern __shared__ uint8_t merge_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)merge_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *sA = smem, *sB = smem + kMergeA;
    uint64_t* a_full = (uint64_t*)(sB + kMergeB);
    uint64_t* d_full = a_full + 1;
    uint32_t* tmem_slot = (uint32_t*)(d_full + 1);
    const Shape& s = src.s;
    const int h = blockIdx.x, n0 = blockIdx.y * per, NV = s.B * s.q_len;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        ptx::mbar_init(a_full, 1);
        ptx::mbar_init(d_full, 1);
        ptx::fence_mbar_init();
        ptx::mbar_expect_tx(a_full, kMergeA);
#pragma unroll
        for (int kc = 0; kc < 8; ++kc) ptx::tma_load_2d(sA + kc * 16384, &tm_w, a_full, 64 * kc, h * 128);
        pdl_trigger();
    }
    if (warp == 1) {
        ptx::tmem_alloc(tmem_slot, 2 * kMergeN);
        ptx::tmem_relinquish();
    }
    // More than 16 queries: rows warp and warp + 16, both rows' requests in flight together.
    // 8 or fewer: `shares` warps take every shares-th piece of one row each (a row of one long
    // sequence has a piece per CTA).
    const int rows = min(per, NV - n0);
    const int shares = rows > 8 ? 1 : rows > 4 ? 2 : rows > 2 ? 4 : rows > 1 ? 8 : 16, share = warp % shares, mine = rows > 16 ? 2 : 1;
    int item[2], rin[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int v = min(n0 + (shares > 1 ? warp / shares : warp + 16 * k), NV - 1);
        const int b = v / s.q_len, row = (v - b * s.q_len) * s.H + h, g = row / s.R;
        item[k] = b * s.G + g;
        rin[k] = row - g * s.R;
    }
    pdl_wait();   // the partials come from the attention kernel
    int2 pc[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (k < mine) pc[k] = ws.pieces[item[k]];
    auto at = [&](int k, int p) -> size_t {   // row of part_o and part_ml
        return (size_t)(p == 0 ? item[k] : pc[k].x + (p - 1) * s.sib) * s.R + rin[k];
    };
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 ml[2];        // statistics of the first 32 pieces (lane p)
    uint4 x[2][4][2];    // this warp's first four pieces
    auto fetch = [&](int k, int q, size_t row) {
        const uint4* from = (const uint4*)(ws.part_o + row * kDc + 16 * lane);
        x[k][q][0] = from[0];
        x[k][q][1] = from[1];
    };
    auto request = [&](int k, int i0) {   // pieces share + shares (i0 .. i0 + 3)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int p = share + shares * (i0 + q);
            if (p > 0 && p < pc[k].y) fetch(k, q, at(k, p));
        }
    };
    // the first piece's place is known without `pieces` (and holds nothing if there is none)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (k >= mine) break;
        ml[k] = ws.part_ml[at(k, 0)];
        if (share == 0) fetch(k, 0, at(k, 0));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (k >= mine) break;
        if (lane >= pc[k].y) ml[k] = none;
        else if (lane > 0) ml[k] = ws.part_ml[at(k, lane)];
        request(k, 0);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (k >= mine) break;
        const int r = shares > 1 ? warp / shares : warp + 16 * k, np = pc[k].y;
        float acc[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.f;
        // a piece without a key of this row (sum 0) has no reference
        float M = ml[k].y != 0.f ? ml[k].x : -INFINITY;
#pragma unroll 1
        for (int p = 32 + lane; p < np; p += 32) {
            const float4 o = ws.part_ml[at(k, p)];
            if (o.y != 0.f) M = fmaxf(M, o.x);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float sum = 0.f;
#pragma unroll 1
        for (int p0 = 0; p0 < np; p0 += 32) {   // lane i: weight of piece p0 + i
            if (p0 > 0) ml[k] = p0 + lane < np ? ws.part_ml[at(k, p0 + lane)] : none;
            const float e = ml[k].y != 0.f ? exp2f(ml[k].x - M) * ml[k].y : 0.f, w = e * ml[k].z;
            sum += e;
            const int n = min(32, np - p0);   // (shares divides 32)
#pragma unroll 1
            for (int q0 = share; q0 < n; q0 += 4 * shares) {
                if (p0 + q0 > share) request(k, (p0 + q0) / shares);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int i = q0 + q * shares;
                    const float wq = __shfl_sync(0xffffffffu, w, i & 31);
                    if (i < n && wq != 0.f) {
                        const uint32_t word[8] = {x[k][q][0].x, x[k][q][0].y, x[k][q][0].z, x[k][q][0].w,
                                                  x[k][q][1].x, x[k][q][1].y, x[k][q][1].z, x[k][q][1].w};
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&word[c]));
                            acc[2 * c] = fmaf(wq, f.x, acc[2 * c]);
                            acc[2 * c + 1] = fmaf(wq, f.y, acc[2 * c + 1]);
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] *= inv;
        if (shares > 1) {   // the shares of a row meet in shared memory, and are added in order
            float4* to4 = (float4*)(sB + warp * 2048) + lane;
#pragma unroll
            for (int i = 0; i < 4; ++i) to4[32 * i] = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
            __syncthreads();
            // words share * 512 / shares .. of the row are this warp's
            const int n = 16 / shares, w0 = share * (512 / shares) + lane;
            const float* all = (const float*)(sB + (warp - share) * 2048) + w0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                acc[i] = 0.f;
                if (i < n) {
#pragma unroll 4
                    for (int o = 0; o < shares; ++o) acc[i] += all[512 * o + 32 * i];
                }
            }
            __syncthreads();   // the shares are read
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) {   // word 128 u + 4 l + e is column 16 l + 4 u + e
                    const int w = w0 + 32 * i, c = 16 * ((w >> 2) & 31) + 4 * (w >> 7) + (w & 3);
                    const __nv_bfloat16 hi = __float2bfloat16_rn(acc[i]), lo = __float2bfloat16_rn(acc[i] - __bfloat162float(hi));
                    __nv_bfloat16* to = (__nv_bfloat16*)(sB + (c >> 6) * kMergeRows + r * 128 + ((((c >> 3) & 7) ^ (r & 7)) << 4)) + (c & 7);
                    to[0] = hi;
                    to[kMergeN * 64] = lo;
                }
            break;
        }
        // columns 16 lane .. +15 of row r: chunk lane / 4, 16-byte units 2 (lane % 4) and + 1
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            hi[i] = ptx::pack_bf16(acc[2 * i], acc[2 * i + 1]);
            lo[i] = ptx::pack_bf16(acc[2 * i] - __uint_as_float(hi[i] << 16),
                                   acc[2 * i + 1] - __uint_as_float(hi[i] & 0xFFFF0000u));
        }
        uint8_t* to = sB + (lane >> 2) * kMergeRows + r * 128;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int u = ((2 * (lane & 3) + q) ^ (r & 7)) << 4;
            *(uint4*)(to + u) = make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
            *(uint4*)(to + kMergeN * 128 + u) = make_uint4(lo[4 * q], lo[4 * q + 1], lo[4 * q + 2], lo[4 * q + 3]);
        }
    }
    ptx::fence_proxy_async_smem();   // read by the tensor cores
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
    if (warp == 1) {
        const bool landed = ptx::mbar_wait(a_full, 0, nullptr);
        if (!landed) latch(err, kErrTimeout, 9400000 + h);
        ptx::tc_fence_after();
        if (landed && elect()) {
            constexpr uint32_t idesc = ptx::idesc_bf16_f32(128, 2 * kMergeN, 0, 0);
#pragma unroll 1
            for (int kc = 0; kc < 8; ++kc)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    ptx::mma_ss(tmem, ptx::desc_kmajor_sw128(ptx::smem_u32(sA + kc * 16384) + 32 * k),
                                ptx::desc_kmajor_sw128(ptx::smem_u32(sB + kc * kMergeRows) + 32 * k), idesc, (kc | k) != 0);
        }
        if (elect()) ptx::mma_commit(d_full);
    }
    __syncwarp();
    if (warp < 4) {
        const bool done = __all_sync(0xffffffffu, ptx::mbar_wait(d_full, 0, nullptr));
        if (!done && lane == 0) latch(err, kErrTimeout, 9500000 + h);
        ptx::tc_fence_after();
        // D (lane = output column, column = query) -> rows of 128 in the A buffer, then whole
        // 256-byte rows out[v, h, :]
        __nv_bfloat16* stage = (__nv_bfloat16*)sA;
        uint32_t r[32], r2[32];
        ptx::tmem_ld32(tmem + ((uint32_t)(warp * 32) << 16), r);
        ptx::tmem_ld32(tmem + ((uint32_t)(warp * 32) << 16) + kMergeN, r2);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j)
            stage[j * 128 + warp * 32 + lane] = __float2bfloat16_rn(__uint_as_float(r[j]) + __uint_as_float(r2[j]));
        ptx::named_barrier_sync(1, 128);
        for (int i = threadIdx.x; i < kMergeN * 16; i += 128) {
            const int v = n0 + (i >> 4);
            if ((i >> 4) < rows) ((uint4*)(out + ((size_t)v * s.H + h) * 128))[i & 15] = ((const uint4*)sA)[i];
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) ptx::tmem_dealloc(tmem, 2 * kMergeN);
}

// Dynamic shared memory and the largest carve-out, once per kernel and device
template <typename K>
cudaError_t set_smem(K kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

template <int R>
cudaError_t launch_attn(const CUtensorMap& ml, const CUtensorMap& mr, const Src& src, const Problem& p, const Ws& ws,
                        DevErr err, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = set_smem(attn_kernel<R>, Cfg<R>::kSmem, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_kernel<R>, dim3(src.s.ctas), dim3(Cfg<R>::kThreads), Cfg<R>::kSmem, st, ml, mr, src, p.block_table,
                      p.scales, p.num_pages, p.scale * 1.4426950408889634f, ws, err);
}

}  // namespace

// Rows per group: 16 where that holds a sequence's rows, else 32 (the most whose scores and O, three
// terms each with its own accumulator, fit the tensor memory).  Groups of 64 rows, O in one
// accumulator for two E4M3 terms, were quicker (128 heads, 32 x 4096 tokens: 60.9 us against 71.2), but
// left nothing of a probability below 2^-11 of its tile's largest.
Shape make_shape(int B, int q_len, int H, int num_sms) {
    const int rows = q_len * H;
    Shape s{B, q_len, H, rows <= 16 ? 16 : 32, 1, 1, num_sms};
    s.G = (rows + s.R - 1) / s.R;
    s.sib = s.G <= kMaxSib && s.G <= num_sms ? s.G : 1;
    return s;
}

Ws carve(char* base, const Shape& s) {
    const size_t items = (size_t)s.B * s.G, slots = items + s.ctas;
    Ws w{};
    size_t off = 0;
    auto take = [&](size_t bytes) -> char* {
        char* p = base ? base + off : nullptr;
        off += (bytes + 255) & ~(size_t)255;
        return p;
    };
    w.q_img = (uint8_t*)take(items * 2 * s.R * kRow);
    w.q_scale = (float*)take(items * s.R * 4);
    w.part_o = (__half*)take(slots * s.R * kDc * 2);
    w.part_ml = (float4*)take(slots * s.R * 16);
    w.start = (int4*)take((size_t)s.ctas * 16);
    w.pieces = (int2*)take(items * 8);
    w.bytes = off;
    return w;
}

cudaError_t decode(const Problem& p, const Shape& s, const Ws& ws, DevErr err, cudaStream_t st) {
    const Src src{p.seq_lens, p.max_blocks, s};
    const uint64_t NV = (uint64_t)s.B * s.q_len, H = s.H;
    cudaError_t e;
    CUtensorMap mq, mk, ml, mr, mv;
    {
        ProfScope ps(st, "q8_absorb");
        const uint64_t dq[3] = {128, NV, H}, sq[2] = {H * 256, 256};
        const uint32_t bq[3] = {64, 32, 1};
        const uint64_t dw[2] = {128, H * kDc}, sw[1] = {256};
        const uint32_t bw[2] = {64, 256};
        if (!make_tmap_bf16(&mq, p.q_nope, 3, dq, sq, bq) || !make_tmap_bf16(&mk, p.W_UKT, 2, dw, sw, bw))
            return cudaErrorInvalidValue;
        static std::atomic<uint64_t> done{0};
        if ((e = set_smem(absorb_kernel, kAbsorbSmem, done)) != cudaSuccess) return e;
        e = launch_pdl(absorb_kernel, dim3(kAbsorbCluster * (s.H + 1), (unsigned)((NV + 127) / 128)),
                       dim3(kAbsorbThreads), kAbsorbSmem, st, mq, mk, p.q_rope, src, ws, err);
        if (e != cudaSuccess) return e;
    }
    {
        ProfScope ps(st, "q8_attention");
        const uint64_t dc[2] = {kRow, (uint64_t)p.num_pages * kPageRows}, sc[1] = {kRow};
        const uint32_t bl[2] = {128, kPageRows}, br[2] = {kDr, kPageRows};
        if (!make_tmap(&ml, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.codes, 2, dc, sc, bl, 128) ||
            !make_tmap(&mr, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.codes, 2, dc, sc, br, 64))
            return cudaErrorInvalidValue;
        e = s.R == 16 ? launch_attn<16>(ml, mr, src, p, ws, err, st) : launch_attn<32>(ml, mr, src, p, ws, err, st);
        if (e != cudaSuccess) return e;
    }
    ProfScope ps(st, "q8_merge_w_uv");
    const uint64_t dv[2] = {kDc, H * 128}, sv[1] = {kDc * 2};
    const uint32_t bv[2] = {64, 128};
    if (!make_tmap_bf16(&mv, p.W_UV, 2, dv, sv, bv)) return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    if ((e = set_smem(merge_kernel, kMergeSmem, done)) != cudaSuccess) return e;
    int per = kMergeN;
    while (per > 8 && (long long)s.H * ((NV + per / 2 - 1) / (per / 2)) <= s.ctas) per /= 2;
    return launch_pdl(merge_kernel, dim3(s.H, (unsigned)((NV + per - 1) / per)), dim3(kMergeThreads), kMergeSmem, st, mv,
                      src, ws, p.out, per, err);
}

cudaError_t set_wait_limit_decode_q8(uint32_t polls) { return ptx::set_wait_limit_of_this_file(polls); }
cudaError_t set_starve_decode_q8(int on) { return cudaMemcpyToSymbol(g_starve_loads, &on, sizeof on); }

}  // namespace q8
}  // namespace mla
