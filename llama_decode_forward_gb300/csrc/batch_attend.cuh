// What the attention kernels of a batch share (batch_attend.cu, which has the whole picture, and
// batch_attend_q4.cu): their arguments, how scores and probabilities are kept, and the deal
// of the pages' rows to warps.
#pragma once

#include "batch_ops.cuh"

namespace llm {

struct AttendDev {
    int n_heads, gq;
    int rows;                       // query rows per kv head: n_seqs * n_new * gq
    float sc;                       // scale * log2(e)
    const void* q;
    long long q_stride;
    int q_f16;
    void* out;
    long long out_stride;
    int out_f16;
    float* prefix_o;                // [n_kv * row tiles + blocks][2 groups][128][hd]
    float2* prefix_ml;              // [n_kv * row tiles + blocks][2][128]: Y, l
    float* suffix_o;                // [units of all sequences + workers][up to 16 rows, of 4-bit pages 24][hd]
    float2* suffix_ml;
    int* starts;                    // [n_seqs + 1]: pieces of the sequences before each
    int prefix_blocks, suffix_workers;
    int unit_rows;                          // query rows of a unit of the pages' kernel
    Div by_heads, by_new, by_gq;            // the join's divisions
    Q4Dev q4;                               // pages of 4-bit values
    int* timeout;                   // a handle's word for waits that gave up, or nullptr
    int wait_limit;                 // probes before the prefix kernel's waits give up; below kWaitLimit
                                    // (a test's) it makes no copies either, so that they do
};

// Probabilities are kept as 2^(y - Y + kHead) with Y = (scale log2(e)) R and R a recent
// maximum of the scores, so that the largest is about 2^kHead: F16 then resolves those
// 2^-33 of it (its subnormal step 2^-24, halved by rounding), and R may lag behind the
// running maximum by kLag / (scale log2(e)) before 2^(kHead + kLag) nears F16's 2^16.
// The scores' difference is taken first and then scaled: as fma(score, scale, kHead - Y)
// every exponent would keep the half step by which Y was rounded, and with |y| above 2^27
// the largest probability be infinite or zero.  (256 rows behind 16,000 shared ones 79 us
// that way, 81.5 us this way; a branch that keeps the difference to rows that need it
// took no less.)  Parts give Y to the join; their common 2^kHead cancels there.
// Each meets V as two F16 parts, its first 22 bits, whatever the output's type:
// with one part (11 bits) F16 outputs were 1.4 times as far from the exact ones as
// one rounding leaves them; the second part costs 256 rows behind 16,000 shared ones
// 10 us of 81, 64 rows behind 32,000 3.5 us of 51, and next to nothing where the pages
// are the larger part.
constexpr float kHead = 8.f, kLag = 6.f;
constexpr float kLow = -3e38f;               // R, or Y, where there is no key: low, but a number

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two F32 values as a pair of F16 (low half first), and what is left of them.
__device__ __forceinline__ uint32_t pack_hi(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t pack_lo(float a, float b, uint32_t hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return pack_hi(a - f.x, b - f.y);
}

// Eight consecutive elements of a query row, as F32.
__device__ __forceinline__ void load_q8(const AttendDev& a, long long at, float (&x)[8]) {
    if (a.q_f16) {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const __half*>(a.q) + at);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&ws[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    } else {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
        const float4 u = p[0], v = p[1];
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
        x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    }
}

// An F32 row of q is multiplied by a power of two that brings its largest element to
// 2^14 .. 2^15, so that its two F16 parts hold 22 bits of every element down to 2^-39 of
// the largest, whatever the row's magnitude; its scores are multiplied by the inverse.
struct PowerOfTwo {
    float up, down;                 // the factor of q and that of the scores
};
__device__ __forceinline__ float largest8(const float (&x)[8], float m) {
#pragma unroll
    for (int k = 0; k < 8; k += 2) m = max3(m, fabsf(x[k]), fabsf(x[k + 1]));
    return m;
}
__device__ __forceinline__ PowerOfTwo power_of(int exponent) {         // the largest element's
    const int e = max(15, exponent);         // (15: the factor stays below 2^127; infinity has 255)
    return {__uint_as_float((uint32_t)(268 - e) << 23), __uint_as_float((uint32_t)(e - 14) << 23)};
}

// Element offset of row r (of kv head g's rows) in q.
__device__ __forceinline__ long long q_offset(const AttendDev& a, int hd, int g, int r) {
    return (long long)(r / a.gq) * a.q_stride + (long long)(g * a.gq + r % a.gq) * hd;
}

// ------------------------------------------------------------- deals --
// Work in units of equal or unequal size, laid out in a row, is cut into `total`
// pieces and dealt to workers evenly: worker w takes pieces [w T / W, (w + 1) T /
// W), whatever units they belong to.  A worker leaves one part per unit that it
// touches, in slot unit + worker: each step of that walk raises one or both, so no
// two parts share a slot.  Piece x is worker ((x + 1) W - 1) / T's.
__device__ __forceinline__ long long owner_of(long long x, int workers, long long total) {
    const long long y = (x + 1) * workers - 1;
    return (unsigned long long)(total * workers) >> 32 ? y / total : (long long)((uint32_t)y / (uint32_t)total);
}

// -------------------------------------------------- pages of a batch --
// A unit is up to 8 NT query rows (row tile j % rt of kv head j / rt, j < units of
// a sequence) of one sequence against its pages, a piece 16 of its cached rows, a
// worker one warp: ragged lengths leave no warp waiting.
constexpr int kSuffixWarps = 4, kMaxSeqs = 4096;
constexpr int kQuantum = 2;                  // pieces that are worth a worker of their own
// A unit's own cost in pieces (its query rows, its part).  48 sequences of 1 to 512 rows
// and 32 heads: 66 to 77 us when only pieces counted (a worker of one-piece units ran twice as
// long as the others), 62 us.
constexpr int kUnit = 1;

// Query rows of a unit.
__host__ __device__ constexpr int unit_rows(int srows) { return srows <= 8 ? 8 : 16; }

// Row counts of the sequences (clipped to their pages) and the sums of their
// pieces before each: the suffix kernel's blocks compute them, block 0 leaves
// them for the join.
struct Deal {
    long long total;                         // pieces of all units
    int workers;
    int units;                               // of a sequence
};
__device__ __forceinline__ Deal deal_of(int pieces, int units, int max_workers) {
    Deal d;
    d.units = units;
    d.total = (long long)pieces * units;
    d.workers = (int)min((long long)max_workers, (d.total + kQuantum - 1) / kQuantum);
    return d;
}
__device__ __forceinline__ int clipped_len(const PagesDev& p, int s) {
    return (int)max(0ll, min((long long)p.lens[s], (long long)p.max_pages << p.page_shift));
}

// Pieces of `len` rows (unsigned: len may be 2^31 - 1).
__device__ __forceinline__ int pieces_of(int len) { return (int)(((uint32_t)len + 15) / 16); }

// What a unit of a sequence of `len` rows counts in the deal: its pieces, then kUnit
// empty ones.
__device__ __forceinline__ int weight(int len) { return len > 0 ? pieces_of(len) + kUnit : 0; }

// The sequences' row counts, and the sums of their weights before each.
__device__ __forceinline__ void count_pieces(const PagesDev& p, const AttendDev& a, int* starts, int* lens) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ int sums[kSuffixWarps];
    const int each = (p.n_seqs + 32 * kSuffixWarps - 1) / (32 * kSuffixWarps), s0 = threadIdx.x * each;
    int mine = 0;
    for (int s = s0; s < min(p.n_seqs, s0 + each); s++) {
        lens[s] = clipped_len(p, s);
        mine += weight(lens[s]);
    }
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    int at = sum - mine;
    for (int w = 0; w < warp; w++) at += sums[w];
    for (int s = s0; s < min(p.n_seqs, s0 + each); s++) {
        starts[s] = at;
        at += weight(lens[s]);
        if (blockIdx.x == 0) a.starts[s + 1] = at;
    }
    if (threadIdx.x == 0) {
        int all = 0;
        for (int w = 0; w < kSuffixWarps; w++) all += sums[w];
        starts[p.n_seqs] = all;
        if (blockIdx.x == 0) a.starts[0] = 0;
    }
    __syncthreads();
}

// An 8 x 8 matrix of F16 pairs, transposed across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

typedef void (*PagesKernel)(PagesDev, AttendDev, int);

// The kernel for pages of 4-bit values (batch_attend_q4.cu): query rows of a unit, blocks that
// an SM holds at once, shared memory behind the sequences' counts; and the kernel itself,
// *e saying whether it may have that much.
int unit_rows_q4(int srows, int head_dim);
int suffix_ctas_q4(int unit_rows, int head_dim);
int suffix_smem_q4(int n_seqs, int head_dim);
PagesKernel suffix_kernel_q4(int srows, int head_dim, bool split_q, cudaError_t* e);

}  // namespace llm
