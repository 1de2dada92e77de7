// Attention of a batch that shares a prefix (llm_attend_batch, include/llm.h):
// out = sum_t softmax_t(scale q.k_t) v_t over the prefix's rows and the row's
// own sequence's pages.
//
// The softmax splits over the keys: a part keeps, per query row, a reference
// Y, l = sum 2^(y_t - Y) and O = sum 2^(y_t - Y) v_t over its keys (y =
// scale log2(e) q.k), and parts join as out = sum_i w_i O_i / sum_i w_i l_i,
// w_i = 2^(Y_i - max Y).  Three kernels, chained by programmatic dependent
// launches:
//   prefix_kernel  every query row of the batch against the shared rows: the
//                  rows (new token, head of the kv head's group) of all
//                  sequences fill the 128 rows of a tensor-core tile, so the
//                  prefix is read once for 128 rows;
//   suffix_kernel  each sequence's rows against its own pages;
//   join_kernel    the parts of a row into its output.
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "batch_ops.cuh"

namespace llm {

namespace {

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
    float* suffix_o;                // [units of all sequences + workers][up to 16 rows][hd]
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

// ------------------------------------------------------------- prefix --
constexpr int kKT = 64;                      // keys per tile

template <int HDP>
struct PrefixPlan {
    // score buffers of 64 columns, half of them each softmax group's; with the two
    // groups' O (HDP columns each) and Q (HDP / 2 columns a part) they fill at most the
    // 512 columns of tensor memory
    static constexpr int kScores = HDP == 64 ? 4 : 2;
    static constexpr int kO = kScores * 64, kQ = kO + 2 * HDP, kTmemCols = 512;

    static constexpr int kSlabs = HDP / 64;                        // 64-column (128-byte) slabs of a row
    static constexpr int kTileBytes = kKT * HDP * 2;               // K or V
    // more than half of an SM's shared memory: a second block there would only wait
    // for the first one's tensor memory
    static constexpr int kStages = HDP == 64 ? 8 : 5;
    // behind the ring: the barriers and the tensor memory's address, then a byte per softmax thread
    static constexpr int kBars = 8 * (2 * kStages + 3 * kScores + 4) + 16;
    static constexpr int kSmem = kStages * 2 * kTileBytes + kBars + 256 + 1024;
};

constexpr int kSoftmaxWarps = 8, kPrefixThreads = 32 * (kSoftmaxWarps + 3);
// A quarter of the SM (16,384 registers) holds up to three of this kernel's warps (7,680)
// and then two of the suffix kernel's 128 x 32: two of its blocks run beside a block of
// this one.  With 88 registers here only one did: 256 rows of 250 pages behind 16,000
// shared ones 91 us, 81 us with 80.
constexpr int kPrefixRegs = 80;

constexpr int kWaitLimit = 10000000;         // probes (each suspends the warp for a while) before a wait gives up
// A whole warp's bounded wait for a phase.  The first probe stands outside the loop
// and every branch is the warp's: a completed phase costs 75 cycles (a loop of each
// lane's own took 250).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t par, const AttendDev& a) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, par))) return true;
    for (int i = 0; i < a.wait_limit; i++)
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, par))) return true;
    return false;
}

// One lane of the warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// Descriptor of a 128-byte-swizzled tile: K-major rows of 64 F16 values, 8-row
// groups 1024 bytes apart; or the same bytes read with the rows as the K
// dimension (MN-major), whose 64-value slabs lie `slab` bytes apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr, uint32_t slab) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)(slab >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void tm_ld32(uint32_t a, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(a));
}
__device__ __forceinline__ void tm_ld16(uint32_t a, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(a));
}
__device__ __forceinline__ void tm_st16(uint32_t a, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// The prefix's tiles against tiles of 128 query rows.  Unit u is row tile u % mt of
// kv head u / mt, a piece is one of its 64-key tiles, a worker is a block (one per
// SM).  Of a block's warps
//   0-3, 4-7  two groups do the softmax of the block's even and odd tiles, one query
//        row per thread (its lane of tensor memory), each with a maximum, a sum and
//        an O of its own: one group's exponentials run beside the other's waits and
//        maxima.  A thread reads the row's 64 scores in halves, writes the
//        probabilities over each half as two F16 parts, and rescales O when the row's
//        maximum has moved by more than kLag;
//   8, 9 issue a group's products each, S = Q K^T (a tile ahead, where its score
//        buffers allow) and O += P V;
//   10   loads 64-key tiles of K and V into a ring (TMA).
// Q and P are operands in tensor memory: an MMA whose 128-row operand comes from
// shared memory takes 48 cycles at this width, for 32 of work.  The MMA warps walk
// their loops whole and one elected lane issues: counters and descriptors stay in
// uniform registers (a loop of one lane took 90 to 140 cycles an instruction); a
// wait costs them 75 cycles and the MMAs of a product 200 to 400.  Halving the scores keeps a
// thread within kPrefixRegs.  SPLITQ: Q as two F16 parts.
template <int HDP, bool SPLITQ>
__global__ void __maxnreg__(kPrefixRegs)
    prefix_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                  const __grid_constant__ PagesDev p, const __grid_constant__ AttendDev a) {
    using G = PrefixPlan<HDP>;
    constexpr int NS = G::kStages, kScores = G::kScores;
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~(uintptr_t)1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + NS * 2 * G::kTileBytes);
    uint64_t* empty = full + NS;
    uint64_t* sfull = empty + NS;            // [kScores] scores of a tile are in buffer b
    uint64_t* pfull = sfull + kScores;       // [kScores] its probabilities are
    uint64_t* pvdone = pfull + kScores;      // [kScores] its P V has been added
    // [2] a unit's Q is in tensor memory, units taking turns: the softmax warps may be done with a
    // unit that has no tile of a group (one of a single tile) before that group's MMA warp has looked
    // at it, but not with the next one, whose scores it issues.  With one barrier such a warp could
    // miss two phases and wait for a third that needs its own scores
    uint64_t* qfull = pvdone + kScores;
    uint64_t* fin = qfull + 2;               // [2] every MMA of a group has completed
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(fin + 2);
    uint8_t* q_exponent = reinterpret_cast<uint8_t*>(full) + G::kBars;     // [256] of the largest element that each softmax thread has loaded
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mt = (a.rows + 127) / 128, ntiles = (p.prefix_len + kKT - 1) / kKT;
    const long long total = (long long)mt * p.n_kv * ntiles;
    const long long x0 = total * blockIdx.x / gridDim.x;
    const int n = (int)(total * (blockIdx.x + 1) / gridDim.x - x0);          // this block's pieces
    const int u0 = (int)(x0 / ntiles), t0 = (int)(x0 % ntiles);              // unit and tile of the first
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < kScores; b++) {
            mbar_init(&sfull[b], 1);
            mbar_init(&pfull[b], kSoftmaxWarps / 2);
            mbar_init(&pvdone[b], 1);
        }
        mbar_init(&qfull[0], kSoftmaxWarps);
        mbar_init(&qfull[1], kSoftmaxWarps);
        mbar_init(&fin[0], 1);
        mbar_init(&fin[1], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kSoftmaxWarps) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(G::kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tm_fence_before();
    __syncthreads();
    tm_fence_after();
    const uint32_t tmem = *tmem_slot;
    // the suffix kernel may start once every CTA here has seen the work before
    // this kernel complete: it needs that work, but nothing of this kernel's
    griddep_wait();
    griddep_launch();

    bool ok = true;                          // no wait of this warp has given up
    if (warp == kSoftmaxWarps || warp == kSoftmaxWarps + 1) {
        // ---- the products of one group's tiles.  F16 operands, F32 accumulators, M 128.  Scores:
        // N 64, K is K-major; sums: N HDP, V has the keys (the MMA's K) as rows, so it is MN-major
        constexpr uint32_t is = (1u << 4) | ((uint32_t)(kKT >> 3) << 17) | (8u << 24);
        constexpr uint32_t io = (1u << 4) | (1u << 16) | ((uint32_t)(HDP >> 3) << 17) | (8u << 24);
        constexpr int AHEAD = kScores / 2 - 1;                         // tiles that the scores run ahead of the sums
        const int group = warp - kSoftmaxWarps;
        const uint64_t dk = desc_sw128(smem_addr(ring), 16), dv = desc_sw128(smem_addr(ring) + G::kTileBytes, kKT * 128);
        const uint32_t o = tmem + G::kO + group * HDP;
        auto scores = [&](int it) {
            // they go where tile it - kScores's probabilities were
            if (!warp_wait(&full[it % NS], (uint32_t)((it / NS) & 1), a)) return false;
            if (it >= kScores && !warp_wait(&pvdone[it % kScores], (uint32_t)((it / kScores - 1) & 1), a)) return false;
            tm_fence_after();
            const uint64_t k = dk + (uint64_t)((it % NS) * (2 * G::kTileBytes >> 4));
            if (elect_one()) {
#pragma unroll
                for (int part = 0; part < (SPLITQ ? 2 : 1); part++)
#pragma unroll
                    for (int kk = 0; kk < HDP / 16; kk++)
                        mma_ts(tmem + (uint32_t)((it % kScores) * 64), tmem + G::kQ + part * (HDP / 2) + kk * 8,
                               k + (((kk / 4) * kKT * 128 + (kk % 4) * 32) >> 4), is, part + kk > 0);
                mma_commit(&sfull[it % kScores]);
            }
            __syncwarp();
            return true;
        };
        for (int begin = 0, tile0 = t0, unit = 0; begin < n && ok; tile0 = 0, unit++) {
            const int end = min(n, begin + ntiles - tile0), first = begin + ((begin ^ group) & 1);
            ok = warp_wait(&qfull[unit & 1], (uint32_t)((unit >> 1) & 1), a);
            if (ok && AHEAD > 0 && first < end) ok = scores(first);
            for (int it = first; it < end && ok; it += 2) {
                if (it + 2 * AHEAD < end && !(ok = scores(it + 2 * AHEAD))) break;
                if (!(ok = warp_wait(&pfull[it % kScores], (uint32_t)((it / kScores) & 1), a))) break;
                tm_fence_after();
                const uint64_t v = dv + (uint64_t)((it % NS) * (2 * G::kTileBytes >> 4));
                const uint32_t pa = tmem + (uint32_t)((it % kScores) * 64), more = it > first;
                if (elect_one()) {
#pragma unroll
                    for (int part = 0; part < 2; part++)
#pragma unroll
                        for (int kk = 0; kk < kKT / 16; kk++)
                            mma_ts(o, pa + kk * 16 + part * 8, v + (kk * 16 * 128 >> 4), io, part + kk > 0 ? 1u : more);
                    mma_commit(&pvdone[it % kScores]);
                    mma_commit(&empty[it % NS]);
                }
                __syncwarp();
            }
            begin = end;
        }
        // every MMA issued has completed before the tensor memory is freed
        if (elect_one()) mma_commit(&fin[group]);
        __syncwarp();
        ok = warp_wait(&fin[group], 0, a) && ok;
    } else if (warp == kSoftmaxWarps + 2) {
        // ---- copies
        const int copies = a.wait_limit < kWaitLimit ? 0 : n;
        int lt = t0, lu = u0, it = 0;
        for (; it < copies; it++) {
            if (it >= NS && !(ok = warp_wait(&empty[it % NS], (uint32_t)((it / NS - 1) & 1), a))) break;
            uint8_t* st = ring + (it % NS) * 2 * G::kTileBytes;
            if (elect_one()) {
                mbar_arrive_expect_tx(&full[it % NS], 2 * G::kTileBytes);
#pragma unroll
                for (int c = 0; c < G::kSlabs; c++) tma_3d_g2s(st + c * kKT * 128, &mk, c * 64, lu / mt, lt * kKT, &full[it % NS]);
#pragma unroll
                for (int c = 0; c < G::kSlabs; c++)
                    tma_3d_g2s(st + G::kTileBytes + c * kKT * 128, &mv, c * 64, lu / mt, lt * kKT, &full[it % NS]);
            }
            __syncwarp();
            if (++lt == ntiles) lt = 0, lu++;
        }
        // every copy has landed before the block can end (at once, unless a wait gave up)
        for (int k = it - 1; k >= 0 && k >= it - NS; k--) ok = warp_wait(&full[k % NS], (uint32_t)((k / NS) & 1), a) && ok;
    } else {
        // ---- softmax
        const int group = warp >> 2, lrow = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, to = tmem + lanes + G::kO + group * HDP;
        float R = 0.f, l = 0.f, sc = a.sc;   // sc: the factor of the row's scores
        // after a wait that gave up the warp goes on without waiting, to no result
        for (int begin = 0, tile0 = t0, unit = u0; begin < n; tile0 = 0, unit++) {
            // ---- a unit's tiles, `begin` to `end` of the block's: first this group's half of the
            // row's Q into tensor memory, once the last scores of both groups are there: they read all of it
            const int end = min(n, begin + ntiles - tile0), r = unit % mt * 128 + lrow, g = unit / mt;
            for (int it = max(0, begin - 2); it < begin; it++) ok = ok && warp_wait(&sfull[it % kScores], (uint32_t)((it / kScores) & 1), a);
            tm_fence_after();
            const long long q_at = r < a.rows ? q_offset(a, p.hd, g, r) : 0;
            float up = 1.f;
            if (SPLITQ) {
                // the largest of this group's columns, and the other group's
                float m = 0.f;
#pragma unroll
                for (int c = 0; c < HDP / 16; c++) {
                    float x[8];
                    if (r < a.rows && group * (HDP / 2) + c * 8 < p.hd) {
                        load_q8(a, q_at + group * (HDP / 2) + c * 8, x);
                        m = largest8(x, m);
                    }
                }
                const int e = (int)(__float_as_uint(m) >> 23);
                q_exponent[threadIdx.x] = (uint8_t)e;
                asm volatile("bar.sync 1, %0;" ::"n"(32 * kSoftmaxWarps) : "memory");
                const PowerOfTwo two = power_of(max(e, (int)q_exponent[threadIdx.x ^ 128]));
                up = two.up;
                sc = a.sc * two.down;
            }
#pragma unroll
            for (int h = 0; h < HDP / 64; h++) {
                const int c0 = group * (HDP / 2) + h * 32;             // 32 columns from here
                uint32_t hi[16], lo[SPLITQ ? 16 : 1];
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    if (r < a.rows && c0 + c * 8 < p.hd) load_q8(a, q_at + c0 + c * 8, x);
                    if (SPLITQ)
#pragma unroll
                        for (int k = 0; k < 8; k++) x[k] *= up;
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        hi[4 * c + k] = pack_hi(x[2 * k], x[2 * k + 1]);
                        if (SPLITQ) lo[SPLITQ ? 4 * c + k : 0] = pack_lo(x[2 * k], x[2 * k + 1], hi[4 * c + k]);
                    }
                }
                tm_st16(tmem + lanes + G::kQ + c0 / 2, hi);
                if (SPLITQ) tm_st16(tmem + lanes + G::kQ + HDP / 2 + c0 / 2, lo);
            }
            tm_wait_st();
            tm_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&qfull[(unit - u0) & 1]);
            const int first = begin + ((begin ^ group) & 1);           // the group's first tile of the unit
            for (int it = first; it < end; it += 2) {
                const uint32_t sb = tmem + lanes + (uint32_t)((it % kScores) * 64);
                const int left = p.prefix_len - (tile0 + it - begin) * kKT;      // keys from this tile on
                ok = ok && warp_wait(&sfull[it % kScores], (uint32_t)((it / kScores) & 1), a);
                tm_fence_after();
                // 32 scores, keys behind the prefix at -infinity
                auto scores = [&](int h, uint32_t (&s)[32]) {
                    tm_ld32(sb + h * 32, s);
                    tm_wait_ld();
                    if (left < h * 32 + 32) {
#pragma unroll
                        for (int c = 0; c < 32; c++)
                            if (h * 32 + c >= left) s[c] = 0xFF800000u;
                    }
                };
                auto largest = [&](const uint32_t (&s)[32]) {
                    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};       // four chains side by side
#pragma unroll
                    for (int c = 0; c < 32; c += 2) m[c / 2 & 3] = max3(m[c / 2 & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
                    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
                };
                float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                auto probabilities = [&](int h, const uint32_t (&s)[32]) {
                    const float2 sc2 = make_float2(sc, sc), r2 = make_float2(-R, -R), head2 = make_float2(kHead, kHead);
#pragma unroll
                    for (int k = 0; k < 32; k += 16) {       // one MMA's keys: eight columns of high parts, eight of low ones
                        uint32_t p2[16];
#pragma unroll
                        for (int c = 0; c < 8; c++) {
                            const float2 d = __fadd2_rn(make_float2(__uint_as_float(s[k + 2 * c]), __uint_as_float(s[k + 2 * c + 1])), r2);
                            const float2 y = __ffma2_rn(d, sc2, head2);
                            const float2 e = make_float2(exp2_fast(y.x), exp2_fast(y.y));
                            l2[c & 1] = __fadd2_rn(l2[c & 1], e);
                            p2[c] = pack_hi(e.x, e.y);
                            p2[8 + c] = pack_lo(e.x, e.y, p2[c]);
                        }
                        tm_st16(sb + h * 32 + k, p2);
                    }
                };
                uint32_t s[32];
                scores(0, s);
                float mx = largest(s);
                scores(1, s);
                mx = fmaxf(mx, largest(s));
                mx = fmaxf(mx, kLow);
                if (it == first) {
                    R = mx;
                    l = 0.f;
                } else if (__any_sync(0xffffffffu, (mx - R) * sc > kLag)) {
                    float c = 1.f;
                    if ((mx - R) * sc > kLag) {
                        c = exp2_fast((R - mx) * sc);
                        R = mx;
                    }
                    l *= c;
                    ok = ok && warp_wait(&pvdone[(it - 2) % kScores], (uint32_t)(((it - 2) / kScores) & 1), a);
                    tm_fence_after();
#pragma unroll 1
                    for (int h = 0; h < HDP; h += 16) {
                        uint32_t o[16];
                        tm_ld16(to + h, o);
                        tm_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; k++) o[k] = __float_as_uint(__uint_as_float(o[k]) * c);
                        tm_st16(to + h, o);
                    }
                }
                probabilities(1, s);
                scores(0, s);                // read a second time: 64 scores at once would not leave the registers
                probabilities(0, s);
                l += (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
                tm_wait_st();
                tm_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[it % kScores]);
            }
            // ---- this group's part of the unit; without a tile of its own an empty one
            const int last = end - 1 - ((end - 1 - first) & 1);
            const bool any = first < end;
            if (any) ok = ok && warp_wait(&pvdone[last % kScores], (uint32_t)((last / kScores) & 1), a);
            tm_fence_after();
            const long long at = (((long long)unit + blockIdx.x) * 2 + group) * 128 + lrow;
#pragma unroll 1
            for (int h = 0; h < HDP; h += 16) {
                uint32_t o[16];
                tm_ld16(to + h, o);
                tm_wait_ld();
                if (r < a.rows)
#pragma unroll
                    for (int k = 0; k < 16; k += 4)
                        if (h + k < p.hd)
                            *reinterpret_cast<uint4*>(a.prefix_o + at * p.hd + h + k) =
                                any ? make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]) : make_uint4(0, 0, 0, 0);
            }
            if (r < a.rows) a.prefix_ml[at] = any ? make_float2(fmaxf(R * sc, kLow), l) : make_float2(kLow, 0.f);
            // O has been read before the next unit's first P V, which waits for these warps' probabilities
            tm_fence_before();
            begin = end;
        }
    }
    if (!ok && lane == 0) {
        flag(p.err, LLM_PAGES_TIMEOUT);
        flag(a.timeout, kErrTimeout);
    }
    tm_fence_before();
    __syncthreads();
    if (warp == kSoftmaxWarps)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(G::kTmemCols));
}

// ------------------------------------------------------------- suffix --
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

// Blocks that an SM holds at once, by their registers: the pieces are dealt to
// as many, so that all run together.
__host__ __device__ constexpr int suffix_ctas(int hdp, int nt) { return hdp == 64 ? (nt == 1 ? 4 : 3) : 2; }

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

// What a unit of a sequence of `len` rows counts in the deal: its pieces, then kUnit
// empty ones.
__device__ __forceinline__ int weight(int len) { return len > 0 ? (len + 15) / 16 + kUnit : 0; }

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

// Each warp walks its pieces alone: the rows of the next piece are on their way
// to registers (and the pages of the one behind it are being looked up) while
// one is multiplied, across units.  The products are mma.sync m16n8k16 with the
// cached rows as the 16 (scores S^T = K q^T, sums O^T = V^T P^T), so 8 query rows
// waste none of them, and the operands need no shared memory:
// - lane (r, t) = (lane / 4, lane % 4) loads 16-byte chunks t, t + 4, ... of cached
//   rows r and r + 8, 64 contiguous bytes of a row per instruction.  The order of
//   the dims in a dot product is free, so MMA k-step 2 i + h takes dims 8 (t + 4 i) +
//   4 h + {0, 1 | 2, 3} of each lane, as they lie in its registers; q is loaded in
//   the same order;
// - V's registers become V^T's by 8 x 8 transposes across the warp (movmatrix):
//   register w of chunk i of row r turns into dim 8 (r / 2) + 32 i + 2 w + r % 2, r
//   now counting dims.
// The stream of rows is the bound.  At 64 continuations of 2048 rows each (268 MB)
// a ring of TMA boxes (16 rows x 128 bytes a request) brought 3.6 TB/s, plain
// loads 5.5 TB/s, the join and the launches included; 805 MB with heads of 128
// values 6.4 TB/s.
template <int HDP, int NT, bool SPLITQ>
__global__ void __launch_bounds__(32 * kSuffixWarps, suffix_ctas(HDP, NT))
    suffix_kernel(const __grid_constant__ PagesDev p, const __grid_constant__ AttendDev a, int first) {
    constexpr int CH = HDP / 32, RU = 8 * NT;                // 16-byte chunks of a row in a lane
    extern __shared__ int seqs[];
    if (first) griddep_wait();               // otherwise the prefix kernel has waited for the work before it
    griddep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int srows = p.n_new * a.gq, rt = (srows + RU - 1) / RU, units = p.n_kv * rt;
    int* starts = seqs;                      // [n_seqs + 1]
    int* lens = starts + p.n_seqs + 1;       // [n_seqs]
    count_pieces(p, a, starts, lens);
    const Deal deal = deal_of(starts[p.n_seqs], units, (int)gridDim.x * kSuffixWarps);
    const int me = blockIdx.x * kSuffixWarps + warp;
    if (me < deal.workers) {
        const long long x0 = deal.total * me / deal.workers, x1 = deal.total * (me + 1) / deal.workers;
        // where the first piece lies: the last sequence that starts at or before it
        int s = 0;
        for (int lo = 0, hi = p.n_seqs; hi - lo > 1;) {
            const int mid = (lo + hi) / 2;
            ((long long)starts[mid] * units <= x0 ? lo : hi) = mid;
            s = lo;
        }
        auto next = [&](int& s, int& j, int& pc, int& np) {      // the unit behind one, at its first piece
            pc = 0;
            if (++j < units) return;
            j = 0;
            do s++;
            while (lens[s] == 0);
            np = (lens[s] + 15) / 16;
        };
        int np = (lens[s] + 15) / 16;
        const long long in_seq = x0 - (long long)starts[s] * units;
        int j = (int)(in_seq / (np + kUnit)), pc = (int)(in_seq % (np + kUnit)), left = (int)(x1 - x0);
        if (pc >= np) {                      // it starts with empty pieces
            left -= np + kUnit - pc;
            if (left > 0) next(s, j, pc, np);
        }
        const int r = lane >> 2, t = lane & 3;
        const long long pitch = (long long)p.n_kv * p.hd;

        // the pages of this lane's rows r and r + 8 of the piece that is loaded next
        int ls = s, lj = j, lpc = pc, lnp = np, lleft = left, page[2] = {-1, -1};
        auto look = [&]() {
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const int e = lpc * 16 + r + 8 * k;
                page[k] = e < lens[ls] ? p.table[(long long)ls * p.max_pages + (e >> p.page_shift)] : INT_MIN;
            }
        };
        uint4 kx[2][CH], vx[2][CH];          // rows r and r + 8 of the piece on its way
        bool there_x[2];                     // neither behind the sequence's last row nor on a bad page
        auto load = [&]() {                  // requests the piece, moves on and looks the next one up
#pragma unroll
            for (int k = 0; k < 2; k++) {
                there_x[k] = page[k] >= 0 && page[k] < p.n_pages;
                if (!there_x[k] && page[k] != INT_MIN) flag(p.err, LLM_PAGES_BAD_PAGE);
                const int e = lpc * 16 + r + 8 * k;
                const long long at = (((long long)page[k] << p.page_shift) + (e & ((1 << p.page_shift) - 1))) * pitch +
                                     (long long)(lj / rt) * p.hd + 8 * t;
#pragma unroll
                for (int i = 0; i < CH; i++) {
                    kx[k][i] = vx[k][i] = make_uint4(0, 0, 0, 0);
                    if (there_x[k] && 8 * (t + 4 * i) < p.hd) {
                        kx[k][i] = __ldcs(reinterpret_cast<const uint4*>(p.k + at + 32 * i));
                        vx[k][i] = __ldcs(reinterpret_cast<const uint4*>(p.v + at + 32 * i));
                    }
                }
            }
            lleft--;
            if (++lpc == lnp) {
                lleft -= kUnit;
                if (lleft > 0) {
                    next(ls, lj, lpc, lnp);
                }
            }
            if (lleft > 0) look();
        };
        if (left > 0) {
            look();
            load();
        }
        while (left > 0) {
            // ---- one unit: pieces pc .. of its np, as far as this worker goes
            const int tile = j % rt, g = j / rt, count = min(left, np - pc);
            const int last = p.lens[s] - p.n_new, e_min = last + tile * RU / a.gq;
            // q as the second operand: query row r of each eight; rows behind the last repeat it (never stored)
            uint32_t qhi[NT][2 * CH][2], qlo[NT][SPLITQ ? 2 * CH : 1][2];
            int e[NT][2];                    // the last cached row that query rows 2t and 2t + 1 see
            float qs[NT][2];                 // and the factor of their scores
#pragma unroll
            for (int q = 0; q < NT; q++) {
                const long long at = q_offset(a, p.hd, g, s * srows + min(tile * RU + q * 8 + r, srows - 1));
#pragma unroll
                for (int k = 0; k < 2; k++) e[q][k] = last + min(tile * RU + q * 8 + 2 * t + k, srows - 1) / a.gq;
                float up = 1.f;
                qs[q][0] = qs[q][1] = a.sc;
                if (SPLITQ) {
                    float m = 0.f;
#pragma unroll
                    for (int i = 0; i < CH; i++) {
                        float x[8];
                        if (8 * (t + 4 * i) < p.hd) {
                            load_q8(a, at + 8 * (t + 4 * i), x);
                            m = largest8(x, m);
                        }
                    }
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                    const PowerOfTwo two = power_of((int)(__float_as_uint(fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2))) >> 23));
                    up = two.up;
#pragma unroll
                    for (int k = 0; k < 2; k++) qs[q][k] = a.sc * __shfl_sync(0xffffffffu, two.down, 4 * (2 * t + k));
                }
#pragma unroll
                for (int i = 0; i < CH; i++) {
                    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    if (8 * (t + 4 * i) < p.hd) load_q8(a, at + 8 * (t + 4 * i), x);
                    if (SPLITQ)
#pragma unroll
                        for (int k = 0; k < 8; k++) x[k] *= up;
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const uint32_t hi = pack_hi(x[2 * k], x[2 * k + 1]);
                        qhi[q][2 * i + k / 2][k % 2] = hi;
                        if (SPLITQ) qlo[q][SPLITQ ? 2 * i + k / 2 : 0][k % 2] = pack_lo(x[2 * k], x[2 * k + 1], hi);
                    }
                }
            }
            float o[NT][2 * CH][4], R[NT][2], l[NT][2];
#pragma unroll
            for (int q = 0; q < NT; q++) {
#pragma unroll
                for (int d = 0; d < 2 * CH; d++) o[q][d][0] = o[q][d][1] = o[q][d][2] = o[q][d][3] = 0.f;
                R[q][0] = R[q][1] = kLow;    // no key seen yet
                l[q][0] = l[q][1] = 0.f;
            }
            for (int i0 = 0; i0 < count; i0++) {
                uint32_t k0[4 * CH], k1[4 * CH], v0[4 * CH], v1[4 * CH];     // rows r (0) and r + 8 (1)
#pragma unroll
                for (int i = 0; i < CH; i++) {
                    k0[4 * i] = kx[0][i].x; k0[4 * i + 1] = kx[0][i].y; k0[4 * i + 2] = kx[0][i].z; k0[4 * i + 3] = kx[0][i].w;
                    k1[4 * i] = kx[1][i].x; k1[4 * i + 1] = kx[1][i].y; k1[4 * i + 2] = kx[1][i].z; k1[4 * i + 3] = kx[1][i].w;
                    v0[4 * i] = vx[0][i].x; v0[4 * i + 1] = vx[0][i].y; v0[4 * i + 2] = vx[0][i].z; v0[4 * i + 3] = vx[0][i].w;
                    v1[4 * i] = vx[1][i].x; v1[4 * i + 1] = vx[1][i].y; v1[4 * i + 2] = vx[1][i].z; v1[4 * i + 3] = vx[1][i].w;
                }
                const bool there[2] = {there_x[0], there_x[1]};
                if (lleft > 0) load();
                float sc[NT][4];
#pragma unroll
                for (int q = 0; q < NT; q++) {
                    sc[q][0] = sc[q][1] = sc[q][2] = sc[q][3] = 0.f;
#pragma unroll
                    for (int ks = 0; ks < 2 * CH; ks++) {
                        const uint32_t k[4] = {k0[2 * ks], k1[2 * ks], k0[2 * ks + 1], k1[2 * ks + 1]};
                        mma16816(sc[q], k, qhi[q][ks][0], qhi[q][ks][1]);
                        if (SPLITQ) mma16816(sc[q], k, qlo[q][SPLITQ ? ks : 0][0], qlo[q][SPLITQ ? ks : 0][1]);
                    }
                }
                // rows that are not there, and those that some query rows do not see
                const int e0 = (pc + i0) * 16;
#pragma unroll
                for (int q = 0; q < NT; q++)
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        if (!there[k >> 1] || e0 + r + (k >> 1) * 8 > e[q][k & 1]) sc[q][k] = -INFINITY;
                uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
                for (int q = 0; q < NT; q++) {
                    float top[2];
                    bool move = false;
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        float m = fmaxf(sc[q][k], sc[q][2 + k]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                        top[k] = fmaxf(m, kLow);
                        move |= (top[k] - R[q][k]) * qs[q][k] > kLag;
                    }
                    if (__any_sync(0xffffffffu, move)) {
                        float c[2];
#pragma unroll
                        for (int k = 0; k < 2; k++) {
                            // (a row's own maximum decides: its bits do not depend on its neighbours)
                            const float up = (top[k] - R[q][k]) * qs[q][k] > kLag ? top[k] : R[q][k];
                            c[k] = exp2_fast((R[q][k] - up) * qs[q][k]);
                            R[q][k] = up;
                            l[q][k] *= c[k];
                        }
#pragma unroll
                        for (int d = 0; d < 2 * CH; d++) {
                            o[q][d][0] *= c[0];
                            o[q][d][1] *= c[1];
                            o[q][d][2] *= c[0];
                            o[q][d][3] *= c[1];
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        sc[q][k] = exp2_fast(fmaf(sc[q][k] - R[q][k & 1], qs[q][k & 1], kHead));
                        l[q][k & 1] += sc[q][k];          // this thread's cached rows; all are added at the end
                    }
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        const uint32_t hi = pack_hi(sc[q][2 * k], sc[q][2 * k + 1]);
                        ph[q][k] = transpose8(hi);
                        pl[q][k] = transpose8(pack_lo(sc[q][2 * k], sc[q][2 * k + 1], hi));
                    }
                }
                // a row that some new tokens see and others do not: where its V is not
                // finite, 0 * V would reach those that do not, so it is added to the
                // others alone and taken out of the product
                if (p.n_new > 1 && e0 + 15 > e_min) {
                    bool wild[2] = {false, false};
#pragma unroll
                    for (int i = 0; i < 4 * CH; i++) {
                        wild[0] |= (v0[i] & 0x7C00u) == 0x7C00u || (v0[i] & 0x7C000000u) == 0x7C000000u;
                        wild[1] |= (v1[i] & 0x7C00u) == 0x7C00u || (v1[i] & 0x7C000000u) == 0x7C000000u;
                    }
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        const uint32_t who = __ballot_sync(0xffffffffu, wild[k]);
                        for (int kr = 0; kr < 8 && who; kr++) {
                            if (!((who >> (4 * kr)) & 15u)) continue;
#pragma unroll
                            for (int q = 0; q < NT; q++) {
                                const float pa = __shfl_sync(0xffffffffu, sc[q][2 * k], 4 * kr + t), pb = __shfl_sync(0xffffffffu, sc[q][2 * k + 1], 4 * kr + t);
#pragma unroll
                                for (int i = 0; i < 4 * CH; i++) {
                                    const uint32_t w = __shfl_sync(0xffffffffu, k ? v1[i] : v0[i], 4 * kr + (r >> 1));
                                    const float v = __half2float(__ushort_as_half((unsigned short)(r & 1 ? w >> 16 : w & 0xFFFFu)));
                                    if (pa != 0.f) o[q][i / 2][2 * (i & 1)] = fmaf(pa, v, o[q][i / 2][2 * (i & 1)]);
                                    if (pb != 0.f) o[q][i / 2][2 * (i & 1) + 1] = fmaf(pb, v, o[q][i / 2][2 * (i & 1) + 1]);
                                }
                            }
                            if (r == kr)
#pragma unroll
                                for (int i = 0; i < 4 * CH; i++) (k ? v1[i] : v0[i]) = 0u;
                        }
                    }
                }
#pragma unroll
                for (int d = 0; d < 2 * CH; d++) {
                    const uint32_t v[4] = {transpose8(v0[2 * d]), transpose8(v0[2 * d + 1]), transpose8(v1[2 * d]), transpose8(v1[2 * d + 1])};
#pragma unroll
                    for (int q = 0; q < NT; q++) {
                        mma16816(o[q][d], v, ph[q][0], ph[q][1]);
                        mma16816(o[q][d], v, pl[q][0], pl[q][1]);
                    }
                }
            }
            // ---- this worker's part of the unit
            const long long slot = ((long long)s * units + j + me) * min(srows, RU);
#pragma unroll
            for (int q = 0; q < NT; q++)
#pragma unroll
                for (int k = 0; k < 2; k++) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[q][k] += __shfl_xor_sync(0xffffffffu, l[q][k], d);
                    const int row = q * 8 + 2 * t + k;
                    if (tile * RU + row >= srows) continue;
                    float* dst = a.suffix_o + (slot + row) * p.hd;
#pragma unroll
                    for (int i = 0; i < 4 * CH; i++) {
                        const int d = 8 * (r >> 1) + 32 * (i / 4) + 2 * (i % 4) + (r & 1);
                        if (d < p.hd) dst[d] = o[q][i / 2][2 * (i & 1) + k];
                    }
                    if (r == 0) a.suffix_ml[slot + row] = make_float2(fmaxf(R[q][k] * qs[q][k], kLow), l[q][k]);
                }
            left -= count + kUnit;
            if (left > 0) next(s, j, pc, np);
        }
    }
    // this grid's end is the prefix kernel's too, for the join; only the last block waits for it, so
    // that the others make room for the next while the prefix kernel runs
    if (!first && blockIdx.x + 1 == gridDim.x) griddep_wait();
}

// ---------------------------------------------- suffix, 4-bit pages --
// The suffix kernel for pages of 4-bit values: the same pieces, deal and parts.
// A value is made where it is used: numbers become F16 by their bits (0x6400 | n is
// 1024 + n, 0x6400 | 16 n is 1024 + 16 n; one exact operation takes the 1024 away) and
// one fused multiply-add rounds d n + m to the F16 that it stands for.
// - K is the products' first operand: lane (r, t) holds dims 64 c + 16 t + {0 .. 15} of
//   cached rows r and r + 8, two words of numbers.  Their half-words pair dims 0 and 4, 1
//   and 5, ... of a word, so q is loaded in that order.
// - V^T is the other product's first operand, and needs pairs of cached rows: lane (r, t)
//   loads dims 8 C r .. of rows 2t, 2t + 1 (and those eight behind), and a byte permutation
//   joins the two rows' numbers, so no transpose is needed.  An MMA's rows r and r + 8 are
//   dims 8 C r + 2 i and + 1.
// A step is H pieces.  Eight rows in a row lie in one page (page_size >= 8): an octet.  Each
// warp has a ring of steps in shared memory, filled by asynchronous 16-byte copies: an
// octet's numbers lie in a row, and so do its pairs, so a step of 32 rows of heads of 64
// values takes five copies of a warp where loads into registers took 24.
// PACK: up to four query rows.  The eight columns of a product hold each of them twice;
// the second four take the probabilities' second parts, so one product adds both.
// FULL: head_dim is HDP, so that the distances of rows and pairs are constants.
// What bounds it: making the values.  A step of 32 rows of heads of 64 values takes a warp some 560
// instructions, 230 of them for the 4096 values; the logical and the half-precision operations together keep their
// two units busy 95 % of the time (one half each).  64 sequences of 1 to 8192 rows, 8 heads of 64 (194 MB): 58 us, 3.3 TB/s, 95 us
// as first written; 32 of 1 to 4096, 32 heads of 128 (390 MB): 103 us, 3.8 TB/s, from 179 us.  F16 pages of the
// same rows would be 3.2 times the bytes.  Steps of 16 rows take 5 to 20 % longer; of 64 rows, 3 % less on the
// first, 20 % more where sequences are short.  Neither more blocks on an SM nor fewer (12 to 20 warps), nor an order of rows
// without bank conflicts, changed these by more than 4 %.
constexpr int kQ4Pieces = 2, kQ4Stages = 2;
// Shared memory of a block's rings.
__host__ __device__ constexpr int q4_rings(int hdp) { return kSuffixWarps * kQ4Stages * 2 * (2 * kQ4Pieces) * 5 * hdp; }

// A 16-byte asynchronous copy to shared memory, or zeros.
__device__ __forceinline__ void cp_async16_or_zero(void* dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}
// Waits until at most N groups of this thread's copies are on their way.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__host__ __device__ constexpr int suffix_q4_ctas(int hdp, int nt) { return hdp == 64 ? (nt == 1 ? 4 : nt == 2 ? 3 : 2) : (nt == 1 ? 3 : 2); }

// Query rows of a unit: more than 16 are taken at once (up to 24, where the registers allow) as
// long as one unit then does, since every unit makes the values anew.
__host__ __device__ constexpr int unit_rows_q4(int srows, int hd) { return srows <= 8 ? 8 : srows > 16 && srows <= 24 && hd <= 64 ? 24 : 16; }

// Pairs of numbers of a word, as F16 pairs.  (x & m | c in one instruction: left to itself the compiler takes
// two, each with a constant of its own; a step of 32 rows then had 145 logical operations, of 777.)
__device__ __forceinline__ __half2 half2_of(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t m, uint32_t c) {
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(m), "r"(c));
    return y;
}
__device__ __forceinline__ __half2 q4_low(uint32_t x, uint32_t c) {            // numbers at bits 0 and 16
    return __hsub2(half2_of(and_or(x, 0x000F000Fu, c)), __float2half2_rn(1024.f));
}
__device__ __forceinline__ __half2 q4_high(uint32_t x, uint32_t c) {           // numbers at bits 4 and 20
    return __hfma2(half2_of(and_or(x, 0x00F000F0u, c)), __float2half2_rn(0.0625f), __float2half2_rn(-64.f));
}
__device__ __forceinline__ uint32_t q4_value(__half2 n, __half2 d, __half2 m) {
    const __half2 v = __hfma2(n, d, m);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <int HDP, int NT, bool SPLITQ, bool PACK, bool FULL>
__global__ void __launch_bounds__(32 * kSuffixWarps, suffix_q4_ctas(HDP, NT))
    suffix_q4_kernel(const __grid_constant__ PagesDev p, const __grid_constant__ AttendDev a, int first) {
    static_assert(!PACK || NT == 1, "four query rows");
    constexpr int C = HDP / 64, KS = HDP / 16, RU = 8 * NT;  // chunks of 64 dims; MMA steps of a dot product, and MMA tiles of the sums
    constexpr int H = kQ4Pieces, OCT = 2 * H;                // pieces and octets of a step
    constexpr int S = kQ4Stages, NUMBERS = OCT * 4 * HDP, PAIRS = OCT * HDP, STAGE = 2 * (NUMBERS + PAIRS);
    extern __shared__ __align__(16) int seqs[];
    if (first) griddep_wait();
    griddep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int srows = p.n_new * a.gq, rt = (srows + RU - 1) / RU, units = p.n_kv * rt;
    int* starts = seqs;
    int* lens = starts + p.n_seqs + 1;
    count_pieces(p, a, starts, lens);
    const Deal deal = deal_of(starts[p.n_seqs], units, (int)gridDim.x * kSuffixWarps);
    const int me = blockIdx.x * kSuffixWarps + warp;
    if (me < deal.workers) {
        const long long x0 = deal.total * me / deal.workers, x1 = deal.total * (me + 1) / deal.workers;
        int s = 0;
        for (int lo = 0, hi = p.n_seqs; hi - lo > 1;) {
            const int mid = (lo + hi) / 2;
            ((long long)starts[mid] * units <= x0 ? lo : hi) = mid;
            s = lo;
        }
        // the unit behind one (row tile `tile` of kv head g of sequence s), at its first piece
        auto next = [&](int& s, int& g, int& tile, int& pc, int& np) {
            pc = 0;
            if (++tile < rt) return;
            tile = 0;
            if (++g < p.n_kv) return;
            g = 0;
            do s++;
            while (lens[s] == 0);
            np = (lens[s] + 15) / 16;
        };
        int np = (lens[s] + 15) / 16;
        const long long in_seq = x0 - (long long)starts[s] * units;
        const int j0 = (int)(in_seq / (np + kUnit));
        int g = j0 / rt, tile = j0 % rt, pc = (int)(in_seq % (np + kUnit)), left = (int)(x1 - x0);
        if (pc >= np) {                      // it starts with empty pieces
            left -= np + kUnit - pc;
            if (left > 0) next(s, g, tile, pc, np);
        }
        const int r = lane >> 2, t = lane & 3;
        const uint32_t pitch = (FULL ? HDP : (uint32_t)p.hd) / 2, pairs = FULL ? HDP / 8 : 4u * a.q4.groups, page_bytes = (uint32_t)a.q4.page_bytes,
                       mask = (1u << p.page_shift) - 1;
        // the warp's ring of steps: numbers of K, of V, pairs of K, of V
        uint8_t* ring = reinterpret_cast<uint8_t*>(seqs) + ((2 * p.n_seqs + 1) * 4 + 15) / 16 * 16 + warp * (S * STAGE);
        // 16-byte words of an octet's numbers, two octets of heads of up to 64 values to a copy of the whole warp; those of
        // its pairs, K's and V's of four octets (two, of heads of up to 128)
        constexpr int NW = HDP / 4, NO = 32 / NW, PW = HDP / 16, PO = 16 / PW;
        const int n_oct = lane / NW, n_word = lane % NW, p_oct = lane % 16 / PW, p_word = lane % PW;
        const bool n_in = FULL || 4 * n_word < p.hd, p_in = FULL || 4 * p_word < (int)pairs * 2;
        const uint8_t *kp = reinterpret_cast<const uint8_t*>(p.k) + 16 * n_word, *vp = reinterpret_cast<const uint8_t*>(p.v) + 16 * n_word,
                      *dp = reinterpret_cast<const uint8_t*>(lane < 16 ? p.k : p.v) + a.q4.scales + 16 * p_word;
        uint8_t* n_to = ring + n_oct * (8 * pitch) + 16 * n_word;
        uint8_t* p_to = ring + 2 * NUMBERS + (lane < 16 ? 0 : PAIRS) + p_oct * (8 * pairs) + 16 * p_word;
        const bool k_in[2] = {FULL || 16 * t < p.hd, FULL || 64 + 16 * t < p.hd}, v_in = FULL || 8 * C * r < p.hd;
        const float second = t >= 2 ? -1.f : 0.f;                // PACK: which part of the probabilities this lane's columns take
        uint32_t k1024;                      // (a register: see and_or)
        asm volatile("mov.u32 %0, 0x64006400;" : "=r"(k1024));

        // the step that is loaded next: octet lane % OCT's page (-1: nothing to read there), looked up ahead
        int ls = s, lg = g, ltile = tile, lpc = pc, lnp = np, lleft = left, page = -1, lend = 0;
        auto look = [&]() {
            const int e = lpc * 16 + 8 * (lane % OCT);
            lend = min(lens[ls], 16 * (lpc + min(lleft, H)));
            page = -1;
            if (e < lend) {
                page = p.table[(long long)ls * p.max_pages + (e >> p.page_shift)];
                if (page < 0 || page >= p.n_pages) {
                    flag(p.err, LLM_PAGES_BAD_PAGE);
                    page = -1;
                }
            }
        };
        uint32_t pages_ok = 0;               // four bits for each step in the ring: its octets that have a page
        // requests the step into a place of the ring, moves on and looks the next one up.  An octet without a page is zero;
        // rows of its page that are not the sequence's come along
        auto load = [&](int to) {
            const int e0 = lpc * 16, first_row = lg << p.page_shift;
            pages_ok |= (__ballot_sync(0xffffffffu, page >= 0) & ((1u << OCT) - 1)) << (4 * to);
#pragma unroll
            for (int i = 0; i < OCT; i += NO) {
                const int pg = __shfl_sync(0xffffffffu, page, i + n_oct);
                const unsigned long long off = (unsigned long long)(uint32_t)max(pg, 0) * page_bytes +
                                               (unsigned long long)(uint32_t)(first_row + ((e0 + 8 * (i + n_oct)) & (int)mask)) * pitch;
                if (n_in) {
                    cp_async16_or_zero(n_to + to * STAGE + i * (8 * pitch), kp + off, pg >= 0);
                    cp_async16_or_zero(n_to + to * STAGE + NUMBERS + i * (8 * pitch), vp + off, pg >= 0);
                }
            }
#pragma unroll
            for (int i = 0; i < OCT; i += PO) {
                const int oc = i + p_oct, pg = __shfl_sync(0xffffffffu, page, oc % OCT);
                const unsigned long long off = (unsigned long long)(uint32_t)max(pg, 0) * page_bytes +
                                               (unsigned long long)(uint32_t)(first_row + ((e0 + 8 * oc) & (int)mask)) * pairs;
                if (p_in && oc < OCT) cp_async16_or_zero(p_to + to * STAGE + i * (8 * pairs), dp + off, pg >= 0);
            }
            const int n = min(min(lleft, H), lnp - lpc);
            lleft -= n;
            lpc += n;
            if (lpc == lnp) {
                lleft -= kUnit;
                if (lleft > 0) next(ls, lg, ltile, lpc, lnp);
            }
            if (lleft > 0) look();
        };
        if (left > 0) look();
#pragma unroll
        for (int i = 0; i < S - 1; i++) {
            if (lleft > 0) load(i);
            cp_async_commit();
        }
        int cur = 0;                         // the step's place in the ring
        while (left > 0) {
            // ---- one unit: pieces pc .. of its np, as far as this worker goes
            const int count = min(left, np - pc);
            const int last = p.lens[s] - p.n_new, e_min = last + tile * RU / a.gq;
            // q as the second operand: query row r of each eight; rows behind the last repeat it (never stored)
            uint32_t qhi[NT][KS][2], qlo[NT][SPLITQ ? KS : 1][2];
            int e[NT][2];                    // the last cached row that query rows 2t and 2t + 1 see
            float qs[NT][2];                 // and the factor of their scores
#pragma unroll
            for (int q = 0; q < NT; q++) {
                const long long at = q_offset(a, p.hd, g, s * srows + min(tile * RU + q * 8 + (PACK ? r & 3 : r), srows - 1));
#pragma unroll
                for (int k = 0; k < 2; k++) e[q][k] = last + min(tile * RU + q * 8 + (PACK ? (2 * t + k) & 3 : 2 * t + k), srows - 1) / a.gq;
                float up = 1.f;
                qs[q][0] = qs[q][1] = a.sc;
                if (SPLITQ) {
                    float m = 0.f;
#pragma unroll
                    for (int i = 0; i < 2 * C; i++) {
                        float x[8];
                        const int d = 64 * (i / 2) + 16 * t + 8 * (i % 2);
                        if (d < p.hd) {
                            load_q8(a, at + d, x);
                            m = largest8(x, m);
                        }
                    }
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                    const PowerOfTwo two = power_of((int)(__float_as_uint(fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2))) >> 23));
                    up = two.up;
#pragma unroll
                    for (int k = 0; k < 2; k++) qs[q][k] = a.sc * __shfl_sync(0xffffffffu, two.down, 4 * (2 * t + k));
                }
#pragma unroll
                for (int i = 0; i < 2 * C; i++) {
                    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    const int d = 64 * (i / 2) + 16 * t + 8 * (i % 2);
                    if (d < p.hd) load_q8(a, at + d, x);
                    if (SPLITQ)
#pragma unroll
                        for (int k = 0; k < 8; k++) x[k] *= up;
#pragma unroll
                    for (int k = 0; k < 4; k++) {                // dims k and k + 4
                        const uint32_t hi = pack_hi(x[k], x[k + 4]);
                        qhi[q][2 * i + k / 2][k % 2] = hi;
                        if (SPLITQ) qlo[q][SPLITQ ? 2 * i + k / 2 : 0][k % 2] = pack_lo(x[k], x[k + 4], hi);
                    }
                }
            }
            float o[NT][KS][4], R[NT][2], l[NT][2];
#pragma unroll
            for (int q = 0; q < NT; q++) {
#pragma unroll
                for (int d = 0; d < KS; d++) o[q][d][0] = o[q][d][1] = o[q][d][2] = o[q][d][3] = 0.f;
                R[q][0] = R[q][1] = kLow;    // no key seen yet
                l[q][0] = l[q][1] = 0.f;
            }
            for (int i0 = 0; i0 < count; i0 += H) {
                cp_async_wait<S - 2>();
                __syncwarp();                // the step is there, and every lane has read the one before
                if (lleft > 0) load(cur == 0 ? S - 1 : cur - 1);
                cp_async_commit();
                const uint8_t* st = ring + cur * STAGE;
                const uint32_t has_page = (pages_ok >> (4 * cur)) & ((1u << OCT) - 1);
                pages_ok &= ~(15u << (4 * cur));
                cur = cur == S - 1 ? 0 : cur + 1;
                // ---- scores
                float sc[H][NT][4];
#pragma unroll
                for (int h = 0; h < H; h++) {
#pragma unroll
                    for (int q = 0; q < NT; q++) sc[h][q][0] = sc[h][q][1] = sc[h][q][2] = sc[h][q][3] = 0.f;
#pragma unroll
                    for (int c = 0; c < C; c++) {
                        __half2 d[2], m[2];
                        uint2 kw[2] = {make_uint2(0, 0), make_uint2(0, 0)};
#pragma unroll
                        for (int x = 0; x < 2; x++) {
                            const int row = 8 * (2 * h + x) + r;
                            uint32_t dm = 0;
                            if (k_in[c]) {
                                kw[x] = *reinterpret_cast<const uint2*>(st + row * pitch + 32 * c + 8 * t);
                                dm = *reinterpret_cast<const uint32_t*>(st + 2 * NUMBERS + row * pairs + 4 * (2 * c + (t >> 1)));
                            }
                            d[x] = __low2half2(half2_of(dm));
                            m[x] = __high2half2(half2_of(dm));
                        }
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            uint32_t y[2][4];
#pragma unroll
                            for (int x = 0; x < 2; x++) {
                                const uint32_t w = i == 0 ? kw[x].x : kw[x].y;
                                y[x][0] = q4_value(q4_low(w, k1024), d[x], m[x]);
                                y[x][1] = q4_value(q4_high(w, k1024), d[x], m[x]);
                                y[x][2] = q4_value(q4_low(w >> 8, k1024), d[x], m[x]);
                                y[x][3] = q4_value(q4_high(w >> 8, k1024), d[x], m[x]);
                            }
#pragma unroll
                            for (int u = 0; u < 2; u++) {
                                const uint32_t k[4] = {y[0][2 * u], y[1][2 * u], y[0][2 * u + 1], y[1][2 * u + 1]};
                                const int ks = 4 * c + 2 * i + u;
#pragma unroll
                                for (int q = 0; q < NT; q++) {
                                    mma16816(sc[h][q], k, qhi[q][ks][0], qhi[q][ks][1]);
                                    if (SPLITQ) mma16816(sc[h][q], k, qlo[q][SPLITQ ? ks : 0][0], qlo[q][SPLITQ ? ks : 0][1]);
                                }
                            }
                        }
                    }
                }
                const int e0 = (pc + i0) * 16, end = min(lens[s], e0 + 16 * min(H, count - i0));
                const bool whole = e0 + 16 * H <= end && has_page == (1u << OCT) - 1;
                // rows that are not there, and those that some query rows do not see
                if (!whole || e0 + 16 * H - 1 > e_min) {
#pragma unroll
                    for (int h = 0; h < H; h++)
#pragma unroll
                        for (int q = 0; q < NT; q++)
#pragma unroll
                            for (int k = 0; k < 4; k++) {
                                const int at = e0 + 16 * h + r + (k >> 1) * 8;
                                if (!((has_page >> (2 * h + (k >> 1))) & 1u) || at >= end || at > e[q][k & 1]) sc[h][q][k] = -INFINITY;
                            }
                }
                uint32_t ph[H][NT][2], pl[H][NT][2];
#pragma unroll
                for (int q = 0; q < NT; q++) {
                    float top[2];
                    bool move = false;
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        float m = fmaxf(sc[0][q][k], sc[0][q][2 + k]);
                        if (H == 2) m = max3(m, sc[H - 1][q][k], sc[H - 1][q][2 + k]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                        top[k] = fmaxf(m, kLow);
                        move |= (top[k] - R[q][k]) * qs[q][k] > kLag;
                    }
                    if (__any_sync(0xffffffffu, move)) {
                        float c[2];
#pragma unroll
                        for (int k = 0; k < 2; k++) {
                            // (a row's own maximum decides: its bits do not depend on its neighbours)
                            const float up = (top[k] - R[q][k]) * qs[q][k] > kLag ? top[k] : R[q][k];
                            c[k] = exp2_fast((R[q][k] - up) * qs[q][k]);
                            R[q][k] = up;
                            l[q][k] *= c[k];
                        }
#pragma unroll
                        for (int d = 0; d < KS; d++) {
                            o[q][d][0] *= c[0];
                            o[q][d][1] *= c[1];
                            o[q][d][2] *= c[0];
                            o[q][d][3] *= c[1];
                        }
                    }
#pragma unroll
                    for (int h = 0; h < H; h++) {
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            sc[h][q][k] = exp2_fast(fmaf(sc[h][q][k] - R[q][k & 1], qs[q][k & 1], kHead));
                            l[q][k & 1] += sc[h][q][k];          // this thread's cached rows; all are added at the end
                        }
#pragma unroll
                        for (int k = 0; k < 2; k++) {
                            const uint32_t hi = pack_hi(sc[h][q][2 * k], sc[h][q][2 * k + 1]);
                            if (PACK) {      // the first part, or what it leaves
                                const float2 f = __half22float2(half2_of(hi));
                                ph[h][q][k] = transpose8(pack_hi(fmaf(f.x, second, sc[h][q][2 * k]), fmaf(f.y, second, sc[h][q][2 * k + 1])));
                            } else {
                                ph[h][q][k] = transpose8(hi);
                                pl[h][q][k] = transpose8(pack_lo(sc[h][q][2 * k], sc[h][q][2 * k + 1], hi));
                            }
                        }
                    }
                }
                // ---- sums
#pragma unroll
                for (int h = 0; h < H; h++) {
                    uint32_t v[KS][4];       // tile i: dims 2i and 2i + 1 of this lane's, of rows 2t, 2t + 1 and of the eight behind
                    uint32_t vw[4][C], vd[4];
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const int row = 16 * h + 8 * (k / 2) + 2 * t + k % 2;
                        const uint8_t* w = st + NUMBERS + row * pitch + 4 * C * r;
                        vd[k] = 0;
#pragma unroll
                        for (int c = 0; c < C; c++) vw[k][c] = 0;
                        if (!v_in) continue;
                        if (C == 1) {
                            vw[k][0] = *reinterpret_cast<const uint32_t*>(w);
                        } else {
                            const uint2 y = *reinterpret_cast<const uint2*>(w);
                            vw[k][0] = y.x;
                            vw[k][C - 1] = y.y;
                        }
                        vd[k] = *reinterpret_cast<const uint32_t*>(st + 2 * NUMBERS + PAIRS + row * pairs + 4 * (C * r >> 2));
                    }
                    if (!whole)              // rows behind the last: whatever is there, their values are 0
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            if (e0 + 16 * h + 8 * (k / 2) + 2 * t + k % 2 >= end) vd[k] = 0;
#pragma unroll
                    for (int x = 0; x < 2; x++) {
                        const __half2 d = half2_of(__byte_perm(vd[2 * x], vd[2 * x + 1], 0x5410)), m = half2_of(__byte_perm(vd[2 * x], vd[2 * x + 1], 0x7632));
#pragma unroll
                        for (int i = 0; i < KS; i++) {
                            const uint32_t b = i % 4, w = __byte_perm(vw[2 * x][i / 4], vw[2 * x + 1][i / 4], b | b << 4 | (4 + b) << 8 | (4 + b) << 12);
                            v[i][2 * x] = q4_value(q4_low(w, k1024), d, m);
                            v[i][2 * x + 1] = q4_value(q4_high(w, k1024), d, m);
                        }
                    }
                    // a row that some new tokens see and others do not: where its V is not
                    // finite, 0 * V would reach those that do not, so it is added to the
                    // others alone and taken out of the product
                    if (p.n_new > 1 && e0 + 16 * h + 15 > e_min) {
#pragma unroll
                        for (int x = 0; x < 2; x++)
#pragma unroll
                            for (int k = 0; k < 2; k++) {
                                bool wild = false;
#pragma unroll
                                for (int i = 0; i < KS; i++)
#pragma unroll
                                    for (int z = 0; z < 2; z++) wild |= ((v[i][2 * x + z] >> (16 * k)) & 0x7C00u) == 0x7C00u;
                                const uint32_t who = __ballot_sync(0xffffffffu, wild);
                                for (int tt = 0; tt < 4 && who; tt++) {
                                    if (!(who & (0x11111111u << tt))) continue;
#pragma unroll
                                    for (int q = 0; q < NT; q++) {
                                        float pa = __shfl_sync(0xffffffffu, sc[h][q][2 * x], 4 * (2 * tt + k) + t),
                                              pb = __shfl_sync(0xffffffffu, sc[h][q][2 * x + 1], 4 * (2 * tt + k) + t);
                                        if (PACK && t >= 2) pa = pb = 0.f;       // (the first four columns' are whole)
#pragma unroll
                                        for (int i = 0; i < KS; i++)
#pragma unroll
                                            for (int z = 0; z < 2; z++) {
                                                const uint32_t w = __shfl_sync(0xffffffffu, v[i][2 * x + z], 4 * r + tt);
                                                const float y = __half2float(__ushort_as_half((unsigned short)(w >> (16 * k))));
                                                if (pa != 0.f) o[q][i][2 * z] = fmaf(pa, y, o[q][i][2 * z]);
                                                if (pb != 0.f) o[q][i][2 * z + 1] = fmaf(pb, y, o[q][i][2 * z + 1]);
                                            }
                                    }
                                    if (t == tt)
#pragma unroll
                                        for (int i = 0; i < KS; i++)
#pragma unroll
                                            for (int z = 0; z < 2; z++) v[i][2 * x + z] &= k ? 0x0000FFFFu : 0xFFFF0000u;
                                }
                            }
                    }
#pragma unroll
                    for (int i = 0; i < KS; i++)
#pragma unroll
                        for (int q = 0; q < NT; q++) {
                            mma16816(o[q][i], v[i], ph[h][q][0], ph[h][q][1]);
                            if (!PACK) mma16816(o[q][i], v[i], pl[h][q][0], pl[h][q][1]);
                        }
                }
            }
            // ---- this worker's part of the unit
            const long long slot = ((long long)s * units + (g * rt + tile) + me) * min(srows, RU);
            if (PACK)
#pragma unroll
                for (int i = 0; i < KS; i++)
#pragma unroll
                    for (int k = 0; k < 4; k++) o[0][i][k] += __shfl_xor_sync(0xffffffffu, o[0][i][k], 2);
#pragma unroll
            for (int q = 0; q < NT; q++)
#pragma unroll
                for (int k = 0; k < 2; k++) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[q][k] += __shfl_xor_sync(0xffffffffu, l[q][k], d);
                    const int row = q * 8 + 2 * t + k;
                    if (tile * RU + row >= srows || (PACK && t >= 2)) continue;
                    float* dst = a.suffix_o + (slot + row) * p.hd + 8 * C * r;
                    if (v_in)
#pragma unroll
                        for (int i = 0; i < KS; i += 2)
                            *reinterpret_cast<float4*>(dst + 2 * i) = make_float4(o[q][i][k], o[q][i][2 + k], o[q][i + 1][k], o[q][i + 1][2 + k]);
                    if (r == 0) a.suffix_ml[slot + row] = make_float2(fmaxf(R[q][k] * qs[q][k], kLow), l[q][k]);
                }
            left -= count + kUnit;
            if (left > 0) next(s, g, tile, pc, np);
        }
    }
    if (!first && blockIdx.x + 1 == gridDim.x) griddep_wait();   // (as the suffix kernel above)
}

// --------------------------------------------------------------- join --
// One warp per (row, head): the prefix's parts, then the sequence's.  LP lanes
// hold the hd values of a part, four each, and the warp's 32 / LP groups take
// the parts in turn, eight of them in flight per group.
template <int LP>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ PagesDev p, const __grid_constant__ AttendDev a) {
    constexpr int GROUPS = 32 / LP, AHEAD = 8;
    griddep_launch();
    const int w = blockIdx.x * 4 + (threadIdx.x >> 5);         // (rows of all heads: at most 2^25)
    const int lane = threadIdx.x & 31, grp = lane / LP, d = 4 * (lane % LP);
    if (w >= p.n_seqs * p.n_new * a.n_heads) {
        griddep_wait();                      // (every path: this grid must not end before those it follows)
        return;
    }
    if (a.prefix_blocks == 0 && a.suffix_workers == 0) griddep_wait();       // the lengths, otherwise known (below)
    const int token = a.by_heads.of(w), h = w - token * a.n_heads, s = a.by_new.of(token), i = token - s * p.n_new;
    const int g = a.by_gq.of(h), hq = h - g * a.gq;
    const int len = p.lens[s];
    if (len < p.n_new - i) {                 // padding
        griddep_wait();
        return;
    }
    if (lane == 0 && len > clipped_len(p, s)) flag(p.err, LLM_PAGES_BAD_LEN);
    const int srows = p.n_new * a.gq, ru = a.unit_rows, rt = (srows + ru - 1) / ru, row = i * a.gq + hq;
    int np = 0, ns = 0;                      // the row's parts of the prefix and of its pages
    int pre = 0, suf = 0;                    // the first ones' rows
    if (a.prefix_blocks > 0) {
        const int mt = (a.rows + 127) / 128, ntiles = (p.prefix_len + kKT - 1) / kKT, r = token * a.gq + hq, u = g * mt + r / 128;
        const long long total = (long long)mt * p.n_kv * ntiles, x = (long long)u * ntiles;
        const int w0 = (int)owner_of(x, a.prefix_blocks, total);
        np = 2 * ((int)(owner_of(x + ntiles - 1, a.prefix_blocks, total) - w0) + 1);       // a part of each softmax group
        pre = (u + w0) * 256 + r % 128;
    }
    // the lengths (written before this kernel's predecessors began) and the prefix's parts are known
    // by now; the rest comes from those
    griddep_wait();
    const int step = min(srows, ru);
    if (a.suffix_workers > 0) {
        const int b = a.starts[s], pieces = a.starts[s + 1] - b;
        const Deal deal = deal_of(a.starts[p.n_seqs], p.n_kv * rt, a.suffix_workers);
        if (pieces > 0) {
            const int j = g * rt + row / ru;
            const long long x = (long long)b * deal.units + (long long)j * pieces;           // (pieces: kUnit empty ones among them)
            // (the bounds hold by themselves; they keep the reads within the workspace where another
            // call has written into it, which the caller must not let happen)
            const int w0 = max(0, min((int)owner_of(x, deal.workers, deal.total), a.suffix_workers - 1));
            ns = max(0, min((int)owner_of(x + pieces - kUnit - 1, deal.workers, deal.total) - w0 + 1, a.suffix_workers - w0));
            suf = (s * deal.units + j + w0) * step + row % ru;
        }
    }
    const int n = np + ns;
    auto part = [&](int k) { return k < np ? pre + k * 128 : suf + (k - np) * step; };
    float M = -INFINITY, L = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < n; k0 += GROUPS * AHEAD) {
        // the parts' statistics and values are requested together
        float2 ml[(GROUPS * AHEAD + 31) / 32];
        float4 v[AHEAD];
#pragma unroll
        for (int c = 0; c < (GROUPS * AHEAD + 31) / 32; c++) {
            const int k = k0 + c * 32 + lane;
            ml[c] = make_float2(-INFINITY, 0.f);
            if (k < n && c * 32 + lane < GROUPS * AHEAD) ml[c] = (k < np ? a.prefix_ml : a.suffix_ml)[part(k)];
        }
#pragma unroll
        for (int q = 0; q < AHEAD; q++) {
            const int k = k0 + q * GROUPS + grp;
            v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k < n && d < p.hd) v[q] = *reinterpret_cast<const float4*>((k < np ? a.prefix_o : a.suffix_o) + (long long)part(k) * p.hd + d);
        }
        float top = M;
#pragma unroll
        for (int c = 0; c < (GROUPS * AHEAD + 31) / 32; c++) top = fmaxf(top, ml[c].x);
        top = warp_max(top);
        const float c0 = M == -INFINITY ? 0.f : exp2_fast(M - top);
        M = top;
        L *= c0;
        x.x *= c0;
        x.y *= c0;
        x.z *= c0;
        x.w *= c0;
        float wk[(GROUPS * AHEAD + 31) / 32];
#pragma unroll
        for (int c = 0; c < (GROUPS * AHEAD + 31) / 32; c++) {
            wk[c] = exp2_fast(ml[c].x - M);
            L += wk[c] * ml[c].y;
        }
#pragma unroll
        for (int q = 0; q < AHEAD; q++) {
            const float c = __shfl_sync(0xffffffffu, wk[q * GROUPS / 32], (q * GROUPS + grp) & 31);
            x.x = fmaf(c, v[q].x, x.x);
            x.y = fmaf(c, v[q].y, x.y);
            x.z = fmaf(c, v[q].z, x.z);
            x.w = fmaf(c, v[q].w, x.w);
        }
    }
    L = warp_sum(L);
#pragma unroll
    for (int o = LP; o < 32; o <<= 1) {
        x.x += __shfl_xor_sync(0xffffffffu, x.x, o);
        x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
        x.z += __shfl_xor_sync(0xffffffffu, x.z, o);
        x.w += __shfl_xor_sync(0xffffffffu, x.w, o);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;                // a row without any key is zero
    if (d >= p.hd || grp > 0) return;
    const long long at = (long long)token * a.out_stride + (long long)h * p.hd + d;
    if (a.out_f16)
        *reinterpret_cast<uint2*>(static_cast<__half*>(a.out) + at) = make_uint2(pack_hi(x.x * inv, x.y * inv), pack_hi(x.z * inv, x.w * inv));
    else
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
}

// --------------------------------------------------------------- host --
struct Plan {
    int prefix_blocks, suffix_blocks, unit_rows;
    long long prefix_rows, suffix_rows;      // parts of one row each
    size_t off_pml, off_so, off_sml, off_starts, bytes;
};

Plan make_plan(const llm_pages* p, const llm_attend* a, int sms, bool q4) {
    Plan pl{};
    const int gq = a->n_heads / p->n_kv_heads;
    const long long srows = (long long)p->n_new * gq, rows = srows * p->n_seqs;
    if (p->prefix_len > 0) {
        // a block per SM, but none with less than two tiles
        const long long units = (rows + 127) / 128 * p->n_kv_heads, tiles = units * ((p->prefix_len + kKT - 1) / kKT);
        pl.prefix_blocks = (int)std::max<long long>(1, std::min<long long>(sms, tiles / 2));
        pl.prefix_rows = (units + pl.prefix_blocks) * 256;
    }
    if (p->max_pages > 0) {
        // workers for as many blocks as an SM holds at once, but no more than the
        // longest sequences could keep busy
        const int ru = q4 ? unit_rows_q4((int)srows, p->head_dim) : unit_rows((int)srows);
        pl.unit_rows = ru;
        const long long units = (long long)p->n_kv_heads * ((srows + ru - 1) / ru),
                        most = units * p->n_seqs * (((long long)p->max_pages * p->page_size + 15) / 16 + kUnit),
                        blocks = (most + kQuantum * kSuffixWarps - 1) / (kQuantum * kSuffixWarps);
        const int hdp = p->head_dim <= 64 ? 64 : 128, ctas = q4 ? suffix_q4_ctas(hdp, ru / 8) : suffix_ctas(hdp, ru / 8);
        pl.suffix_blocks = (int)std::max<long long>(1, std::min<long long>(blocks, (long long)ctas * sms));
        pl.suffix_rows = (units * p->n_seqs + pl.suffix_blocks * kSuffixWarps) * std::min<long long>(srows, ru);
    }
    auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
    size_t at = up((size_t)pl.prefix_rows * p->head_dim * 4);
    pl.off_pml = at;
    at += up((size_t)pl.prefix_rows * 8);
    pl.off_so = at;
    at += up((size_t)pl.suffix_rows * p->head_dim * 4);
    pl.off_sml = at;
    at += up((size_t)pl.suffix_rows * 8);
    pl.off_starts = at;
    if (pl.suffix_blocks > 0) at += up((size_t)(p->n_seqs + 1) * 4);
    pl.bytes = at;
    return pl;
}

// Cached rows as {hd, n_kv, rows}, `stride` elements apart, in boxes of
// box_rows: columns behind hd and rows behind the last read as zero.
bool rows_map(CUtensorMap* m, const uint16_t* base, int hd, int n_kv, long long rows, int64_t stride, int box_rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dim[3] = {(cuuint64_t)hd, (cuuint64_t)n_kv, (cuuint64_t)(rows > 0 ? rows : 1)};
    cuuint64_t step[2] = {(cuuint64_t)hd * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<uint16_t*>(base), dim, step, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Percent of an SM's memory as shared memory for the prefix kernel and a suffix
// kernel that runs beside it: an SM that holds a block of one takes none of the
// other under another division.  (A suffix kernel alone wants the cache: 268 MB of
// pages 65 us, 49 us with the default.)
constexpr int kCarveout = 72;
// The page kernel's rings want all of it, beside the prefix kernel or alone.
constexpr int kCarveoutQ4 = 100;

void launch_attributes(cudaLaunchAttribute (&at)[2], int carveout) {
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
    at[1].val.sharedMemCarveout = carveout;
}

template <int HDP, bool SPLITQ>
cudaError_t launch_prefix(cudaStream_t st, const CUtensorMap& mk, const CUtensorMap& mv, const PagesDev& pd, const AttendDev& ad, int carveout) {
    auto k = prefix_kernel<HDP, SPLITQ>;
    static OncePerDevice once;
    const cudaError_t e = once([&] { return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, PrefixPlan<HDP>::kSmem); });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ad.prefix_blocks);
    cfg.blockDim = dim3(kPrefixThreads);
    cfg.dynamicSmemBytes = (size_t)PrefixPlan<HDP>::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    launch_attributes(at, carveout);
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k, mk, mv, pd, ad);
}

// Shared memory of a block of the pages' kernel: row counts and sums of the sequences, the rings.
constexpr int suffix_smem(int n_seqs, int hdp, bool q4) { return q4 ? ((2 * n_seqs + 1) * 4 + 15) / 16 * 16 + q4_rings(hdp) : (2 * n_seqs + 1) * 4; }
// (within the 48 KB that need no opt-in)
static_assert(suffix_smem(kMaxSeqs, 128, false) <= 47 * 1024, "shared memory of the sequences");

typedef void (*PagesKernel)(PagesDev, AttendDev, int);
template <int HDP, int NT>
PagesKernel pages_kernel(bool splitq) { return splitq ? suffix_kernel<HDP, NT, true> : suffix_kernel<HDP, NT, false>; }
// (*e: whether it may have the shared memory that it needs)
template <int HDP, int NT, bool PACK, bool FULL>
PagesKernel pages_q4_kernel(bool splitq, cudaError_t* e) {
    const PagesKernel one = suffix_q4_kernel<HDP, NT, false, PACK, FULL>, two = suffix_q4_kernel<HDP, NT, true, PACK, FULL>;
    static OncePerDevice once;
    *e = once([&] {
        const int most = suffix_smem(kMaxSeqs, HDP, true);
        const cudaError_t r = cudaFuncSetAttribute(one, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        return r != cudaSuccess ? r : cudaFuncSetAttribute(two, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    });
    return splitq ? two : one;
}

// carveout 0: the driver's choice.
cudaError_t launch_suffix(PagesKernel k, cudaStream_t st, const PagesDev& pd, const AttendDev& ad, int first, int blocks, int smem, int carveout) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(32 * kSuffixWarps);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    launch_attributes(at, carveout);
    cfg.attrs = at;
    cfg.numAttrs = carveout ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, pd, ad, first);
}

int check_attend(const llm_pages* p, const llm_attend* a) {
    if (!a) return fail_op(LLM_ERR_INVALID_ARG, "the attention arguments are NULL");
    if (a->n_heads < 1 || a->n_heads % p->n_kv_heads)
        return fail_op(LLM_ERR_INVALID_ARG, "n_heads %d is not a multiple of n_kv_heads %d", a->n_heads, p->n_kv_heads);
    if (((long long)p->max_pages * p->page_size / 16 + 1) > (1ll << 50) / std::max(1ll, (long long)p->n_seqs * p->n_new * a->n_heads))
        return fail_op(LLM_ERR_UNSUPPORTED, "the sequences' pages hold too many rows for that many heads");
    if (p->prefix_len > INT_MAX - kKT) return fail_op(LLM_ERR_UNSUPPORTED, "prefix_len %d exceeds 2^31 - 65", p->prefix_len);
    if (p->n_seqs > kMaxSeqs) return fail_op(LLM_ERR_UNSUPPORTED, "n_seqs %d exceeds %d", p->n_seqs, kMaxSeqs);
    if ((long long)p->n_seqs * ((long long)p->max_pages * p->page_size / 16 + 1) > INT_MAX / 2)
        return fail_op(LLM_ERR_UNSUPPORTED, "the sequences' pages hold more than 2^34 rows together");
    if (p->n_kv_heads > 65535) return fail_op(LLM_ERR_UNSUPPORTED, "n_kv_heads %d exceeds 65535", p->n_kv_heads);
    if ((long long)p->n_seqs * p->n_new * a->n_heads > INT_MAX / 64)
        return fail_op(LLM_ERR_UNSUPPORTED, "more than 2^25 rows of all heads");
    // a block's share of the prefix's tiles and a warp's of the pages' pieces are counted in 32 bits
    const long long gq = a->n_heads / p->n_kv_heads, srows = p->n_new * gq, ru = unit_rows((int)srows);
    if ((srows * p->n_seqs + 127) / 128 * p->n_kv_heads * ((p->prefix_len + (long long)kKT - 1) / kKT) > 1ll << 38)
        return fail_op(LLM_ERR_UNSUPPORTED, "the prefix is too long for that many rows and heads");
    if ((srows + ru - 1) / ru * p->n_kv_heads * p->n_seqs * (((long long)p->max_pages * p->page_size + 15) / 16 + kUnit) > 1ll << 41)
        return fail_op(LLM_ERR_UNSUPPORTED, "the sequences' pages hold too many rows for that many heads");
    if (!type_bytes(a->q_dtype) || !type_bytes(a->out_dtype))
        return fail_op(LLM_ERR_UNSUPPORTED, "q or out is neither LLM_F32 nor LLM_F16");
    if (!(a->scale >= 0.f) || !(a->scale < INFINITY)) return fail_op(LLM_ERR_INVALID_ARG, "scale is not a finite number >= 0");
    return LLM_OK;
}

}  // namespace

namespace {

// llm_attend_batch; q4: over pages of 4-bit values.
int attend(const llm_pages* pages, const llm_attend* a, cudaStream_t stream, int* timeout, int wait_limit, bool q4) {
    Q4Dev f{};
    int rc = q4 ? check_pages_q4(pages, true, &f) : check_pages(pages, true);
    if (rc || (rc = check_attend(pages, a))) return rc;
    if (pages->n_seqs == 0) return LLM_OK;
    const long long rows = (long long)pages->n_seqs * pages->n_new, width = (long long)a->n_heads * pages->head_dim,
                    kv = (long long)pages->n_kv_heads * pages->head_dim;
    if ((rc = check_rows("q", a->q, a->q_dtype, a->q_stride, width, rows)) ||
        (rc = check_rows("out", a->out, a->out_dtype, a->out_stride, width, rows)))
        return rc;
    const bool prefix = pages->prefix_len > 0;
    if (prefix && ((rc = check_rows("prefix_k", a->prefix_k, LLM_F16, a->prefix_stride, kv, 2)) ||
                   (rc = check_rows("prefix_v", a->prefix_v, LLM_F16, a->prefix_stride, kv, 2))))
        return rc;
    if (prefix && a->prefix_stride >= (1ll << 39)) return fail_op(LLM_ERR_UNSUPPORTED, "prefix_stride is too large");
    const Plan pl = make_plan(pages, a, sm_count(), q4);
    if (pl.bytes > 0 && (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < (int64_t)pl.bytes))
        return fail_op(LLM_ERR_INVALID_ARG, "workspace: NULL, not 256-byte aligned, or below %zu bytes", pl.bytes);
    const PagesDev pd = pages_dev(pages);
    const float scale = a->scale == 0.f ? (float)(1.0 / sqrt((double)pages->head_dim)) : a->scale;
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    AttendDev ad{};
    ad.n_heads = a->n_heads;
    ad.gq = a->n_heads / pages->n_kv_heads;
    ad.rows = (int)(rows * ad.gq);
    ad.sc = (float)((double)scale * 1.4426950408889634);
    ad.q = a->q; ad.q_stride = a->q_stride; ad.q_f16 = a->q_dtype == LLM_F16;
    ad.out = a->out; ad.out_stride = a->out_stride; ad.out_f16 = a->out_dtype == LLM_F16;
    ad.prefix_o = reinterpret_cast<float*>(ws);
    ad.prefix_ml = reinterpret_cast<float2*>(ws + pl.off_pml);
    ad.suffix_o = reinterpret_cast<float*>(ws + pl.off_so);
    ad.suffix_ml = reinterpret_cast<float2*>(ws + pl.off_sml);
    ad.prefix_blocks = pl.prefix_blocks;
    ad.by_heads = Div((uint32_t)a->n_heads);
    ad.by_new = Div((uint32_t)pages->n_new);
    ad.by_gq = Div((uint32_t)ad.gq);
    ad.starts = reinterpret_cast<int*>(ws + pl.off_starts);
    ad.suffix_workers = pl.suffix_blocks * kSuffixWarps;
    ad.unit_rows = pl.unit_rows;
    ad.q4 = f;
    ad.timeout = timeout;
    ad.wait_limit = wait_limit > 0 ? wait_limit : kWaitLimit;
    const bool sq = !ad.q_f16;
    const int hd = pages->head_dim;
    const int carveout = q4 ? kCarveoutQ4 : kCarveout;
    cudaError_t e = cudaSuccess;
    if (prefix) {
        CUtensorMap mk, mv;
        if (!rows_map(&mk, a->prefix_k, hd, pages->n_kv_heads, pages->prefix_len, a->prefix_stride, kKT) ||
            !rows_map(&mv, a->prefix_v, hd, pages->n_kv_heads, pages->prefix_len, a->prefix_stride, kKT))
            return fail_op(LLM_ERR_CUDA, "a tensor map of the prefix");
#define LLM_PREFIX(HDP) (sq ? launch_prefix<HDP, true>(stream, mk, mv, pd, ad, carveout) : launch_prefix<HDP, false>(stream, mk, mv, pd, ad, carveout))
        e = hd <= 64 ? LLM_PREFIX(64) : LLM_PREFIX(128);
#undef LLM_PREFIX
        if (e != cudaSuccess) return launched(e, "llm_attend_batch (prefix)");
    }
    if (pl.suffix_blocks > 0) {
        const int first = prefix ? 0 : 1;
        PagesKernel k;
        const int tiles = pl.unit_rows / 8;
        if (!q4) {
            k = hd <= 64 ? (tiles == 1 ? pages_kernel<64, 1>(sq) : pages_kernel<64, 2>(sq)) : (tiles == 1 ? pages_kernel<128, 1>(sq) : pages_kernel<128, 2>(sq));
        } else if (pages->n_new * ad.gq <= 4) {
            k = hd == 64    ? pages_q4_kernel<64, 1, true, true>(sq, &e)
                : hd < 64   ? pages_q4_kernel<64, 1, true, false>(sq, &e)
                : hd == 128 ? pages_q4_kernel<128, 1, true, true>(sq, &e)
                            : pages_q4_kernel<128, 1, true, false>(sq, &e);
        } else if (hd <= 64) {
            k = tiles == 1   ? pages_q4_kernel<64, 1, false, false>(sq, &e)
                : tiles == 2 ? pages_q4_kernel<64, 2, false, false>(sq, &e)
                             : pages_q4_kernel<64, 3, false, false>(sq, &e);
        } else {
            k = tiles == 1 ? pages_q4_kernel<128, 1, false, false>(sq, &e) : pages_q4_kernel<128, 2, false, false>(sq, &e);
        }
        if (e == cudaSuccess)
            e = launch_suffix(k, stream, pd, ad, first, pl.suffix_blocks, suffix_smem(pages->n_seqs, hd <= 64 ? 64 : 128, q4),
                              q4 || !first ? carveout : 0);
        if (e != cudaSuccess) return launched(e, "llm_attend_batch (suffix)");
    }
    const dim3 grid((unsigned)((rows * a->n_heads + 3) / 4));
    return launched(hd <= 32   ? launch_dep(join_kernel<8>, grid, dim3(128), 0, stream, pd, ad)
                    : hd <= 64 ? launch_dep(join_kernel<16>, grid, dim3(128), 0, stream, pd, ad)
                               : launch_dep(join_kernel<32>, grid, dim3(128), 0, stream, pd, ad),
                    "llm_attend_batch (join)");
}

int64_t attend_workspace(const llm_pages* pages, const llm_attend* a, bool q4) {
    Q4Dev f{};
    int rc = q4 ? check_pages_q4(pages, false, &f) : check_pages(pages, false);
    if (rc || (rc = check_attend(pages, a))) return rc;
    return (int64_t)make_plan(pages, a, sm_count(), q4).bytes;
}

}  // namespace

int attend_batch(const llm_pages* pages, const llm_attend* a, cudaStream_t stream, int* timeout, int wait_limit) {
    return attend(pages, a, stream, timeout, wait_limit, false);
}

}  // namespace llm

using namespace llm;

extern "C" int64_t llm_attend_batch_workspace(const llm_pages* pages, const llm_attend* a) { return attend_workspace(pages, a, false); }
extern "C" int64_t llm_attend_batch_q4_workspace(const llm_pages* pages, const llm_attend* a) { return attend_workspace(pages, a, true); }

extern "C" int llm_attend_batch(const llm_pages* pages, const llm_attend* a, llm_stream_t stream) {
    return attend_batch(pages, a, stream, nullptr, 0);
}
extern "C" int llm_attend_batch_q4(const llm_pages* pages, const llm_attend* a, llm_stream_t stream) {
    return attend(pages, a, stream, nullptr, 0, true);
}
