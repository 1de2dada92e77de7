// Attention of a batch that shares a prefix (llm_attend_batch, include/llm.h):
// out = sum_t softmax_t(scale q.k_t) v_t over the prefix's rows and the row's
// own sequence's pages.
//
// The softmax splits over the keys: a part keeps, per query row, a reference
// M, l = sum 2^(y_t - M) and O = sum 2^(y_t - M) v_t over its keys (y =
// scale log2(e) q.k), and parts join as out = sum_i w_i O_i / sum_i w_i l_i,
// w_i = 2^(M_i - max M).  Three kernels, chained by programmatic dependent
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
    float* prefix_o;                // [prefix splits][n_kv][rows][hd]
    float2* prefix_ml;              // [prefix splits][n_kv][rows]: M, l
    float* suffix_o;                // [n_seqs][n_kv][suffix splits][n_new * gq][hd]
    float2* suffix_ml;
    int prefix_splits, suffix_splits;
};

// Probabilities are kept as 2^(y - M) with M = (a recent maximum) - kHead, so
// that the largest is about 2^kHead: F16 then resolves those 2^-33 of it
// (its subnormal step 2^-24, halved by rounding), and the reference may lag
// behind the running maximum by kLag before 2^(kHead + kLag) nears F16's 2^16.
constexpr float kHead = 8.f, kLag = 6.f;

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

// Element offset of row r (of kv head g's rows) in q.
__device__ __forceinline__ long long q_offset(const AttendDev& a, int hd, int g, int r) {
    return (long long)(r / a.gq) * a.q_stride + (long long)(g * a.gq + r % a.gq) * hd;
}

// ------------------------------------------------------------- prefix --
constexpr int kKT = 64;                      // keys per tile

// Blocks of an SM: two of head sizes up to 64 overlap one's softmax with the
// other's waits; the tiles of larger heads fill an SM's shared memory at one.
constexpr int prefix_ctas(int hd) { return hd <= 64 ? 2 : 1; }

template <int HDP, bool SPLITQ>
struct PrefixPlan {
    static constexpr int kSlabs = HDP / 64;                        // 64-column (128-byte) slabs of a row
    static constexpr bool kQInTmem = HDP == 64;
    static constexpr int kQBytes = kQInTmem ? 0 : 128 * HDP * 2;   // the query tile (twice with SPLITQ)
    static constexpr int kTileBytes = kKT * HDP * 2;               // K or V
    static constexpr int kCtas = prefix_ctas(HDP);                 // per SM
    static constexpr int kStages = HDP == 64 ? 6 : SPLITQ ? 4 : 5;
    static constexpr int kBarBytes = 256;
    static constexpr int kSmem = kQBytes * (SPLITQ ? 2 : 1) + kStages * 2 * kTileBytes + kBarBytes + 1024;
    static constexpr int kTmemCols = 256;                          // S0 | S1 (64 each) | O (HDP) | Q (32 a part)
};

constexpr int kPrefixThreads = 192;

__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t par, int* err) {
    for (long long i = 0; i < kSpinLimit / 16; i++)
        if (mbar_try_wait(bar, par)) return true;
    flag(err, LLM_PAGES_TIMEOUT);
    return false;
}

// The same for a whole warp that goes on to warp-wide instructions.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t par, int* err) {
    return __all_sync(0xffffffffu, bar_wait(bar, par, err));
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

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
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
__device__ __forceinline__ void tm_st32(uint32_t a, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(a),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
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

// 128 query rows of kv head g against one split of the prefix:
//   warps 0-3  softmax, one query row per thread (its TMEM lane): reads the
//              row's 64 scores, writes its probabilities back over them as
//              F16 (with SPLITP the rounded-off rest beside them), and rescales
//              O when the row's maximum has moved by more than kLag;
//   warp 4     MMA: S = Q K^T into one of two score buffers, one tile ahead;
//   warp 5     TMA: 64-key tiles of K and V into a ring; MMA: O += P V, P from
//              tensor memory.
// Two MMA warps, because each wait and each issue takes one of them 150 to 200
// cycles; a seventh warp for the copies would leave two blocks of an SM 128
// registers a thread, and the scores would spill.
// Q is read from tensor memory too where it fits (head sizes up to 64): an MMA
// whose 128-row operand comes from shared memory takes 48 cycles at this width,
// for 32 of work.
// SPLITQ: Q as two F16 parts; SPLITP: P as two F16 parts.
template <int HDP, bool SPLITQ, bool SPLITP>
__global__ void __launch_bounds__(kPrefixThreads, PrefixPlan<HDP, SPLITQ>::kCtas)
    prefix_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                  const __grid_constant__ PagesDev p, const __grid_constant__ AttendDev a) {
    using G = PrefixPlan<HDP, SPLITQ>;
    constexpr int NS = G::kStages;
    extern __shared__ __align__(1024) uint8_t smraw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~(uintptr_t)1023);
    uint8_t* qs = sm;
    uint8_t* ring = sm + G::kQBytes * (SPLITQ ? 2 : 1);
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + NS * 2 * G::kTileBytes);
    uint64_t* empty = full + NS;
    uint64_t* sfull = empty + NS;            // [2] scores of a tile are in buffer b
    uint64_t* pfull = sfull + 2;             // [2] probabilities of a tile are in buffer b
    uint64_t* pvdone = pfull + 2;            // [2] the P V of a tile in buffer b has been added
    uint64_t* qfull = pvdone + 2;
    uint64_t* fin = qfull + 1;               // every P V has been added
    uint64_t* qfin = fin + 1;                // every MMA of the scores has completed
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(qfin + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mtiles = (a.rows + 127) / 128;
    const int m0 = (int)(blockIdx.x % mtiles) * 128, sp = (int)(blockIdx.x / mtiles), g = blockIdx.y;
    const int ntiles = (p.prefix_len + kKT - 1) / kKT;
    const int t0 = (int)((long long)ntiles * sp / a.prefix_splits), n = (int)((long long)ntiles * (sp + 1) / a.prefix_splits) - t0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(&sfull[b], 1);
            mbar_init(&pfull[b], 4);
            mbar_init(&pvdone[b], 1);
        }
        mbar_init(qfull, 4);
        mbar_init(fin, 1);
        mbar_init(qfin, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 4) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(G::kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tm_fence_before();
    __syncthreads();
    tm_fence_after();
    const uint32_t tmem = *tmem_slot, to = tmem + 128;
    // the suffix kernel may start once every CTA here has seen the work before
    // this kernel complete: it needs that work, but nothing of this kernel's
    griddep_wait();
    griddep_launch();

    if (warp == 4) {
        // The whole warp walks the loop and one elected lane issues: the tile
        // counters and descriptors stay in uniform registers (a loop of one
        // lane alone took 90 to 140 cycles per MMA to issue, and set the pace).
        // F16 operands, F32 accumulators, M 128, N 64, both K-major.
        constexpr uint32_t is = (1u << 4) | ((uint32_t)(kKT >> 3) << 17) | (8u << 24);
        const uint64_t dq = desc_sw128(smem_addr(qs), 16), dk = desc_sw128(smem_addr(ring), 16);
        bool ok = warp_wait(qfull, 0, p.err);
        for (int it = 0; it < n && ok; it++) {
            if (!(ok = warp_wait(&full[it % NS], (uint32_t)((it / NS) & 1), p.err))) break;
            // these scores go where tile it - 2's probabilities were
            if (it > 1 && !(ok = warp_wait(&pvdone[it & 1], (uint32_t)(((it >> 1) - 1) & 1), p.err))) break;
            tm_fence_after();
            const uint64_t k = dk + (uint64_t)((it % NS) * (2 * G::kTileBytes >> 4));
            const uint32_t d = tmem + (uint32_t)((it & 1) * 64);
            if (elect_one()) {
#pragma unroll
                for (int part = 0; part < (SPLITQ ? 2 : 1); part++)
#pragma unroll
                    for (int kk = 0; kk < HDP / 16; kk++) {
                        const uint64_t kd = k + (((kk / 4) * kKT * 128 + (kk % 4) * 32) >> 4);
                        if (G::kQInTmem)
                            mma_ts(d, tmem + 192 + part * 32 + kk * 8, kd, is, part + kk > 0);
                        else
                            mma_ss(d, dq + ((part * G::kQBytes + (kk / 4) * 128 * 128 + (kk % 4) * 32) >> 4), kd, is, part + kk > 0);
                    }
                mma_commit(&sfull[it & 1]);
            }
            __syncwarp();
        }
        // every MMA issued has completed before the tensor memory is freed
        if (elect_one()) mma_commit(qfin);
        __syncwarp();
        warp_wait(qfin, 0, p.err);
    } else if (warp == 5) {
        // N HDP; V has the keys (the MMA's K) as rows, so it is MN-major
        constexpr uint32_t io = (1u << 4) | (1u << 16) | ((uint32_t)(HDP >> 3) << 17) | (8u << 24);
        const uint64_t dv = desc_sw128(smem_addr(ring) + G::kTileBytes, kKT * 128);
        auto load = [&](int it) {            // tile it into its stage
            uint8_t* st = ring + (it % NS) * 2 * G::kTileBytes;
            if (elect_one()) {
                mbar_arrive_expect_tx(&full[it % NS], 2 * G::kTileBytes);
#pragma unroll
                for (int c = 0; c < G::kSlabs; c++) tma_3d_g2s(st + c * kKT * 128, &mk, c * 64, g, (t0 + it) * kKT, &full[it % NS]);
#pragma unroll
                for (int c = 0; c < G::kSlabs; c++)
                    tma_3d_g2s(st + G::kTileBytes + c * kKT * 128, &mv, c * 64, g, (t0 + it) * kKT, &full[it % NS]);
            }
            __syncwarp();
        };
        int loaded = 0;
        for (; loaded < min(n, NS); loaded++) load(loaded);
        for (int it = 0; it < n; it++) {
            // tile it - 1's stage is free when its P V is done, while the softmax of tile it runs
            if (it > 0 && loaded < n) {
                if (!warp_wait(&empty[(it - 1) % NS], (uint32_t)(((it - 1) / NS) & 1), p.err)) break;
                load(loaded++);
            }
            if (!warp_wait(&pfull[it & 1], (uint32_t)((it >> 1) & 1), p.err)) break;
            tm_fence_after();
            const uint64_t v = dv + (uint64_t)((it % NS) * (2 * G::kTileBytes >> 4));
            const uint32_t pa = tmem + (uint32_t)((it & 1) * 64);
            if (elect_one()) {
#pragma unroll
                for (int part = 0; part < (SPLITP ? 2 : 1); part++)
#pragma unroll
                    for (int kk = 0; kk < kKT / 16; kk++)
                        mma_ts(to, pa + part * 32 + kk * 8, v + (kk * 16 * 128 >> 4), io, it > 0 || part + kk > 0);
                mma_commit(&pvdone[it & 1]);
                mma_commit(&empty[it % NS]);
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(fin);
        __syncwarp();
        warp_wait(fin, 0, p.err);
        // every copy has landed before the block can end (at once, unless a wait gave up)
        for (int k = loaded - 1; k >= 0 && k >= loaded - NS; k--) warp_wait(&full[k % NS], (uint32_t)((k / NS) & 1), p.err);
    } else {
        // ---- Q into tensor memory, this thread's row, or into shared memory,
        // swizzled as the descriptors say
        if constexpr (G::kQInTmem) {
            const int r = m0 + warp * 32 + lane;
            const long long at = r < a.rows ? q_offset(a, p.hd, g, r) : 0;
            const uint32_t tq = tmem + ((uint32_t)(warp * 32) << 16) + 192;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                uint32_t hi[16], lo[SPLITQ ? 16 : 1];
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    if (r < a.rows && h * 32 + c * 8 < p.hd) load_q8(a, at + h * 32 + c * 8, x);
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        hi[4 * c + k] = pack_hi(x[2 * k], x[2 * k + 1]);
                        if (SPLITQ) lo[SPLITQ ? 4 * c + k : 0] = pack_lo(x[2 * k], x[2 * k + 1], hi[4 * c + k]);
                    }
                }
                tm_st16(tq + h * 16, hi);
                if (SPLITQ) tm_st16(tq + 32 + h * 16, lo);
            }
            tm_wait_st();
            tm_fence_before();
        }
        for (int i = threadIdx.x; !G::kQInTmem && i < 128 * (HDP / 8); i += 128) {
            const int r = i / (HDP / 8), c = i % (HDP / 8);
            float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (m0 + r < a.rows && c * 8 < p.hd) load_q8(a, q_offset(a, p.hd, g, m0 + r) + c * 8, x);
            const uint4 hi = make_uint4(pack_hi(x[0], x[1]), pack_hi(x[2], x[3]), pack_hi(x[4], x[5]), pack_hi(x[6], x[7]));
            uint8_t* at = qs + (c / 8) * 128 * 128 + r * 128 + (((c % 8) ^ (r & 7)) << 4);
            *reinterpret_cast<uint4*>(at) = hi;
            if (SPLITQ)
                *reinterpret_cast<uint4*>(at + G::kQBytes) = make_uint4(pack_lo(x[0], x[1], hi.x), pack_lo(x[2], x[3], hi.y),
                                                                         pack_lo(x[4], x[5], hi.z), pack_lo(x[6], x[7], hi.w));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(qfull);
        // ---- softmax of row m0 + 32 warp + lane
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        float M = 0.f, l = 0.f;              // M: the reference less kHead
        bool ok = true;
        for (int it = 0; it < n; it++) {
            const uint32_t sb = tmem + lanes + (uint32_t)((it & 1) * 64);
            if (!(ok = warp_wait(&sfull[it & 1], (uint32_t)((it >> 1) & 1), p.err))) break;
            tm_fence_after();
            uint32_t s[64];
            tm_ld32(sb, s);
            tm_ld32(sb + 32, s + 32);
            tm_wait_ld();
            const int valid = p.prefix_len - (t0 + it) * kKT;
            if (valid < kKT) {
#pragma unroll
                for (int c = 0; c < 64; c++)
                    if (c >= valid) s[c] = 0xFF800000u;           // -infinity
            }
            float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};      // four chains side by side
#pragma unroll
            for (int c = 0; c < 64; c++) mx4[c & 3] = fmaxf(mx4[c & 3], __uint_as_float(s[c]));
            const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
            const float top = fmaxf(mx * a.sc, -1e30f) - kHead;
            if (it == 0) {
                M = top;
            } else if (__any_sync(0xffffffffu, top > M + kLag)) {
                float c = 1.f;
                if (top > M + kLag) {
                    c = exp2_fast(M - top);
                    M = top;
                }
                l *= c;
                if (!(ok = warp_wait(&pvdone[(it - 1) & 1], (uint32_t)(((it - 1) >> 1) & 1), p.err))) break;
                tm_fence_after();
#pragma unroll
                for (int h = 0; h < HDP; h += 32) {
                    uint32_t o[32];
                    tm_ld32(to + lanes + h, o);
                    tm_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; k++) o[k] = __float_as_uint(__uint_as_float(o[k]) * c);
                    tm_st32(to + lanes + h, o);
                }
            }
            float l0 = 0.f, l1 = 0.f;
#pragma unroll
            for (int h = 0; h < 32; h += 16) {
                uint32_t hi[16], lo[SPLITP ? 16 : 1];
#pragma unroll
                for (int c = 0; c < 16; c++) {
                    const float x = exp2_fast(fmaf(__uint_as_float(s[2 * (h + c)]), a.sc, -M));
                    const float y = exp2_fast(fmaf(__uint_as_float(s[2 * (h + c) + 1]), a.sc, -M));
                    l0 += x;
                    l1 += y;
                    hi[c] = pack_hi(x, y);
                    if (SPLITP) lo[SPLITP ? c : 0] = pack_lo(x, y, hi[c]);
                }
                tm_st16(sb + h, hi);
                if (SPLITP) tm_st16(sb + 32 + h, lo);
            }
            l += l0 + l1;
            tm_wait_st();
            tm_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pfull[it & 1]);
        }
        if (ok) ok = warp_wait(fin, 0, p.err);
        tm_fence_after();
        if (ok) {
            const int r = m0 + warp * 32 + lane;
            const long long at = ((long long)sp * p.n_kv + g) * a.rows + r;
#pragma unroll
            for (int h = 0; h < HDP; h += 32) {
                uint32_t o[32];
                tm_ld32(to + lanes + h, o);
                tm_wait_ld();
                if (r < a.rows)
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        if (h + k < p.hd)
                            *reinterpret_cast<uint4*>(a.prefix_o + at * p.hd + h + k) = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
            }
            if (r < a.rows) a.prefix_ml[at] = make_float2(M, l);
        }
    }
    tm_fence_before();
    __syncthreads();
    if (warp == 4)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(G::kTmemCols));
}

// ------------------------------------------------------------- suffix --
constexpr int kSuffixWarps = 4, kSuffixBufs = 3;

// Rows of a sequence's pages that its new tokens see, and how its splits share
// them: `per` 64-row tiles each.
struct SuffixCut {
    int len, per, parts;
};
__device__ __forceinline__ SuffixCut suffix_cut(const PagesDev& p, int s, int splits) {
    SuffixCut c;
    const long long cap = (long long)p.max_pages << p.page_shift;
    c.len = (int)max(0ll, min((long long)p.lens[s], cap));
    const int tiles = (c.len + 63) / 64;
    c.per = max(1, (tiles + splits - 1) / max(1, splits));
    c.parts = (tiles + c.per - 1) / c.per;
    return c;
}

// 16 query rows of one kv head of one sequence against one split of its pages.
// Each warp takes every fourth 16-row piece of the split with a running
// softmax of its own; its rows arrive by cp.async, three pieces in flight, in
// rows padded to HDP + 8 halves (ldmatrix without bank conflicts), so the warps
// only meet at the end.  Scores and sums are mma.sync m16n8k16 products.
template <int HDP, bool SPLITQ, bool SPLITP>
__global__ void __launch_bounds__(32 * kSuffixWarps) suffix_kernel(const __grid_constant__ PagesDev p,
                                                                   const __grid_constant__ AttendDev a, int first) {
    constexpr int PITCH = HDP + 8;
    extern __shared__ __align__(16) uint8_t smraw[];
    if (first) griddep_wait();               // otherwise the prefix kernel has waited for the work before it
    griddep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int srows = p.n_new * a.gq, rt = (srows + 15) / 16;
    const int sp = (int)(blockIdx.x % a.suffix_splits), tile = (int)(blockIdx.x / a.suffix_splits) % rt;
    const int s = (int)(blockIdx.x / a.suffix_splits) / rt, g = blockIdx.y;
    const SuffixCut cut = suffix_cut(p, s, a.suffix_splits);
    const int k0 = sp * cut.per * 64, k1 = min(cut.len, k0 + cut.per * 64);
    if (k0 < k1) {
        __half* mine = reinterpret_cast<__half*>(smraw) + warp * kSuffixBufs * 2 * 16 * PITCH;
        if (p.hd < HDP) {
            // columns behind hd: zero once, never written again
            const int w = (HDP - p.hd) / 8;
            for (int i = lane; i < kSuffixBufs * 32 * w; i += 32)
                *reinterpret_cast<uint4*>(mine + (i / w) * PITCH + p.hd + (i % w) * 8) = make_uint4(0, 0, 0, 0);
        }
        const int r = lane >> 2, t = lane & 3;
        // this thread's two rows of the tile; rows behind the last repeat it (never stored)
        const int ra = min(tile * 16 + r, srows - 1), rb = min(tile * 16 + r + 8, srows - 1);
        // the last row each of them sees (a padding row: none)
        const int ea = p.lens[s] - p.n_new + ra / a.gq, eb = p.lens[s] - p.n_new + rb / a.gq;
        uint32_t qhi[HDP / 16][4], qlo[SPLITQ ? HDP / 16 : 1][4];
        {
            const long long oa = q_offset(a, p.hd, g, s * srows + ra), ob = q_offset(a, p.hd, g, s * srows + rb);
#pragma unroll
            for (int ks = 0; ks < HDP / 16; ks++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int col = ks * 16 + (j >> 1) * 8 + 2 * t;
                    const long long at = ((j & 1) ? ob : oa) + col;
                    float2 x = make_float2(0.f, 0.f);
                    if (col < p.hd)
                        x = a.q_f16 ? __half22float2(*reinterpret_cast<const __half2*>(static_cast<const __half*>(a.q) + at))
                                    : *reinterpret_cast<const float2*>(static_cast<const float*>(a.q) + at);
                    qhi[ks][j] = pack_hi(x.x, x.y);
                    if (SPLITQ) qlo[SPLITQ ? ks : 0][j] = pack_lo(x.x, x.y, qhi[ks][j]);
                }
        }
        float o[HDP / 8][4];
#pragma unroll
        for (int i = 0; i < HDP / 8; i++) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float Ma = -INFINITY, Mb = -INFINITY, la = 0.f, lb = 0.f;
        const int w8 = p.hd / 8;
        // rows of this warp's pieces: k0 + 16 (warp + 4 i); a row on a bad page is
        // marked and its bytes are zero
        unsigned long long bad = 0;          // 16 bits per buffer
        auto load = [&](int piece, int buf) {
            const int e0 = k0 + piece * 16;
            __half* kb = mine + buf * 2 * 16 * PITCH;
            // lanes 0..15 look their row up, then all lanes copy
            long long row = -1;
            if (lane < 16 && e0 + lane < k1) row = page_row(p, s, e0 + lane);
            const unsigned long long out = __ballot_sync(0xffffffffu, row < 0) & 0xFFFFu;
            bad = (bad & ~(0xFFFFull << (16 * buf))) | out << (16 * buf);
            for (int i0 = 0; i0 < 16 * w8; i0 += 32) {
                const int i = i0 + lane, rr = i / w8, c = i % w8;
                const long long at = __shfl_sync(0xffffffffu, row, rr & 15);
                if (rr >= 16) continue;
                __half *kd = kb + rr * PITCH + c * 8, *vd = kd + 16 * PITCH;
                if (at >= 0) {
                    const long long src = (at * p.n_kv + g) * p.hd + c * 8;
                    cp_async16(kd, p.k + src);
                    cp_async16(vd, p.v + src);
                } else {
                    *reinterpret_cast<uint4*>(kd) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(vd) = make_uint4(0, 0, 0, 0);
                }
            }
            cp_async_commit();
        };
        const int pieces = (k1 - k0 + 15) / 16;
        int next = warp;
#pragma unroll
        for (int b = 0; b < kSuffixBufs - 1; b++) {
            if (next < pieces) load(next, b);
            else cp_async_commit();
            next += kSuffixWarps;
        }
        int buf = 0;
        for (int piece = warp; piece < pieces; piece += kSuffixWarps) {
            // the buffer read last turn takes the piece two turns ahead
            int nb = buf + kSuffixBufs - 1;
            if (nb >= kSuffixBufs) nb -= kSuffixBufs;
            __syncwarp();
            if (next < pieces) load(next, nb);
            else cp_async_commit();
            next += kSuffixWarps;
            asm volatile("cp.async.wait_group %0;" ::"n"(kSuffixBufs - 1) : "memory");
            __syncwarp();
            const __half* kb = mine + buf * 2 * 16 * PITCH;
            const uint32_t kbase = smem_addr(kb), vbase = smem_addr(kb + 16 * PITCH);
            float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            const int mi = lane >> 3, ri = lane & 7;
            {
                const uint32_t krow = kbase + (uint32_t)((ri + (mi >= 2 ? 8 : 0)) * PITCH * 2);
#pragma unroll
                for (int ks = 0; ks < HDP / 16; ks++) {
                    uint32_t b0, b1, b2, b3;
                    ldsm_x4(krow + (uint32_t)((ks * 16 + (mi & 1) * 8) * 2), b0, b1, b2, b3);
                    mma16816(sc[0], qhi[ks], b0, b1);
                    mma16816(sc[1], qhi[ks], b2, b3);
                    if (SPLITQ) {
                        mma16816(sc[0], qlo[SPLITQ ? ks : 0], b0, b1);
                        mma16816(sc[1], qlo[SPLITQ ? ks : 0], b2, b3);
                    }
                }
            }
            const int e0 = k0 + piece * 16;
            const uint32_t gone = (uint32_t)(bad >> (16 * buf)) & 0xFFFFu;
            float ma = -INFINITY, mb = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < 2; nt++)
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    const int rr = nt * 8 + 2 * t + k;
                    const bool there = !((gone >> rr) & 1u);
                    sc[nt][k] = there && e0 + rr <= ea ? sc[nt][k] * a.sc : -INFINITY;
                    sc[nt][2 + k] = there && e0 + rr <= eb ? sc[nt][2 + k] * a.sc : -INFINITY;
                    ma = fmaxf(ma, sc[nt][k]);
                    mb = fmaxf(mb, sc[nt][2 + k]);
                }
            ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, 1));
            ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, 2));
            mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
            mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
            // new references; -1e30 in place of -infinity (no key seen yet) keeps the differences numbers
            const float na = fmaxf(Ma, fmaxf(ma, -1e30f) - kHead), nb2 = fmaxf(Mb, fmaxf(mb, -1e30f) - kHead);
            const float ca = exp2_fast(Ma - na), cb = exp2_fast(Mb - nb2);
            Ma = na;
            Mb = nb2;
            float sa = 0.f, sb = 0.f;
#pragma unroll
            for (int nt = 0; nt < 2; nt++)
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    sc[nt][k] = exp2_fast(sc[nt][k] - Ma);
                    sc[nt][2 + k] = exp2_fast(sc[nt][2 + k] - Mb);
                    sa += sc[nt][k];
                    sb += sc[nt][2 + k];
                }
            la = la * ca + sa;               // this thread's columns; the quad's are added at the end
            lb = lb * cb + sb;
#pragma unroll
            for (int i = 0; i < HDP / 8; i++) {
                o[i][0] *= ca;
                o[i][1] *= ca;
                o[i][2] *= cb;
                o[i][3] *= cb;
            }
            uint32_t ph[4], pl[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float x = sc[j >> 1][(j & 1) * 2], y = sc[j >> 1][(j & 1) * 2 + 1];
                ph[j] = pack_hi(x, y);
                if (SPLITP) pl[j] = pack_lo(x, y, ph[j]);
            }
            // a row that some new tokens see and others do not: where its V is not
            // finite, 0 * V would reach those that do not, so it is added to the
            // others alone and taken out of the product
            if (p.n_new > 1 && e0 + 15 > p.lens[s] - p.n_new + tile * 16 / a.gq) {
                uint32_t odd = 0;
                for (int i = lane; i < 16 * w8; i += 32) {
                    const uint4 v = *reinterpret_cast<const uint4*>(kb + (16 + i / w8) * PITCH + (i % w8) * 8);
                    auto wild = [](uint32_t x) { return (x & 0x7C00u) == 0x7C00u || (x & 0x7C000000u) == 0x7C000000u; };
                    if (wild(v.x) || wild(v.y) || wild(v.z) || wild(v.w)) odd |= 1u << (i / w8);
                }
                odd = __reduce_or_sync(0xffffffffu, odd);
                for (uint32_t left = odd; left; left &= left - 1) {
                    const int kk = __ffs(left) - 1, from = (lane & ~3) | ((kk & 7) >> 1);
                    const float xa = kk < 8 ? (kk & 1 ? sc[0][1] : sc[0][0]) : (kk & 1 ? sc[1][1] : sc[1][0]);
                    const float xb = kk < 8 ? (kk & 1 ? sc[0][3] : sc[0][2]) : (kk & 1 ? sc[1][3] : sc[1][2]);
                    const float pa = __shfl_sync(0xffffffffu, xa, from), pb = __shfl_sync(0xffffffffu, xb, from);
#pragma unroll
                    for (int i = 0; i < HDP / 8; i++) {
                        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(kb + (16 + kk) * PITCH + i * 8 + 2 * t));
                        if (pa != 0.f) { o[i][0] = fmaf(pa, v.x, o[i][0]); o[i][1] = fmaf(pa, v.y, o[i][1]); }
                        if (pb != 0.f) { o[i][2] = fmaf(pb, v.x, o[i][2]); o[i][3] = fmaf(pb, v.y, o[i][3]); }
                    }
                }
                __syncwarp();
                for (int i = lane; odd && i < 16 * w8; i += 32)
                    if ((odd >> (i / w8)) & 1u)
                        *reinterpret_cast<uint4*>(const_cast<__half*>(kb) + (16 + i / w8) * PITCH + (i % w8) * 8) = make_uint4(0, 0, 0, 0);
                __syncwarp();
            }
            const uint32_t vrow = vbase + (uint32_t)((ri + (mi & 1) * 8) * PITCH * 2);
#pragma unroll
            for (int i = 0; i < HDP / 8; i += 2) {
                uint32_t b0, b1, b2, b3;
                ldsm_x4_t(vrow + (uint32_t)(((i + (mi >> 1)) * 8) * 2), b0, b1, b2, b3);
                mma16816(o[i], ph, b0, b1);
                mma16816(o[i + 1], ph, b2, b3);
                if (SPLITP) {
                    mma16816(o[i], pl, b0, b1);
                    mma16816(o[i + 1], pl, b2, b3);
                }
            }
            buf = buf + 1 == kSuffixBufs ? 0 : buf + 1;
        }
        la += __shfl_xor_sync(0xffffffffu, la, 1);
        la += __shfl_xor_sync(0xffffffffu, la, 2);
        lb += __shfl_xor_sync(0xffffffffu, lb, 1);
        lb += __shfl_xor_sync(0xffffffffu, lb, 2);
        cp_async_wait_all();
        __syncthreads();                     // every warp is done with its rows: their memory takes the parts
        float* po = reinterpret_cast<float*>(smraw);                  // [warps][16][HDP]
        float2* pm = reinterpret_cast<float2*>(po + kSuffixWarps * 16 * HDP);   // [warps][16]
        if (t == 0) {
            pm[warp * 16 + r] = make_float2(Ma, la);
            pm[warp * 16 + r + 8] = make_float2(Mb, lb);
        }
#pragma unroll
        for (int i = 0; i < HDP / 8; i++) {
            *reinterpret_cast<float2*>(po + (warp * 16 + r) * HDP + i * 8 + 2 * t) = make_float2(o[i][0], o[i][1]);
            *reinterpret_cast<float2*>(po + (warp * 16 + r + 8) * HDP + i * 8 + 2 * t) = make_float2(o[i][2], o[i][3]);
        }
        __syncthreads();
        const long long part = (((long long)s * p.n_kv + g) * a.suffix_splits + sp) * srows + tile * 16;
        for (int i = threadIdx.x; i < 16 * p.hd; i += 32 * kSuffixWarps) {
            const int rr = i / p.hd, d = i % p.hd;
            if (tile * 16 + rr >= srows) break;
            float M = -INFINITY, L = 0.f, x = 0.f;
#pragma unroll
            for (int w = 0; w < kSuffixWarps; w++) M = fmaxf(M, pm[w * 16 + rr].x);
#pragma unroll
            for (int w = 0; w < kSuffixWarps; w++) {
                const float2 ml = pm[w * 16 + rr];
                const float c = exp2_fast(ml.x - M);          // a warp without a piece: 2^-infinity = 0
                L += c * ml.y;
                x = fmaf(c, po[(w * 16 + rr) * HDP + d], x);
            }
            a.suffix_o[(part + rr) * p.hd + d] = x;
            if (d == 0) a.suffix_ml[part + rr] = make_float2(M, L);
        }
    }
    if (!first) griddep_wait();              // this grid's end is the prefix kernel's too, for the join
}

// --------------------------------------------------------------- join --
// One warp per (row, head): the prefix's parts, then the sequence's.
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ PagesDev p, const __grid_constant__ AttendDev a) {
    griddep_entry();
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int token = (int)(w / a.n_heads), h = (int)(w % a.n_heads);
    if (token >= p.n_seqs * p.n_new) return;
    const int s = token / p.n_new, i = token % p.n_new, g = h / a.gq, hq = h % a.gq;
    if (p.lens[s] - p.n_new + i < 0) return;                   // padding
    const SuffixCut cut = suffix_cut(p, s, a.suffix_splits);
    if (lane == 0 && p.lens[s] > cut.len) flag(p.err, LLM_PAGES_BAD_LEN);
    const int np = a.prefix_splits, n = np + cut.parts, srows = p.n_new * a.gq;
    const long long pre = (long long)g * a.rows + (long long)token * a.gq + hq, pre_step = (long long)p.n_kv * a.rows;
    const long long suf = ((long long)s * p.n_kv + g) * a.suffix_splits * srows + i * a.gq + hq;
    auto ml_of = [&](int k) { return k < np ? a.prefix_ml[pre + k * pre_step] : a.suffix_ml[suf + (long long)(k - np) * srows]; };
    float M = -INFINITY;
    for (int k = lane; k < n; k += 32) M = fmaxf(M, ml_of(k).x);
    M = warp_max(M);
    const int d = 4 * lane;
    float L = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < n; k0 += 32) {
        float wk = 0.f;
        if (k0 + lane < n) {
            const float2 ml = ml_of(k0 + lane);
            wk = exp2_fast(ml.x - M);
            L += wk * ml.y;
        }
#pragma unroll 4
        for (int k = 0; k < min(32, n - k0); k++) {
            const float c = __shfl_sync(0xffffffffu, wk, k);
            if (d < p.hd) {
                const int kk = k0 + k;
                const float4 v = *reinterpret_cast<const float4*>((kk < np ? a.prefix_o + (pre + kk * pre_step) * p.hd
                                                                           : a.suffix_o + (suf + (long long)(kk - np) * srows) * p.hd) + d);
                x.x = fmaf(c, v.x, x.x);
                x.y = fmaf(c, v.y, x.y);
                x.z = fmaf(c, v.z, x.z);
                x.w = fmaf(c, v.w, x.w);
            }
        }
    }
    L = warp_sum(L);
    const float inv = L == 0.f ? 0.f : 1.f / L;                // a row without any key is zero
    if (d >= p.hd) return;
    const long long at = (long long)token * a.out_stride + (long long)h * p.hd + d;
    if (a.out_f16)
        *reinterpret_cast<uint2*>(static_cast<__half*>(a.out) + at) = make_uint2(pack_hi(x.x * inv, x.y * inv), pack_hi(x.z * inv, x.w * inv));
    else
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
}

// --------------------------------------------------------------- host --
struct Plan {
    int prefix_splits, suffix_splits, mtiles;
    long long prefix_rows, suffix_rows;      // parts of one row each
    size_t off_pml, off_so, off_sml, bytes;
};

Plan make_plan(const llm_pages* p, const llm_attend* a, int sms) {
    Plan pl{};
    const int gq = a->n_heads / p->n_kv_heads;
    const long long srows = (long long)p->n_new * gq, rows = srows * p->n_seqs;
    pl.mtiles = (int)((rows + 127) / 128);
    const int slots = prefix_ctas(p->head_dim) * sms;
    if (p->prefix_len > 0) {
        const long long ntiles = (p->prefix_len + kKT - 1) / kKT, base = (long long)pl.mtiles * p->n_kv_heads;
        const long long want = std::max<long long>(1, slots / base);
        pl.prefix_splits = (int)std::max<long long>(1, std::min<long long>(want, ntiles / 2));
    }
    if (p->max_pages > 0) {
        const long long units = (long long)p->n_seqs * p->n_kv_heads * ((srows + 15) / 16);
        const long long tiles = ((long long)p->max_pages * p->page_size + 63) / 64;
        pl.suffix_splits = (int)std::max<long long>(1, std::min<long long>({32, 4 * sms / std::max(1ll, units), tiles}));
    }
    pl.prefix_rows = (long long)pl.prefix_splits * p->n_kv_heads * rows;
    pl.suffix_rows = (long long)p->n_seqs * p->n_kv_heads * pl.suffix_splits * srows;
    auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
    size_t at = up((size_t)pl.prefix_rows * p->head_dim * 4);
    pl.off_pml = at;
    at += up((size_t)pl.prefix_rows * 8);
    pl.off_so = at;
    at += up((size_t)pl.suffix_rows * p->head_dim * 4);
    pl.off_sml = at;
    at += up((size_t)pl.suffix_rows * 8);
    pl.bytes = at;
    return pl;
}

// K or V rows of the prefix as {hd, n_kv, rows}: columns behind hd and rows
// behind the prefix read as zero.
bool prefix_map(CUtensorMap* m, const uint16_t* base, const llm_pages* p, int64_t stride) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dim[3] = {(cuuint64_t)p->head_dim, (cuuint64_t)p->n_kv_heads, (cuuint64_t)p->prefix_len};
    cuuint64_t step[2] = {(cuuint64_t)p->head_dim * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, 1, kKT}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<uint16_t*>(base), dim, step, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HDP, bool SPLITQ, bool SPLITP>
cudaError_t launch_prefix(cudaStream_t st, const CUtensorMap& mk, const CUtensorMap& mv, const PagesDev& pd,
                          const AttendDev& ad, int mtiles) {
    using G = PrefixPlan<HDP, SPLITQ>;
    auto k = prefix_kernel<HDP, SPLITQ, SPLITP>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem);
    if (e != cudaSuccess) return e;
    return launch_dep(k, dim3((unsigned)mtiles * ad.prefix_splits, pd.n_kv), dim3(kPrefixThreads), (size_t)G::kSmem, st, mk, mv, pd, ad);
}

template <int HDP, bool SPLITQ, bool SPLITP>
cudaError_t launch_suffix(cudaStream_t st, const PagesDev& pd, const AttendDev& ad, int first) {
    auto k = suffix_kernel<HDP, SPLITQ, SPLITP>;
    constexpr int rows = kSuffixWarps * kSuffixBufs * 2 * 16 * (HDP + 8) * 2, parts = kSuffixWarps * 16 * (HDP + 2) * 4;
    constexpr int smem = rows > parts ? rows : parts;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const long long rt = (pd.n_new * ad.gq + 15) / 16;
    return launch_dep(k, dim3((unsigned)(ad.suffix_splits * rt * pd.n_seqs), pd.n_kv), dim3(32 * kSuffixWarps), (size_t)smem, st, pd, ad, first);
}

int check_attend(const llm_pages* p, const llm_attend* a) {
    if (!a) return fail_op(LLM_ERR_INVALID_ARG, "the attention arguments are NULL");
    if (a->n_heads < 1 || a->n_heads % p->n_kv_heads)
        return fail_op(LLM_ERR_INVALID_ARG, "n_heads %d is not a multiple of n_kv_heads %d", a->n_heads, p->n_kv_heads);
    if (p->n_kv_heads > 65535) return fail_op(LLM_ERR_UNSUPPORTED, "n_kv_heads %d exceeds 65535", p->n_kv_heads);
    if ((long long)p->n_seqs * p->n_new * a->n_heads > INT_MAX / 64)
        return fail_op(LLM_ERR_UNSUPPORTED, "more than 2^25 rows of all heads");
    if (!type_bytes(a->q_dtype) || !type_bytes(a->out_dtype))
        return fail_op(LLM_ERR_UNSUPPORTED, "q or out is neither LLM_F32 nor LLM_F16");
    if (!(a->scale >= 0.f) || !(a->scale < INFINITY)) return fail_op(LLM_ERR_INVALID_ARG, "scale is not a finite number >= 0");
    return LLM_OK;
}

}  // namespace

}  // namespace llm

using namespace llm;

extern "C" int64_t llm_attend_batch_workspace(const llm_pages* pages, const llm_attend* a) {
    int rc = check_pages(pages, false);
    if (rc || (rc = check_attend(pages, a))) return rc;
    return (int64_t)make_plan(pages, a, sm_count()).bytes;
}

extern "C" int llm_attend_batch(const llm_pages* pages, const llm_attend* a, llm_stream_t stream) {
    int rc = check_pages(pages, true);
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
    const Plan pl = make_plan(pages, a, sm_count());
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
    ad.prefix_splits = pl.prefix_splits;
    ad.suffix_splits = pl.suffix_splits;
    const bool sq = !ad.q_f16, so = !ad.out_f16;
    const int hd = pages->head_dim;
    cudaError_t e = cudaSuccess;
    if (prefix) {
        CUtensorMap mk, mv;
        if (!prefix_map(&mk, a->prefix_k, pages, a->prefix_stride) || !prefix_map(&mv, a->prefix_v, pages, a->prefix_stride))
            return fail_op(LLM_ERR_CUDA, "a tensor map of the prefix");
#define LLM_PREFIX(HDP)                                                                                          \
    (sq ? (so ? launch_prefix<HDP, true, true>(stream, mk, mv, pd, ad, pl.mtiles)                                 \
              : launch_prefix<HDP, true, false>(stream, mk, mv, pd, ad, pl.mtiles))                               \
        : (so ? launch_prefix<HDP, false, true>(stream, mk, mv, pd, ad, pl.mtiles)                                \
              : launch_prefix<HDP, false, false>(stream, mk, mv, pd, ad, pl.mtiles)))
        e = hd <= 64 ? LLM_PREFIX(64) : LLM_PREFIX(128);
#undef LLM_PREFIX
        if (e != cudaSuccess) return launched(e, "llm_attend_batch (prefix)");
    }
    if (pl.suffix_splits > 0) {
        const int first = prefix ? 0 : 1;
#define LLM_SUFFIX(HDP)                                                                                          \
    (sq ? (so ? launch_suffix<HDP, true, true>(stream, pd, ad, first) : launch_suffix<HDP, true, false>(stream, pd, ad, first)) \
        : (so ? launch_suffix<HDP, false, true>(stream, pd, ad, first) : launch_suffix<HDP, false, false>(stream, pd, ad, first)))
        e = hd <= 32 ? LLM_SUFFIX(32) : hd <= 64 ? LLM_SUFFIX(64) : LLM_SUFFIX(128);
#undef LLM_SUFFIX
        if (e != cudaSuccess) return launched(e, "llm_attend_batch (suffix)");
    }
    const long long warps = rows * a->n_heads;
    return launched(launch_dep(join_kernel, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, stream, pd, ad), "llm_attend_batch (join)");
}
