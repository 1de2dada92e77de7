// Page tables of a batch: sequences forked, reordered, cut and extended
// (llm_pages_update), and the pages in use moved to the front of their pool
// (llm_pages_compact).  include/llm.h defines what each computes.
//
// Each is two kernels.  A plan (one cluster of blocks, whose barriers separate its
// phases) works out in the workspace which page goes where; everything it decides by
// atomics is a sum, a minimum or an OR of whole numbers, so the order of its threads
// does not matter.  Then a grid over all SMs copies pages and writes the tables.  The
// plan changes nothing that the caller sees before every check has passed.
#include <limits.h>

#include <algorithm>

#include "batch_ops.cuh"

namespace llm {

namespace {

constexpr int kPlanBlocks = 8, kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
constexpr int kMoveThreads = 256, kMoveVecs = 4;                       // 16-byte words of a thread per item
constexpr int kMoveBytes = kMoveThreads * kMoveVecs * 16;

struct PoolDev {
    int n_seqs, page_shift, n_pages, max_pages, n_layers;
    int *table, *lens, *refs, *err;
    uint8_t *k, *v;
    long long page_bytes, row_bytes, layer_stride;
};

// What the plan of an update leaves for the move.
struct UpdateWork {
    int* header;                             // [2]: whether the update goes on; copies
    int* refs;                               // [n_pages]: holders of whole pages
    int* first;                              // [n_pages]: the first sequence that keeps the page in part
    int* fresh;                              // [n_pages]: pages given out, ascending
    int* copies;                             // [n_seqs]: the sequences whose page is copied
    int4* rows;                              // [n_seqs]: whole pages kept, rows of the page kept in part, that page, all rows
    int4* pages;                             // [n_seqs]: pages held before, parent, whether the page kept in part stays, first of its fresh pages
    int* source;                             // [n_seqs][max_pages]: whole pages of sequences that go on from another
};

struct CompactWork {
    int* header;                             // [2]: pages to be moved
    int *from, *to;                          // [n_pages]
};

// A plan runs as one block (ONE), whose working arrays are in shared memory, or as a cluster
// of kPlanBlocks.
template <bool ONE>
__device__ __forceinline__ int plan_rank() {
    if (ONE) return 0;
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return (int)r;
}
// (of the cluster's global memory too: what a block wrote before it is seen behind it by the others, which read around L1)
template <bool ONE>
__device__ __forceinline__ void plan_barrier() {
    if (ONE) __syncthreads();
    else asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
template <bool ONE>
__device__ __forceinline__ int read(const int* p) { return ONE ? *static_cast<const volatile int*>(p) : __ldcg(p); }
template <bool ONE>
__device__ __forceinline__ void write(int* p, int v) {
    if (ONE) *static_cast<volatile int*>(p) = v;
    else __stcg(p, v);
}
// A shared-memory word of block `rank`.
template <bool ONE>
__device__ __forceinline__ int plan_peer(const int* p, uint32_t rank) {
    if (ONE) return *static_cast<const volatile int*>(p);
    uint32_t a;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
template <bool ONE>
__device__ __forceinline__ long long plan_peer(const long long* p, uint32_t rank) {
    if (ONE) return *static_cast<const volatile long long*>(p);
    uint32_t a;
    long long v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}
// ORs bits into block 0's word.
template <bool ONE>
__device__ __forceinline__ void plan_or(int* p, int bits) {
    if (ONE) {
        atomicOr(p, bits);
        return;
    }
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_addr(p)));
    asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(a), "r"(bits) : "memory");
}

// Sum of `x` over the block's threads before this one; the whole sum in *all.  `tmp`: kPlanWarps words.
template <class N>
__device__ __forceinline__ N block_scan(N x, N* tmp, N* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    N s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const N v = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += v;
    }
    __syncthreads();
    if (lane == 31) tmp[warp] = s;
    __syncthreads();
    N t = tmp[lane];                         // (as many warps as lanes)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const N v = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += v;
    }
    *all = __shfl_sync(0xffffffffu, t, 31);
    const N before = __shfl_sync(0xffffffffu, t, max(warp - 1, 0));
    return (warp > 0 ? before : 0) + s - x;
}
static_assert(kPlanWarps == 32, "a warp adds up the warps' sums");

// The run of `n` things that block `rank` handles: whole warps' words of 32.
__device__ __forceinline__ void share_of(int n, int rank, int blocks, int* lo, int* hi) {
    const long long w = (n + 31ll) / 32;
    *lo = (int)min((long long)n, w * rank / blocks * 32);
    *hi = (int)min((long long)n, w * (rank + 1) / blocks * 32);
}

__device__ __forceinline__ int pages_of(long long rows, int shift) { return (int)((rows + (1ll << shift) - 1) >> shift); }

// ------------------------------------------------------------- update --
// Phases: 0 copies of the counts, and what each sequence keeps (a thread each); 1 the pages that
// it gives up and takes (a warp each); 2 which pages stay, how many are wanted and free; 3
// the free ones in order, the counts.
template <bool ONE>
__global__ void __launch_bounds__(kPlanThreads, 1)
    update_plan_kernel(const __grid_constant__ PoolDev p, const __grid_constant__ UpdateWork w, const int* __restrict__ parents,
                       const int* __restrict__ rows) {
    constexpr int BLOCKS = ONE ? 1 : kPlanBlocks;
    extern __shared__ int arrays[];          // ONE: refs, first
    __shared__ int tmp[kPlanWarps], bad[2], copied, unheld;
    __shared__ long long tmp_wide[kPlanWarps], wanted;           // (the pages that all sequences want may pass 32 bits)
    __shared__ int4 todo[kPlanThreads];      // of the block's sequences: whole pages, pages held, parent (-2: nothing to do)
    const int rank = plan_rank<ONE>(), lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gtid = rank * kPlanThreads + (int)threadIdx.x;
    const int shift = p.page_shift, ps = 1 << shift;
    int *refs = ONE ? arrays : w.refs, *first = ONE ? arrays + p.n_pages : w.first;
    if (threadIdx.x == 0) bad[0] = bad[1] = 0;
    griddep_entry();
    // the block's sequences: a thread has at most one (n_seqs <= BLOCKS * kPlanThreads)
    const int each = (p.n_seqs + BLOCKS - 1) / BLOCKS, s0 = rank * each, s = s0 + (int)threadIdx.x;
    const int mine_n = min(each, p.n_seqs - s0);
    const bool one = (int)threadIdx.x < mine_n;
    int parent = -1, was = 0, had = 0, now = 0, part = -1, wrong = 0;
    if (one) {
        parent = parents ? parents[s] : s;
        was = p.lens[s];
        now = rows ? rows[s] : 0;
        if (parent < -1 || parent >= p.n_seqs) wrong = LLM_PAGES_BAD_SEQ;
        had = wrong || parent < 0 ? 0 : p.lens[parent];
        if (!rows) now = had;
        const long long room = (long long)p.max_pages << shift;
        if (was < 0 || was > room || had < 0 || had > room || now < 0 || now > room) wrong |= LLM_PAGES_BAD_LEN;
    }
    const int keep = wrong ? 0 : min(had, now), full = keep >> shift, tail = keep & (ps - 1), held = wrong ? 0 : pages_of(was, shift);
    if (one) {
        todo[threadIdx.x] = make_int4(full, held, wrong ? -2 : parent, 0);
        if (tail > 0) part = p.table[(long long)parent * p.max_pages + full];
    }
    // (unsigned: the step behind the last of up to 2^31 - 65 pages passes 2^31)
    for (uint32_t j = gtid; j < (uint32_t)p.n_pages; j += BLOCKS * kPlanThreads) {
        write<ONE>(refs + j, p.refs[j]);
        write<ONE>(first + j, INT_MAX);
    }
    plan_barrier<ONE>();                     // (bad[] is zero, too)

    if (tail > 0) {
        if (part < 0 || part >= p.n_pages) wrong |= LLM_PAGES_BAD_PAGE;
        else atomicMin(first + part, s);
    }
    for (int i0 = warp; i0 < mine_n; i0 += kPlanWarps) {
        const int4 q = todo[i0];
        if (q.z == -2) continue;
        const int* mine = p.table + (long long)(s0 + i0) * p.max_pages;
        // (a sequence that goes on from itself keeps its whole pages: only the others change hands)
        // (entries are unsigned in every loop: with pages of one row a sequence has up to 2^31 - 2, and the step behind
        // them passes 2^31)
        for (uint32_t i = (uint32_t)(q.z == s0 + i0 ? q.x : 0) + lane; i < (uint32_t)q.y; i += 32) {
            const int j = mine[i];
            if (j < 0 || j >= p.n_pages) wrong |= LLM_PAGES_BAD_PAGE;
            else atomicSub(refs + j, 1);
        }
        if (q.z == s0 + i0) continue;
        const int* theirs = p.table + (long long)max(q.z, 0) * p.max_pages;
        for (uint32_t i = lane; i < (uint32_t)q.x; i += 32) {
            const int j = theirs[i];
            w.source[(long long)(s0 + i0) * p.max_pages + i] = j;
            if (j < 0 || j >= p.n_pages) wrong |= LLM_PAGES_BAD_PAGE;
            else atomicAdd(refs + j, 1);
        }
    }
    if (wrong) plan_or<ONE>(&bad[0], wrong);
    plan_barrier<ONE>();

    wrong = plan_peer<ONE>(&bad[0], 0);
    if (wrong) {                             // every block alike: nothing has been changed
        if (gtid == 0) {
            flag(p.err, wrong);
            w.header[0] = 0;
        }
        plan_barrier<ONE>();                 // (a block's shared memory stays until it has been read)
        return;
    }
    int need = 0, copy = 0, stays = 0;
    if (one) {
        // a page kept in part stays where no one holds it whole, with the first sequence that keeps it
        stays = tail > 0 && read<ONE>(refs + part) == 0 && read<ONE>(first + part) == s;
        copy = tail > 0 && !stays;
        need = pages_of(now, shift) - full - stays;
        // (a sequence that wants more pages than there are is refused without the sum below)
        if (need > p.n_pages) plan_or<ONE>(&bad[1], LLM_PAGES_FULL);
    }
    // both sums in one: copies in the lower bits (a thread has at most one)
    long long both;
    const long long both_before = block_scan((long long)need << 12 | copy, tmp_wide, &both);
    const long long all_need = both >> 12, need_before = both_before >> 12;
    const int all_copy = (int)(both & 4095), copy_before = (int)(both_before & 4095);
    // pages, in runs of 32: free ones are held by no sequence, in whole or in part
    int lo, hi;
    share_of(p.n_pages, rank, BLOCKS, &lo, &hi);
    const int words = (hi - lo + 31) / 32, w0 = (int)((long long)words * warp / kPlanWarps), w1 = (int)((long long)words * (warp + 1) / kPlanWarps);
    int mine = 0, below = 0;
    for (int k = w0; k < w1; k++) {
        const int j = lo + 32 * k + lane;
        bool none = false;
        if (j < hi) {
            const int held = read<ONE>(refs + j);
            below |= held < 0;
            none = held == 0 && read<ONE>(first + j) == INT_MAX;
        }
        mine += __popc(__ballot_sync(0xffffffffu, none));
    }
    if (below) plan_or<ONE>(&bad[1], LLM_PAGES_BAD_PAGE);        // fewer counted holders than there are
    int all_free;
    const int free_before = __shfl_sync(0xffffffffu, block_scan(lane == 0 ? mine : 0, tmp, &all_free), 0);
    if (threadIdx.x == 0) {
        wanted = all_need;
        copied = all_copy;
        unheld = all_free;
    }
    plan_barrier<ONE>();

    long long need0 = 0, needs = 0;
    int copy0 = 0, at = free_before, copies = 0, frees = 0;
    for (int b = 0; b < BLOCKS; b++) {
        const long long n = plan_peer<ONE>(&wanted, b);
        const int c = plan_peer<ONE>(&copied, b), f = plan_peer<ONE>(&unheld, b);
        if (b < rank) {
            need0 += n;
            copy0 += c;
            at += f;
        }
        needs += n;
        copies += c;
        frees += f;
    }
    const int stop = plan_peer<ONE>(&bad[1], 0) | (needs > frees ? LLM_PAGES_FULL : 0);
    if (!ONE) plan_barrier<ONE>();           // (the same)
    if (gtid == 0) {
        if (stop) flag(p.err, stop);
        w.header[0] = stop == 0;
        w.header[1] = copies;
    }
    if (stop) return;
    if (one) {
        w.rows[s] = make_int4(full, tail, part, now);
        w.pages[s] = make_int4(held, parent, stays, (int)(need0 + need_before));
        if (copy) w.copies[copy0 + copy_before] = s;
    }
    for (int k = w0; k < w1; k++) {
        const int j = lo + 32 * k + lane;
        int held = 0;
        bool part = false;
        if (j < hi) {
            held = read<ONE>(refs + j);
            part = read<ONE>(first + j) != INT_MAX;
        }
        const bool none = j < hi && held == 0 && !part;
        const uint32_t who = __ballot_sync(0xffffffffu, none);
        const int nth = at + __popc(who & ((1u << lane) - 1));
        const bool given = none && nth < needs;
        if (given) w.fresh[nth] = j;
        if (j < hi) p.refs[j] = held > 0 ? held : part || given ? 1 : 0;
        at += __popc(who);
    }
}

// One item of a move: kMoveBytes of a page's first `bytes` (a multiple of 16).
__device__ __forceinline__ void copy_part(uint8_t* dst, const uint8_t* src, long long bytes, int part) {
    const long long at = (long long)part * kMoveBytes + (long long)threadIdx.x * 16;
    uint4 x[kMoveVecs];
#pragma unroll
    for (int k = 0; k < kMoveVecs; k++)
        if (at + k * kMoveThreads * 16 < bytes) x[k] = __ldcs(reinterpret_cast<const uint4*>(src + at + k * kMoveThreads * 16));
#pragma unroll
    for (int k = 0; k < kMoveVecs; k++)
        if (at + k * kMoveThreads * 16 < bytes) __stcs(reinterpret_cast<uint4*>(dst + at + k * kMoveThreads * 16), x[k]);
}
// The items of `pairs` page pairs: each of every layer's K and V pages in `parts` parts.  page_pair(i, &from, &to)
// returns how many bytes of pair i are copied.
template <class Pair>
__device__ __forceinline__ void move_pages(const PoolDev& p, int pairs, int parts, Pair page_pair) {
    const uint32_t per_pair = (uint32_t)(2 * p.n_layers * parts);
    const long long items = (long long)pairs * per_pair;
    for (long long x = blockIdx.x; x < items; x += gridDim.x) {
        const int i = (int)(items >> 32 ? x / per_pair : (uint32_t)x / per_pair), rest = (int)(x - (long long)i * per_pair);
        const int plane = rest / parts, part = rest - plane * parts;
        int from, to;
        const long long bytes = page_pair(i, &from, &to);
        uint8_t* base = (plane & 1 ? p.v : p.k) + (plane >> 1) * p.layer_stride;
        copy_part(base + to * p.page_bytes, base + from * p.page_bytes, bytes, part);
    }
}

__global__ void __launch_bounds__(kMoveThreads) update_move_kernel(const __grid_constant__ PoolDev p, const __grid_constant__ UpdateWork w, int parts) {
    griddep_entry();
    if (w.header[0] == 0) return;
    const int shift = p.page_shift, lane = threadIdx.x & 31;
    // tables: a warp per sequence
    for (int s = (blockIdx.x * kMoveThreads + threadIdx.x) >> 5; s < p.n_seqs; s += gridDim.x * (kMoveThreads / 32)) {
        const int4 r = w.rows[s], q = w.pages[s];
        const int total = pages_of(r.w, shift), given = r.x + q.z;                 // the first entry with a fresh page
        int* mine = p.table + (long long)s * p.max_pages;
        if (q.y != s)
            for (uint32_t i = lane; i < (uint32_t)r.x; i += 32) mine[i] = w.source[(long long)s * p.max_pages + i];
        for (uint32_t i = (uint32_t)r.x + lane; i < (uint32_t)max(total, q.x); i += 32)
            mine[i] = i < (uint32_t)given ? r.z : i < (uint32_t)total ? w.fresh[(uint32_t)q.w + (i - given)] : -1;
        if (lane == 0) p.lens[s] = r.w;
    }
    if (p.n_layers == 0) return;
    move_pages(p, w.header[1], parts, [&](int i, int* from, int* to) {
        const int s = w.copies[i];
        const int4 r = w.rows[s];
        *from = r.z;
        *to = w.fresh[w.pages[s].w];
        return p.row_bytes > 0 ? r.y * p.row_bytes : p.page_bytes;
    });
}

// ------------------------------------------------------------ compact --
// Phases: 1 how many pages are in use; 2 the pages in use by their rank, and the free
// places before the last of them; 3 the pairs: the pages in use behind the first
// n_live places, ascending, go to the free ones among those, ascending.
template <bool ONE>
__global__ void __launch_bounds__(kPlanThreads, 1)
    compact_plan_kernel(const __grid_constant__ PoolDev p, const __grid_constant__ CompactWork w, int* refs_out, int* moved, int* n_live) {
    constexpr int BLOCKS = ONE ? 1 : kPlanBlocks;
    __shared__ int tmp[kPlanWarps], live_here, free_before_end;
    const int rank = plan_rank<ONE>(), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gtid = rank * kPlanThreads + (int)threadIdx.x;
    griddep_entry();
    int lo, hi;
    share_of(p.n_pages, rank, BLOCKS, &lo, &hi);
    const int words = (hi - lo + 31) / 32, w0 = (int)((long long)words * warp / kPlanWarps), w1 = (int)((long long)words * (warp + 1) / kPlanWarps);
    int mine = 0;
    for (int k = w0; k < w1; k++) {
        const int j = lo + 32 * k + lane;
        mine += __popc(__ballot_sync(0xffffffffu, j < hi && p.refs[j] > 0));
    }
    int all;
    int at = __shfl_sync(0xffffffffu, block_scan(lane == 0 ? mine : 0, tmp, &all), 0);
    if (threadIdx.x == 0) {
        live_here = all;
        free_before_end = 0;
    }
    plan_barrier<ONE>();
    int live = 0;
    for (int b = 0; b < BLOCKS; b++) {
        const int n = plan_peer<ONE>(&live_here, b);
        if (b < rank) at += n;
        live += n;
    }
    // page j: `at` pages in use lie before it
    int holes = 0;
    for (int k = w0; k < w1; k++) {
        const int j = lo + 32 * k + lane;
        const int r = j < hi ? p.refs[j] : 0;
        const uint32_t who = __ballot_sync(0xffffffffu, r > 0);
        const int before = at + __popc(who & ((1u << lane) - 1));
        if (j < hi) {
            if (r > 0) {
                __stcg(w.from + before, j);
                moved[j] = j;                                    // (those that move: below, behind the barrier)
                refs_out[j] = r;
            } else {
                if (j < live) {
                    __stcg(w.to + (j - before), j);
                    holes++;
                }
                moved[j] = -1;
                refs_out[j] = 0;
            }
        }
        at += __popc(who);
    }
    int all_holes;
    block_scan(holes, tmp, &all_holes);
    if (threadIdx.x == 0) free_before_end = all_holes;
    plan_barrier<ONE>();
    int pairs = 0;
    for (int b = 0; b < BLOCKS; b++) pairs += plan_peer<ONE>(&free_before_end, b);
    plan_barrier<ONE>();                          // (a block's shared memory stays until it has been read)
    for (int k = gtid; k < pairs; k += BLOCKS * kPlanThreads) {
        const int from = __ldcg(w.from + live - pairs + k), to = __ldcg(w.to + k), r = __ldcg(refs_out + from);
        moved[from] = to;
        refs_out[to] = r;
        refs_out[from] = 0;
    }
    if (gtid == 0) {
        w.header[0] = live - pairs;
        w.header[1] = pairs;
        *n_live = live;
    }
}

__global__ void __launch_bounds__(kMoveThreads)
    compact_move_kernel(const __grid_constant__ PoolDev p, const __grid_constant__ CompactWork w, const int* moved, int* table_out, int parts) {
    griddep_entry();
    const int lane = threadIdx.x & 31;
    for (int s = (blockIdx.x * kMoveThreads + threadIdx.x) >> 5; s < p.n_seqs; s += gridDim.x * (kMoveThreads / 32)) {
        const int len = p.lens[s];
        const long long room = (long long)p.max_pages << p.page_shift;
        if (lane == 0 && len > room) flag(p.err, LLM_PAGES_BAD_LEN);
        const int held = pages_of(max(0ll, min((long long)len, room)), p.page_shift);
        for (uint32_t i = lane; i < (uint32_t)held; i += 32) {
            const long long x = (long long)s * p.max_pages + i;
            const int j = p.table[x], to = j >= 0 && j < p.n_pages ? moved[j] : -1;
            if (to < 0) flag(p.err, LLM_PAGES_BAD_PAGE);
            table_out[x] = to < 0 ? j : to;
        }
    }
    if (p.n_layers == 0) return;
    const int first = w.header[0];
    move_pages(p, w.header[1], parts, [&](int i, int* from, int* to) {
        *from = w.from[first + i];
        *to = w.to[i];
        return p.page_bytes;
    });
}

// --------------------------------------------------------------- host --
int check_pool(const llm_pool* p, bool pointers) {
    if (!p) return fail_op(LLM_ERR_INVALID_ARG, "pool is NULL");
    if (p->n_seqs < 0 || p->n_pages < 0 || p->max_pages < 0 || p->n_layers < 0)
        return fail_op(LLM_ERR_INVALID_ARG, "a size of the pool is negative");
    if (p->page_size < 1 || (p->page_size & (p->page_size - 1)))
        return fail_op(LLM_ERR_INVALID_ARG, "page_size %d is not a power of two", p->page_size);
    if (p->n_seqs > 4096) return fail_op(LLM_ERR_UNSUPPORTED, "n_seqs %d exceeds 4096", p->n_seqs);
    if ((long long)p->max_pages * p->page_size > INT_MAX - p->page_size)
        return fail_op(LLM_ERR_UNSUPPORTED, "a sequence's capacity exceeds 2^31 - 1 rows less a page");
    if (p->n_pages > INT_MAX - 64 || p->n_layers > 1 << 16) return fail_op(LLM_ERR_UNSUPPORTED, "n_pages or n_layers is too large");
    if (p->n_layers > 0) {
        if (p->page_bytes < 16 || p->page_bytes % 16 || p->page_bytes > 1ll << 32 || p->layer_stride % 16 || p->row_bytes < 0 || p->row_bytes % 16)
            return fail_op(LLM_ERR_INVALID_ARG, "page_bytes, row_bytes or layer_stride is not a multiple of 16, or out of range");
        if (p->row_bytes > p->page_bytes / p->page_size) return fail_op(LLM_ERR_INVALID_ARG, "page_size rows of row_bytes exceed page_bytes");
        if (2ll * p->n_layers * ((p->page_bytes + kMoveBytes - 1) / kMoveBytes) > INT_MAX)
            return fail_op(LLM_ERR_UNSUPPORTED, "a page of all layers is too large");
        if (p->n_layers > 1 && p->layer_stride / p->page_bytes < p->n_pages)
            return fail_op(LLM_ERR_INVALID_ARG, "layer_stride is below the layer's pages");
    }
    if (!pointers) return LLM_OK;
    if ((p->n_seqs > 0 && (!p->lens || (p->max_pages > 0 && !p->page_table))) || (p->n_pages > 0 && !p->refs) ||
        (p->n_layers > 0 && p->n_pages > 0 && (!p->k_pages || !p->v_pages)))
        return fail_op(LLM_ERR_INVALID_ARG, "a pointer of the pool is NULL");
    if (!aligned(p->page_table, 4) || !aligned(p->lens, 4) || !aligned(p->refs, 4) || !aligned(p->err, 4) || !aligned(p->k_pages, 16) ||
        !aligned(p->v_pages, 16))
        return fail_op(LLM_ERR_INVALID_ARG, "a pointer of the pool is not aligned");
    return LLM_OK;
}

PoolDev pool_dev(const llm_pool* p) {
    int shift = 0;
    while ((1 << shift) < p->page_size) shift++;
    return {p->n_seqs, shift, p->n_pages, p->max_pages, p->n_layers, p->page_table, p->lens, p->refs, p->err,
            static_cast<uint8_t*>(p->k_pages), static_cast<uint8_t*>(p->v_pages), p->page_bytes, p->row_bytes, p->layer_stride};
}

// Parts of a page, and the blocks of a move: eight for each SM, where there may be work for them.
int parts_of(const llm_pool* p) { return p->n_layers ? (int)((p->page_bytes + kMoveBytes - 1) / kMoveBytes) : 1; }
int move_blocks(const llm_pool* p, long long most_pairs) {
    const long long items = most_pairs * 2 * p->n_layers * parts_of(p), warps = (p->n_seqs + kMoveThreads / 32 - 1) / (kMoveThreads / 32);
    return (int)std::max(1ll, std::min((long long)8 * sm_count(), std::max(items, warps)));
}

// One block plans for pools whose counts fit its shared memory: a barrier of a cluster takes some 0.5 us more.
constexpr int kOnePages = 16384, kOneSeqs = kPlanThreads;
constexpr long long kOneEntries = 1 << 16;
bool one_block(const llm_pool* p) {
    return p->n_pages <= kOnePages && p->n_seqs <= kOneSeqs && (long long)p->n_seqs * p->max_pages <= kOneEntries;
}

// A plan: one block, or a cluster.
template <class... KArgs, class... Args>
cudaError_t launch_plan(void (*one)(KArgs...), void (*cluster)(KArgs...), bool is_one, size_t smem, cudaStream_t st, Args... args) {
    if (is_one) return launch_dep(one, dim3(1), dim3(kPlanThreads), smem, st, args...);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kPlanBlocks);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = kPlanBlocks;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, cluster, static_cast<KArgs>(args)...);
}

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

size_t update_work(const llm_pool* p, uint8_t* ws, UpdateWork* w) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        uint8_t* q = ws ? ws + at : nullptr;
        at += up256(bytes);
        return q;
    };
    const size_t pages = (size_t)p->n_pages * 4, seqs = (size_t)p->n_seqs;
    w->header = reinterpret_cast<int*>(take(8));
    w->refs = reinterpret_cast<int*>(take(pages));
    w->first = reinterpret_cast<int*>(take(pages));
    w->fresh = reinterpret_cast<int*>(take(pages));
    w->copies = reinterpret_cast<int*>(take(seqs * 4));
    w->rows = reinterpret_cast<int4*>(take(seqs * 16));
    w->pages = reinterpret_cast<int4*>(take(seqs * 16));
    w->source = reinterpret_cast<int*>(take(seqs * p->max_pages * 4));
    return at;
}
size_t compact_work(const llm_pool* p, uint8_t* ws, CompactWork* w) {
    const size_t pages = up256((size_t)p->n_pages * 4);
    w->header = reinterpret_cast<int*>(ws);
    w->from = reinterpret_cast<int*>(ws + 256);
    w->to = reinterpret_cast<int*>(ws + 256 + pages);
    return 256 + 2 * pages;
}

int check_workspace(const void* ws, int64_t bytes, size_t need) {
    if (!ws || !aligned(ws, 256) || bytes < (int64_t)need)
        return fail_op(LLM_ERR_INVALID_ARG, "workspace: NULL, not 256-byte aligned, or below %zu bytes", need);
    return LLM_OK;
}

}  // namespace

}  // namespace llm

using namespace llm;

extern "C" int64_t llm_pages_update_workspace(const llm_pool* pool) {
    const int rc = check_pool(pool, false);
    UpdateWork w;
    return rc ? rc : (int64_t)update_work(pool, nullptr, &w);
}

extern "C" int llm_pages_update(const llm_pool* pool, const int32_t* parents, const int32_t* rows, void* workspace,
                                int64_t workspace_bytes, llm_stream_t stream) {
    int rc = check_pool(pool, true);
    if (rc) return rc;
    if (!aligned(parents, 4) || !aligned(rows, 4)) return fail_op(LLM_ERR_INVALID_ARG, "parents or rows is not aligned");
    UpdateWork w;
    if ((rc = check_workspace(workspace, workspace_bytes, update_work(pool, static_cast<uint8_t*>(workspace), &w)))) return rc;
    if (pool->n_seqs == 0) return LLM_OK;
    const PoolDev d = pool_dev(pool);
    static OncePerDevice once;
    cudaError_t e = once([] { return cudaFuncSetAttribute(update_plan_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kOnePages * 8); });
    if (e == cudaSuccess)
        e = launch_plan(update_plan_kernel<true>, update_plan_kernel<false>, one_block(pool), (size_t)pool->n_pages * 8, stream, d, w, parents, rows);
    if (e == cudaSuccess)
        e = launch_dep(update_move_kernel, dim3((unsigned)move_blocks(pool, pool->n_seqs)), dim3(kMoveThreads), 0, stream, d, w, parts_of(pool));
    return launched(e, "llm_pages_update");
}

extern "C" int64_t llm_pages_compact_workspace(const llm_pool* pool) {
    const int rc = check_pool(pool, false);
    CompactWork w;
    return rc ? rc : (int64_t)compact_work(pool, nullptr, &w);
}

extern "C" int llm_pages_compact(const llm_pool* pool, int32_t* table_out, int32_t* refs_out, int32_t* moved, int32_t* n_live,
                                 void* workspace, int64_t workspace_bytes, llm_stream_t stream) {
    int rc = check_pool(pool, true);
    if (rc) return rc;
    if (!n_live || (pool->n_pages > 0 && (!refs_out || !moved)) || (pool->n_seqs > 0 && pool->max_pages > 0 && !table_out))
        return fail_op(LLM_ERR_INVALID_ARG, "a result's pointer is NULL");
    if (!aligned(table_out, 4) || !aligned(refs_out, 4) || !aligned(moved, 4) || !aligned(n_live, 4))
        return fail_op(LLM_ERR_INVALID_ARG, "a result's pointer is not aligned");
    if (pool->n_pages > 0 && (moved == pool->refs || moved == refs_out)) return fail_op(LLM_ERR_INVALID_ARG, "moved needs memory of its own");
    CompactWork w;
    if ((rc = check_workspace(workspace, workspace_bytes, compact_work(pool, static_cast<uint8_t*>(workspace), &w)))) return rc;
    const PoolDev d = pool_dev(pool);
    cudaError_t e = launch_plan(compact_plan_kernel<true>, compact_plan_kernel<false>, one_block(pool), 0, stream, d, w, refs_out, moved, n_live);
    if (e == cudaSuccess)
        e = launch_dep(compact_move_kernel, dim3((unsigned)move_blocks(pool, pool->n_pages / 2)), dim3(kMoveThreads), 0, stream, d, w,
                       static_cast<const int*>(moved), table_out, parts_of(pool));
    return launched(e, "llm_pages_compact");
}
