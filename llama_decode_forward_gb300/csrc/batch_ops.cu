// Operators of batched decoding: the paged K/V append with RoPE on the way,
// and log probabilities (declared in include/llm.h, which defines what each
// computes).
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "batch_ops.cuh"

namespace llm {

namespace {

// ------------------------------------------------------------- append --
struct AppendDev {
    int n_heads, half, neox, table_rows;
    int group;                               // elements of an item's two groups
    int q_blocks, row_blocks;                // blocks of a row's q, and of all of it
    Div by_row_blocks, by_head, by_new;      // divisions by row_blocks, a head's items and n_new
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    void* q_out;
    long long q_out_stride;
    const float2* cs;
};

// N (4 or 8) consecutive elements, as F32.
template <int N>
__device__ __forceinline__ void load_n(const float* p, float (&x)[N]) {
#pragma unroll
    for (int k = 0; k < N; k += 4) {
        const float4 v = *reinterpret_cast<const float4*>(p + k);
        x[k] = v.x; x[k + 1] = v.y; x[k + 2] = v.z; x[k + 3] = v.w;
    }
}
template <int N>
__device__ __forceinline__ void load_n(const __half* p, float (&x)[N]) {
    __align__(16) uint32_t w[N / 2];
    if (N == 8) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
    else *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
#pragma unroll
    for (int k = 0; k < N / 2; k++) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
    }
}
template <int N>
__device__ __forceinline__ void store_n(float* p, const float (&x)[N]) {
#pragma unroll
    for (int k = 0; k < N; k += 4) *reinterpret_cast<float4*>(p + k) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
}
template <int N>
__device__ __forceinline__ void store_n(__half* p, const float (&x)[N]) {
    __align__(16) uint32_t w[N / 2];
#pragma unroll
    for (int k = 0; k < N / 2; k++) w[k] = h2_bits(__float2half_rn(x[2 * k]), __float2half_rn(x[2 * k + 1]));
    if (N == 8) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(w);
    else *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(w);
}
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(__half* p, float x) { *p = __float2half_rn(x); }

// One pair (x0, x1) turned by the angle with cosine r.x and sine r.y, each
// product and sum rounded once, as the decode step rotates.
__device__ __forceinline__ void turn(float& x0, float& x1, float2 r) {
    const float a = x0, b = x1;
    x0 = __fsub_rn(__fmul_rn(a, r.x), __fmul_rn(b, r.y));
    x1 = __fadd_rn(__fmul_rn(a, r.y), __fmul_rn(b, r.x));
}

// The two groups of N elements of a head that item i handles: NEOX pairs join
// element j of the first half with element j of the second, so an item takes N of
// each; otherwise, and behind the rotated elements, 2 N in a row.
struct Groups {
    int a, b, j;                             // first elements; first pair, or -1: not rotated
};
template <int N>
__device__ __forceinline__ Groups groups_of(int i, int half, int neox) {
    if (2 * N * i >= 2 * half) return {2 * N * i, 2 * N * i + N, -1};
    return neox ? Groups{N * i, half + N * i, N * i} : Groups{2 * N * i, 2 * N * i + N, N * i};
}

// One thread per item of a head of q, k or v; a row has blocks of its own for q and
// for k and v, so its sequence, place and angles are the block's.  The elements are
// loaded before the row's place is known: the chain length -> page -> store runs
// beside that load.  N: elements of an item's two groups, 8 where head_dim and
// rope_dims are multiples of 16, else 4 where rope_dims is one of 8, else 0: eight
// elements taken pair by pair.  Bound by the stream of rows, and close behind it by
// instructions: 8000 rows of 4 KB (F16) take 20.8 us (4.8 TB/s) with groups of eight,
// 26.4 us with groups of four.
constexpr int kAppendThreads = 128;
constexpr int append_item(int n) { return n ? 2 * n : 8; }
template <class T, class U, int N>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ PagesDev p,
                                                                const __grid_constant__ AppendDev a) {
    griddep_entry();
    const int row = a.by_row_blocks.of(blockIdx.x), block = blockIdx.x - row * a.row_blocks, per_head = p.hd / append_item(N);
    const bool is_q = block < a.q_blocks;
    const int item = (is_q ? block : block - a.q_blocks) * kAppendThreads + (int)threadIdx.x;
    const int h = a.by_head.of(item), i = item - h * per_head;
    if (h >= (is_q ? a.n_heads : 2 * p.n_kv)) return;
    const bool is_v = !is_q && h >= p.n_kv;
    const int g = is_v ? h - p.n_kv : h, half = is_v ? 0 : a.half;
    const T* x = is_q ? static_cast<const T*>(a.q) + row * a.q_stride
                      : is_v ? static_cast<const T*>(a.v) + row * a.v_stride : static_cast<const T*>(a.k) + row * a.k_stride;
    x += g * p.hd;
    constexpr int W = N ? N : 4;
    const Groups f = groups_of<W>(i, half, a.neox);
    float u[W], w[W];
    if (N) {
        load_n<W>(x + f.a, u);
        load_n<W>(x + f.b, w);
    }
    const int s = a.by_new.of(row), len = p.lens[s], behind = p.n_new - (row - s * p.n_new);
    if (len < behind) return;                // padding
    const int e = len - behind;
    const long long pos = (long long)p.prefix_len + e;
    if (pos >= a.table_rows && a.half > 0) {
        flag(p.err, LLM_PAGES_BAD_LEN);
        return;
    }
    U* yq = nullptr;
    __half* yk = nullptr;
    if (is_q) {
        yq = static_cast<U*>(a.q_out) + row * a.q_out_stride + (long long)g * p.hd;
    } else {
        const long long slot = page_row(p, s, e);
        if (slot < 0) return;
        yk = (is_v ? p.v : p.k) + (slot * p.n_kv + g) * p.hd;
    }
    const float2* cs = a.cs + pos * a.half;
    if (N) {
        if (f.j >= 0) {
            float2 r[W];                     // W pairs: two to a 16-byte load (rows of the table are multiples of 32 bytes)
#pragma unroll
            for (int k = 0; k < W; k += 2) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(cs + f.j + k));
                r[k] = make_float2(v.x, v.y);
                r[k + 1] = make_float2(v.z, v.w);
            }
#pragma unroll
            for (int k = 0; k < W; k++) {
                if (a.neox) turn(u[k], w[k], r[k]);
                else if (k < W / 2) turn(u[(2 * k) % W], u[(2 * k) % W + 1], r[k]);
                else turn(w[(2 * k) % W], w[(2 * k) % W + 1], r[k]);
            }
        }
        if (is_q) {
            store_n<W>(yq + f.a, u);
            store_n<W>(yq + f.b, w);
        } else {
            store_n<W>(yk + f.a, u);
            store_n<W>(yk + f.b, w);
        }
    } else {
        for (int k = 0; k < 4; k++) {
            const int j = 4 * i + k;
            const int c = j >= half ? 2 * j : a.neox ? j : 2 * j, d = j >= half ? 2 * j + 1 : a.neox ? j + half : 2 * j + 1;
            float x0 = to_f32(x[c]), x1 = to_f32(x[d]);
            if (j < half) turn(x0, x1, cs[j]);
            if (is_q) {
                store1(yq + c, x0);
                store1(yq + d, x1);
            } else {
                store1(yk + c, x0);
                store1(yk + d, x1);
            }
        }
    }
}

template <class T, class U>
cudaError_t launch_append(cudaStream_t st, const PagesDev& pd, const AppendDev& ad, long long rows) {
    auto k = ad.group == 8 ? append_kernel<T, U, 8> : ad.group == 4 ? append_kernel<T, U, 4> : append_kernel<T, U, 0>;
    return launch_dep(k, dim3((unsigned)(rows * ad.row_blocks)), dim3(kAppendThreads), 0, st, pd, ad);
}

// --------------------------------------------------- log probabilities --
// One pass over a row: every thread keeps the running maximum m of its logits,
// s = sum e^(x - m) and t = sum e^(x - m) (x - m) (from which the entropy is
// ln s - t / s), every warp the keys that may be among the row's `top` largest.
// A row is shared by a cluster of 1 to 16 blocks, so that few rows still occupy
// every SM; the blocks' results meet in the first one's shared memory.  Bound by
// the stream of logits; for one row by the chain of its steps.
//
// A key (argmax_key) orders by value, then by the lower index.  A warp looks at
// its logits one by one only when one of them reaches the floor: a key that at
// least `top` keys of the row are known to reach.  For a warp's first logits that
// is the top-th largest of its lanes' largest; later its own top-th key, or the
// block's, through shared memory.  Keys that reach it wait in shared memory; 32 of
// them are sorted into the warp's list (lane i the i-th) at a time.  After steps 1,
// 4, 16, ... and at the end the keys of a block that reach its floor are ranked by
// counting the larger ones, and the top-th becomes its floor.  512 rows of 151,936
// with eight alternatives: 77 us without those ranks (a warp then meets some 37 keys
// that reach its floor, in every other step), 68 us with them.
constexpr int kLpElems = 16;                 // logits of a lane per step
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kDown = 1.f / 16384.f;       // a power of two: x * kDown is exact

struct LpStat {
    float m, s, t;
};

__device__ __forceinline__ LpStat lp_join(LpStat a, LpStat b) {
    LpStat r;
    r.m = fmaxf(a.m, b.m);
    // a side without any logit above -infinity has s = 0 (or NaN, which stays)
    const float da = a.m - r.m, db = b.m - r.m;
    const float ca = a.s == 0.f ? 0.f : exp2f(da * kLog2e), cb = b.s == 0.f ? 0.f : exp2f(db * kLog2e);
    r.s = (a.s == 0.f ? 0.f : ca * a.s) + (b.s == 0.f ? 0.f : cb * b.s);
    r.t = (ca == 0.f ? 0.f : ca * (a.t + a.s * da)) + (cb == 0.f ? 0.f : cb * (b.t + b.s * db));
    return r;
}
template <int FROM>
__device__ __forceinline__ LpStat lp_join_warp(LpStat st) {
#pragma unroll
    for (int o = FROM; o > 0; o >>= 1)
        st = lp_join(st, LpStat{__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.s, o),
                                __shfl_xor_sync(0xffffffffu, st.t, o)});
    return st;
}

typedef unsigned long long u64;

// Lane i's value of two descending lists' merge, the 32 largest.
template <class K>
__device__ __forceinline__ K merge32(K a, K b, int lane) {
    K k = max(a, __shfl_xor_sync(0xffffffffu, b, 31));         // b reversed: a bitonic sequence of the 32 largest
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const K o = __shfl_xor_sync(0xffffffffu, k, d);
        k = (lane & d) ? min(k, o) : max(k, o);
    }
    return k;
}
// The lanes' values in descending order.
template <class K>
__device__ __forceinline__ K sort32(K k, int lane) {
#pragma unroll
    for (int n = 2; n <= 32; n <<= 1)
#pragma unroll
        for (int d = n >> 1; d > 0; d >>= 1) {
            const K o = __shfl_xor_sync(0xffffffffu, k, d);
            const bool up = (lane & n) != 0;                   // ascending halves build the bitonic sequences
            k = (((lane & d) != 0) == up) ? max(k, o) : min(k, o);
        }
    return k;
}

// The upper half of a value's key, and the value of an upper half (0: below everything).
__device__ __forceinline__ uint32_t order_of(float v) {
    const uint32_t b = __float_as_uint(v);
    return v != v ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return o == 0 ? -INFINITY : __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of a shared-memory word in block `rank` of the cluster.
__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float peer_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ u64 peer_u64(uint32_t a) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}

// How many of the n keys of `list` are larger than key: eight at a time, the list
// (16-byte aligned) with zeros behind its n keys up to a multiple of eight.
__device__ __forceinline__ int rank_of(u64 key, const u64* list, int n) {
    const uint32_t at = smem_addr(list);
    int c = 0;
    for (int i = 0; i < n; i += 8) {
        u64 k[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2)
            asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(k[j]), "=l"(k[j + 1]) : "r"(at + (uint32_t)((i + j) * 8)));
#pragma unroll
        for (int j = 0; j < 8; j++) c += k[j] > key;
    }
    return c;
}

// The `top` largest of list's n keys into best[], in order.  All threads, with the
// list complete but for the zeros behind it.
template <int NT>
__device__ __forceinline__ void put_in_order(u64* list, int n, int top, u64* best) {
    if (threadIdx.x < 8) list[n + threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += NT) {
        const int k = rank_of(list[i], list, n);
        if (k < top) best[k] = list[i];
    }
}

// NT threads a block: 512 for few rows (the shortest chain), 256 for many (512 rows of
// 151,936: 68 us, 74 us with 128 threads and two blocks a row, 77 us with 512 threads).
template <class T, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) logprobs_kernel(const __grid_constant__ llm_logprobs_args a) {
    constexpr int VE = 16 / sizeof(T), NV = kLpElems / VE;     // elements of a 16-byte load, loads of a lane per step
    constexpr int NW = NT / 32;
    const int rank = (int)cluster_rank(), blocks = (int)cluster_size();
    const long long r = blockIdx.x / (unsigned)blocks;
    const T* x = static_cast<const T*>(a.logits) + r * a.stride;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, top = a.top;
    __shared__ LpStat stat[NW];
    __shared__ __align__(16) u64 wait[NW][64 + 8];   // keys that reached the floor and are not in the warp's list yet
    __shared__ __align__(16) u64 list[(NW * 64 > 512 ? NW * 64 : 512) + 8], best[32];   // the block's keys that reach its floor; its largest in order
    __shared__ u64 floor_all;
    __shared__ int count;
    if (threadIdx.x == 0) {
        floor_all = 0;
        count = 0;
    }
    if (threadIdx.x < 32) best[threadIdx.x] = 0;
    __syncthreads();
    griddep_entry();
    // 16-byte words of the row, from the aligned one that holds its first element
    const int lead = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const uint4* words = reinterpret_cast<const uint4*>(x - lead);
    const int n_words = (lead + a.vocab + VE - 1) / VE;
    constexpr int STEP = 32 * NV;            // words of a warp's step; a block's words are whole steps
    const int steps = (n_words + STEP - 1) / STEP;
    const int w0 = (int)((long long)steps * rank / blocks) * STEP, w1 = min(n_words, (int)((long long)steps * (rank + 1) / blocks) * STEP);
    uint4 raw[NV];
    // a step that lies within the row and this block's words is plain loads; in the others, at the
    // ends, each word and its elements are looked at
    auto whole = [&](int b) { return b * VE >= lead && (b + STEP) * VE - lead <= a.vocab && b + STEP <= w1; };
    auto fetch = [&](int b) {
#pragma unroll
        for (int k = 0; k < NV; k++) raw[k] = __ldcs(words + b + k * 32 + lane);
    };
    LpStat st{-INFINITY, 0.f, 0.f};
    // the targets' logits are wanted at the end: the first block asks for them now
    float of_target = 0.f;
    if (rank == 0 && (int)threadIdx.x < a.n_targets) {
        const int id = a.targets[r * a.n_targets + threadIdx.x];
        if (id >= 0 && id < a.vocab) of_target = to_f32(x[id]);
    }
    u64 keys = 0, floor = 0;
    int waiting = 0;
    float floor_v = -INFINITY;
    auto raise = [&](u64 f) {
        floor = max(floor, f);
        floor_v = value_of((uint32_t)(floor >> 32));
    };
    auto sort_in = [&](u64 k) {              // 32 keys into the warp's list
        keys = merge32(keys, sort32(k, lane), lane);
        const u64 last = __shfl_sync(0xffffffffu, keys, top - 1);
        if (last > floor && lane == 0) atomicMax(&floor_all, last);
        raise(last);
    };
    auto take = [&](u64 key, u64 f) {        // a warp's keys that reach f into the block's list
        const uint32_t who = __ballot_sync(0xffffffffu, key != 0 && key >= f);
        int at = 0;
        if (lane == 0 && who) at = atomicAdd(&count, __popc(who));
        at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1));
        if ((who >> lane) & 1u) list[at] = key;
    };
    const int first = w0 + warp * STEP;
    if (first < w1 && whole(first)) fetch(first);
    // (every warp walks as many steps: the last of one may lie behind the block's words)
    for (int b = first, step = 0, next = 0; w0 + step * NW * STEP < w1; b += NW * STEP, step++) {
        if (b < w1) {
            float v[kLpElems];
            const bool inside = whole(b);
            if (inside) {
#pragma unroll
                for (int k = 0; k < NV; k++) {
                    const uint32_t us[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        if (sizeof(T) == 4) {
                            v[k * VE + i] = __uint_as_float(us[i]);
                        } else {
                            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&us[i]));
                            v[k * VE + 2 * i] = f.x;
                            v[k * VE + (VE == 8 ? 2 * i + 1 : 0)] = f.y;
                        }
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < NV; k++)
#pragma unroll
                    for (int i = 0; i < VE; i++) {
                        const int w = b + k * 32 + lane, e = w * VE - lead + i;
                        v[k * VE + i] = w < w1 && e >= 0 && e < a.vocab ? to_f32(x[e]) : -INFINITY;
                    }
            }
            if (b + NW * STEP < w1 && whole(b + NW * STEP)) fetch(b + NW * STEP);
            float bm = max3_nan(v[0], v[1], v[2]);
#pragma unroll
            for (int i = 3; i < kLpElems; i += 2) bm = max3_nan(bm, v[i], i + 1 < kLpElems ? v[i + 1] : v[i]);
            if (bm != bm) {                      // a NaN makes the row's sum one; the largest is the numbers'
                st.s = NAN;
                bm = -INFINITY;
#pragma unroll
                for (int i = 0; i < kLpElems; i++) bm = fmaxf(bm, v[i]);
            }
            if (bm > st.m) {
                // (a maximum that was very low, or none, leaves nothing: there s d may be -infinity, or NaN)
                const float d = st.m - bm, c = exp2f(d * kLog2e);
                st.t = c == 0.f ? 0.f : c * (st.t + st.s * d);
                st.s *= c;
                st.m = bm;
            }
            if (st.m > -INFINITY) {
                // two pairs of sums side by side.  w = (m - x) / 2^14, cut off at 1 by the rounding's
                // saturation: an x of -infinity gives e = 0 and a product of 0 (with a maximum for
                // each x instead 512 rows of 151,936 took 1.3 us more)
                float2 s[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}, t[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                const float md = st.m * kDown;
                const float2 up2 = make_float2(-kLog2e / kDown, -kLog2e / kDown);
#pragma unroll
                for (int i = 0; i < kLpElems; i += 2) {
                    const float2 w = make_float2(__saturatef(fmaf(v[i], -kDown, md)), __saturatef(fmaf(v[i + 1], -kDown, md)));
                    const float2 y = __fmul2_rn(w, up2);
                    float2 e;
                    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(y.x));
                    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(y.y));
                    s[(i >> 1) & 1] = __fadd2_rn(s[(i >> 1) & 1], e);
                    t[(i >> 1) & 1] = __ffma2_rn(e, w, t[(i >> 1) & 1]);
                }
                st.s += (s[0].x + s[0].y) + (s[1].x + s[1].y);
                st.t = fmaf((t[0].x + t[0].y) + (t[1].x + t[1].y), -1.f / kDown, st.t);
            }
            if (top == 0) continue;
            if (step == 0) {
                // (+ 0: a largest of -0 stands for equal +0s too.)  Many alternatives: of the lanes' two
                // largest each, or the last lanes' poor ones would let half of the logits through
                // (a lane without an element of the row has -infinity and counts as none)
                uint32_t near = sort32(inside || bm > -INFINITY ? order_of(bm + 0.f) : 0u, lane);
                if (top > 24) {
                    float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
                    for (int i = 0; i < kLpElems; i++) {
                        const float z = v[i] == v[i] ? v[i] : -INFINITY;       // (fminf(m1, NaN) is m1: it would count twice)
                        m2 = fmaxf(m2, fminf(m1, z));
                        m1 = fmaxf(m1, z);
                    }
                    near = merge32(near, sort32(inside || m2 > -INFINITY ? order_of(m2 + 0.f) : 0u, lane), lane);
                }
                const uint32_t bound = __shfl_sync(0xffffffffu, near, top - 1);
                raise((u64)bound << 32);
                if (bound && lane == 0) atomicMax(&floor_all, floor);
            }
            uint32_t mask = 0;
            if (__any_sync(0xffffffffu, bm >= floor_v)) {
                raise(*static_cast<volatile u64*>(&floor_all));       // (only here: the other warps' floor seldom matters sooner)
#pragma unroll
                for (int i = 0; i < kLpElems; i++) mask |= v[i] >= floor_v ? 1u << i : 0u;
            }
            while (__any_sync(0xffffffffu, mask)) {
                const int i = __ffs(mask) - 1;
                u64 key = 0;
                if (mask) {
                    float z = v[0];
#pragma unroll
                    for (int k = 1; k < kLpElems; k++) z = k == i ? v[k] : z;
                    const int e = (b + (i / VE) * 32 + lane) * VE - lead + i % VE;
                    if (inside || (b + (i / VE) * 32 + lane < w1 && e >= 0 && e < a.vocab))
                        key = argmax_key(z + 0.f, e);              // -0 + 0 = +0: equal values, equal order
                    mask &= mask - 1;
                }
                const bool in = key != 0 && key >= floor;
                const uint32_t who = __ballot_sync(0xffffffffu, in);
                if (in) wait[warp][waiting + __popc(who & ((1u << lane) - 1))] = key;
                waiting += __popc(who);
                __syncwarp();
                if (waiting >= 32) {
                    sort_in(wait[warp][lane]);
                    const u64 rest = wait[warp][32 + lane];
                    __syncwarp();
                    wait[warp][lane] = rest;
                    waiting -= 32;
                    __syncwarp();
                }
            }
        }
        if (step == next && w0 + (step + 1) * NW * STEP < w1) {
            // after steps 1, 4, 16, ... the top-th largest key that the block knows becomes its floor
            next = 4 * next + 3;
            __syncthreads();
            const u64 f = floor_all;
            take(keys, f);
            take(lane < waiting ? wait[warp][lane] : 0ull, f);
            __syncthreads();
            const int n = count;
            if (threadIdx.x < 8) list[n + threadIdx.x] = 0;
            __syncthreads();
            if (threadIdx.x == 0) count = 0;
            for (int i = threadIdx.x; i < n; i += NT)
                if (rank_of(list[i], list, n) == top - 1) floor_all = list[i];
            __syncthreads();
            raise(floor_all);
        }
    }
    // many alternatives: the warp's own top-th key as a floor leaves the block fewer to rank
    if (top > 8 && waiting > 0) {
        const u64 listed = __shfl_sync(0xffffffffu, keys, 0);
        if (listed) {
            sort_in(lane < waiting ? wait[warp][lane] : 0ull);
            waiting = 0;
        } else {
            if (lane < 8) wait[warp][waiting + lane] = 0;
            __syncwarp();
            for (int i = lane; i < waiting; i += 32)
                if (rank_of(wait[warp][i], wait[warp], waiting) == top - 1) atomicMax(&floor_all, wait[warp][i]);
        }
    }
    if (st.m == INFINITY) st.s = NAN;        // (+infinity less itself was cut off too)
    st = lp_join_warp<16>(st);
    if (lane == 0) stat[warp] = st;
    __syncthreads();                         // the floor is the block's now
    if (top > 0) {
        // the keys that reach it, from the lists and the waiting ones; of these the largest in order
        const u64 f = floor_all;
        take(keys, f);
        take(lane < waiting ? wait[warp][lane] : 0ull, f);
        __syncthreads();
        put_in_order<NT>(list, count, top, best);
    }
    if (warp == 0) {
        st = lp_join_warp<16>(lane < NW ? stat[lane] : LpStat{-INFINITY, 0.f, 0.f});
        if (lane == 0) stat[0] = st;
    }
    __syncthreads();
    if (blocks > 1) {
        cluster_barrier();
        if (rank == 0) {
            // the blocks' sums, and of their largest keys those that reach the largest top-th one
            if (warp == 0) {
                st = LpStat{-INFINITY, 0.f, 0.f};
                u64 f = 0;
                if (lane < blocks) {
                    const uint32_t at = peer(&stat[0], lane);
                    st = LpStat{peer_f32(at), peer_f32(at + 4), peer_f32(at + 8)};
                    if (top > 0) f = peer_u64(peer(&best[top - 1], lane));
                }
                st = lp_join_warp<8>(st);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) f = max(f, __shfl_xor_sync(0xffffffffu, f, o));
                if (lane == 0) {
                    floor_all = f;
                    count = 0;
                }
            }
            constexpr int C = 16 * 32 / NT;
            u64 mine[C];                     // key i % 32 of block i / 32
#pragma unroll
            for (int c = 0; c < C; c++) {
                const int i = c * NT + threadIdx.x;
                mine[c] = i / 32 < blocks && i % 32 < top ? peer_u64(peer(&best[i % 32], i / 32)) : 0ull;
            }
            __syncthreads();
            if (threadIdx.x == 0) stat[0] = st;
            if (top > 0) {
                const u64 f = floor_all;
#pragma unroll
                for (int c = 0; c < C; c++)
                    if (mine[c] != 0 && mine[c] >= f) list[atomicAdd(&count, 1)] = mine[c];
                __syncthreads();
                put_in_order<NT>(list, count, top, best);
            }
            __syncthreads();
        }
        cluster_barrier();                                     // a block's shared memory stays until it has been read
        if (rank != 0) return;
    }
    st = stat[0];
    const float ls = logf(st.s);
    auto logp = [&](float z) { return st.s == 0.f || (z == -INFINITY && st.s == st.s) ? -INFINITY : (z - st.m) - ls; };
    if (threadIdx.x == 0 && a.entropy) a.entropy[r] = st.s == 0.f ? 0.f : ls - st.t / st.s;
    for (int k = threadIdx.x; k < a.n_targets; k += NT) {
        const int id = a.targets[r * a.n_targets + k];
        a.logprob[r * a.n_targets + k] = id == -1 ? 0.f : id < 0 || id >= a.vocab ? NAN : logp(k < NT ? of_target : to_f32(x[id]));
    }
    if (threadIdx.x < top) {
        const u64 key = best[threadIdx.x];
        a.top_id[r * top + threadIdx.x] = key ? argmax_key_index(key) : -1;
        a.top_logprob[r * top + threadIdx.x] = key ? logp(value_of((uint32_t)(key >> 32))) : NAN;
    }
}

template <class T, int NT>
cudaError_t launch_logprobs(const llm_logprobs_args& a, int blocks, cudaStream_t st) {
    static OncePerDevice once;
    const cudaError_t e = once([] { return cudaFuncSetAttribute(logprobs_kernel<T, NT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1); });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)a.n_rows * blocks);
    cfg.blockDim = dim3(NT);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = blocks;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, NT>, a);
}

// Few rows (not one for each SM): blocks of 512 threads, enough of them to give
// every SM two, none with less than one step's logits, at most 16 a row (beyond 8
// by opt-in).  More rows: blocks of 256, three or more for each SM.
template <class T>
cudaError_t launch_logprobs(const llm_logprobs_args& a, cudaStream_t st) {
    const int sms = sm_count();
    int blocks = 1;
    if (a.n_rows < sms) {
        while (blocks < 16 && (long long)a.n_rows * blocks < 2 * sms && a.vocab > blocks * 512 * kLpElems) blocks *= 2;
        return launch_logprobs<T, 512>(a, blocks, st);
    }
    while (blocks < 16 && (long long)a.n_rows * blocks < 3 * sms && a.vocab > blocks * 256 * kLpElems) blocks *= 2;
    return launch_logprobs<T, 256>(a, blocks, st);
}

}  // namespace

}  // namespace llm

using namespace llm;

extern "C" int llm_rope_table(float* cos_sin, int32_t pos0, int32_t n_pos, int32_t rope_dims, float rope_base,
                              const float* rope_freqs, llm_stream_t stream) {
    if (!cos_sin || pos0 < 0 || n_pos < 0 || (long long)pos0 + n_pos > INT_MAX || rope_dims < 2 || rope_dims % 2 ||
        !(rope_base > 0.f) || !aligned(cos_sin, 4) || !aligned(rope_freqs, 4))
        return fail_op(LLM_ERR_INVALID_ARG, "llm_rope_table: bad argument");
    // (an angle is a chain of rope_dims / 2 products at most)
    if (rope_dims > 1024) return fail_op(LLM_ERR_UNSUPPORTED, "llm_rope_table: rope_dims %d exceeds 1024", rope_dims);
    if ((long long)n_pos * (rope_dims / 2) > INT_MAX - 256) return fail_op(LLM_ERR_UNSUPPORTED, "llm_rope_table: the table is too large");
    if (n_pos == 0) return LLM_OK;
    return launched(rope_table(stream, cos_sin, n_pos, pos0, rope_dims, rope_theta_scale(rope_base, rope_dims), rope_freqs), "llm_rope_table");
}

extern "C" int llm_kv_append(const llm_pages* pages, const llm_append* a, llm_stream_t stream) {
    int rc = check_pages(pages, true);
    if (rc) return rc;
    if (!a) return fail_op(LLM_ERR_INVALID_ARG, "the append arguments are NULL");
    if (a->n_heads < 0 || a->table_rows < 0) return fail_op(LLM_ERR_INVALID_ARG, "n_heads or table_rows is negative");
    if (a->rope_dims < 0 || a->rope_dims % 2 || a->rope_dims > pages->head_dim)
        return fail_op(LLM_ERR_INVALID_ARG, "rope_dims must be even and in [0, head_dim]");
    if (pages->n_seqs == 0) return LLM_OK;
    const long long rows = (long long)pages->n_seqs * pages->n_new, kv = (long long)pages->n_kv_heads * pages->head_dim,
                    qw = (long long)a->n_heads * pages->head_dim;
    if ((rc = check_rows("k", a->k, a->dtype, a->k_stride, kv, rows)) || (rc = check_rows("v", a->v, a->dtype, a->v_stride, kv, rows)))
        return rc;
    if (a->n_heads > 0 && ((rc = check_rows("q", a->q, a->dtype, a->q_stride, qw, rows)) ||
                           (rc = check_rows("q_out", a->q_out, a->q_out_dtype, a->q_out_stride, qw, rows))))
        return rc;
    if (a->rope_dims > 0 && (!a->cos_sin || !aligned(a->cos_sin, 16)))
        return fail_op(LLM_ERR_INVALID_ARG, "cos_sin is NULL or not 16-byte aligned");
    if (a->n_heads > 0 && a->q == a->q_out && (a->dtype != a->q_out_dtype || a->q_stride != a->q_out_stride))
        return fail_op(LLM_ERR_INVALID_ARG, "q_out is q with another type or stride");
    const PagesDev pd = pages_dev(pages);
    const int half = a->rope_dims / 2, group = pages->head_dim % 16 == 0 && half % 8 == 0 ? 8 : half % 4 == 0 ? 4 : 0;
    const long long per_head = pages->head_dim / append_item(group), q_blocks = (a->n_heads * per_head + kAppendThreads - 1) / kAppendThreads,
                    row_blocks = q_blocks + (2 * pages->n_kv_heads * per_head + kAppendThreads - 1) / kAppendThreads;
    if (qw > INT_MAX || rows * row_blocks > INT_MAX)
        return fail_op(LLM_ERR_UNSUPPORTED, "more than 2^31 blocks of %d threads", kAppendThreads);
    const AppendDev ad{a->n_heads, half, a->rope_neox, a->table_rows, group, (int)q_blocks, (int)row_blocks,
                       Div((uint32_t)row_blocks), Div((uint32_t)per_head), Div((uint32_t)pages->n_new), a->q, a->k, a->v, a->q_stride,
                       a->k_stride, a->v_stride, a->q_out, a->q_out_stride, reinterpret_cast<const float2*>(a->cos_sin)};
    const bool h = a->dtype == LLM_F16, qh = a->n_heads > 0 && a->q_out_dtype == LLM_F16;
    return launched(h ? (qh ? launch_append<__half, __half>(stream, pd, ad, rows) : launch_append<__half, float>(stream, pd, ad, rows))
                      : (qh ? launch_append<float, __half>(stream, pd, ad, rows) : launch_append<float, float>(stream, pd, ad, rows)),
                    "llm_kv_append");
}

extern "C" int llm_logprobs(const llm_logprobs_args* a, llm_stream_t stream) {
    if (!a) return fail_op(LLM_ERR_INVALID_ARG, "the arguments are NULL");
    if (a->n_rows < 0 || a->vocab < 1 || a->n_targets < 0 || a->top < 0 || a->top > a->vocab)
        return fail_op(LLM_ERR_INVALID_ARG, "n_rows, vocab, n_targets or top is out of range");
    if (a->vocab > 1 << 30) return fail_op(LLM_ERR_UNSUPPORTED, "vocab %d exceeds 2^30", a->vocab);
    if (a->top > 32) return fail_op(LLM_ERR_UNSUPPORTED, "top %d exceeds 32", a->top);
    const int b = type_bytes(a->dtype);
    if (!b) return fail_op(LLM_ERR_UNSUPPORTED, "logits of type %d", a->dtype);
    if (a->n_rows == 0) return LLM_OK;
    if (!a->logits || (a->n_targets > 0 && (!a->targets || !a->logprob)) || (a->top > 0 && (!a->top_id || !a->top_logprob)))
        return fail_op(LLM_ERR_INVALID_ARG, "a pointer is NULL");
    if (!aligned(a->logits, b) || !aligned(a->targets, 4) || !aligned(a->logprob, 4) || !aligned(a->entropy, 4) ||
        !aligned(a->top_id, 4) || !aligned(a->top_logprob, 4))
        return fail_op(LLM_ERR_INVALID_ARG, "a pointer is not aligned to its type");
    if (a->n_rows > 1 && a->stride < a->vocab)
        return fail_op(LLM_ERR_INVALID_ARG, "stride %lld below vocab %d", (long long)a->stride, a->vocab);
    if (a->n_rows > INT_MAX / 16) return fail_op(LLM_ERR_UNSUPPORTED, "more than 2^27 rows");
    return launched(a->dtype == LLM_F16 ? launch_logprobs<__half>(*a, stream) : launch_logprobs<float>(*a, stream), "llm_logprobs");
}
