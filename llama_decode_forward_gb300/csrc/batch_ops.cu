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
    int row_blocks;                          // blocks of one row
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    void* q_out;
    long long q_out_stride;
    const float2* cs;
};

// Four consecutive elements, as F32.
__device__ __forceinline__ void load4(const float* p, float (&x)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void load4(const __half* p, float (&x)[4]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__half* p, const float (&x)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(h2_bits(__float2half_rn(x[0]), __float2half_rn(x[1])),
                                              h2_bits(__float2half_rn(x[2]), __float2half_rn(x[3])));
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

// The two groups of four elements of a head that item i (of hd / 8) handles:
// NEOX pairs join element j of the first half with element j of the second, so
// an item takes four of each; otherwise, and behind the rotated elements, eight
// in a row.
struct Fours {
    int a, b, j;                             // first elements; first pair, or -1: not rotated
};
__device__ __forceinline__ Fours fours(int i, int half, int neox) {
    if (8 * i >= 2 * half) return {8 * i, 8 * i + 4, -1};
    return neox ? Fours{4 * i, half + 4 * i, 4 * i} : Fours{8 * i, 8 * i + 4, 4 * i};
}

// One thread per eight elements of a head of q, k or v; a row's blocks are
// whole, so its sequence, place and angles are the block's.  The elements are
// loaded before the row's place is known: the chain length -> page -> store
// runs beside that load.  VEC: rope_dims / 2 is a multiple of four, so items
// are two groups of four; otherwise the pairs are taken one at a time.  Bound
// by the stream of rows.
constexpr int kAppendThreads = 128;
template <class T, class U, bool VEC>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ PagesDev p,
                                                                const __grid_constant__ AppendDev a) {
    griddep_entry();
    const int row = (int)(blockIdx.x / (unsigned)a.row_blocks), per_head = p.hd / 8;
    const int item = (int)(blockIdx.x % (unsigned)a.row_blocks) * kAppendThreads + (int)threadIdx.x;
    const int h = item / per_head, i = item % per_head;
    if (h >= a.n_heads + 2 * p.n_kv) return;
    const bool is_q = h < a.n_heads, is_v = h >= a.n_heads + p.n_kv;
    const int g = is_q ? h : is_v ? h - a.n_heads - p.n_kv : h - a.n_heads, half = is_v ? 0 : a.half;
    const T* x = static_cast<const T*>(is_q ? a.q : is_v ? a.v : a.k) +
                 row * (is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride) + (long long)g * p.hd;
    const Fours f = fours(i, half, a.neox);
    float u[4], w[4];
    if (VEC) {
        load4(x + f.a, u);
        load4(x + f.b, w);
    }
    const int s = row / p.n_new, e = p.lens[s] - p.n_new + row % p.n_new;
    if (e < 0) return;                       // padding
    const long long pos = (long long)p.prefix_len + e;
    if (pos >= a.table_rows) {
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
    if (VEC) {
        if (f.j >= 0) {
            float2 r[4];
#pragma unroll
            for (int k = 0; k < 4; k++) r[k] = __ldg(cs + f.j + k);
            if (a.neox) {
#pragma unroll
                for (int k = 0; k < 4; k++) turn(u[k], w[k], r[k]);
            } else {
                turn(u[0], u[1], r[0]);
                turn(u[2], u[3], r[1]);
                turn(w[0], w[1], r[2]);
                turn(w[2], w[3], r[3]);
            }
        }
        if (is_q) {
            store4(yq + f.a, u);
            store4(yq + f.b, w);
        } else {
            store4(yk + f.a, u);
            store4(yk + f.b, w);
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
    auto k = ad.half % 4 == 0 ? append_kernel<T, U, true> : append_kernel<T, U, false>;
    return launch_dep(k, dim3((unsigned)(rows * ad.row_blocks)), dim3(kAppendThreads), 0, st, pd, ad);
}

// --------------------------------------------------- log probabilities --
// One pass over a row: every thread keeps the running maximum m of its logits,
// s = sum e^(x - m) and t = sum e^(x - m) (x - m) (from which the entropy is
// ln s - t / s), every warp the `top` largest keys it has met (lane i the
// i-th).  A row is shared by a cluster of 1 to 16 blocks, so that few rows
// still occupy every SM; the blocks' results meet in the first one's shared
// memory.  Bound by the stream of logits.
//
// A key (argmax_key) orders by value, then by the lower index.  A warp looks
// at its logits one by one only when one of them reaches the floor: a key that
// at least `top` keys of the row are known to reach (the warp's own last key,
// or another warp's, through shared memory).  In its first block of logits, when
// no list is filled yet, the floor is the top-th of the 32 lanes' best keys.
constexpr int kLpThreads = 512, kLpWarps = kLpThreads / 32, kLpElems = 16;   // elements of a lane per block
constexpr float kLog2e = 1.4426950408889634f;

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

typedef unsigned long long u64;

// Lane i's key of two descending lists' merge, the 32 largest.
__device__ __forceinline__ u64 merge32(u64 a, u64 b, int lane) {
    u64 k = max(a, __shfl_xor_sync(0xffffffffu, b, 31));       // b reversed: a bitonic sequence of the 32 largest
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const u64 o = __shfl_xor_sync(0xffffffffu, k, d);
        k = (lane & d) ? min(k, o) : max(k, o);
    }
    return k;
}
__device__ __forceinline__ u64 sort32(u64 k, int lane) {
#pragma unroll
    for (int n = 2; n <= 32; n <<= 1)
#pragma unroll
        for (int d = n >> 1; d > 0; d >>= 1) {
            const u64 o = __shfl_xor_sync(0xffffffffu, k, d);
            const bool up = (lane & n) != 0;                   // ascending halves build the bitonic sequences
            k = (((lane & d) != 0) == up) ? max(k, o) : min(k, o);
        }
    return k;
}

// The value a key stands for (0: below everything).
__device__ __forceinline__ float key_value(u64 k) {
    const uint32_t o = (uint32_t)(k >> 32);
    return k == 0 ? -INFINITY : __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
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

template <class T>
__global__ void __launch_bounds__(kLpThreads, 2) logprobs_kernel(const __grid_constant__ llm_logprobs_args a) {
    constexpr int VE = 16 / sizeof(T), NV = kLpElems / VE;     // elements of a 16-byte load, loads of a lane per block
    const uint32_t rank = cluster_rank(), blocks = cluster_size();
    const long long r = blockIdx.x / blocks;
    const T* x = static_cast<const T*>(a.logits) + r * a.stride;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, top = a.top;
    __shared__ LpStat stat[kLpWarps];
    __shared__ u64 list[kLpWarps][32];
    __shared__ u64 floor_all;
    if (threadIdx.x == 0) floor_all = 0;
    __syncthreads();
    griddep_entry();
    // 16-byte words of the row, from the aligned one that holds its first element
    const int lead = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const uint4* words = reinterpret_cast<const uint4*>(x - lead);
    const long long n_words = ((long long)lead + a.vocab + VE - 1) / VE;
    const long long w0 = n_words * rank / blocks, w1 = n_words * (rank + 1) / blocks;
    LpStat st{-INFINITY, 0.f, 0.f};
    u64 keys = 0, floor = 0;
    bool first = true;
    for (long long b = w0 + (long long)warp * 32 * NV; b < w1; b += (long long)kLpWarps * 32 * NV) {
        float v[kLpElems];
        bool inside = true;                                    // every element of this lane is one of the row's
#pragma unroll
        for (int k = 0; k < NV; k++) {
            const long long w = b + k * 32 + lane, e = w * VE - lead;
            if (w < w1 && e >= 0 && e + VE <= a.vocab) {
                const uint4 u = __ldcs(words + w);
                const uint32_t us[4] = {u.x, u.y, u.z, u.w};
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
            } else {
                inside = false;
#pragma unroll
                for (int i = 0; i < VE; i++)
                    v[k * VE + i] = w < w1 && e + i >= 0 && e + i < a.vocab ? to_f32(x[e + i]) : -INFINITY;
            }
        }
        float bm = v[0];
#pragma unroll
        for (int i = 1; i < kLpElems; i++) bm = fmaxf(bm, v[i]);
        if (bm > st.m) {
            const float d = st.m - bm, c = exp2f(d * kLog2e);
            st.t = st.s == 0.f ? 0.f : c * (st.t + st.s * d);
            st.s *= c;
            st.m = bm;
        }
        if (st.m > -INFINITY) {
            // four sums side by side; -infinity - m gives e = 0, whose (x - m) is cut off at a number
            float s[4] = {0.f, 0.f, 0.f, 0.f}, t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kLpElems; i++) {
                const float d = v[i] - st.m;
                float e;
                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(d * kLog2e));
                s[i & 3] += e;
                t[i & 3] = fmaf(e, fmaxf(d, -1e4f), t[i & 3]);
            }
            st.s += (s[0] + s[1]) + (s[2] + s[3]);
            st.t += (t[0] + t[1]) + (t[2] + t[3]);
        } else {
#pragma unroll
            for (int i = 0; i < kLpElems; i++)
                if (v[i] != v[i]) st.s = NAN;
        }
        if (top == 0) continue;
        auto key_of = [&](int i) {
            const long long e = (b + (i / VE) * 32 + lane) * VE - lead + i % VE;
            const bool there = inside || (b + (i / VE) * 32 + lane < w1 && e >= 0 && e < a.vocab);
            return there ? argmax_key(v[i] + 0.f, (int)e) : 0ull;          // -0 + 0 = +0: equal values, equal order
        };
        if (first) {
            first = false;
            u64 best = 0;
#pragma unroll
            for (int i = 0; i < kLpElems; i++) best = max(best, key_of(i));
            const u64 bound = __shfl_sync(0xffffffffu, sort32(best, lane), top - 1);
            if (bound) floor = max(floor, bound - 1);
        }
        floor = max(floor, *static_cast<volatile u64*>(&floor_all));
        if (!__any_sync(0xffffffffu, bm >= key_value(floor))) continue;
        const u64 before = floor;
#pragma unroll
        for (int i = 0; i < kLpElems; i++) {
            const u64 key = key_of(i);
            for (uint32_t who = __ballot_sync(0xffffffffu, key > floor); who; who &= who - 1) {
                const u64 c = __shfl_sync(0xffffffffu, key, __ffs(who) - 1);
                if (c <= floor) continue;
                const u64 up = __shfl_up_sync(0xffffffffu, keys, 1);
                const bool above = keys > c, shift = lane > 0 && !(up > c);
                keys = above ? keys : shift ? up : c;
                floor = max(floor, __shfl_sync(0xffffffffu, keys, top - 1));
            }
        }
        if (floor > before && lane == 0) atomicMax(&floor_all, floor);
    }
    // the warps' results, then the cluster's
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        st = lp_join(st, LpStat{__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.s, o),
                                __shfl_xor_sync(0xffffffffu, st.t, o)});
    if (lane >= top) keys = 0;
    if (lane == 0) stat[warp] = st;
    list[warp][lane] = keys;
    __syncthreads();
    for (int n = kLpWarps / 2; n > 0 && top > 0; n >>= 1) {
        if (warp < n) list[warp][lane] = merge32(list[warp][lane], list[warp + n][lane], lane);
        __syncthreads();
    }
    if (warp == 0) {
        st = lane < kLpWarps ? stat[lane] : LpStat{-INFINITY, 0.f, 0.f};
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            st = lp_join(st, LpStat{__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.s, o),
                                    __shfl_xor_sync(0xffffffffu, st.t, o)});
        if (lane == 0) stat[0] = st;
    }
    if (blocks > 1) {
        __syncwarp();
        cluster_barrier();
        if (rank == 0) {
            // warp w takes block w's list, lane w of warp 0 its sums
            u64 k = 0;
            if (warp < blocks) k = peer_u64(peer(&list[0][lane], warp));
            if (warp == 0) {
                st = LpStat{-INFINITY, 0.f, 0.f};
                if (lane < blocks) {
                    const uint32_t at = peer(&stat[0], lane);
                    st = LpStat{peer_f32(at), peer_f32(at + 4), peer_f32(at + 8)};
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1)
                    st = lp_join(st, LpStat{__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.s, o),
                                            __shfl_xor_sync(0xffffffffu, st.t, o)});
            }
            __syncthreads();
            list[warp][lane] = k;
            if (threadIdx.x == 0) stat[0] = st;
            __syncthreads();
            for (int n = kLpWarps / 2; n > 0 && top > 0; n >>= 1) {
                if (warp < n && n <= (int)blocks) list[warp][lane] = merge32(list[warp][lane], list[warp + n][lane], lane);
                __syncthreads();
            }
        }
        cluster_barrier();                                     // a block's shared memory stays until it has been read
        if (rank != 0) return;
    }
    __syncthreads();
    st = stat[0];
    const float ls = logf(st.s);
    auto logp = [&](float z) { return st.s == 0.f || (z == -INFINITY && st.s == st.s) ? -INFINITY : (z - st.m) - ls; };
    if (threadIdx.x == 0 && a.entropy) a.entropy[r] = st.s == 0.f ? 0.f : ls - st.t / st.s;
    for (int k = threadIdx.x; k < a.n_targets; k += kLpThreads) {
        const int id = a.targets[r * a.n_targets + k];
        a.logprob[r * a.n_targets + k] = id == -1 ? 0.f : id < 0 || id >= a.vocab ? NAN : logp(to_f32(x[id]));
    }
    if (threadIdx.x < top) {
        const u64 key = list[0][threadIdx.x];
        a.top_id[r * top + threadIdx.x] = key ? argmax_key_index(key) : -1;
        a.top_logprob[r * top + threadIdx.x] = key ? logp(key_value(key)) : NAN;
    }
}

template <class T>
cudaError_t launch_logprobs(const llm_logprobs_args& a, cudaStream_t st) {
    // blocks of a row: enough to give every SM two, none with less than one
    // block of its lanes' elements, at most 16 (beyond 8 by opt-in)
    const int sms = sm_count();
    int blocks = 1;
    while (blocks < 16 && (long long)a.n_rows * blocks < 2 * sms && a.vocab > blocks * kLpThreads * kLpElems) blocks *= 2;
    const cudaError_t e = cudaFuncSetAttribute(logprobs_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)a.n_rows * blocks);
    cfg.blockDim = dim3(kLpThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = blocks;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, a);
}

}  // namespace

}  // namespace llm

using namespace llm;

extern "C" int llm_rope_table(float* cos_sin, int32_t pos0, int32_t n_pos, int32_t rope_dims, float rope_base,
                              const float* rope_freqs, llm_stream_t stream) {
    if (!cos_sin || pos0 < 0 || n_pos < 0 || (long long)pos0 + n_pos > INT_MAX || rope_dims < 2 || rope_dims % 2 ||
        !(rope_base > 0.f))
        return fail_op(LLM_ERR_INVALID_ARG, "llm_rope_table: bad argument");
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
    if (a->rope_dims > 0 && (!a->cos_sin || !aligned(a->cos_sin, 8)))
        return fail_op(LLM_ERR_INVALID_ARG, "cos_sin is NULL or not 8-byte aligned");
    if (a->n_heads > 0 && a->q == a->q_out && (a->dtype != a->q_out_dtype || a->q_stride != a->q_out_stride))
        return fail_op(LLM_ERR_INVALID_ARG, "q_out is q with another type or stride");
    const PagesDev pd = pages_dev(pages);
    const long long items = (a->n_heads + 2LL * pages->n_kv_heads) * (pages->head_dim / 8), row_blocks = (items + kAppendThreads - 1) / kAppendThreads;
    if (items > INT_MAX / 2 || rows * row_blocks > INT_MAX)
        return fail_op(LLM_ERR_UNSUPPORTED, "more than 2^31 blocks of %d threads", kAppendThreads);
    const AppendDev ad{a->n_heads, a->rope_dims / 2, a->rope_neox, a->table_rows, (int)row_blocks, a->q, a->k, a->v, a->q_stride,
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
