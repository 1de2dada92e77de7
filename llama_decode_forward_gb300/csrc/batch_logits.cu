// Penalties, biases and masks on logits (llm_logits_adjust, include/llm.h).
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "batch_ops.cuh"

namespace llm {

namespace {

// One row is a cluster of 1 to 16 blocks with a run of `span` tokens each.  A block keeps
// in shared memory how often each of its tokens was counted, and the last entry of the
// bias list that names it: whole numbers, so the order of the atomics does not matter.
// The row's history is read once by the cluster, each block a share of it, and counted
// where the token lives (distributed shared memory).  Then the logits stream through.
// A span that is too large for shared memory is taken in tiles, each with a pass over the
// history.  Bound by the stream of logits.
constexpr int kAdjThreads = 512, kAdjVals = 4, kAdjSteps = 4;    // values of a lane per 128-token chunk; chunks of a warp per step
constexpr int kAdjChunk = 32 * kAdjVals;
constexpr int kAdjWords = 24 * 1024;                             // words of counts and entries that a block keeps: two blocks per SM

struct AdjustDev {
    int vocab, span, tile;                   // span: a multiple of kAdjChunk; tile: tokens counted at a time
    const void* x;
    long long x_stride;
    void* y;
    long long y_stride;
    const int* history;
    long long history_stride;
    const int* history_lens;
    int max_history, window;
    const float *repetition, *frequency, *presence;
    const int* bias_ids;
    const float* bias;
    int n_bias;
    const uint32_t* masks;
    long long mask_stride;
    int n_masks;
    const int* mask_of;
    int in_place;
    Div by_span;
};

__device__ __forceinline__ uint32_t block_of_cluster() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t blocks_of_cluster() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void whole_cluster() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A shared-memory word of block `rank`.
__device__ __forceinline__ uint32_t word_of(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}

// The four values of a lane, from consecutive addresses (one load) or 32 apart.
__device__ __forceinline__ void load4(const float* p, bool vec, uint32_t in, float (&x)[4]) {
    if (vec) {
        if (in) {
            const float4 v = __ldcs(reinterpret_cast<const float4*>(p));
            x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; k++)
            if ((in >> k) & 1u) x[k] = __ldcs(p + 32 * k);
    }
}
__device__ __forceinline__ void load4(const __half* p, bool vec, uint32_t in, float (&x)[4]) {
    if (vec) {
        if (in) {
            const uint2 w = __ldcs(reinterpret_cast<const uint2*>(p));
            const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
            x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; k++)
            if ((in >> k) & 1u) x[k] = __half2float(__ldcs(p + 32 * k));
    }
}
__device__ __forceinline__ void store4(float* p, bool vec, uint32_t in, const float (&x)[4]) {
    if (vec) {
        if (in) __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
    } else {
#pragma unroll
        for (int k = 0; k < 4; k++)
            if ((in >> k) & 1u) __stcs(p + 32 * k, x[k]);
    }
}
__device__ __forceinline__ void store4(__half* p, bool vec, uint32_t in, const float (&x)[4]) {
    if (vec) {
        if (in)
            __stcs(reinterpret_cast<uint2*>(p), make_uint2(h2_bits(__float2half_rn(x[0]), __float2half_rn(x[1])),
                                                           h2_bits(__float2half_rn(x[2]), __float2half_rn(x[3]))));
    } else {
#pragma unroll
        for (int k = 0; k < 4; k++)
            if ((in >> k) & 1u) __stcs(p + 32 * k, __float2half_rn(x[k]));
    }
}

template <class T, class U>
__global__ void __launch_bounds__(kAdjThreads, 2) adjust_kernel(const __grid_constant__ AdjustDev a) {
    extern __shared__ __align__(16) uint32_t words[];
    griddep_entry();
    const int rank = (int)block_of_cluster(), blocks = (int)blocks_of_cluster();
    const long long r = blockIdx.x / (unsigned)blocks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t* counts = words;                                    // [tile], where there is a history
    uint32_t* entry = a.history ? words + a.tile : words;        // [tile], where there are biases
    const int per_tile = (a.history ? a.tile : 0) + (a.n_bias > 0 ? a.tile : 0);
    const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
    U* y = static_cast<U*>(a.y) + r * a.y_stride;
    // a chunk of 128 tokens: four in a row for each lane where that is one aligned load and store, else 32 apart
    const bool vec = (reinterpret_cast<uintptr_t>(x) & (4 * sizeof(T) - 1)) == 0 && (reinterpret_cast<uintptr_t>(y) & (4 * sizeof(U) - 1)) == 0;
    const int mine = vec ? 4 * lane : lane, apart = vec ? 1 : 32;
    const int first = rank * a.span, end = min(a.vocab, first + a.span);
    int h0 = 0, h1 = 0;
    float rho = 1.f, freq = 0.f, pres = 0.f;
    if (a.history) {
        h1 = max(0, min(a.history_lens[r], a.max_history));
        h0 = a.window > 0 ? max(0, h1 - a.window) : 0;
        if (a.repetition) rho = a.repetition[r];
        if (a.frequency) freq = a.frequency[r];
        if (a.presence) pres = a.presence[r];
    }
    const uint32_t* mask = nullptr;
    if (a.masks) {
        const long long m = a.mask_of ? a.mask_of[r] : r;
        if (m >= 0 && m < a.n_masks) mask = a.masks + m * a.mask_stride;
    }
    // (the tiles of all blocks are passed together: tile t is tokens [t tile, (t + 1) tile) of each span)
    for (int t0 = 0; t0 < a.span; t0 += a.tile) {
        if (per_tile > 0) {
            if (t0 > 0) whole_cluster();                         // the last tile's counts have been used
            for (int i = threadIdx.x * 4; i < per_tile; i += 4 * kAdjThreads) *reinterpret_cast<uint4*>(words + i) = make_uint4(0, 0, 0, 0);
            whole_cluster();
            for (int i = h0 + rank * kAdjThreads + (int)threadIdx.x; i < h1; i += blocks * kAdjThreads) {
                const int id = a.history[r * a.history_stride + i];
                if (id < 0 || id >= a.vocab) continue;
                const int b = a.by_span.of(id), at = id - b * a.span - t0;
                if (at >= 0 && at < a.tile)
                    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], 1;" ::"r"(word_of(counts + at, (uint32_t)b)) : "memory");
            }
            for (int i = rank * kAdjThreads + (int)threadIdx.x; i < a.n_bias; i += blocks * kAdjThreads) {
                const int id = a.bias_ids[r * a.n_bias + i];
                if (id < 0 || id >= a.vocab) continue;
                const int b = a.by_span.of(id), at = id - b * a.span - t0;
                if (at >= 0 && at < a.tile)
                    asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(word_of(entry + at, (uint32_t)b)), "r"(i + 1) : "memory");
            }
            whole_cluster();
        }
        const int tile_end = min(end, first + min(a.span, t0 + a.tile));
        for (int base = first + t0 + warp * (kAdjSteps * kAdjChunk); base < tile_end; base += (kAdjThreads / 32) * kAdjSteps * kAdjChunk) {
            float v[kAdjSteps][4];
            uint32_t in[kAdjSteps], banned[kAdjSteps], c[kAdjSteps][4], e[kAdjSteps][4];
#pragma unroll
            for (int s = 0; s < kAdjSteps; s++) {
                const int at = base + s * kAdjChunk + mine;      // this lane's first token of the chunk
                in[s] = 0;
#pragma unroll
                for (int k = 0; k < 4; k++) in[s] |= at + k * apart < tile_end ? 1u << k : 0u;
                banned[s] = 0;
#pragma unroll
                for (int k = 0; k < 4; k++) c[s][k] = e[s][k] = 0;
                if (mask) {
                    // (a chunk begins at a multiple of 128 tokens: four words of the mask)
                    if (vec) {
                        if (in[s]) banned[s] = ~(__ldg(mask + (at >> 5)) >> (at & 31)) & 15u;
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            if ((in[s] >> k) & 1u) banned[s] |= (~(__ldg(mask + ((at + 32 * k) >> 5)) >> lane) & 1u) << k;
                    }
                }
                const int l = at - first - t0;                   // (within the tile where in[s] says so)
                if (a.history && in[s]) {
                    if (vec) {
                        const uint4 w = *reinterpret_cast<const uint4*>(counts + l);
                        c[s][0] = w.x; c[s][1] = w.y; c[s][2] = w.z; c[s][3] = w.w;
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            if ((in[s] >> k) & 1u) c[s][k] = counts[l + 32 * k];
                    }
                }
                if (a.n_bias > 0 && in[s]) {
                    if (vec) {
                        const uint4 w = *reinterpret_cast<const uint4*>(entry + l);
                        e[s][0] = w.x; e[s][1] = w.y; e[s][2] = w.z; e[s][3] = w.w;
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            if ((in[s] >> k) & 1u) e[s][k] = entry[l + 32 * k];
                    }
                }
                // in place, what stays as it is is neither read nor written
                if (a.in_place && (c[s][0] | c[s][1] | c[s][2] | c[s][3] | e[s][0] | e[s][1] | e[s][2] | e[s][3] | banned[s]) == 0) in[s] = 0;
                const bool whole = in[s] == 15u;                 // (the last tokens of a row one by one)
                v[s][0] = v[s][1] = v[s][2] = v[s][3] = 0.f;
                if (vec && !whole) {
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        if ((in[s] >> k) & 1u) v[s][k] = to_f32(x[at + k]);
                } else {
                    load4(x + at, vec, in[s], v[s]);
                }
            }
#pragma unroll
            for (int s = 0; s < kAdjSteps; s++) {
                const int at = base + s * kAdjChunk + mine;
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    float z = v[s][k];
                    if (c[s][k] > 0) {
                        z = z > 0.f ? __fdiv_rn(z, rho) : __fmul_rn(z, rho);
                        z = __fsub_rn(z, __fadd_rn(__fmul_rn(freq, (float)c[s][k]), pres));
                    }
                    if (e[s][k] > 0) z = __fadd_rn(z, a.bias[r * a.n_bias + (e[s][k] - 1)]);
                    v[s][k] = (banned[s] >> k) & 1u ? -INFINITY : z;
                }
                if (vec && in[s] != 15u) {
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        if ((in[s] >> k) & 1u) {
                            if (sizeof(U) == 4) *reinterpret_cast<float*>(y + at + k) = v[s][k];
                            else *reinterpret_cast<__half*>(y + at + k) = __float2half_rn(v[s][k]);
                        }
                } else {
                    store4(y + at, vec, in[s], v[s]);
                }
            }
        }
    }
}

template <class T, class U>
cudaError_t launch_adjust(const AdjustDev& a, int n_rows, int blocks, size_t smem, cudaStream_t st) {
    static OncePerDevice once;
    const cudaError_t e = once([] {
        const cudaError_t r = cudaFuncSetAttribute(adjust_kernel<T, U>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        return r != cudaSuccess ? r : cudaFuncSetAttribute(adjust_kernel<T, U>, cudaFuncAttributeMaxDynamicSharedMemorySize, kAdjWords * 4);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)n_rows * blocks);
    cfg.blockDim = dim3(kAdjThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = blocks;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, adjust_kernel<T, U>, a);
}

}  // namespace

}  // namespace llm

using namespace llm;

extern "C" int llm_logits_adjust(const llm_adjust* a, llm_stream_t stream) {
    if (!a) return fail_op(LLM_ERR_INVALID_ARG, "the arguments are NULL");
    if (a->n_rows < 0 || a->vocab < 1 || a->max_history < 0 || a->window < 0 || a->n_bias < 0 || a->n_masks < 0)
        return fail_op(LLM_ERR_INVALID_ARG, "n_rows, vocab, max_history, window, n_bias or n_masks is out of range");
    if (a->vocab > 1 << 30) return fail_op(LLM_ERR_UNSUPPORTED, "vocab %d exceeds 2^30", a->vocab);
    const int b = type_bytes(a->dtype), ob = type_bytes(a->out_dtype);
    if (!b || !ob) return fail_op(LLM_ERR_UNSUPPORTED, "logits of type %d into type %d", a->dtype, a->out_dtype);
    if (a->n_rows == 0) return LLM_OK;
    if (!a->logits || !a->out || (a->history && !a->history_lens) || (a->n_bias > 0 && (!a->bias_ids || !a->bias)) ||
        (a->n_masks > 0 && !a->masks))
        return fail_op(LLM_ERR_INVALID_ARG, "a pointer is NULL");
    if (!aligned(a->logits, b) || !aligned(a->out, ob) || !aligned(a->history, 4) || !aligned(a->history_lens, 4) ||
        !aligned(a->repetition, 4) || !aligned(a->frequency, 4) || !aligned(a->presence, 4) || !aligned(a->bias_ids, 4) ||
        !aligned(a->bias, 4) || !aligned(a->masks, 4) || !aligned(a->mask_of, 4))
        return fail_op(LLM_ERR_INVALID_ARG, "a pointer is not aligned to its type");
    if (a->n_rows > 1 && (a->stride < a->vocab || a->out_stride < a->vocab))
        return fail_op(LLM_ERR_INVALID_ARG, "a stride of the logits is below vocab %d", a->vocab);
    if (a->history && a->n_rows > 1 && a->history_stride < a->max_history)
        return fail_op(LLM_ERR_INVALID_ARG, "history_stride %lld below max_history %d", (long long)a->history_stride, a->max_history);
    if (a->n_masks > 1 && a->mask_stride < (a->vocab + 31ll) / 32)
        return fail_op(LLM_ERR_INVALID_ARG, "mask_stride %lld below the %d words of a mask", (long long)a->mask_stride, (a->vocab + 31) / 32);
    if (a->out == a->logits && (a->dtype != a->out_dtype || (a->n_rows > 1 && a->stride != a->out_stride)))
        return fail_op(LLM_ERR_INVALID_ARG, "out is logits with another type or stride");
    if (a->n_rows > INT_MAX / 16) return fail_op(LLM_ERR_UNSUPPORTED, "more than 2^27 rows");
    // The smallest cluster whose counts fit and that gives every SM two blocks, as long as each has a step's
    // tokens for its threads; at most 16 blocks (beyond 8 by opt-in).
    const bool counted = a->history && a->max_history > 0;
    const int arrays = (counted ? 1 : 0) + (a->n_bias > 0 ? 1 : 0), sms = sm_count();
    const int most = arrays ? kAdjWords / arrays / kAdjChunk * kAdjChunk : INT_MAX;
    int blocks = 1;
    while (blocks < 16 && ((a->vocab + blocks - 1) / blocks > most ||
                           ((long long)a->n_rows * blocks < 2 * sms && a->vocab > blocks * kAdjThreads * kAdjVals * kAdjSteps)))
        blocks *= 2;
    AdjustDev d{};
    d.vocab = a->vocab;
    d.span = (int)(((a->vocab + (long long)blocks - 1) / blocks + kAdjChunk - 1) / kAdjChunk * kAdjChunk);
    d.tile = std::min(d.span, most);
    d.x = a->logits; d.x_stride = a->stride;
    d.y = a->out; d.y_stride = a->out_stride;
    if (counted) {
        d.history = a->history;
        d.history_stride = a->history_stride;
        d.history_lens = a->history_lens;
        d.max_history = a->max_history;
        d.window = a->window;
        d.repetition = a->repetition;
        d.frequency = a->frequency;
        d.presence = a->presence;
    }
    d.bias_ids = a->bias_ids;
    d.bias = a->bias;
    d.n_bias = a->n_bias;
    if (a->n_masks > 0) d.masks = a->masks;
    d.mask_stride = a->mask_stride;
    d.n_masks = a->n_masks;
    d.mask_of = a->mask_of;
    d.in_place = a->out == a->logits;
    d.by_span = Div((uint32_t)d.span);
    const size_t smem = (size_t)arrays * d.tile * 4;
    const bool h = a->dtype == LLM_F16, oh = a->out_dtype == LLM_F16;
    return launched(h ? (oh ? launch_adjust<__half, __half>(d, a->n_rows, blocks, smem, stream) : launch_adjust<__half, float>(d, a->n_rows, blocks, smem, stream))
                      : (oh ? launch_adjust<float, __half>(d, a->n_rows, blocks, smem, stream) : launch_adjust<float, float>(d, a->n_rows, blocks, smem, stream)),
                    "llm_logits_adjust");
}
