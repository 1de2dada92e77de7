// Penalties, biases and masks on logits (llm_logits_adjust, include/llm.h).
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "batch_ops.cuh"

namespace llm {

namespace {

// A block takes 8192 tokens of a row.  It keeps a word in shared memory for each of them:
// how often it was counted, and above that the last entry of the bias list that names it
// (in words of their own where the two do not fit one).  It reads the row's whole lists and
// keeps what is its own; whoever finds a word zero puts its token on the block's list.
// All are whole numbers, so the order of the atomics does not matter.  The logits stream
// through beside that, copied or banned by the mask; then the listed tokens are made from
// their logits once more.  Bound by the stream of logits, and by instructions where lists are long.
// 256 rows of 151,936, F32: 46 us alone (6.8 TB/s), 66 us with 1024 tokens counted, 50 biases and
// a mask (97 us when each word was looked at within the stream: most warps met a touched token in
// most steps, one lane at a time), 78 us with 8000 tokens counted and 120 us with 30,000 (196 us and 400 us as
// clusters of blocks that share the reading of the lists and count in each other's shared memory).
constexpr int kAdjThreads = 512, kAdjSteps = 4;                  // chunks of 128 tokens (four for each lane) of a warp
constexpr int kAdjChunk = 128, kAdjSpan = kAdjThreads / 32 * kAdjSteps * kAdjChunk;      // tokens of a block
constexpr int kAdjCountBits = 20;                                // of a word that holds a bias entry too

struct AdjustDev {
    int vocab, two;                          // two: bias entries in words of their own
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
    Div by_blocks = Div(1);                  // division by a row's blocks
};

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
        if (in) {
            const __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
            __stcs(reinterpret_cast<uint2*>(p), make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b)));
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; k++)
            if ((in >> k) & 1u) __stcs(p + 32 * k, __float2half_rn(x[k]));
    }
}

__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(__half* p, float x) { *p = __float2half_rn(x); }

// What becomes of a logit whose token's word is not zero.
struct RowParams {
    float rho, freq, pres;
    const float* bias;                       // the row's
};
__device__ __forceinline__ float adjusted(float z, uint32_t count, uint32_t entry, const RowParams& r) {
    if (count > 0) {
        z = z > 0.f ? __fdiv_rn(z, r.rho) : __fmul_rn(z, r.rho);
        z = __fsub_rn(z, __fadd_rn(__fmul_rn(r.freq, (float)count), r.pres));
    }
    return entry > 0 ? __fadd_rn(z, r.bias[entry - 1]) : z;
}

template <class T, class U>
__global__ void __launch_bounds__(kAdjThreads, 3) adjust_kernel(const __grid_constant__ AdjustDev a, int row_blocks) {
    extern __shared__ __align__(16) uint32_t words[];
    griddep_entry();
    const int row = a.by_blocks.of((int)blockIdx.x), first = ((int)blockIdx.x - row * row_blocks) * kAdjSpan;
    const int n_here = min(a.vocab - first, kAdjSpan);           // tokens of this block
    const long long r = row;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool counted = a.history != nullptr, biased = a.n_bias > 0;
    const int n_words = counted || biased ? kAdjSpan << a.two : 0;
    uint32_t* second = words + kAdjSpan;                         // two: the bias entries
    uint32_t* listed = words + n_words;                          // how many tokens are listed; two: those that a bias put there
    uint16_t* list = reinterpret_cast<uint16_t*>(listed + 4);    // [kAdjSpan << two]
    const T* x = static_cast<const T*>(a.x) + r * a.x_stride + first;
    U* y = static_cast<U*>(a.y) + r * a.y_stride + first;
    const uint32_t* mask = nullptr;
    if (a.masks) {
        const long long m = a.mask_of ? a.mask_of[r] : r;
        if (m >= 0 && m < a.n_masks) mask = a.masks + m * a.mask_stride + (first >> 5);
    }
    // a chunk of 128 tokens: four in a row for each lane where that is one aligned load and store, else 32 apart
    const bool vec = (reinterpret_cast<uintptr_t>(x) & (4 * sizeof(T) - 1)) == 0 && (reinterpret_cast<uintptr_t>(y) & (4 * sizeof(U) - 1)) == 0;
    const int apart = vec ? 1 : 32, mine = warp * (kAdjSteps * kAdjChunk) + (vec ? 4 * lane : lane);
    // this lane's tokens of chunk s: bit k says that token at + k * apart is one of the row's
    auto inside = [&](int at) {
        uint32_t in = at + 3 * apart < n_here ? 15u : 0u;
        if (in == 0)
#pragma unroll
            for (int k = 0; k < 3; k++) in |= at + k * apart < n_here ? 1u << k : 0u;
        return in;
    };
    float v[kAdjSteps][4];
    if (!a.in_place)
#pragma unroll
        for (int s = 0; s < kAdjSteps; s++) {
            const int at = mine + s * kAdjChunk;
            const uint32_t in = inside(at);
            if (!vec || in == 15u) {
                load4(x + at, vec, in, v[s]);
            } else {
#pragma unroll
                for (int k = 0; k < 3; k++)
                    if ((in >> k) & 1u) v[s][k] = to_f32(x[at + k]);
            }
        }
    if (n_words > 0) {
        for (int i = threadIdx.x * 4; i < n_words + 4; i += 4 * kAdjThreads) *reinterpret_cast<uint4*>(words + i) = make_uint4(0, 0, 0, 0);
        __syncthreads();
        // take(i, place) for the entries i of a list that name a token of this block, four of them requested at a time
        // (unsigned: a list has up to 2^31 - 1 entries, and the step behind the last one passes that)
        auto walk = [&](const int* ids, uint32_t n, auto take) {
            for (uint32_t i = threadIdx.x; i < n; i += 4 * kAdjThreads) {
                uint32_t at[4];
#pragma unroll
                for (int k = 0; k < 4; k++) at[k] = i + k * kAdjThreads < n ? (uint32_t)ids[i + k * kAdjThreads] - (uint32_t)first : UINT_MAX;
#pragma unroll
                for (int k = 0; k < 4; k++)
                    if (at[k] < (uint32_t)n_here) take(i + k * kAdjThreads, (int)at[k]);
            }
        };
        if (counted) {
            const int h1 = max(0, min(a.history_lens[r], a.max_history)), h0 = a.window > 0 ? max(0, h1 - a.window) : 0;
            walk(a.history + r * a.history_stride + h0, (uint32_t)(h1 - h0), [&](uint32_t, int at) {
                if (atomicAdd(words + at, 1u) == 0) list[atomicAdd(listed, 1u)] = (uint16_t)at;
            });
        }
        // the larger entry takes the place above the count
        const uint32_t low = counted && !a.two ? (1u << kAdjCountBits) - 1 : 0u;
        walk(a.bias_ids + r * a.n_bias, (uint32_t)a.n_bias, [&](uint32_t i, int at) {
            const uint32_t e = (i + 1) << (low ? kAdjCountBits : 0);
            uint32_t old = 0, seen;
            for (;; old = seen) {
                seen = atomicCAS((a.two ? second : words) + at, old, e | (old & low));
                if (seen == old || (seen & ~low) >= e) break;
            }
            if (seen == 0) list[(a.two ? kAdjSpan : 0) + atomicAdd(listed + a.two, 1u)] = (uint16_t)at;
        });
    }
#pragma unroll
    for (int s = 0; s < kAdjSteps; s++) {
        const int at = mine + s * kAdjChunk;
        uint32_t in = inside(at), banned = 0;
        if (mask && in) {
            // (a chunk begins at a multiple of 128 tokens: four words of the mask)
            if (vec) {
                banned = ~(__ldg(mask + (at >> 5)) >> (at & 31)) & in;
            } else {
#pragma unroll
                for (int k = 0; k < 4; k++)
                    if ((in >> k) & 1u) banned |= (~(__ldg(mask + ((at + 32 * k) >> 5)) >> lane) & 1u) << k;
            }
        }
        if (a.in_place) in = banned;         // what stays as it is is neither read nor written
        if (banned)
#pragma unroll
            for (int k = 0; k < 4; k++) v[s][k] = (banned >> k) & 1u ? -INFINITY : v[s][k];
        if (!vec || in == 15u) {
            store4(y + at, vec, in, v[s]);
        } else if (in) {
#pragma unroll
            for (int k = 0; k < 4; k++)
                if ((in >> k) & 1u) store1(y + at + k, v[s][k]);
        }
    }
    if (n_words == 0) return;
    __syncthreads();                         // the lists are complete; what the stream wrote of their tokens goes
    RowParams params{1.f, 0.f, 0.f, a.bias + r * a.n_bias};
    if (a.repetition) params.rho = a.repetition[r];
    if (a.frequency) params.freq = a.frequency[r];
    if (a.presence) params.pres = a.presence[r];
    for (int kind = 0; kind <= a.two; kind++)
        for (int j = threadIdx.x; j < (int)listed[kind]; j += kAdjThreads) {
            const int at = list[kind * kAdjSpan + j];
            const float z = to_f32(x[at]);
            const uint32_t w = words[at];
            if ((kind && w != 0) || (mask && !((__ldg(mask + (at >> 5)) >> (at & 31)) & 1u))) continue;      // (two: it is on the other list too)
            const uint32_t n = !counted ? 0u : biased && !a.two ? w & ((1u << kAdjCountBits) - 1) : w;
            const uint32_t e = !biased ? 0u : a.two ? second[at] : counted ? w >> kAdjCountBits : w;
            store1(y + at, adjusted(z, n, e, params));
        }
}

template <class T, class U>
cudaError_t launch_adjust(const AdjustDev& a, int n_rows, int row_blocks, cudaStream_t st) {
    static OncePerDevice once;
    const cudaError_t e = once([] {
        return cudaFuncSetAttribute(adjust_kernel<T, U>, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * kAdjSpan * 6 + 16);
    });
    if (e != cudaSuccess) return e;
    const size_t smem = a.history || a.n_bias > 0 ? (size_t)(kAdjSpan << a.two) * 6 + 16 : 0;
    return launch_dep(adjust_kernel<T, U>, dim3((unsigned)(n_rows * row_blocks)), dim3(kAdjThreads), smem, st, a, row_blocks);
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
    const bool counted = a->history && a->max_history > 0, biased = a->n_bias > 0;
    const int most = a->window > 0 ? std::min(a->window, a->max_history) : a->max_history;     // tokens counted
    AdjustDev d{};
    d.two = counted && biased && (most >= 1 << kAdjCountBits || a->n_bias >= 1 << (32 - kAdjCountBits));
    const long long blocks = (a->vocab + (long long)kAdjSpan - 1) / kAdjSpan;
    if (a->n_rows * blocks > INT_MAX) return fail_op(LLM_ERR_UNSUPPORTED, "more than 2^31 blocks of %d tokens", kAdjSpan);
    d.vocab = a->vocab;
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
    d.by_blocks = Div((uint32_t)blocks);
    const bool h = a->dtype == LLM_F16, oh = a->out_dtype == LLM_F16;
    return launched(h ? (oh ? launch_adjust<__half, __half>(d, a->n_rows, (int)blocks, stream) : launch_adjust<__half, float>(d, a->n_rows, (int)blocks, stream))
                      : (oh ? launch_adjust<float, __half>(d, a->n_rows, (int)blocks, stream) : launch_adjust<float, float>(d, a->n_rows, (int)blocks, stream)),
                    "llm_logits_adjust");
}
