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
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    void* q_out;
    long long q_out_stride;
    const float2* cs;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f32(float& y, float x) { y = x; }
__device__ __forceinline__ void from_f32(__half& y, float x) { y = __float2half_rn(x); }

template <class T, class U>
__device__ __forceinline__ void rotate_head(const T* x, U* y, const float2* cs, int half, int neox, int hd, int d0) {
    for (int d = d0; d < hd && d < d0 + 8; d += 2) {
        // elements d, d + 1: one pair (or two dims behind the rotated ones)
        const int j = d / 2;
        if (j < half) {
            const int a = neox ? j : 2 * j, b = neox ? j + half : 2 * j + 1;
            const float2 r = cs[j];
            const float x0 = to_f32(x[a]), x1 = to_f32(x[b]);
            from_f32(y[a], __fsub_rn(__fmul_rn(x0, r.x), __fmul_rn(x1, r.y)));
            from_f32(y[b], __fadd_rn(__fmul_rn(x0, r.y), __fmul_rn(x1, r.x)));
        } else {
            from_f32(y[d], to_f32(x[d]));
            from_f32(y[d + 1], to_f32(x[d + 1]));
        }
    }
}

template <class T, class U>
__global__ void append_kernel(const __grid_constant__ PagesDev p, const __grid_constant__ AppendDev a) {
    griddep_entry();
    const int per_head = p.hd / 8, heads = a.n_heads + 2 * p.n_kv;
    const long long items = (long long)p.n_seqs * p.n_new * heads * per_head;
    for (long long it = blockIdx.x * (long long)blockDim.x + threadIdx.x; it < items;
         it += (long long)gridDim.x * blockDim.x) {
        const int d0 = (int)(it % per_head) * 8;
        const long long rest = it / per_head;
        const int h = (int)(rest % heads);
        const long long row = rest / heads;
        const int s = (int)(row / p.n_new), e = p.lens[s] - p.n_new + (int)(row % p.n_new);
        if (e < 0) continue;
        const long long pos = (long long)p.prefix_len + e;
        if (pos >= a.table_rows) {
            flag(p.err, LLM_PAGES_BAD_LEN);
            continue;
        }
        const float2* cs = a.cs + pos * a.half;
        if (h < a.n_heads) {
            rotate_head(static_cast<const T*>(a.q) + row * a.q_stride + (long long)h * p.hd,
                        static_cast<U*>(a.q_out) + row * a.q_out_stride + (long long)h * p.hd, cs, a.half, a.neox, p.hd, d0);
            continue;
        }
        const long long slot = page_row(p, s, e);
        if (slot < 0) continue;
        const int g = (h - a.n_heads) % p.n_kv;
        const long long at = (slot * p.n_kv + g) * p.hd;
        if (h < a.n_heads + p.n_kv)
            rotate_head(static_cast<const T*>(a.k) + row * a.k_stride + g * p.hd, p.k + at, cs, a.half, a.neox, p.hd, d0);
        else
            rotate_head(static_cast<const T*>(a.v) + row * a.v_stride + g * p.hd, p.v + at, cs, 0, 0, p.hd, d0);
    }
}

// --------------------------------------------------- log probabilities --
// One block per row: the statistics, then one pass per alternative for the
// largest key below the one found before.
template <class T>
__global__ void __launch_bounds__(512) logprobs_kernel(const __grid_constant__ llm_logprobs_args a) {
    griddep_entry();
    const long long r = blockIdx.x;
    const T* x = static_cast<const T*>(a.logits) + r * a.stride;
    __shared__ float red[16][2];
    __shared__ unsigned long long best[16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float m = -INFINITY;
    for (int i = threadIdx.x; i < a.vocab; i += 512) m = fmaxf(m, to_f32(x[i]));
    m = warp_max(m);
    if (lane == 0) red[warp][0] = m;
    __syncthreads();
    for (int w = 0; w < 16; w++) m = fmaxf(m, red[w][0]);
    __syncthreads();
    float s = 0.f, t = 0.f;
    for (int i = threadIdx.x; i < a.vocab; i += 512) {
        const float v = to_f32(x[i]);
        if (v == -INFINITY) continue;
        const float d = v - m, e = expf(d);
        s += e;
        t += e == 0.f ? 0.f : e * d;
    }
    s = warp_sum(s);
    t = warp_sum(t);
    if (lane == 0) {
        red[warp][0] = s;
        red[warp][1] = t;
    }
    __syncthreads();
    s = t = 0.f;
    for (int w = 0; w < 16; w++) {
        s += red[w][0];
        t += red[w][1];
    }
    const float ls = logf(s);
    auto logp = [&](float v) { return s == 0.f ? -INFINITY : v == -INFINITY && s == s ? v : (v - m) - ls; };
    if (threadIdx.x == 0 && a.entropy) a.entropy[r] = s == 0.f ? 0.f : ls - t / s;
    for (int k = threadIdx.x; k < a.n_targets; k += 512) {
        const int id = a.targets[r * a.n_targets + k];
        a.logprob[r * a.n_targets + k] = id == -1 ? 0.f : id < 0 || id >= a.vocab ? NAN : logp(to_f32(x[id]));
    }
    unsigned long long below = ~0ull;
    for (int k = 0; k < a.top; k++) {
        unsigned long long key = 0ull;
        for (int i = threadIdx.x; i < a.vocab; i += 512) {
            const unsigned long long c = argmax_key(to_f32(x[i]) + 0.f, i);   // -0 + 0 = +0: equal values, equal keys
            if (c < below && c > key) key = c;
        }
        for (int o = 16; o > 0; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
        __syncthreads();
        if (lane == 0) best[warp] = key;
        __syncthreads();
        for (int w = 0; w < 16; w++) key = max(key, best[w]);
        below = key;
        if (threadIdx.x == 0) {
            const int id = key ? argmax_key_index(key) : -1;
            a.top_id[r * a.top + k] = id;
            a.top_logprob[r * a.top + k] = id < 0 ? NAN : logp(to_f32(x[id]));
        }
    }
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
    const AppendDev ad{a->n_heads, a->rope_dims / 2, a->rope_neox, a->table_rows, a->q, a->k, a->v, a->q_stride, a->k_stride,
                       a->v_stride, a->q_out, a->q_out_stride, reinterpret_cast<const float2*>(a->cos_sin)};
    const long long items = rows * (a->n_heads + 2LL * pages->n_kv_heads) * (pages->head_dim / 8);
    const dim3 grid((unsigned)std::min<long long>((items + 255) / 256, 1 << 30)), block(256);
    const bool h = a->dtype == LLM_F16, qh = a->n_heads > 0 && a->q_out_dtype == LLM_F16;
    return launched(h ? (qh ? launch_dep(append_kernel<__half, __half>, grid, block, 0, stream, pd, ad)
                            : launch_dep(append_kernel<__half, float>, grid, block, 0, stream, pd, ad))
                      : (qh ? launch_dep(append_kernel<float, __half>, grid, block, 0, stream, pd, ad)
                            : launch_dep(append_kernel<float, float>, grid, block, 0, stream, pd, ad)),
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
    const dim3 grid(a->n_rows), block(512);
    return launched(a->dtype == LLM_F16 ? launch_dep(logprobs_kernel<__half>, grid, block, 0, stream, *a)
                                        : launch_dep(logprobs_kernel<float>, grid, block, 0, stream, *a),
                    "llm_logprobs");
}
