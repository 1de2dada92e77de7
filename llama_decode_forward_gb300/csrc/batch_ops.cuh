// What the operators of batched decoding share: the paged batch on the device
// and the checks of the arguments.
#pragma once

#include <limits.h>

#include <atomic>

#include "llm_internal.cuh"

namespace llm {

// What the kernels need of an llm_pages.
struct PagesDev {
    int n_seqs, n_new, prefix_len, page_shift, n_pages, max_pages, n_kv, hd;
    __half *k, *v;
    const int* table;
    const int* lens;
    int* err;
};

__device__ __forceinline__ void flag(int* err, int bit) {
    if (err) atomicOr(err, bit);
}

// The page that holds row e >= 0 of sequence s; a bad place is flagged and gives -1.
__device__ __forceinline__ int page_of(const PagesDev& p, int s, int e) {
    const int i = e >> p.page_shift;
    if (i >= p.max_pages) {
        flag(p.err, LLM_PAGES_BAD_LEN);
        return -1;
    }
    const int page = p.table[(long long)s * p.max_pages + i];
    if (page < 0 || page >= p.n_pages) {
        flag(p.err, LLM_PAGES_BAD_PAGE);
        return -1;
    }
    return page;
}
// Its row of the pool's n_pages * page_size rows, or -1.
__device__ __forceinline__ long long page_row(const PagesDev& p, int s, int e) {
    const int page = page_of(p, s, e);
    return page < 0 ? -1 : ((long long)page << p.page_shift) + (e & ((1 << p.page_shift) - 1));
}

// Pages of 4-bit values (include/llm.h): [n_kv][page_size][hd / 2] bytes of numbers, then
// [n_kv][page_size][groups] pairs d, m, in whole words of 16 bytes.
struct Q4Dev {
    int groups;                              // of a head's row
    long long page_bytes, scales;            // bytes of a page, and where its pairs begin
};
constexpr int kQ4Group = 32;

// Byte offsets of a row's numbers and of its pairs: row `in` (of the page) of kv head g.  (page_bytes is below 2^32 and
// a page has at most 2^25 rows of all heads: each product is one instruction.)
__device__ __forceinline__ long long q4_numbers(const PagesDev& p, const Q4Dev& f, int page, int g, int in) {
    return (long long)((unsigned long long)(uint32_t)page * (uint32_t)f.page_bytes + (unsigned long long)(uint32_t)((g << p.page_shift) + in) * (uint32_t)(p.hd / 2));
}
__device__ __forceinline__ long long q4_pairs(const PagesDev& p, const Q4Dev& f, int page, int g, int in) {
    return (long long)((unsigned long long)(uint32_t)page * (uint32_t)f.page_bytes + (unsigned long long)(uint32_t)((g << p.page_shift) + in) * (uint32_t)(4 * f.groups)) + f.scales;
}

// Division of numbers below 2^31 by a fixed one (Granlund and Montgomery, "Division by
// Invariant Integers using Multiplication", 1994): with 2^s >= d and m = floor(2^32
// (2^s - d) / d) + 1, n / d = (floor(m n / 2^32) + n) >> s.
struct Div {
    uint32_t d, m, s;
    explicit Div(uint32_t by = 1) : d(by), s(0) {
        while ((1ull << s) < by) s++;
        m = (uint32_t)(((1ull << 32) * ((1ull << s) - by)) / by + 1);
    }
    __device__ __forceinline__ int of(int n) const { return (int)((__umulhi(m, (uint32_t)n) + (uint32_t)n) >> s); }
};

// max(a, b, c) in one instruction; a NaN counts as no value.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

__device__ __forceinline__ float min3(float a, float b, float c) {
    float y;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// max3, but NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

// ------------------------------------------------------------- checks --
inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int type_bytes(int t) { return t == LLM_F32 ? 4 : t == LLM_F16 ? 2 : 0; }

// The sizes of a batch's pages; the pointers too when they are going to be used.
inline int check_pages(const llm_pages* p, bool pointers) {
    if (!p) return fail_op(LLM_ERR_INVALID_ARG, "pages is NULL");
    if (p->n_seqs < 0 || p->n_new < 1 || p->prefix_len < 0 || p->n_pages < 0 || p->max_pages < 0 || p->n_kv_heads < 1 ||
        p->head_dim < 1)
        return fail_op(LLM_ERR_INVALID_ARG, "a size of the batch is out of range");
    if (p->page_size < 1 || (p->page_size & (p->page_size - 1)))
        return fail_op(LLM_ERR_INVALID_ARG, "page_size %d is not a power of two", p->page_size);
    if (p->head_dim % 8 || p->head_dim > 128)
        return fail_op(LLM_ERR_UNSUPPORTED, "head_dim %d is not a multiple of 8 up to 128", p->head_dim);
    if ((long long)p->n_seqs * p->n_new > INT_MAX || (long long)p->max_pages * p->page_size > INT_MAX ||
        (long long)p->n_kv_heads * p->head_dim > INT_MAX)
        return fail_op(LLM_ERR_UNSUPPORTED, "rows, a sequence's capacity or a cache row exceed 2^31 - 1");
    if (!pointers || p->n_seqs == 0) return LLM_OK;
    if (!p->lens || (p->max_pages > 0 && (!p->page_table || !p->k_pages || !p->v_pages)))
        return fail_op(LLM_ERR_INVALID_ARG, "a pointer of the pages is NULL");
    if (!aligned(p->k_pages, 16) || !aligned(p->v_pages, 16) || !aligned(p->page_table, 4) || !aligned(p->lens, 4) ||
        !aligned(p->err, 4))
        return fail_op(LLM_ERR_INVALID_ARG, "a pointer of the pages is not aligned");
    return LLM_OK;
}

// The same for pages of 4-bit values, and their layout.
inline int check_pages_q4(const llm_pages* p, bool pointers, Q4Dev* f) {
    const int rc = check_pages(p, pointers);
    if (rc) return rc;
    if (p->head_dim % 16) return fail_op(LLM_ERR_UNSUPPORTED, "pages of 4-bit values: head_dim %d is not a multiple of 16", p->head_dim);
    if (p->page_size < 8) return fail_op(LLM_ERR_UNSUPPORTED, "pages of 4-bit values: page_size %d is below 8", p->page_size);
    const long long rows = (long long)p->page_size * p->n_kv_heads;
    if (rows > INT_MAX / 64) return fail_op(LLM_ERR_UNSUPPORTED, "a page of 4-bit values has more than 2^25 rows of all heads");
    f->groups = (p->head_dim + kQ4Group - 1) / kQ4Group;
    f->scales = rows * (p->head_dim / 2);
    f->page_bytes = (f->scales + rows * 4 * f->groups + 15) / 16 * 16;
    return LLM_OK;
}

// One strided operand: type, alignment, stride of at least `width` elements.
inline int check_rows(const char* name, const void* p, int dtype, int64_t stride, long long width, long long rows) {
    const int b = type_bytes(dtype);
    if (!b) return fail_op(LLM_ERR_UNSUPPORTED, "%s: type %d is neither LLM_F32 nor LLM_F16", name, dtype);
    if (!p) return fail_op(LLM_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, 16) || stride % (16 / b)) return fail_op(LLM_ERR_INVALID_ARG, "%s: pointer or stride not 16-byte aligned", name);
    if (rows > 1 && stride < width) return fail_op(LLM_ERR_INVALID_ARG, "%s: stride %lld below a row's %lld", name, (long long)stride, width);
    return LLM_OK;
}

inline PagesDev pages_dev(const llm_pages* p) {
    int shift = 0;
    while ((1 << shift) < p->page_size) shift++;
    return {p->n_seqs, p->n_new, p->prefix_len, shift, p->n_pages, p->max_pages, p->n_kv_heads, p->head_dim,
            reinterpret_cast<__half*>(p->k_pages), reinterpret_cast<__half*>(p->v_pages), p->page_table, p->lens, p->err};
}

inline int launched(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return LLM_OK;
    cudaGetLastError();
    return fail_op(LLM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// The current device, 0 where there is none to ask.
inline int device_now() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return dev;
}
constexpr int kDevicesKept = 64;             // devices whose answers are kept; others are asked every time

// SMs of the current device (152 where there is none to ask).
inline int sm_count() {
    static std::atomic<int> known[kDevicesKept];
    const int dev = device_now();
    int n = dev < kDevicesKept ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 152;
    }
    if (dev < kDevicesKept) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Runs `set` (the attributes of one kernel) the first time on each device; one
// static array of flags per kernel.
struct OncePerDevice {
    std::atomic<bool> done[kDevicesKept];
    template <class Set>
    cudaError_t operator()(Set set) {
        const int dev = device_now();
        if (dev < kDevicesKept && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
        const cudaError_t e = set();
        if (e == cudaSuccess && dev < kDevicesKept) done[dev].store(true, std::memory_order_release);
        return e;
    }
};

}  // namespace llm
