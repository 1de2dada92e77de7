// Attention of a batch's new rows over pages of 4-bit values: the part of llm_attend_batch_q4
// (include/llm.h, which defines the format) that reads the pages.  Units, pieces, deal and parts are those of
// batch_attend.cu's suffix_kernel; its prefix and join kernels do the rest.
#include "batch_attend.cuh"

namespace llm {

namespace {

// A value is made where it is used: numbers become F16 by their bits (0x6400 | n is
// 1024 + n, 0x6400 | 16 n is 1024 + 16 n; one exact operation takes the 1024 away: Kim,
// Henry, Fahim and Awadalla, "Who Says Elephants Can't Run: Bringing Large Scale MoE Models into
// Cloud Scale Production", 2022) and one fused multiply-add rounds d n + m to the F16 that it stands for.
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
// A piece's product is a sum of its own, added to the unit's in F32.  The matrix instruction cuts what it adds to
// its accumulator off towards zero, so a sum that went through it all the way fell short by some 2^-25 of itself
// a piece: 32 sequences of 1 to 4096 rows, heads of 128, F32, came out 1.8e-6 of the answer away from the exact one,
// 8e-7 this way (a plain form in F32: 5e-7); one sequence of 2^26 rows 2e-4 to 4e-4 away.  It costs 1 to 2 %.
// PACK: up to four query rows.  The eight columns of a product hold each of them twice;
// the second four take the probabilities' second parts, so one product adds both.
// FULL: head_dim is HDP, so that the distances of rows and pairs are constants.
// What bounds it: its instructions, no unit of them alone.  A step of 32 rows of heads of 64 values takes a warp 571
// (smsp__inst_executed over the steps); making the 4096 values is 224 of them by this source (three for each of a lane's
// 64 pairs, 8 shifts, 24 permutations).  64 sequences of 1 to 8192 rows, 8 heads of 64: issue 66 %, ALU 49 %, FMA (which
// has the half-precision operations) 49 %, DRAM 40 %; a loop of independent logical and half-precision operations in
// turn reaches 73 and 72 % of what each does alone, so the two units do not wait for one another.
// That case (194 MB) takes 59 us, 3.3 TB/s, 95 us as first written; 32 sequences of 1 to 4096, 32 heads of 128 (390 MB)
// 102 to 105 us, 3.7 TB/s, from 179 us.  F16 pages of the same rows would be 3.2 times the bytes.  Steps of 16 rows take 5 to 20 % longer; of 64 rows, 3 % less on the
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

// Pairs of numbers of a word, as F16 pairs.  (x & m | c as one instruction: written as an expression, the 64
// sequences above take 62.3 us for 59.1, the 32 with heads of 128 110.1 us for 101.8.)
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
            np = pieces_of(lens[s]);
        };
        int np = pieces_of(lens[s]);
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
        int ls = s, lg = g, ltile = tile, lpc = pc, lnp = np, lleft = left, page = -1;
        // (rows of a step are counted from its first one: a row behind the last of 2^31 - 1 has no number)
        auto look = [&]() {
            const int in = 8 * (lane % OCT);
            page = -1;
            if (in < min(lens[ls] - lpc * 16, 16 * min(lleft, H))) {
                page = p.table[(long long)ls * p.max_pages + ((lpc * 16 + in) >> p.page_shift)];
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
            const uint32_t e0 = (uint32_t)lpc * 16, first_row = (uint32_t)lg << p.page_shift;
            pages_ok |= (__ballot_sync(0xffffffffu, page >= 0) & ((1u << OCT) - 1)) << (4 * to);
#pragma unroll
            for (int i = 0; i < OCT; i += NO) {
                const int pg = __shfl_sync(0xffffffffu, page, i + n_oct);
                const unsigned long long off = (unsigned long long)(uint32_t)max(pg, 0) * page_bytes +
                                               (unsigned long long)(first_row + ((e0 + 8 * (i + n_oct)) & mask)) * pitch;
                if (n_in) {
                    cp_async16_or_zero(n_to + to * STAGE + i * (8 * pitch), kp + off, pg >= 0);
                    cp_async16_or_zero(n_to + to * STAGE + NUMBERS + i * (8 * pitch), vp + off, pg >= 0);
                }
            }
#pragma unroll
            for (int i = 0; i < OCT; i += PO) {
                const int oc = i + p_oct, pg = __shfl_sync(0xffffffffu, page, oc % OCT);
                const unsigned long long off = (unsigned long long)(uint32_t)max(pg, 0) * page_bytes +
                                               (unsigned long long)(first_row + ((e0 + 8 * oc) & mask)) * pairs;
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
                const int e0 = (pc + i0) * 16, rest = min(lens[s] - e0, 16 * min(H, count - i0));
                const bool whole = rest >= 16 * H && has_page == (1u << OCT) - 1;
                // rows that are not there, and those that some query rows do not see
                if (!whole || 16 * H - 1 > e_min - e0) {
#pragma unroll
                    for (int h = 0; h < H; h++)
#pragma unroll
                        for (int q = 0; q < NT; q++)
#pragma unroll
                            for (int k = 0; k < 4; k++) {
                                const int at = 16 * h + r + (k >> 1) * 8;
                                if (!((has_page >> (2 * h + (k >> 1))) & 1u) || at >= rest || at > e[q][k & 1] - e0) sc[h][q][k] = -INFINITY;
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
                    float2 add = make_float2(0.f, 0.f);          // of this thread's cached rows; all are added at the end
#pragma unroll
                    for (int h = 0; h < H; h++) {
#pragma unroll
                        for (int k = 0; k < 4; k++) sc[h][q][k] = exp2_fast(fmaf(sc[h][q][k] - R[q][k & 1], qs[q][k & 1], kHead));
                        const float2 two = __fadd2_rn(make_float2(sc[h][q][0], sc[h][q][1]), make_float2(sc[h][q][2], sc[h][q][3]));
                        add = h == 0 ? two : __fadd2_rn(add, two);
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
                    add = __fadd2_rn(make_float2(l[q][0], l[q][1]), add);
                    l[q][0] = add.x;
                    l[q][1] = add.y;
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
                            if (16 * h + 8 * (k / 2) + 2 * t + k % 2 >= rest) vd[k] = 0;
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
                    if (p.n_new > 1 && 16 * h + 15 > e_min - e0) {
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
                            // (a piece's own sum first, see the top)
                            float z[4] = {0.f, 0.f, 0.f, 0.f};
                            mma16816(z, v[i], ph[h][q][0], ph[h][q][1]);
                            if (!PACK) mma16816(z, v[i], pl[h][q][0], pl[h][q][1]);
#pragma unroll
                            for (int k = 0; k < 4; k += 2) {
                                const float2 y = __fadd2_rn(make_float2(o[q][i][k], o[q][i][k + 1]), make_float2(z[k], z[k + 1]));
                                o[q][i][k] = y.x;
                                o[q][i][k + 1] = y.y;
                            }
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
    if (!first && blockIdx.x + 1 == gridDim.x) griddep_wait();   // (as batch_attend.cu's suffix_kernel)
}

// (*e: whether it may have the shared memory that it needs)
template <int HDP, int NT, bool PACK, bool FULL>
PagesKernel one_of(bool split_q, cudaError_t* e) {
    const PagesKernel one = suffix_q4_kernel<HDP, NT, false, PACK, FULL>, two = suffix_q4_kernel<HDP, NT, true, PACK, FULL>;
    static OncePerDevice once;
    *e = once([&] {
        const int most = suffix_smem_q4(kMaxSeqs, HDP);
        const cudaError_t r = cudaFuncSetAttribute(one, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        return r != cudaSuccess ? r : cudaFuncSetAttribute(two, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    });
    return split_q ? two : one;
}
template <int HDP, bool FULL>
PagesKernel one_of(int srows, int rows, bool split_q, cudaError_t* e) {
    if (srows <= 4) return one_of<HDP, 1, true, FULL>(split_q, e);
    if (rows == 8) return one_of<HDP, 1, false, FULL>(split_q, e);
    if (HDP == 64 && rows == 24) return one_of<HDP, HDP == 64 ? 3 : 2, false, FULL>(split_q, e);
    return one_of<HDP, 2, false, FULL>(split_q, e);
}

int padded(int head_dim) { return head_dim <= 64 ? 64 : 128; }

}  // namespace

// More than 16 query rows are taken at once (up to 24, where the registers allow) as long as one unit then does,
// since every unit makes the values anew.  64 sequences of up to 8192 rows: 20 rows of heads of 64 25.2 us, 28.9 us as two
// units of 16; 24 rows of heads of 48 26.5 and 31.7 us; 12 sequences of 20 rows in F32 behind a prefix 42.1 and 43.1 us.
// For 33 to 48 rows two units of 24 for three of 16 give nothing for sure: 40 rows in F16 128.4 us for 130.8 (64
// sequences of 10 new tokens), 48 rows 137.3 us for 134.8, 40 rows in F32 53.3 us for 52.3 (12 sequences).
int unit_rows_q4(int srows, int head_dim) { return srows <= 8 ? 8 : srows > 16 && srows <= 24 && head_dim <= 64 ? 24 : 16; }
int suffix_ctas_q4(int unit_rows, int head_dim) { return suffix_q4_ctas(padded(head_dim), unit_rows / 8); }
int suffix_smem_q4(int n_seqs, int head_dim) { return ((2 * n_seqs + 1) * 4 + 15) / 16 * 16 + q4_rings(padded(head_dim)); }

PagesKernel suffix_kernel_q4(int srows, int head_dim, bool split_q, cudaError_t* e) {
    const int rows = unit_rows_q4(srows, head_dim);
    return head_dim == 64    ? one_of<64, true>(srows, rows, split_q, e)
           : head_dim < 64   ? one_of<64, false>(srows, rows, split_q, e)
           : head_dim == 128 ? one_of<128, true>(srows, rows, split_q, e)
                             : one_of<128, false>(srows, rows, split_q, e);
}

}  // namespace llm
