// segments.cuh -- what a call's new tokens touch, found on the GPU: every CTA
// scans the sequences' counts and takes its share of the pieces.
#pragma once

#include "dsa_internal.cuh"

namespace dsa {

// exclusive sum over the CTA's threads; `total` gets the sum of all.  `red` is
// shared scratch of THREADS / 32 + 1 values; ends in a barrier.
template <int THREADS, typename T>
__device__ __forceinline__ T cta_scan(T mine, T* red, T& total) {
    constexpr int W = THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();  // the last scan's sums are no longer read
    if (lane == 31) red[warp] = incl;
    __syncthreads();
    T before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const T x = red[w];
        if (w < warp) before += x;
        total += x;
    }
    return before + incl - mine;
}

// Sequences in pieces, a chunk of them at a time: first[i] pieces lie before
// sequence i of the chunk.
template <int THREADS, int PER = 4>
struct Pieces {
    static constexpr int kPer = PER, kChunk = THREADS * kPer;
    int first[kChunk + 1];
    int red[THREADS / 32 + 1];
    // counts of sequences c0 .. ; count(b) >= 0.  Returns the chunk's pieces.
    template <typename F>
    __device__ __forceinline__ int scan(int c0, int num_seqs, F count) {
        const int left = min(kChunk, num_seqs - c0);
        const int per = (left + THREADS - 1) / THREADS;
        int v[kPer];
        int mine = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = (int)threadIdx.x * per + k;
            v[k] = k < per && i < left ? count(c0 + i) : 0;
            mine += v[k];
        }
        int total;
        int at = cta_scan<THREADS>(mine, red, total);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = (int)threadIdx.x * per + k;
            if (k < per && i < left) first[i] = at;
            at += v[k];
        }
        if (threadIdx.x == 0) first[left] = total;
        __syncthreads();
        return total;
    }
    // the sequence of the chunk that piece x lies in
    __device__ __forceinline__ int find(int x, int left) const {
        int lo = 0, hi = left - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= x) lo = mid; else hi = mid - 1;
        }
        return lo;
    }
};

// phys_row with the page size as a power of two (a 64-bit division takes as long as a tile's products),
// and in two steps, so that the page's load can be under way while other work is done: its result must
// not be touched before, not even widened.
__device__ __forceinline__ int page_at(const dsa_seqs& s, int page_shift, int b, int64_t j) {
    const int64_t p = j >> page_shift;
    return s.page_table && p < s.max_pages ? __ldg(s.page_table + (int64_t)b * s.max_pages + p) : -1;
}
__device__ __forceinline__ int64_t first_row(const dsa_seqs& s, int b) { return s.page_table ? 0 : __ldg(s.seq_base + b); }
__device__ __forceinline__ int64_t row_in(const dsa_seqs& s, int page_shift, int page, int64_t first, int64_t j) {
    const int64_t row = s.page_table ? ((int64_t)page << page_shift) + (j & ((1 << page_shift) - 1)) : first + j;
    return (page >= 0 || !s.page_table) && row >= 0 && row < s.num_rows ? row : -1;
}
__device__ __forceinline__ int64_t row_at(const dsa_seqs& s, int page_shift, int b, int64_t j) {
    return row_in(s, page_shift, page_at(s, page_shift, b, j), first_row(s, b), j);
}
inline int page_shift_of(const dsa_seqs& s) { return s.page_table ? 31 - __builtin_clz((unsigned)s.page_size) : 0; }

// Sequence b's new tokens: rows [q0, q0 + nq) at positions p0, p0 + 1, ..;
// nq = 0 where there is nothing to do (p0 = -1: refused tokens).
struct NewTokens {
    int q0, nq, p0, ctx;
    bool bad;
};
__device__ __forceinline__ NewTokens new_tokens(const dsa_seqs& s, int b, int num_q) {
    NewTokens r;
    r.ctx = __ldg(s.ctx_len + b);
    r.q0 = __ldg(s.q_start + b);
    const int qe = __ldg(s.q_start + b + 1);
    r.nq = qe - r.q0;
    r.p0 = -1;
    r.bad = !(r.ctx >= 0 && r.ctx <= s.max_ctx && r.q0 >= 0 && qe >= r.q0 && qe <= num_q && r.nq <= s.max_q_per_seq);
    if (r.bad || r.nq == 0) {
        r.nq = 0;
        return r;
    }
    r.p0 = __ldg(s.q_pos + r.q0);
    if (r.p0 < 0 || r.p0 >= r.ctx) {
        r.bad = r.p0 != -1;
        r.nq = 0;
    }
    return r;
}

// the blocks of 2^shift tokens that they lie in
__device__ __forceinline__ int blocks_touched(const NewTokens& n, int shift) {
    return n.nq ? (int)((((int64_t)n.p0 + n.nq - 1) >> shift) - (n.p0 >> shift)) + 1 : 0;
}

// 16 bytes to shared memory, asynchronously, or zeros
__device__ __forceinline__ void copy16(void* dst, const void* src, bool copy) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(copy ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// the least e >= -126 with |x| <= 1.m 2^e max, for max = (1 + limit 2^-23) 2^top: x > 0 finite
__device__ __forceinline__ int scale_exponent(float x, int top, uint32_t limit) {
    const uint32_t u = __float_as_uint(x);
    const int e = (int)(u >> 23) - 127 - top + ((u & 0x7FFFFFu) > limit ? 1 : 0);
    return (u >> 23) == 0 || e < -126 ? -126 : e;  // (a subnormal x lies below 2^-126)
}
__device__ __forceinline__ float two_to(int e) { return __int_as_float((e + 127) << 23); }

}  // namespace dsa
