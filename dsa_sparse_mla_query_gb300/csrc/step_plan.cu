// step_plan.cu -- a step's page tables, positions and cache slots from the
// requests' lengths (sm_103a).
//
// Two exclusive sums over the requests (rows, pages) say where each one's rows
// and new pages lie; everything else follows for each row by itself:
//   pos = cached + row - start,  slot = page(pos) P + pos mod P,
// the page from the table for columns that the request already has, else the
// next ones of the free list, which the row that opens a page writes into the
// table.
//
// Bound by latency (a step of 64 requests moves 2 KB): so one launch, and no
// CTA waits for another: each one sums the requests' lengths for itself, 2,048
// at a time (two barriers a sum), keeps the chunk's starts in shared memory and
// finds its rows' requests there by bisection.  64 requests of one token: 3.9 us in a
// graph, 6.3 with the host's call; 1,000 ragged ones, 50,000 rows: 6.8.
#include <algorithm>

#include "segments.cuh"

namespace dsa {
namespace {

constexpr int kPlanThreads = 512, kPlanPer = 4, kPlanChunk = kPlanThreads * kPlanPer;
constexpr int kPlanRows = 2 * kPlanThreads;  // rows per CTA

struct PlanArgs {
    const int32_t *cached, *fresh, *free_pages, *free_range;
    int32_t *table, *ctx, *q_start, *q_pos, *next;
    int64_t* slot;
    int32_t* d_status;
    int32_t num_seqs, shift, num_pages, max_pages, num_q, free_cap;
};

__global__ void __launch_bounds__(kPlanThreads) step_plan_kernel(const __grid_constant__ PlanArgs a) {
    __shared__ int32_t start[kPlanChunk + 1];  // first row, up to num_q
    __shared__ int32_t held[kPlanChunk];       // cached tokens
    __shared__ int32_t from[kPlanChunk];       // place of its first new page in the free list, -1: refused
    __shared__ int64_t red[kPlanThreads / 32 + 1];
    pdl_enter();
    const int tid = threadIdx.x;
    const int page = 1 << a.shift;
    const int64_t capacity = min((int64_t)a.max_pages << a.shift, (int64_t)1 << 30);  // positions stay below it
    const bool writer = blockIdx.x == 0;
    int f0 = __ldg(a.free_range), f1 = __ldg(a.free_range + 1);
    const bool bad_range = f0 < 0 || f1 < f0 || f1 > a.free_cap;
    if (bad_range) {
        if (writer && tid == 0) report(a.d_status, DSA_ERR_BAD_INPUT);
        f0 = f1 = 0;
    }
    const int row0 = blockIdx.x * kPlanRows;  // (the last CTA's may pass num_q)
    int64_t rows_before = 0, pages_before = 0, taken = 0;
    bool refused = false;
    for (int c0 = 0; c0 < a.num_seqs; c0 += kPlanChunk) {
        const int left = min(kPlanChunk, a.num_seqs - c0);
        const int per = (left + kPlanThreads - 1) / kPlanThreads;
        int had[kPlanPer], n[kPlanPer];
        int64_t sum = 0;
#pragma unroll
        for (int k = 0; k < kPlanPer; ++k) {
            const int i = tid * per + k;
            const bool in = k < per && i < left;
            had[k] = in ? __ldg(a.cached + c0 + i) : 0;
            n[k] = in ? __ldg(a.fresh + c0 + i) : 0;
            sum += max(n[k], 0);
        }
        int64_t rows, at = rows_before + cta_scan<kPlanThreads>(sum, red, rows);
        int64_t need[kPlanPer], first[kPlanPer];
        sum = 0;
#pragma unroll
        for (int k = 0; k < kPlanPer; ++k) {
            first[k] = at;
            at += max(n[k], 0);
            const bool ok = had[k] >= 0 && n[k] >= 0 && (int64_t)had[k] + n[k] <= capacity && at <= a.num_q;
            need[k] = ok ? (((int64_t)had[k] + n[k] + page - 1) >> a.shift) - (((int64_t)had[k] + page - 1) >> a.shift) : -1;
            sum += max(need[k], (int64_t)0);
        }
        int64_t pages, want = pages_before + cta_scan<kPlanThreads>(sum, red, pages);
#pragma unroll
        for (int k = 0; k < kPlanPer; ++k) {
            const int i = tid * per + k;
            if (k >= per || i >= left) continue;
            const int64_t end = want + max(need[k], (int64_t)0);
            const bool ok = need[k] >= 0 && (need[k] == 0 || end <= f1 - f0);
            if (ok && need[k] > 0) taken = end;
            refused = refused || !ok;
            start[i] = (int)min(first[k], (int64_t)a.num_q);
            held[i] = had[k];
            from[i] = ok ? f0 + (int)min(want, (int64_t)(f1 - f0)) : -1;
            want = end;
            if (writer) {
                a.q_start[c0 + i] = start[i];
                a.ctx[c0 + i] = max(0, ok ? had[k] + n[k] : had[k]);
            }
        }
        rows_before += rows;
        pages_before += pages;
        const int end = (int)min(rows_before, (int64_t)a.num_q);
        if (tid == 0) start[left] = end;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kPlanRows / kPlanThreads; ++r) {
            const int t = row0 + r * kPlanThreads + tid;
            if (t < start[0] || t >= end) continue;
            int lo = 0, hi = left - 1;  // the last request that starts at or before the row: one with rows
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (start[mid] <= t) lo = mid; else hi = mid - 1;
            }
            int pos = -1;
            int64_t slot = -1;
            if (from[lo] >= 0) {
                pos = held[lo] + (t - start[lo]);
                const int col = pos >> a.shift;
                const int old = (int)(((int64_t)held[lo] + page - 1) >> a.shift);
                int32_t* cell = a.table + (int64_t)(c0 + lo) * a.max_pages + col;
                const int p = col < old ? *cell : __ldg(a.free_pages + from[lo] + (col - old));
                if (col >= old && (pos & (page - 1)) == 0) *cell = p;
                if (p < 0 || p >= a.num_pages) {
                    report(a.d_status, DSA_ERR_BAD_INPUT);
                    pos = -1;
                } else {
                    slot = ((int64_t)p << a.shift) + (pos & (page - 1));
                }
            }
            a.q_pos[t] = pos;
            a.slot[t] = slot;
        }
        // the other CTAs need no later requests than their rows'
        if (!writer && rows_before >= (int64_t)row0 + kPlanRows) return;
        __syncthreads();  // the chunk's starts are no longer read
    }
    // rows behind the last request: padding
#pragma unroll
    for (int r = 0; r < kPlanRows / kPlanThreads; ++r) {
        const int t = row0 + r * kPlanThreads + tid;
        if (t < a.num_q && t >= rows_before) {
            a.q_pos[t] = -1;
            a.slot[t] = -1;
        }
    }
    if (!writer) return;
    if (refused) report(a.d_status, DSA_ERR_BAD_INPUT);
    // the last place taken: the largest of the threads'
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const int64_t y = __shfl_xor_sync(0xffffffffu, taken, o);
        taken = y > taken ? y : taken;
    }
    if ((tid & 31) == 0) red[tid >> 5] = taken;
    __syncthreads();
    if (tid == 0) {
        for (int w = 0; w < kPlanThreads / 32; ++w) taken = max(taken, red[w]);
        a.q_start[a.num_seqs] = (int)min(rows_before, (int64_t)a.num_q);
        a.next[0] = bad_range ? __ldg(a.free_range) : f0 + (int)taken;
        a.next[1] = __ldg(a.free_range + 1);
    }
}

}  // namespace

cudaError_t launch_step_plan(const int32_t* cached, const int32_t* fresh, int32_t num_seqs, const int32_t* free_pages,
                             int32_t free_cap, const int32_t* free_range, int32_t page_size, int32_t num_pages,
                             int32_t* table, int32_t max_pages, int32_t num_q, int32_t* ctx, int32_t* q_start,
                             int32_t* q_pos, int64_t* slot, int32_t* next, int32_t* d_status, cudaStream_t stream) {
    PlanArgs a;
    a.cached = cached;
    a.fresh = fresh;
    a.free_pages = free_pages;
    a.free_range = free_range;
    a.table = table;
    a.ctx = ctx;
    a.q_start = q_start;
    a.q_pos = q_pos;
    a.next = next;
    a.slot = slot;
    a.d_status = d_status;
    a.num_seqs = num_seqs;
    a.shift = 31 - __builtin_clz((unsigned)page_size);
    a.num_pages = num_pages;
    a.max_pages = max_pages;
    a.num_q = num_q;
    a.free_cap = free_cap;
    const unsigned grid = (unsigned)std::max<int64_t>(1, ((int64_t)num_q + kPlanRows - 1) / kPlanRows);
    return launch_pdl(step_plan_kernel, dim3(grid), dim3(kPlanThreads), 0, stream, 1, a);
}

}  // namespace dsa
