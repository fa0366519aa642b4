// Block tables, token starts and slot maps of the next step, from the lengths of
// the requests, all in device memory.
//
// Request b holds ctx_b + advance_b tokens and brings n_b new ones: it wants
//     want_b = ceil((ctx_b + advance_b + n_b) / page_size)
// pages.  Pages it has beyond those go to the end of the free list, in the order of
// the requests; missing ones come from its end.  Who is served follows from prefix
// sums of what the requests ask for, so the result does not depend on how the work
// is divided, and there are no atomics.
//
// One workgroup does this for all requests: three passes over them (what goes
// back; who is served; tables and starts), kPageThreads at a time, prefix sums by
// lanes and then over the waves in LDS.  It is bound by latency: a pass is a few
// loads and a scan one after the other.  What follows per row (slots and positions)
// is work for the whole chip where there are many rows, in a second launch; with up
// to kPageRows rows the same workgroup does it.
#pragma once

#include "attention.hpp"

namespace df2 {

constexpr uint32_t kFlagServed = 128u;  // a request was left without new tokens
constexpr int kPageThreads = 1024;

struct PagesArgs {
    int32_t* table;         // [B, table_stride]
    int32_t* held;          // [B] pages each request has
    int32_t* free_list;     // [num_pages]
    int32_t* free_count;    // [1]
    const int32_t* ctx;     // [B]
    const int32_t* advance; // [B] or NULL
    const int32_t* n_new;   // [B]
    int32_t* ctx_out;       // [B], may be ctx
    int32_t* start;         // [B + 1]
    int64_t* slot;          // [N] or NULL
    int32_t* pos;           // [N] or NULL
    uint32_t* err;
    int64_t table_stride;
    int B, N, page_shift, num_pages, table_width;
    int rows_here;          // this launch makes the rows' slots too
};

// A request of the batch as it comes in.
struct PageRequest {
    int ctx, n, held, want;     // tokens after advance, new ones asked for, pages held and wanted
    bool wide;                  // more than the table holds
};
__device__ __forceinline__ PageRequest page_request(const PagesArgs& a, int b) {
    PageRequest r = {0, 0, 0, 0, false};
    if (b >= a.B) return r;
    const int n = a.n_new[b], held = a.held[b];
    const int64_t ctx = max((int64_t)a.ctx[b] + (a.advance ? a.advance[b] : 0), (int64_t)0);
    r.held = min(max(held, 0), a.table_width);
    if (n < 0) return r;                    // finished: wants nothing, holds no tokens
    const int64_t want = (ctx + n + ((1 << a.page_shift) - 1)) >> a.page_shift;
    r.ctx = (int)min(ctx, (int64_t)0x7FFFFFFF);
    r.wide = want > a.table_width;
    r.n = r.wide ? 0 : n;
    r.want = r.wide ? r.held : (int)want;
    return r;
}

// Sum over the threads up to this one; all: over the whole workgroup.  In fp64, exact
// to 2^53, so that what 2^20 requests ask for cannot wrap around.
template <int NT>
__device__ __forceinline__ double pages_scan(double x, double* waves, double& all) {
    const double mine = lanes_scan(x);
    __syncthreads();
    if (lane_id() == 63) waves[wave_id()] = mine;
    __syncthreads();
    double before = 0.0;
    all = 0.0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        const double s = waves[w];
        if (w < wave_id()) before += s;
        all += s;
    }
    return before + mine;
}

// The request that has item i of a chunk's items, from the sums up to each request.
template <int NT>
__device__ __forceinline__ int item_owner(const int* upto, int i) {
    int lo = 0;
#pragma unroll
    for (int step = NT / 2; step > 0; step /= 2)
        if (upto[lo + step - 1] <= i) lo += step;
    return lo;
}

__device__ __forceinline__ void write_row(const PagesArgs& a, int row, int b, int pos) {
    const int64_t page = a.table[(int64_t)b * a.table_stride + (pos >> a.page_shift)];
    if (a.slot) a.slot[row] = page < 0 ? -1 : (page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
    if (a.pos) a.pos[row] = pos;
}
__device__ __forceinline__ void write_idle_row(const PagesArgs& a, int row) {
    if (a.slot) a.slot[row] = -1;
    if (a.pos) a.pos[row] = -1;
}

template <int NT>
__global__ __launch_bounds__(NT) void k_plan_pages(PagesArgs a) {
    __shared__ double waves[NT / 64];
    __shared__ int upto[NT], base[NT], first[NT];
    const int tid = threadIdx.x;
    const int chunks = (a.B + NT - 1) / NT;
    PageRequest r = page_request(a, tid);
    int count = min(max(*a.free_count, 0), a.num_pages);

    // what goes back
    for (int c = 0; c < chunks; ++c) {
        if (c > 0) r = page_request(a, c * NT + tid);
        const int gone = max(r.held - r.want, 0);
        double all;
        const double sum = pages_scan<NT>(gone, waves, all);
        if (all == 0.0) continue;
        const int items = (int)fmin(all, 2147483647.0);
        upto[tid] = (int)fmin(sum, 2147483647.0);
        base[tid] = r.want;
        first[tid] = gone;
        __syncthreads();
        for (int i = tid; i < items; i += NT) {
            const int q = item_owner<NT>(upto, i);
            int32_t* entry = a.table + (int64_t)(c * NT + q) * a.table_stride + base[q] + (i - (upto[q] - first[q]));
            const int id = *entry;
            *entry = -1;
            if (i < a.num_pages - count) a.free_list[count + i] = id;
            else atomicOr(a.err, kFlagPage);        // more than there are: a page held twice
        }
        count += min(items, a.num_pages - count);
        __syncthreads();
    }

    // who is served; their pages, starts and rows
    double asked_pages = 0.0, asked_rows = 0.0;
    int taken = 0, start = 0;
    if (tid == 0) a.start[0] = 0;
    for (int c = 0; c < chunks; ++c) {
        const int b = c * NT + tid;
        if (chunks > 1) r = page_request(a, b);
        int ask = max(r.want - r.held, 0), n = r.n;
        double all_pages, all_rows;
        const double pages = asked_pages + pages_scan<NT>(ask, waves, all_pages);
        const double rows = asked_rows + pages_scan<NT>(n, waves, all_rows);
        asked_pages += all_pages;
        asked_rows += all_rows;
        if (pages > count || rows > a.N) {
            if (n > 0 || ask > 0) atomicOr(a.err, kFlagServed);
            n = ask = 0;
        }
        if (r.wide) atomicOr(a.err, kFlagLength);
        double all_taken, all_n;
        const int page_sum = (int)pages_scan<NT>(ask, waves, all_taken);
        const int row_sum = (int)pages_scan<NT>(n, waves, all_n);
        if (b < a.B) {
            a.held[b] = min(r.held, r.want) + ask;
            a.ctx_out[b] = r.ctx;
            a.start[b + 1] = start + row_sum;
        }
        if (all_taken > 0.0) {
            upto[tid] = page_sum;
            base[tid] = r.held;
            first[tid] = ask;
            __syncthreads();
            for (int i = tid; i < (int)all_taken; i += NT) {
                const int q = item_owner<NT>(upto, i);
                a.table[(int64_t)(c * NT + q) * a.table_stride + base[q] + (i - (upto[q] - first[q]))] =
                    a.free_list[count - 1 - taken - i];
            }
            taken += (int)all_taken;
            __syncthreads();
        }
        if (a.rows_here) {
            upto[tid] = row_sum;
            base[tid] = r.ctx;
            first[tid] = n;
            __syncthreads();
            for (int i = tid; i < (int)all_n; i += NT) {
                const int q = item_owner<NT>(upto, i);
                write_row(a, start + i, c * NT + q, base[q] + (i - (upto[q] - first[q])));
            }
            __syncthreads();
        }
        start += (int)all_n;
    }
    if (tid == 0) *a.free_count = count - taken;
    if (a.rows_here)
        for (int i = start + tid; i < a.N; i += NT) write_idle_row(a, i);
}

// Slots and positions, a wave to a stretch of a request's rows; the last "request"
// is the rows behind all of them.
__global__ __launch_bounds__(64) void k_page_rows(PagesArgs a) {
    const int b = blockIdx.x, step = 64 * gridDim.y;
    const int s0 = a.start[b], s1 = b < a.B ? a.start[b + 1] : a.N;
    const int ctx = b < a.B ? a.ctx_out[b] : 0;
    for (int row = s0 + blockIdx.y * 64 + threadIdx.x; row < s1; row += step) {
        if (b < a.B) write_row(a, row, b, ctx + row - s0);
        else write_idle_row(a, row);
    }
}

}  // namespace df2
