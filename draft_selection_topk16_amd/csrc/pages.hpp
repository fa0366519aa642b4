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
// One workgroup does this for all requests: two passes over them (what goes back; who
// is served, with tables and starts), K neighbouring requests a thread, prefix sums by
// lanes and then over the waves in LDS.  It is bound by latency: a pass is a few loads and
// scans one after the other, so with up to 4096 requests they are read once (3000 of them
// with 93 thousand rows, a thousand at a time: 42 us).  What follows per row (slots and
// positions) is work for the whole chip where there are many rows, in a second launch, waves to
// a request; with up to kPageRows rows the same workgroup does it.  (Where one request, or the
// idle rows behind the last, are most of a large step, its waves bound it: 3000 requests in
// a step of 131072 rows with 3000 used 186 us.)
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
template <int N>
__device__ __forceinline__ int item_owner(const int* upto, int i) {
    int lo = 0;
#pragma unroll
    for (int step = N / 2; step > 0; step /= 2)
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

template <int NT, int K>
__global__ __launch_bounds__(NT) void k_plan_pages(PagesArgs a) {
    constexpr int CH = NT * K;              // requests of a chunk
    __shared__ double waves[NT / 64];
    __shared__ int upto[CH], base[CH], many[CH];
    const int tid = threadIdx.x;
    const int chunks = (a.B + CH - 1) / CH;
    PageRequest r[K];
    const auto read = [&](int c) {
#pragma unroll
        for (int k = 0; k < K; ++k) r[k] = page_request(a, c * CH + tid * K + k);
    };
    read(0);
    int count = min(max(*a.free_count, 0), a.num_pages);
    // sums up to each of this thread's requests, and of all
    const auto scan = [&](const int (&x)[K], double (&sum)[K]) {
        double mine = 0.0, all;
#pragma unroll
        for (int k = 0; k < K; ++k) mine += x[k];
        double before = pages_scan<NT>(mine, waves, all) - mine;
#pragma unroll
        for (int k = 0; k < K; ++k) sum[k] = before += x[k];
        return all;
    };
    // a chunk's items one by one: item i is number j of request q's n, which begin at `first`
    const auto each_item = [&](const int (&n)[K], const double (&sum)[K], const int (&first)[K], int items, auto&& f) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            upto[tid * K + k] = (int)fmin(sum[k], 2147483647.0);
            base[tid * K + k] = first[k];
            many[tid * K + k] = n[k];
        }
        __syncthreads();
        // unsigned: `items` may be the largest int, where page counts are wrong
        for (unsigned u = tid; u < (unsigned)items; u += NT) {
            const int i = (int)u, q = item_owner<CH>(upto, i);
            f(i, q, base[q] + (i - (upto[q] - many[q])));
        }
        __syncthreads();
    };

    // what goes back
    for (int c = 0; c < chunks; ++c) {
        if (c > 0) read(c);
        int gone[K], first[K];
        double sum[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            gone[k] = max(r[k].held - r[k].want, 0);
            first[k] = r[k].want;
        }
        const double all = scan(gone, sum);
        if (all == 0.0) continue;
        const int items = (int)fmin(all, 2147483647.0);
        each_item(gone, sum, first, items, [&](int i, int q, int at) {
            int32_t* entry = a.table + (int64_t)(c * CH + q) * a.table_stride + at;
            const int id = *entry;
            *entry = -1;
            if (i < a.num_pages - count) a.free_list[count + i] = id;
            else atomicOr(a.err, kFlagPage);        // more than there are: a page held twice
        });
        count += min(items, a.num_pages - count);
    }

    // who is served; their pages, starts and rows
    double asked_pages = 0.0, asked_rows = 0.0;
    int taken = 0, start = 0;
    if (tid == 0) a.start[0] = 0;
    for (int c = 0; c < chunks; ++c) {
        if (chunks > 1) read(c);
        int ask[K], n[K], first[K];
        double pages[K], rows[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            ask[k] = max(r[k].want - r[k].held, 0);
            n[k] = r[k].n;
        }
        const double all_pages = scan(ask, pages), all_rows = scan(n, rows);
        bool some = false;              // somebody is not served: the sums change
        if (asked_pages + all_pages > count || asked_rows + all_rows > a.N) {
            some = true;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (asked_pages + pages[k] > count || asked_rows + rows[k] > a.N) {
                    if (n[k] > 0 || ask[k] > 0) atomicOr(a.err, kFlagServed);
                    n[k] = ask[k] = 0;
                }
        }
        asked_pages += all_pages;
        asked_rows += all_rows;
        double all_taken = all_pages, all_n = all_rows;
        if (some) {
            all_taken = scan(ask, pages);
            all_n = scan(n, rows);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int b = c * CH + tid * K + k;
            if (r[k].wide) atomicOr(a.err, kFlagLength);
            first[k] = r[k].held;
            if (b < a.B) {
                a.held[b] = min(r[k].held, r[k].want) + ask[k];
                a.ctx_out[b] = r[k].ctx;
                a.start[b + 1] = start + (int)rows[k];
            }
        }
        if (all_taken > 0.0) {
            each_item(ask, pages, first, (int)all_taken, [&](int i, int q, int at) {
                a.table[(int64_t)(c * CH + q) * a.table_stride + at] = a.free_list[count - 1 - taken - i];
            });
            taken += (int)all_taken;
        }
        if (a.rows_here) {
#pragma unroll
            for (int k = 0; k < K; ++k) first[k] = r[k].ctx;
            each_item(n, rows, first, (int)all_n, [&](int i, int q, int at) { write_row(a, start + i, c * CH + q, at); });
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
