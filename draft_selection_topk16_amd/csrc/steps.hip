// Between the steps of a serving loop: the pages, starts and slots of the next one
// (pages.hpp) and what is done to the target's rows before they are verified
// (adjust.hpp).  The C ABI is declared in include/dflash2.h.  Nothing here keeps
// scratch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>
#include <string>

#include "dflash2.h"
#include "host.hpp"
#include "target_host.hpp"
#include "adjust.hpp"
#include "pages.hpp"

using namespace df2;
using namespace df2::host;

namespace {

// An array in memory, and whether two of them meet.
struct Span {
    const void* p;
    int64_t bytes;
    const char* name;
};
bool meet(const Span& a, const Span& b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

// Rows that are written (bytes; sequences hold their rows, which do not meet), and a list of
// words in rows of its own: either may lie between rows of the other.
struct OutRows {
    uintptr_t at;
    int64_t B, R, seq, row, bytes;
};
struct List {
    const void* p;
    int64_t B, R, seq, row, words;
    const char* name;
};
bool rows_meet_list(const OutRows& o, const List& l) {
    if (!l.p || l.words <= 0) return false;
    const int64_t d = (int64_t)((uintptr_t)l.p - o.at);
    const int64_t all = (o.B - 1) * o.seq + (o.R - 1) * o.row + o.bytes;
    const int64_t list = ((l.B - 1) * l.seq + (l.R - 1) * l.row + l.words) * 4;
    if (d >= all || d + list <= 0) return false;
    for (int64_t i = 0; i < (l.seq ? l.B : 1); ++i)
        for (int64_t j = 0; j < (l.row ? l.R : 1); ++j) {
            // the row that its beginning is in or behind, and the next one
            const int64_t x = d + (i * l.seq + j * l.row) * 4, end = x + l.words * 4;
            for (int64_t b = o.seq && x > 0 ? std::min(x / o.seq, o.B - 1) : 0, b1 = std::min(b + 2, o.B); b < b1; ++b)
                for (int64_t y = x - b * o.seq, t = y > 0 ? std::min(y / o.row, o.R - 1) : 0, t1 = std::min(t + 2, o.R); t < t1; ++t)
                    if (x < b * o.seq + t * o.row + o.bytes && end > b * o.seq + t * o.row) return true;
        }
    return false;
}

// ----------------------------------------------------------------------------
// Pages.
// ----------------------------------------------------------------------------
// Rows that the planning workgroup makes itself; more of them are a second launch.
constexpr int kPageRows = 4096;
constexpr int kMostRequests = 1 << 20;

df2_status check_pool(const df2_page_pool* p) {
    if (!p) return fail_with(DF2_EINVAL, "the pool descriptor is NULL");
    if (p->B < 0 || p->N < 0) return fail_with(DF2_EINVAL, "B and N must be >= 0");
    if (p->B > kMostRequests) return fail_with(DF2_EUNSUPPORTED, "B above 2^20");
    if (p->N > 1 << 30) return fail_with(DF2_EUNSUPPORTED, "N above 2^30");
    if (p->page_size < 1 || (p->page_size & (p->page_size - 1)) || p->page_size > 65536)
        return fail_with(DF2_EUNSUPPORTED, "page_size must be a power of two up to 65536");
    if (p->num_pages < 1) return fail_with(DF2_EINVAL, "num_pages < 1");
    if (p->num_pages > 1 << 30) return fail_with(DF2_EUNSUPPORTED, "num_pages above 2^30");
    if (p->table_width < 1 || p->table_stride < p->table_width)
        return fail_with(DF2_EINVAL, "table_width must be >= 1 and at most table_stride");
    if ((int64_t)p->table_width * p->page_size > (1 << 30))
        return fail_with(DF2_EUNSUPPORTED, "table_width * page_size above 2^30");
    return DF2_OK;
}

}  // namespace

extern "C" {

df2_status dflash2_plan_pages(const df2_page_pool* pool, const int32_t* ctx_len, const int32_t* advance,
                              const int32_t* n_new, int32_t* ctx_out, int32_t* tok_start, int64_t* slots,
                              int32_t* positions, hipStream_t stream) {
    clear_error();
    df2_status st = check_pool(pool);
    if (st != DF2_OK || pool->B == 0) return st;
    if (!pool->block_table || !pool->held || !pool->free_list || !pool->free_count || !ctx_len || !n_new || !ctx_out ||
        !tok_start)
        return fail_with(DF2_EINVAL, "NULL pointer argument");
    const int64_t B = pool->B, N = pool->N;
    const Span outs[] = {{pool->block_table, ((B - 1) * pool->table_stride + pool->table_width) * 4, "block_table"},
                         {pool->held, B * 4, "held"},
                         {pool->free_list, (int64_t)pool->num_pages * 4, "free_list"},
                         {pool->free_count, 4, "free_count"},
                         {ctx_out, B * 4, "ctx_out"},
                         {tok_start, (B + 1) * 4, "tok_start"},
                         {slots, N * 8, "slots"},
                         {positions, N * 4, "positions"}};
    const Span ins[] = {{ctx_len, B * 4, "ctx_len"}, {advance, B * 4, "advance"}, {n_new, B * 4, "n_new"}};
    for (const Span& s : outs)
        if (!aligned(s.p, s.p == slots ? 8 : 4)) return fail_with(DF2_EINVAL, std::string(s.name) + " is misaligned");
    for (const Span& s : ins)
        if (!aligned(s.p, 4)) return fail_with(DF2_EINVAL, std::string(s.name) + " is misaligned");
    for (const Span& o : outs) {
        for (const Span& other : outs)
            if (&o < &other && meet(o, other))
                return fail_with(DF2_EINVAL, std::string(o.name) + " must not overlap " + other.name);
        for (const Span& in : ins)
            if (!(o.p == ctx_out && o.p == in.p && &in == ins) && meet(o, in))
                return fail_with(DF2_EINVAL, std::string(o.name) + " must not overlap " + in.name);
    }
    PagesArgs a;
    std::memset(&a, 0, sizeof(a));
    if ((st = device_flag_word(&a.err)) != DF2_OK) return st;
    a.table = pool->block_table;
    a.held = pool->held;
    a.free_list = pool->free_list;
    a.free_count = pool->free_count;
    a.ctx = ctx_len;
    a.advance = advance;
    a.n_new = n_new;
    a.ctx_out = ctx_out;
    a.start = tok_start;
    a.slot = slots;
    a.pos = positions;
    a.table_stride = pool->table_stride;
    a.B = pool->B;
    a.N = pool->N;
    a.page_shift = __builtin_ctz((unsigned)pool->page_size);
    a.num_pages = pool->num_pages;
    a.table_width = pool->table_width;
    const bool rows = slots || positions;
    a.rows_here = rows && pool->N <= kPageRows;
    if (pool->B <= 256 && (!a.rows_here || pool->N <= 1024))
        hipLaunchKernelGGL((k_plan_pages<256, 1>), dim3(1), dim3(256), 0, stream, a);
    else if (pool->B <= kPageThreads)
        hipLaunchKernelGGL((k_plan_pages<kPageThreads, 1>), dim3(1), dim3(kPageThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((k_plan_pages<kPageThreads, 4>), dim3(1), dim3(kPageThreads), 0, stream, a);
    if ((st = launched("dflash2_plan_pages launch")) != DF2_OK || !rows || a.rows_here) return st;
    // some 16 waves a compute unit over the requests' rows
    const int64_t waves = (int64_t)compute_units() * 16;
    const unsigned y = (unsigned)std::max<int64_t>(1, std::min<int64_t>((N + 63) / 64, waves / (B + 1)));
    hipLaunchKernelGGL(k_page_rows, dim3((unsigned)B + 1, y), dim3(64), 0, stream, a);
    return launched("dflash2_plan_pages rows launch");
}

// ----------------------------------------------------------------------------
// Adjusting rows of logits.
// ----------------------------------------------------------------------------
df2_status dflash2_adjust_logits(const df2_adjust* d, const void* logits, void* out, hipStream_t stream) {
    clear_error();
    if (!d) return fail_with(DF2_EINVAL, "the descriptor is NULL");
    if (d->dtype != DF2_F32 && d->dtype != DF2_BF16) return fail_with(DF2_EINVAL, "unknown dtype");
    if (d->B < 0 || d->R < 0) return fail_with(DF2_EINVAL, "B and R must be >= 0");
    if (d->V < 1) return fail_with(DF2_EINVAL, "V < 1");
    if (d->V > (1 << 29)) return fail_with(DF2_EUNSUPPORTED, "V above 2^29");
    if (d->L < 0 || d->M < 0) return fail_with(DF2_EINVAL, "L and M must be >= 0");
    if (d->L >= 1 << 29) return fail_with(DF2_EUNSUPPORTED, "L must be below 2^29");
    if (d->B == 0 || d->R == 0) return DF2_OK;
    if (!logits || !out) return fail_with(DF2_EINVAL, "NULL pointer argument");
    const int size = d->dtype == DF2_BF16 ? 2 : 4;
    if (!aligned(logits, size) || !aligned(out, size)) return fail_with(DF2_EINVAL, "logits or out misaligned for the dtype");
    const bool history = d->history && d->L > 0, path = d->path && d->R > 1, biases = d->M > 0;
    if ((history ? d->L : 0) + (path ? (int64_t)d->R - 1 : 0) >= 1 << 29)
        return fail_with(DF2_EUNSUPPORTED, "L and the drafts together must be below 2^29");
    if (history && !d->history_len) return fail_with(DF2_EINVAL, "history without history_len");
    if (history && d->history_stride < d->L) return fail_with(DF2_EINVAL, "history_stride below L");
    if (biases && (!d->bias_token || !d->bias)) return fail_with(DF2_EINVAL, "M > 0 without bias_token and bias");
    for (const void* p : {(const void*)d->history, (const void*)d->history_len, (const void*)d->prompt_len, (const void*)d->path,
                          (const void*)d->repetition, (const void*)d->frequency, (const void*)d->presence,
                          (const void*)d->bias_token, (const void*)d->bias, (const void*)d->mask})
        if (!aligned(p, 4)) return fail_with(DF2_EINVAL, "lists, penalties and masks must be 4-byte aligned");
    // rows: apart from one another, and those of out apart from those of logits unless they are the same
    const int64_t row = d->R > 1 ? d->row_stride : d->V, seq = d->B > 1 ? d->seq_stride : 0;
    const int64_t out_row = d->R > 1 ? d->out_row_stride : d->V, out_seq = d->B > 1 ? d->out_seq_stride : 0;
    if (row < d->V || out_row < d->V) return fail_with(DF2_EINVAL, "row strides must be at least V");
    const int64_t extent = (d->R - 1) * row + d->V, out_extent = (d->R - 1) * out_row + d->V;
    if ((d->B > 1 && seq < extent) || (d->B > 1 && out_seq < out_extent))
        return fail_with(DF2_EINVAL, "sequence strides must hold a sequence's rows");
    const bool place = out == logits && row == out_row && seq == out_seq;
    if (!place && meet({logits, ((d->B - 1) * seq + extent) * size, ""}, {out, ((d->B - 1) * out_seq + out_extent) * size, ""}))
        return fail_with(DF2_EINVAL, "out must be logits, with the same strides, or not overlap it");
    const int64_t words = ((int64_t)d->V + 31) / 32;
    if (d->mask && ((d->R > 1 && d->mask_row_stride != 0 && d->mask_row_stride < words) ||
                    (d->B > 1 && d->mask_seq_stride != 0 && d->mask_seq_stride < words)))
        return fail_with(DF2_EINVAL, "mask strides must be 0 or hold a row");
    // what is read of the lists while rows are written
    const OutRows rows = {(uintptr_t)out, d->B, d->R, out_seq * size, out_row * size, (int64_t)d->V * size};
    const List lists[] = {{history ? d->history : nullptr, d->B, 1, d->history_stride, 0, d->L, "history"},
                          {history ? d->history_len : nullptr, 1, 1, 0, 0, d->B, "history_len"},
                          {history ? d->prompt_len : nullptr, 1, 1, 0, 0, d->B, "prompt_len"},
                          {path ? d->path : nullptr, 1, 1, 0, 0, (int64_t)d->B * (d->R - 1), "path"},
                          {d->repetition, 1, 1, 0, 0, d->B, "repetition"},
                          {d->frequency, 1, 1, 0, 0, d->B, "frequency"},
                          {d->presence, 1, 1, 0, 0, d->B, "presence"},
                          {biases ? d->bias_token : nullptr, 1, 1, 0, 0, (int64_t)d->B * d->M, "bias_token"},
                          {biases ? d->bias : nullptr, 1, 1, 0, 0, (int64_t)d->B * d->M, "bias"},
                          {d->mask, d->B, d->R, d->mask_seq_stride, d->mask_row_stride, words, "mask"}};
    for (const List& l : lists)
        if (rows_meet_list(rows, l)) return fail_with(DF2_EINVAL, std::string("out must not overlap ") + l.name);
    if (place && !history && !path && !biases && !d->mask) return DF2_OK;

    AdjustArgs a;
    std::memset(&a, 0, sizeof(a));
    a.logits = logits;
    a.out = out;
    a.history = history ? d->history : nullptr;
    a.history_len = d->history_len;
    a.prompt_len = d->prompt_len;
    a.path = path ? d->path : nullptr;
    a.repetition = d->repetition;
    a.frequency = d->frequency;
    a.presence = d->presence;
    a.bias_token = d->bias_token;
    a.bias = d->bias;
    a.mask = reinterpret_cast<const uint32_t*>(d->mask);
    a.seq_stride = seq;
    a.row_stride = d->R > 1 ? row : 0;
    a.out_seq_stride = out_seq;
    a.out_row_stride = d->R > 1 ? out_row : 0;
    a.history_stride = d->history_stride;
    a.mask_seq_stride = d->B > 1 ? d->mask_seq_stride : 0;
    a.mask_row_stride = d->R > 1 ? d->mask_row_stride : 0;
    a.B = d->B;
    a.R = d->R;
    a.V = d->V;
    a.L = d->L;
    a.M = d->M;
    // Segments of 4096 tokens with all rows of a sequence, so that a history is gone
    // through 37 times for 151936 tokens; fewer rows, then shorter segments, until
    // there are two workgroups a compute unit.
    const int64_t want = 2 * (int64_t)compute_units();
    a.seg = 4096;
    a.rows = d->mask ? std::min(d->R, 16) : d->R;       // the masks of 16 rows are 8 KB of LDS
    const auto count = [&] {
        a.nseg = (int)(((int64_t)d->V + a.seg - 1) / a.seg);
        a.row_groups = (d->R + a.rows - 1) / a.rows;
        return (int64_t)a.nseg * a.row_groups * d->B;
    };
    while (a.rows > 1 && count() < want) a.rows = (a.rows + 1) / 2;
    while (a.seg > 1024 && count() < want) a.seg /= 2;     // four words a thread at least
    const int64_t groups = count();
    if (groups * kAdjustThreads > kMostThreads) return fail_with(DF2_EUNSUPPORTED, "B * R * V too large");
    a.max_words = d->mask ? a.rows * (a.seg / 32) : 0;
    // A list of biases is short LDS and a search for each biased token; with many a word for
    // each token (512 rows in place with 16 biases: a table costs 22 us).
    a.table = d->M > kBiasList;
    const size_t lds = ((size_t)a.seg + a.seg / 2 + a.max_words + (a.table ? a.seg : d->M)) * 4;
    const auto go = [&](auto bf16, auto in_place) {
        hipLaunchKernelGGL((k_adjust<decltype(bf16)::value, decltype(in_place)::value>), dim3((unsigned)groups),
                           dim3(kAdjustThreads), lds, stream, a);
        return launched("dflash2_adjust_logits launch");
    };
    using std::false_type;
    using std::true_type;
    if (d->dtype == DF2_BF16) return place ? go(true_type(), true_type()) : go(true_type(), false_type());
    return place ? go(false_type(), true_type()) : go(false_type(), false_type());
}

}  // extern "C"
