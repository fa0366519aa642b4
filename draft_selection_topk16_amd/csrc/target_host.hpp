// Host-side checks that the operators of the target's side share.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <string>
#include <type_traits>

#include "dflash2.h"
#include "host.hpp"
#include "attention.hpp"
#include "kvappend.hpp"

namespace df2 {
namespace host {

// Threads of a launch along one dimension.
constexpr int64_t kMostThreads = 0xFFFFFFFF;

inline bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

inline df2_status launched(const char* what) {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? DF2_OK : hip_failed(e, what);
}

// Checks the sizes of a cache descriptor; fp4: of 4-bit values, whose stride is in bytes.
inline df2_status check_kv_sizes(const df2_paged_kv* kv, bool fp4 = false) {
    if (!kv) return fail_with(DF2_EINVAL, "the cache descriptor is NULL");
    if (kv->dtype != DF2_F32 && kv->dtype != DF2_BF16) return fail_with(DF2_EINVAL, "unknown dtype");
    if (kv->B < 0 || kv->N < 0) return fail_with(DF2_EINVAL, "B and N must be >= 0");
    if (kv->Hkv < 1 || kv->Hq < 1 || kv->Hq % kv->Hkv != 0)
        return fail_with(DF2_EINVAL, "Hq must be a positive multiple of Hkv");
    if (kv->D != 64 && kv->D != 128 && kv->D != 256)
        return fail_with(DF2_EUNSUPPORTED, "D must be 64, 128 or 256");
    if (kv->page_size < 1 || (kv->page_size & (kv->page_size - 1)) || kv->page_size > 65536)
        return fail_with(DF2_EUNSUPPORTED, "page_size must be a power of two up to 65536");
    if (kv->num_pages < 1) return fail_with(DF2_EINVAL, "num_pages < 1");
    if (kv->table_width < 1 || kv->table_stride < kv->table_width)
        return fail_with(DF2_EINVAL, "table_width must be >= 1 and at most table_stride");
    if ((int64_t)kv->table_width * kv->page_size > (1 << 30))
        return fail_with(DF2_EUNSUPPORTED, "table_width * page_size above 2^30");
    if ((int64_t)kv->N * kv->Hq > 0x7FFFFFFF) return fail_with(DF2_EUNSUPPORTED, "N * Hq too large");
    if (fp4) {
        if (kv->page_size < 16) return fail_with(DF2_EUNSUPPORTED, "page_size of a 4-bit cache must be at least 16");
        if (kv->page_stride < (int64_t)kv->Hkv * kv->page_size * (kv->D / 2 + kv->D / 32))
            return fail_with(DF2_EINVAL, "page_stride below Hkv * page_size * (D / 2 + D / 32)");
        if (kv->page_stride % 16 != 0) return fail_with(DF2_EINVAL, "page_stride must be a multiple of 16 bytes");
        return DF2_OK;
    }
    const int64_t page = (int64_t)kv->Hkv * kv->page_size * kv->D;
    if (kv->page_stride < page) return fail_with(DF2_EINVAL, "page_stride below Hkv * page_size * D");
    const int per16 = kv->dtype == DF2_BF16 ? 8 : 4;
    if (kv->page_stride % per16 != 0) return fail_with(DF2_EINVAL, "page_stride must be a multiple of 16 bytes");
    return DF2_OK;
}

// Checks a cache descriptor and fills what the kernels read of it.
inline df2_status read_kv(const df2_paged_kv* kv, PagedKv* out, bool fp4 = false) {
    const df2_status st = check_kv_sizes(kv, fp4);
    if (st != DF2_OK || kv->B == 0 || kv->N == 0) return st;
    if (!kv->k_cache || !kv->v_cache || !kv->block_table || !kv->ctx_len || !kv->tok_start)
        return fail_with(DF2_EINVAL, "NULL pointer in the cache descriptor");
    if (!aligned(kv->k_cache, 16) || !aligned(kv->v_cache, 16))
        return fail_with(DF2_EINVAL, "k_cache and v_cache must be 16-byte aligned");
    if (!aligned(kv->block_table, 4) || !aligned(kv->ctx_len, 4) || !aligned(kv->tok_start, 4))
        return fail_with(DF2_EINVAL, "block_table, ctx_len and tok_start must be 4-byte aligned");
    out->table = kv->block_table;
    out->ctx = kv->ctx_len;
    out->start = kv->tok_start;
    out->page_stride = kv->page_stride;
    out->B = kv->B;
    out->N = kv->N;
    out->Hq = kv->Hq;
    out->Hkv = kv->Hkv;
    out->page_shift = __builtin_ctz((unsigned)kv->page_size);
    out->num_pages = kv->num_pages;
    out->table_width = kv->table_width;
    out->table_stride = kv->table_stride;
    return DF2_OK;
}

// A token's row of `heads` heads: 16-byte aligned and long enough.
inline df2_status check_rows(const df2_paged_kv* kv, const void* p, int64_t stride, int heads, const char* name) {
    const int per16 = kv->dtype == DF2_BF16 ? 8 : 4;
    if (!aligned(p, 16)) return fail_with(DF2_EINVAL, std::string(name) + " must be 16-byte aligned");
    if (stride < (int64_t)heads * kv->D || stride % per16 != 0)
        return fail_with(DF2_EINVAL, std::string(name) + ": the token stride must hold the heads and be a multiple of 16 bytes");
    return DF2_OK;
}

// Token rows as the arguments give them: stride and heads * D in elements.
struct TokenRows {
    const void* p;
    int64_t stride;
    int heads;
};
// Whether some row of one shares memory with a row of the other.  (Rows of both may
// be parts of the same wider rows.)
inline bool rows_meet(const df2_paged_kv* kv, const TokenRows& a, const TokenRows& b) {
    const int64_t size = kv->dtype == DF2_BF16 ? 2 : 4, last = kv->N - 1;
    const int64_t sa = a.stride * size, wa = (int64_t)a.heads * kv->D * size;
    const int64_t sb = b.stride * size, wb = (int64_t)b.heads * kv->D * size;
    const int64_t d = (int64_t)((uintptr_t)b.p - (uintptr_t)a.p);
    if (d >= last * sa + wa || -d >= last * sb + wb) return false;
    if (sa == sb) {
        const int64_t m = ((d % sa) + sa) % sa;         // where b's rows begin within a's stride
        return m < wa || sa - m < wb;
    }
    for (int64_t i = 0; i <= last; ++i) {
        const int64_t x = i * sa - d;                   // a's row against b's first
        const int64_t j = x < wb ? 0 : (x - wb) / sb + 1;       // b's first row that ends behind its beginning
        if (j <= last && j * sb < x + wa) return true;
    }
    return false;
}

// Checks the arguments of an append and fills what its kernels read.
inline df2_status read_append(const df2_paged_kv* kv, bool fp4, const void* q, int64_t q_stride, const void* k,
                              int64_t k_stride, const void* v, int64_t v_stride, const void* q_norm, const void* k_norm,
                              float eps, const double* rope_freq, int32_t rot, int32_t interleaved, void* out_q,
                              int64_t out_q_stride, AppendArgs* a) {
    std::memset(a, 0, sizeof(*a));
    df2_status st = read_kv(kv, &a->kv, fp4);
    if (st != DF2_OK) return st;
    if (rot < 0 || rot > kv->D || rot % 16 != 0)
        return fail_with(DF2_EUNSUPPORTED, "rot must be a multiple of 16 in [0, D]");
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail_with(DF2_EINVAL, "eps must be finite and >= 0");
    if (kv->B == 0 || kv->N == 0) return DF2_OK;
    if (((int64_t)kv->N + 3) / 4 * 256 > kMostThreads) return fail_with(DF2_EUNSUPPORTED, "N above 2^26 - 4");
    if (!k || !v || (rot > 0 && !rope_freq)) return fail_with(DF2_EINVAL, "NULL pointer argument");
    if (!q != !out_q) return fail_with(DF2_EINVAL, "q and out_q come together");
    if (!q && q_norm) return fail_with(DF2_EINVAL, "q_norm without q");
    if ((st = check_rows(kv, k, k_stride, kv->Hkv, "k")) != DF2_OK) return st;
    if ((st = check_rows(kv, v, v_stride, kv->Hkv, "v")) != DF2_OK) return st;
    if (q) {
        if ((st = check_rows(kv, q, q_stride, kv->Hq, "q")) != DF2_OK) return st;
        if ((st = check_rows(kv, out_q, out_q_stride, kv->Hq, "out_q")) != DF2_OK) return st;
        if (q == out_q && q_stride != out_q_stride)
            return fail_with(DF2_EINVAL, "out_q in place of q needs the same stride");
    }
    if (!aligned(q_norm, 16) || !aligned(k_norm, 16))
        return fail_with(DF2_EINVAL, "q_norm and k_norm must be 16-byte aligned");
    if (!aligned(rope_freq, 8)) return fail_with(DF2_EINVAL, "rope_freq must be 8-byte aligned");
    if (q) {
        const TokenRows out = {out_q, out_q_stride, kv->Hq};
        if ((q != out_q && rows_meet(kv, {q, q_stride, kv->Hq}, out)) || rows_meet(kv, {k, k_stride, kv->Hkv}, out) ||
            rows_meet(kv, {v, v_stride, kv->Hkv}, out))
            return fail_with(DF2_EINVAL, "out_q must not overlap q (unless it is q), k or v");
    }
    if ((st = device_flag_word(&a->kv.err)) != DF2_OK) return st;
    a->q = q;
    a->k = k;
    a->v = v;
    a->k_cache = kv->k_cache;
    a->v_cache = kv->v_cache;
    a->out_q = out_q;
    a->q_norm = q_norm;
    a->k_norm = k_norm;
    a->freq = rope_freq;
    a->q_stride = q_stride;
    a->k_stride = k_stride;
    a->v_stride = v_stride;
    a->out_stride = out_q_stride;
    a->rot = rot;
    a->interleaved = interleaved ? 1 : 0;
    a->eps = eps;
    return DF2_OK;
}

// Calls f with the cache's type and head size as constants.
template <typename F>
auto with_type(const df2_paged_kv* kv, F&& f) {
    using std::integral_constant;
    if (kv->dtype == DF2_BF16) {
        if (kv->D == 64) return f(integral_constant<bool, true>(), integral_constant<int, 64>());
        if (kv->D == 128) return f(integral_constant<bool, true>(), integral_constant<int, 128>());
        return f(integral_constant<bool, true>(), integral_constant<int, 256>());
    }
    if (kv->D == 64) return f(integral_constant<bool, false>(), integral_constant<int, 64>());
    if (kv->D == 128) return f(integral_constant<bool, false>(), integral_constant<int, 128>());
    return f(integral_constant<bool, false>(), integral_constant<int, 256>());
}

// max_len as the plan takes it: 0 means what the page table holds.
inline df2_status plan_length(const df2_paged_kv* kv, int32_t max_len, int* out) {
    if (max_len < 0) return fail_with(DF2_EINVAL, "max_len < 0");
    const int cap = kv->table_width * kv->page_size;
    *out = max_len == 0 ? cap : std::min(max_len, cap);
    return DF2_OK;
}

}  // namespace host
}  // namespace df2
