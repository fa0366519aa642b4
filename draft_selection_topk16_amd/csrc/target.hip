// The target's side of a draft-verify cycle: appending new tokens to a paged
// key/value cache, their attention over it, and the verification of drafted
// tokens.  Kernels in kvappend.hpp, attention.hpp and verify.hpp; the C ABI
// is declared in include/dflash2.h.
//
// Nothing here keeps scratch: what a call needs beside its outputs is the
// caller's workspace, so calls on different streams and captured graphs share
// nothing but the device's flag word.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <utility>

#include "dflash2.h"
#include "host.hpp"
#include "common.hpp"
#include "attention.hpp"
#include "kvappend.hpp"
#include "verify.hpp"

using namespace df2;
using namespace df2::host;

namespace {

// Threads of a launch along one dimension.
constexpr int64_t kMostThreads = 0xFFFFFFFF;

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

df2_status launched(const char* what) {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? DF2_OK : hip_failed(e, what);
}

// Checks the sizes of a cache descriptor.
df2_status check_kv_sizes(const df2_paged_kv* kv) {
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
    const int64_t page = (int64_t)kv->Hkv * kv->page_size * kv->D;
    if (kv->page_stride < page) return fail_with(DF2_EINVAL, "page_stride below Hkv * page_size * D");
    const int per16 = kv->dtype == DF2_BF16 ? 8 : 4;
    if (kv->page_stride % per16 != 0) return fail_with(DF2_EINVAL, "page_stride must be a multiple of 16 bytes");
    return DF2_OK;
}

// Checks a cache descriptor and fills what the kernels read of it.
df2_status read_kv(const df2_paged_kv* kv, PagedKv* out) {
    const df2_status st = check_kv_sizes(kv);
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
df2_status check_rows(const df2_paged_kv* kv, const void* p, int64_t stride, int heads, const char* name) {
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
bool rows_meet(const df2_paged_kv* kv, const TokenRows& a, const TokenRows& b) {
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

// ----------------------------------------------------------------------------
// Attention.
// ----------------------------------------------------------------------------
struct AttnPlan {
    int wr = 1;                 // waves of 32 rows in a block
    int bm = 32, kt = 32, gk = 16;
    int wgs = 1, whole = 0;     // workgroups for stretches, or for whole blocks
    int choose = 0, grid = 1;   // the kernel may take whole blocks by itself; workgroups for either
    bool fits = true;           // 32-bit tile numbers
    size_t part = 0, bytes = 0; // workspace: the parts' outputs, all of it
};

// The kernels there are: rows (WR waves of 32), key groups, 32-key steps.  A block
// of few rows gets its waves from groups of keys (one row after 1003 tokens, event
// times: 9.7 us and 6.0 for the join with four groups, 8.8 and 7.4 with one, which
// leaves four times the parts); with 64 rows of head size 128 in bf16 two workgroups
// of two waves a compute unit do as well without groups to meet (128 contexts of a
// thousand tokens 119 + 16 us, two groups 124 + 18, four groups, one workgroup a
// unit, 136 + 11); with many rows each wave reads all keys, and longer tiles meet
// less often (prompt chunks: 128 keys a tile 700 us, 96 712, blocks of 128 rows, two
// a compute unit, 730).
template <bool BF16, int D, typename F>
auto with_shape(int wr, F&& f) {
    constexpr int RB = AttnTile<BF16, D>::kRow;
    if constexpr (RB == 128) {
        if (wr == 1) return f(AttnShape<BF16, D, 1, 4, 1, 2>());
        if (wr == 2) return f(AttnShape<BF16, D, 2, 2, 2, 2>());
        if (wr == 4) return f(AttnShape<BF16, D, 4, 1, 2, 2>());
        return f(AttnShape<BF16, D, 8, 1, 2, 2>());
    } else if constexpr (RB == 256 && BF16) {
        if (wr == 1) return f(AttnShape<BF16, D, 1, 4, 1, 2>());
        if (wr == 2) return f(AttnShape<BF16, D, 2, 1, 2, 2>());
        if (wr == 4) return f(AttnShape<BF16, D, 4, 1, 2, 2>());
        return f(AttnShape<BF16, D, 8, 1, 4, 2>());
    } else if constexpr (RB == 256) {
        if (wr == 1) return f(AttnShape<BF16, D, 1, 4, 1, 2>());
        if (wr == 2) return f(AttnShape<BF16, D, 2, 2, 1, 2>());
        return f(AttnShape<BF16, D, 4, 1, 1, 2>());
    } else if constexpr (RB == 512) {
        if (wr == 1) return f(AttnShape<BF16, D, 1, 2, 1, 2>());
        if (wr == 2) return f(AttnShape<BF16, D, 2, 2, 1, 2>());
        return f(AttnShape<BF16, D, 4, 1, 1, 2>());
    } else {
        return f(AttnShape<BF16, D, 4, 1, 1, 2>());
    }
}

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

// Blocks of as many rows as a sequence has on average, but smaller ones where a
// compute unit then gets less than three tiles: parts of large blocks cost more than
// reading the keys again (event times with the join, blocks of 256, 128, 64 and 32
// rows: one chunk of 1432 tokens after 700, 4 / 2 heads, 48, 36, 35 and 40 us; 2 of 59
// after 1849, 16 / 4 heads, 35, 32, 27 and 28; 4 of 64 after 4000, 32 / 8 heads, 4
// tiles, 49 and 51).  As many workgroups as are resident at once (fewer where max_len
// says that there are fewer tiles).  Whole blocks from two for each resident
// workgroup on: there is then no part to leave and join, and the end is short
// against the rest.  A window is not counted: planned with the tiles that it leaves, 32
// new tokens after 100000 in a window of 1024, 32 / 8 heads, took 20.1 us (blocks of 32
// rows) and not 18.6 (128); a chunk of 2048 in a window of 4096 143 us either way.
AttnPlan plan_attend(const df2_paged_kv* kv, int max_len) {
    AttnPlan pl;
    const int64_t rows = (int64_t)kv->N * (kv->Hq / kv->Hkv);
    const int64_t seqs = std::min(kv->B, kv->N);
    const int64_t each = (rows + seqs - 1) / seqs;
    int per_cu = 1, threads = 64;
    const auto tiles = [&](int64_t len) { return (len + pl.gk + pl.kt - 1) / pl.kt; };
    for (pl.wr = each <= 32 ? 1 : each <= 64 ? 2 : each <= 128 ? 4 : 8;; pl.wr /= 2) {
        with_type(kv, [&](auto bf16, auto d) {
            return with_shape<decltype(bf16)::value, decltype(d)::value>(pl.wr, [&](auto shape) {
                using S = decltype(shape);
                pl.bm = S::BM;
                pl.kt = S::KT;
                pl.gk = S::kGroupKeys;
                per_cu = S::kResident;
                threads = S::kThreads;
                return 0;
            });
        });
        if (pl.wr == 1 || seqs * ((each + pl.bm - 1) / pl.bm) * kv->Hkv * tiles(max_len) >= 3 * compute_units()) break;
    }
    const int64_t blocks = rows / pl.bm + seqs;     // one more in each sequence that has tokens
    const int64_t resident = (int64_t)compute_units() * per_cu;
    pl.fits = blocks * kv->Hkv * tiles((int64_t)kv->table_width * kv->page_size) < (1LL << 31);
    const bool launchable = blocks * kv->Hkv * threads <= kMostThreads;     // a workgroup a block
    pl.whole = pl.wr == 8 && rows / pl.bm * kv->Hkv >= 2 * resident && launchable;
    if (pl.whole) {
        pl.grid = pl.wgs = (int)(blocks * kv->Hkv);
        return pl;
    }
    pl.wgs = (int)std::min(resident, blocks * kv->Hkv * tiles(max_len));
    // with fewer blocks a stretch is shorter than any of them
    pl.choose = blocks * kv->Hkv * 4 >= pl.wgs && launchable;
    pl.grid = pl.choose ? std::max(pl.wgs, (int)(blocks * kv->Hkv)) : pl.wgs;
    pl.part = (size_t)2 * pl.wgs * pl.bm * kv->D;
    pl.bytes = pl.wgs > 1 ? (pl.part + (size_t)(4 * pl.bm + 8) * pl.wgs) * sizeof(float) : 0;
    return pl;
}

// max_len as the plan takes it: 0 means what the page table holds.
df2_status plan_length(const df2_paged_kv* kv, int32_t max_len, int* out) {
    if (max_len < 0) return fail_with(DF2_EINVAL, "max_len < 0");
    const int cap = kv->table_width * kv->page_size;
    *out = max_len == 0 ? cap : std::min(max_len, cap);
    return DF2_OK;
}

template <bool BF16, int D>
df2_status launch_attend(const AttnPlan& pl, const AttnArgs& a, hipStream_t stream) {
    const df2_status st = with_shape<BF16, D>(pl.wr, [&](auto shape) {
        using S = decltype(shape);
        constexpr auto fn = S::kernel();
        if (S::kAllLds > 65536) {
            static std::mutex mu;
            static std::map<int, hipError_t> done;      // per device
            int dev = 0;
            (void)hipGetDevice(&dev);
            std::lock_guard<std::mutex> lock(mu);
            auto it = done.find(dev);
            if (it == done.end())
                it = done.emplace(dev, hipFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                                           hipFuncAttributeMaxDynamicSharedMemorySize, S::kAllLds)).first;
            if (it->second != hipSuccess) return hip_failed(it->second, "hipFuncSetAttribute (attention)");
        }
        hipLaunchKernelGGL(fn, dim3((unsigned)pl.grid), dim3(S::kThreads), S::kAllLds, stream, a);
        return launched("dflash2_paged_attention launch");
    });
    if (st != DF2_OK || !a.join) return st;
    hipLaunchKernelGGL((k_attend_join<BF16, D>), dim3((unsigned)(kJoinWgs * (pl.wgs - 1))),
                       dim3(kJoinThreads), 0, stream, a);
    return launched("dflash2_paged_attention join launch");
}

}  // namespace

extern "C" {

size_t dflash2_paged_attention_workspace(const df2_paged_kv* kv, int32_t max_len) {
    clear_error();
    int len = 0;
    if (check_kv_sizes(kv) != DF2_OK || plan_length(kv, max_len, &len) != DF2_OK) return 0;
    return kv->B == 0 || kv->N == 0 ? 0 : plan_attend(kv, len).bytes;
}

df2_status dflash2_paged_attention(const df2_paged_kv* kv, const void* q, int64_t q_stride, float scale,
                                   int32_t causal, int32_t window, int32_t max_len, void* out,
                                   int64_t out_stride, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
    clear_error();
    AttnArgs a;
    std::memset(&a, 0, sizeof(a));
    df2_status st = read_kv(kv, &a.kv);
    if (st != DF2_OK) return st;
    if (!(scale > 0.f) || !std::isfinite(scale * 1.44269504f))
        return fail_with(DF2_EINVAL, "scale must be positive and finite");
    if (window < 0 || window > (1 << 30)) return fail_with(DF2_EINVAL, "window must be in [0, 2^30]");
    int len = 0;
    if ((st = plan_length(kv, max_len, &len)) != DF2_OK) return st;
    if (kv->B == 0 || kv->N == 0) return DF2_OK;
    if (!q || !out) return fail_with(DF2_EINVAL, "NULL pointer argument");
    if ((st = check_rows(kv, q, q_stride, kv->Hq, "q")) != DF2_OK) return st;
    if ((st = check_rows(kv, out, out_stride, kv->Hq, "out")) != DF2_OK) return st;
    const AttnPlan pl = plan_attend(kv, len);
    if (!pl.fits) return fail_with(DF2_EUNSUPPORTED, "too many tiles (N, Hkv and the page table's width)");
    if (pl.bytes > 0) {
        if (!workspace || workspace_bytes < pl.bytes)
            return fail_with(DF2_EINVAL, "workspace of " + std::to_string(workspace ? workspace_bytes : 0) +
                                             " bytes; the call needs " + std::to_string(pl.bytes));
        if (!aligned(workspace, 16)) return fail_with(DF2_EINVAL, "workspace must be 16-byte aligned");
    }
    if (rows_meet(kv, {q, q_stride, kv->Hq}, {out, out_stride, kv->Hq}))
        return fail_with(DF2_EINVAL, "out must not overlap q");
    if ((st = device_flag_word(&a.kv.err)) != DF2_OK) return st;
    a.q = q;
    a.k = kv->k_cache;
    a.v = kv->v_cache;
    a.out = out;
    a.part = reinterpret_cast<float*>(workspace);
    a.stat = a.part + pl.part;
    a.split = reinterpret_cast<int32_t*>(a.stat + (size_t)4 * pl.wgs * pl.bm);
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.G = kv->Hq / kv->Hkv;
    a.causal = causal ? 1 : 0;
    a.window = window;
    a.bm = pl.bm;
    a.wgs = pl.wgs;
    a.whole = pl.whole;
    a.cus = compute_units();
    a.join = pl.bytes > 0;
    a.choose = pl.choose;
    a.inv_g = 1.0 / a.G;
    a.c = (float)((double)scale * 1.4426950408889634);
    return with_type(kv, [&](auto bf16, auto d) {
        return launch_attend<decltype(bf16)::value, decltype(d)::value>(pl, a, stream);
    });
}

// ----------------------------------------------------------------------------
// Append.
// ----------------------------------------------------------------------------
df2_status dflash2_kv_append(const df2_paged_kv* kv, const void* q, int64_t q_stride, const void* k,
                             int64_t k_stride, const void* v, int64_t v_stride, const void* q_norm,
                             const void* k_norm, float eps, const double* rope_freq, int32_t rot,
                             int32_t interleaved, void* out_q, int64_t out_q_stride, hipStream_t stream) {
    clear_error();
    AppendArgs a;
    std::memset(&a, 0, sizeof(a));
    df2_status st = read_kv(kv, &a.kv);
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
    if ((st = device_flag_word(&a.kv.err)) != DF2_OK) return st;
    a.q = q;
    a.k = k;
    a.v = v;
    a.k_cache = kv->k_cache;
    a.v_cache = kv->v_cache;
    a.out_q = out_q;
    a.q_norm = q_norm;
    a.k_norm = k_norm;
    a.freq = rope_freq;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.out_stride = out_q_stride;
    a.rot = rot;
    a.interleaved = interleaved ? 1 : 0;
    a.eps = eps;
    return with_type(kv, [&](auto bf16, auto d) {
        constexpr int D = decltype(d)::value, heads = 256 / (D / (decltype(bf16)::value ? 8 : 4));
        const int units = (q ? kv->Hq : 0) + 2 * kv->Hkv;
        // four tokens a workgroup from sixteen tokens a compute unit on; below one
        // token a compute unit, a workgroup for every `heads` heads
        if (kv->N >= 16 * compute_units())
            hipLaunchKernelGGL((k_append<decltype(bf16)::value, D, 4>), dim3((unsigned)((kv->N + 3) / 4)), dim3(256), 0,
                               stream, a);
        else
            hipLaunchKernelGGL((k_append<decltype(bf16)::value, D, 1>),
                               dim3((unsigned)kv->N, kv->N <= compute_units() ? (units + heads - 1) / heads : 1),
                               dim3(256), 0, stream, a);
        return launched("dflash2_kv_append launch");
    });
}

}  // extern "C"

// ----------------------------------------------------------------------------
// Verification.
// ----------------------------------------------------------------------------
namespace {

struct VerifyPlan {
    bool sums = false;          // launch 1 makes every row's chunk sums
    int nseg = 1, nseg_log = 0, per = 1;
    int nseg2 = 1, per2 = 1, chunks2 = 1, rounds2 = 1;
    size_t off_seg = 0, off_chunk = 0, off_top = 0, off_cnt = 0, bytes = 0;
};

// Few elements: launch 1 makes the fp64 sums of all rows, so that launch 2 is one
// short step.  Against the other way, both launches, rows of 151936 in bf16, 8 a
// sequence: 11.7 us and 13.7 at one sequence, 17.7 and 19.6 at 8, 24.5 and 26.5 at
// 16, 38.9 and 33.4 at 32; of 32000, 64 sequences, 22.2 and 21.7.  (So a count of
// elements does not part the two exactly: of these, it sends the 16 sequences and the
// 64 to the slower form, by 2 us and 0.5.)  Segments of 2048
// elements, or longer ones where that would be more workgroups than run at once, as
// far as a workgroup holds them.
// Else launch 1 takes fp32 sums, about eight workgroups a compute unit over all
// rows, none under 4 KB, a power of two of them a row (launch 2 takes several rows
// a wave), and launch 2 goes through the one row that a sequence's draw reads: in
// segments of 4096 elements, 16 for each lane, or more where that would be more
// workgroups than run at once; up to 64 chunks for each of a segment's four waves.
constexpr int64_t kFewElements = 1 << 24;
VerifyPlan plan_verify(const df2_verify_dims* d, bool best) {
    VerifyPlan pl;
    const int64_t rows = (int64_t)d->B * (d->P + 1), cus = compute_units();
    const int per16 = d->dtype == DF2_BF16 ? 8 : 4, vectors = d->V / per16;     // one less in some rows that start unaligned
    if (!best && rows * d->V <= kFewElements) {
        const int64_t most = (int64_t)kHold * kWG * per16;
        int64_t each = 2048;
        while (each < most && ((d->V + each - 1) / each > kVerifySegs || rows * ((d->V + each - 1) / each) > 8 * cus))
            each *= 2;
        pl.nseg2 = (int)((d->V + each - 1) / each);
        pl.per2 = std::max(1, (vectors + pl.nseg2 - 1) / pl.nseg2);
        pl.chunks2 = (pl.per2 + kWG - 1) / kWG;
        pl.sums = pl.nseg2 <= kVerifySegs && pl.chunks2 <= kHold;
    }
    if (!pl.sums) {
        const int64_t row_bytes = (int64_t)d->V * (16 / per16);
        while (pl.nseg < kVerifySegs && 2 * pl.nseg * rows <= 8 * cus && 2 * pl.nseg * 4096 <= row_bytes) {
            pl.nseg *= 2;
            ++pl.nseg_log;
        }
        pl.per = std::max(1, (vectors + pl.nseg - 1) / pl.nseg);
        pl.nseg2 = (int)std::max<int64_t>(1, std::min<int64_t>({kVerifySegs, (d->V + 4095) / 4096, 2 * cus / d->B}));
        pl.per2 = std::max(1, (vectors + pl.nseg2 - 1) / pl.nseg2);
        const int rounds = (pl.per2 + kWG - 1) / kWG;
        pl.rounds2 = (rounds + 63) / 64;
        pl.chunks2 = (rounds + pl.rounds2 - 1) / pl.rounds2;
    }
    const size_t segs = (size_t)(pl.sums ? rows : d->B) * pl.nseg2;
    pl.off_seg = pl.sums ? 0 : (size_t)rows * pl.nseg * 8;
    pl.off_chunk = pl.off_seg + segs * 8;
    pl.off_top = pl.off_chunk + segs * kWaves * pl.chunks2 * 8;
    pl.off_cnt = pl.off_top + (pl.sums ? segs * 4 : 0);
    pl.bytes = (pl.off_cnt + (pl.sums ? 0 : (size_t)d->B * 4) + 15) / 16 * 16;
    return pl;
}

df2_status check_verify(const df2_verify_dims* d) {
    if (!d) return fail_with(DF2_EINVAL, "dims is NULL");
    if (d->dtype != DF2_F32 && d->dtype != DF2_BF16) return fail_with(DF2_EINVAL, "unknown dtype");
    if (d->kind != DF2_TARGET_LOGITS && d->kind != DF2_TARGET_PROBS)
        return fail_with(DF2_EINVAL, "unknown kind of target values");
    if (d->B < 0) return fail_with(DF2_EINVAL, "B < 0");
    if (d->P < 1 || d->P > 64) return fail_with(DF2_EINVAL, "P must be in [1, 64]");
    if (d->V < 1) return fail_with(DF2_EINVAL, "V < 1");
    if (d->V > (1 << 29)) return fail_with(DF2_EUNSUPPORTED, "V above 2^29");
    if (d->K < 1 || d->K > 64 || d->K > d->V) return fail_with(DF2_EINVAL, "K must be in [1, min(V, 64)]");
    if ((int64_t)d->B * (d->P + 1) * kWG > kMostThreads)
        return fail_with(DF2_EUNSUPPORTED, "B * (P + 1) too large");
    return DF2_OK;
}

template <bool BF16>
df2_status launch_verify(const df2_verify_dims* d, bool best, const VerifyPlan& pl, const VerifyArgs& a,
                         hipStream_t stream) {
    const dim3 rows((unsigned)((int64_t)d->B * (d->P + 1) * pl.nseg)), draw((unsigned)(d->B * pl.nseg2)), wg(kWG);
    if (best) {
        hipLaunchKernelGGL((k_verify_rows<BF16, kVerifyArgmax>), rows, wg, 0, stream, a);
        hipLaunchKernelGGL((k_verify_best<BF16>), dim3((unsigned)d->B), wg, 0, stream, a);
        return launched("dflash2_verify launch");
    }
    const auto go = [&](auto kind) {
        constexpr int KIND = decltype(kind)::value;
        if (pl.sums) {
            const dim3 all((unsigned)((int64_t)d->B * (d->P + 1) * pl.nseg2));
            hipLaunchKernelGGL((k_verify_sums<BF16, KIND>), all, wg, 0, stream, a);
            hipLaunchKernelGGL((k_verify_pick<BF16, KIND>), dim3((unsigned)d->B), wg, 0, stream, a);
        } else {
            hipLaunchKernelGGL((k_verify_rows<BF16, KIND>), rows, wg, 0, stream, a);
            hipLaunchKernelGGL((k_verify_draw<BF16, KIND>), draw, wg, 0, stream, a);
        }
        return launched("dflash2_verify launch");
    };
    if (d->kind == DF2_TARGET_PROBS) return go(std::integral_constant<int, kVerifyProbs>());
    return go(std::integral_constant<int, kVerifyLogits>());
}

}  // namespace

extern "C" {

size_t dflash2_verify_workspace(const df2_verify_dims* dims) {
    clear_error();
    if (check_verify(dims) != DF2_OK || dims->B == 0) return 0;
    return std::max(plan_verify(dims, false).bytes, plan_verify(dims, true).bytes);
}

df2_status dflash2_verify(const df2_verify_dims* dims, const void* target, const int32_t* path,
                          const int32_t* cand_idx, const float* cand_prob, const int32_t* n_draft,
                          double temperature, const float* u, int32_t* out_tok, int32_t* out_len,
                          float* out_prob, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    clear_error();
    df2_status st = check_verify(dims);
    if (st != DF2_OK) return st;
    if (!(temperature >= 0.0) || temperature > 1e30)
        return fail_with(DF2_EINVAL, "temperature must be in [0, 1e30]");
    const bool best = temperature == 0.0;
    const double c64 = best ? 0.0 : 1.4426950408889634 / temperature;
    if (c64 > 3.0e38) return fail_with(DF2_EINVAL, "temperature too small (1 / temperature overflows fp32)");
    if (dims->B == 0) return DF2_OK;
    if (!target || !path || !out_tok || !out_len || !out_prob) return fail_with(DF2_EINVAL, "NULL pointer argument");
    if (!best && (!cand_idx || !cand_prob || !u)) return fail_with(DF2_EINVAL, "NULL pointer argument");
    if (!aligned(target, dims->dtype == DF2_BF16 ? 2 : 4)) return fail_with(DF2_EINVAL, "target misaligned for its dtype");
    if (!aligned(path, 4) || !aligned(cand_idx, 4) || !aligned(cand_prob, 4) || !aligned(n_draft, 4) ||
        !aligned(u, 4) || !aligned(out_tok, 4) || !aligned(out_len, 4) || !aligned(out_prob, 4))
        return fail_with(DF2_EINVAL, "arguments must be 4-byte aligned");
    const VerifyPlan pl = plan_verify(dims, best);
    if (!workspace || workspace_bytes < pl.bytes)
        return fail_with(DF2_EINVAL, "workspace of " + std::to_string(workspace ? workspace_bytes : 0) +
                                         " bytes; the call needs " + std::to_string(pl.bytes));
    if (!aligned(workspace, 16)) return fail_with(DF2_EINVAL, "workspace must be 16-byte aligned");
    VerifyArgs a;
    std::memset(&a, 0, sizeof(a));
    if ((st = device_flag_word(&a.err)) != DF2_OK) return st;
    char* ws = reinterpret_cast<char*>(workspace);
    a.target = target;
    a.path = path;
    a.cand = cand_idx;
    a.prob = cand_prob;
    a.n_draft = n_draft;
    a.u = u;
    a.out_tok = out_tok;
    a.out_len = out_len;
    a.out_prob = out_prob;
    a.part = reinterpret_cast<uint64_t*>(ws);
    a.seg = reinterpret_cast<double*>(ws + pl.off_seg);
    a.chunk = reinterpret_cast<double*>(ws + pl.off_chunk);
    a.top = reinterpret_cast<float*>(ws + pl.off_top);
    a.cnt = reinterpret_cast<uint32_t*>(ws + pl.off_cnt);
    a.B = dims->B;
    a.P = dims->P;
    a.V = dims->V;
    a.K = dims->K;
    a.nseg_log = pl.nseg_log;
    a.per = pl.per;
    a.nseg2 = pl.nseg2;
    a.per2 = pl.per2;
    a.chunks2 = pl.chunks2;
    a.rounds2 = pl.rounds2;
    a.k_inv = (1u << 20) / (uint32_t)dims->K + 1;
    a.c = (float)c64;
    a.c_low = (float)(c64 - (double)a.c);
    a.d_min = best ? 0.f : (float)(-1000.0 / c64);
    a.c64 = c64;
    return dims->dtype == DF2_BF16 ? launch_verify<true>(dims, best, pl, a, stream)
                                   : launch_verify<false>(dims, best, pl, a, stream);
}

}  // extern "C"
