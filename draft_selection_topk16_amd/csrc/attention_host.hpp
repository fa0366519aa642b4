// The launch plan of paged attention and its entry point, for a cache of the token
// rows' type and (FP4) of 4-bit values.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <map>
#include <mutex>
#include <string>

#include "dflash2.h"
#include "host.hpp"
#include "attention.hpp"
#include "attention_fp4.hpp"
#include "target_host.hpp"

namespace df2 {
namespace host {

struct AttnPlan {
    int wr = 1;                 // waves of 32 rows in a block
    int bm = 32, kt = 32, gk = 16;
    int wgs = 1, whole = 0;     // workgroups for stretches, or for whole blocks
    int choose = 0, grid = 1;   // the kernel may take whole blocks by itself; workgroups for either
    bool fits = true;           // 32-bit tile numbers
    size_t part = 0, bytes = 0; // workspace: the parts' outputs, all of it
};

// Over a 4-bit cache: blocks of 16 and 32 rows (wr 0 and 1) have a kernel of their own.
// Blocks of 64 rows are bound by the products and the instructions around them, not by
// the bytes, and want two waves a SIMD: four waves a workgroup, two workgroups a compute
// unit (32 contexts of 301 to 12007 tokens, 8 new, 64 / 8 heads: two waves 147 us, four
// 116, with one stage of 128 keys and weights of one bf16 part 100).
template <bool BF16, int D, typename F>
auto with_fp4_shape(int wr, F&& f) {
    constexpr int RB = AttnTile<BF16, D>::kRow;
    if (wr == 0) return f(FewShape<BF16, D, 16>());
    if (wr == 1) return f(FewShape<BF16, D, 32>());
    if constexpr (RB == 128) {
        if (wr == 2) return f(AttnShape<BF16, D, 2, 2, 2, 2, true>());
        if (wr == 4) return f(AttnShape<BF16, D, 4, 1, 2, 2, true>());
        return f(AttnShape<BF16, D, 8, 1, 2, 2, true>());
    } else if constexpr (RB == 256 && BF16) {
        if (wr == 2) return f(AttnShape<BF16, D, 2, 2, 2, 1, true>());
        if (wr == 4) return f(AttnShape<BF16, D, 4, 1, 2, 2, true>());
        return f(AttnShape<BF16, D, 8, 1, 4, 2, true>());
    } else if constexpr (RB <= 512) {
        if (wr == 2) return f(AttnShape<BF16, D, 2, 2, 1, 2, true>());
        return f(AttnShape<BF16, D, 4, 1, 1, 2, true>());
    } else {
        return f(AttnShape<BF16, D, 4, 1, 1, 2, true>());
    }
}

// The kernels there are: rows (WR waves of 32), key groups, 32-key steps.  A block
// of few rows gets its waves from groups of keys (one row after 1003 tokens, event
// times: 9.7 us and 6.0 for the join with four groups, 8.8 and 7.4 with one, which
// leaves four times the parts); with 64 rows of head size 128 in bf16 two workgroups
// of two waves a compute unit do as well without groups to meet (128 contexts of a
// thousand tokens 119 + 16 us, two groups 124 + 18, four groups, one workgroup a
// unit, 136 + 11); with many rows each wave reads all keys, and longer tiles meet
// less often (prompt chunks: 128 keys a tile 700 us, 96 712, blocks of 128 rows, two
// a compute unit, 730).
template <bool BF16, int D, bool FP4, typename F>
auto with_shape(int wr, F&& f) {
    constexpr int RB = AttnTile<BF16, D>::kRow;
    if constexpr (FP4) {
        return with_fp4_shape<BF16, D>(wr, f);
    } else if constexpr (RB == 128) {
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
template <bool FP4>
AttnPlan plan_attend(const df2_paged_kv* kv, int max_len) {
    AttnPlan pl;
    const int64_t rows = (int64_t)kv->N * (kv->Hq / kv->Hkv);
    const int64_t seqs = std::min(kv->B, kv->N);
    const int64_t each = (rows + seqs - 1) / seqs;
    int per_cu = 1, threads = 64;
    const auto tiles = [&](int64_t len) { return (len + pl.gk + pl.kt - 1) / pl.kt; };
    for (pl.wr = FP4 && each <= 16 ? 0 : each <= 32 ? 1 : each <= 64 ? 2 : each <= 128 ? 4 : 8;; pl.wr /= 2) {
        with_type(kv, [&](auto bf16, auto d) {
            return with_shape<decltype(bf16)::value, decltype(d)::value, FP4>(pl.wr, [&](auto shape) {
                using S = decltype(shape);
                pl.bm = S::BM;
                pl.kt = S::KT;
                pl.gk = S::kGroupKeys;
                per_cu = S::kResident;
                threads = S::kThreads;
                return 0;
            });
        });
        if (pl.wr <= 1 || seqs * ((each + pl.bm - 1) / pl.bm) * kv->Hkv * tiles(max_len) >= 3 * compute_units()) break;
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

template <bool BF16, int D, bool FP4>
df2_status launch_attend(const AttnPlan& pl, const AttnArgs& a, hipStream_t stream) {
    const df2_status st = with_shape<BF16, D, FP4>(pl.wr, [&](auto shape) {
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
    // workgroups at a boundary: four for parts of up to 32 rows over a 4-bit cache, sixteen
    const auto join = [&](auto each) {
        constexpr int J = decltype(each)::value;
        hipLaunchKernelGGL((k_attend_join<BF16, D, J>), dim3((unsigned)(J * (pl.wgs - 1))), dim3(kJoinThreads), 0, stream, a);
    };
    using std::integral_constant;
    if constexpr (FP4) {
        if (pl.wr <= 1) join(integral_constant<int, 4>());
        else join(integral_constant<int, 16>());
    } else {
        join(integral_constant<int, 16>());
    }
    return launched("dflash2_paged_attention join launch");
}

template <bool FP4>
size_t attend_workspace(const df2_paged_kv* kv, int32_t max_len) {
    clear_error();
    int len = 0;
    if (check_kv_sizes(kv, FP4) != DF2_OK || plan_length(kv, max_len, &len) != DF2_OK) return 0;
    return kv->B == 0 || kv->N == 0 ? 0 : plan_attend<FP4>(kv, len).bytes;
}

template <bool FP4>
df2_status attend(const df2_paged_kv* kv, const void* q, int64_t q_stride, float scale, int32_t causal, int32_t window,
                  int32_t max_len, void* out, int64_t out_stride, void* workspace, size_t workspace_bytes,
                  hipStream_t stream) {
    clear_error();
    AttnArgs a;
    std::memset(&a, 0, sizeof(a));
    df2_status st = read_kv(kv, &a.kv, FP4);
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
    const AttnPlan pl = plan_attend<FP4>(kv, len);
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
        return launch_attend<decltype(bf16)::value, decltype(d)::value, FP4>(pl, a, stream);
    });
}

}  // namespace host
}  // namespace df2
