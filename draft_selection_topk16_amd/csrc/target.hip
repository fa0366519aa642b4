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
#include "target_host.hpp"
#include "attention_host.hpp"

using namespace df2;
using namespace df2::host;

extern "C" {

size_t dflash2_paged_attention_workspace(const df2_paged_kv* kv, int32_t max_len) {
    return attend_workspace<false>(kv, max_len);
}

df2_status dflash2_paged_attention(const df2_paged_kv* kv, const void* q, int64_t q_stride, float scale,
                                   int32_t causal, int32_t window, int32_t max_len, void* out,
                                   int64_t out_stride, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
    return attend<false>(kv, q, q_stride, scale, causal, window, max_len, out, out_stride, workspace, workspace_bytes,
                         stream);
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
    const df2_status st = read_append(kv, false, q, q_stride, k, k_stride, v, v_stride, q_norm, k_norm, eps, rope_freq, rot,
                                      interleaved, out_q, out_q_stride, &a);
    if (st != DF2_OK || kv->B == 0 || kv->N == 0) return st;
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
