// The paged cache of 4-bit values: appending new tokens, attention over it, and what
// it holds as numbers.  Kernels in append_fp4.hpp, attention_fp4.hpp and fp4.hpp (the
// format); the C ABI is declared in include/dflash2.h.  Nothing here keeps scratch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <map>
#include <mutex>
#include <string>

#include "dflash2.h"
#include "host.hpp"
#include "target_host.hpp"
#include "append_fp4.hpp"
#include "attention_host.hpp"
#include "fp4.hpp"

using namespace df2;
using namespace df2::host;

extern "C" {

df2_status dflash2_kv_append_fp4(const df2_paged_kv* kv, const void* q, int64_t q_stride, const void* k,
                                 int64_t k_stride, const void* v, int64_t v_stride, const void* q_norm,
                                 const void* k_norm, float eps, const double* rope_freq, int32_t rot,
                                 int32_t interleaved, void* out_q, int64_t out_q_stride, hipStream_t stream) {
    clear_error();
    AppendArgs a;
    const df2_status st = read_append(kv, true, q, q_stride, k, k_stride, v, v_stride, q_norm, k_norm, eps, rope_freq, rot,
                                      interleaved, out_q, out_q_stride, &a);
    if (st != DF2_OK || kv->B == 0 || kv->N == 0) return st;
    return with_type(kv, [&](auto bf16, auto d) {
        constexpr int D = decltype(d)::value, heads = 256 / (D / (decltype(bf16)::value ? 8 : 4));
        const int units = (q ? kv->Hq : 0) + 2 * kv->Hkv;
        // workgroups as for dflash2_kv_append
        if (kv->N >= 16 * compute_units())
            hipLaunchKernelGGL((k_append_fp4<decltype(bf16)::value, D, 4>), dim3((unsigned)((kv->N + 3) / 4)), dim3(256), 0,
                               stream, a);
        else
            hipLaunchKernelGGL((k_append_fp4<decltype(bf16)::value, D, 1>),
                               dim3((unsigned)kv->N, kv->N <= compute_units() ? (units + heads - 1) / heads : 1),
                               dim3(256), 0, stream, a);
        return launched("dflash2_kv_append_fp4 launch");
    });
}

df2_status dflash2_kv_unpack_fp4(const df2_paged_kv* kv, void* out_k, void* out_v, hipStream_t stream) {
    clear_error();
    df2_status st = check_kv_sizes(kv, true);
    if (st != DF2_OK) return st;
    if (!kv->k_cache || !kv->v_cache || !out_k || !out_v) return fail_with(DF2_EINVAL, "NULL pointer argument");
    if (!aligned(kv->k_cache, 16) || !aligned(kv->v_cache, 16) || !aligned(out_k, 16) || !aligned(out_v, 16))
        return fail_with(DF2_EINVAL, "caches and outputs must be 16-byte aligned");
    UnpackArgs a;
    a.cache[0] = reinterpret_cast<const uint8_t*>(kv->k_cache);
    a.cache[1] = reinterpret_cast<const uint8_t*>(kv->v_cache);
    a.out[0] = out_k;
    a.out[1] = out_v;
    a.page_stride = kv->page_stride;
    a.Hkv = kv->Hkv;
    a.page_shift = __builtin_ctz((unsigned)kv->page_size);
    a.items = (int64_t)kv->num_pages * kv->Hkv * kv->page_size * (kv->D / 8);
    if (a.items > kMostThreads / 2) return fail_with(DF2_EUNSUPPORTED, "more than 2^34 values in a cache");
    const int64_t in_bytes = (int64_t)(kv->num_pages - 1) * kv->page_stride +
                             (int64_t)kv->Hkv * kv->page_size * (kv->D / 2 + kv->D / 32);
    const int64_t out_bytes = a.items * 8 * (kv->dtype == DF2_BF16 ? 2 : 4);
    const auto meet = [](const void* p, int64_t n, const void* q, int64_t m) {
        return (uintptr_t)p < (uintptr_t)q + (uintptr_t)m && (uintptr_t)q < (uintptr_t)p + (uintptr_t)n;
    };
    for (const void* o : {(const void*)out_k, (const void*)out_v})
        if (meet(o, out_bytes, kv->k_cache, in_bytes) || meet(o, out_bytes, kv->v_cache, in_bytes))
            return fail_with(DF2_EINVAL, "outputs must not overlap the cache");
    if (meet(out_k, out_bytes, out_v, out_bytes)) return fail_with(DF2_EINVAL, "outputs must not overlap each other");
    return with_type(kv, [&](auto bf16, auto d) {
        hipLaunchKernelGGL((k_unpack_fp4<decltype(bf16)::value, decltype(d)::value>),
                           dim3((unsigned)((a.items + kUnpackThreads - 1) / kUnpackThreads), 2), dim3(kUnpackThreads), 0,
                           stream, a);
        return launched("dflash2_kv_unpack_fp4 launch");
    });
}

size_t dflash2_paged_attention_fp4_workspace(const df2_paged_kv* kv, int32_t max_len) {
    return attend_workspace<true>(kv, max_len);
}

df2_status dflash2_paged_attention_fp4(const df2_paged_kv* kv, const void* q, int64_t q_stride, float scale,
                                       int32_t causal, int32_t window, int32_t max_len, void* out, int64_t out_stride,
                                       void* workspace, size_t workspace_bytes, hipStream_t stream) {
    return attend<true>(kv, q, q_stride, scale, causal, window, max_len, out, out_stride, workspace, workspace_bytes,
                        stream);
}

}  // extern "C"
