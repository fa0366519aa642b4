// New tokens into a paged key/value cache: the norm of each query and key
// head, the rotation by the token's position and the write, in one pass.
//
//     y = x * rsqrt(mean(x^2) + eps) * w            (per head; w may be absent)
//     (a, b) -> (a cos - b sin, b cos + a sin)      angle = position * freq[i]
//
// over the first `rot` elements of the head, pair i being (i, i + rot / 2) or
// (2 i, 2 i + 1).  Everything is fp32 from the loads to the one rounding at
// the store; the angle is formed and reduced to a turn in fp64, because at
// position 10^5 an fp32 angle is off by 10^-2.
//
// A workgroup takes one token.  D * size / 16 lanes hold a head, 16 bytes each;
// a lane reads its own 16 bytes and its partner's (the same cache lines), so
// the rotation needs no exchange and the norm only the sum of squares.  The
// turns' cosines and sines are made once a token and shared through LDS.
#pragma once

#include "attention.hpp"

namespace df2 {

struct AppendArgs {
    PagedKv kv;
    const void* q;          // may be NULL: keys and values only
    const void* k;
    const void* v;
    void* k_cache;
    void* v_cache;
    void* out_q;
    const void* q_norm;     // [D], may be NULL
    const void* k_norm;
    const double* freq;     // [rot / 2]
    int64_t q_stride, k_stride, v_stride, out_stride;
    int rot, interleaved;
    float eps;
};

// The sequence of new token `tok` (the first whose end lies behind it); false
// if it belongs to none.  The same in the whole wave.
__device__ __forceinline__ bool find_sequence(const PagedKv& kv, int tok, int& b) {
    const int lane = lane_id();
    for (int c0 = 0; c0 < kv.B; c0 += 64) {
        const int i = c0 + lane;
        const int last = i < kv.B ? kv.start[i + 1] : 0;
        const uint64_t hit = __ballot(i < kv.B && last > tok);
        if (hit) {
            b = c0 + __builtin_ctzll(hit);
            return kv.start[b] <= tok;
        }
    }
    return false;
}

// 16 bytes as floats.
template <bool BF16>
struct Vec16 {
    static constexpr int kN = BF16 ? 8 : 4;
    float x[kN];
    __device__ __forceinline__ void load(const void* p) {
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (BF16) {
                x[2 * i] = bf16_lo(w[i]);
                x[2 * i + 1] = bf16_hi(w[i]);
            } else {
                x[i] = __uint_as_float(w[i]);
            }
        }
    }
    __device__ __forceinline__ void store(void* p) const {
        u32x4_t w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (BF16)
                w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){x[2 * i], x[2 * i + 1]}, bf16x2_t));
            else
                w[i] = __float_as_uint(x[i]);
        }
        *reinterpret_cast<u32x4_t*>(p) = w;
    }
};

template <bool BF16, int D>
__global__ __launch_bounds__(256) void k_append(AppendArgs a) {
    constexpr int E = BF16 ? 8 : 4, SZ = BF16 ? 2 : 4;
    constexpr int L = D / E;                // lanes a head
    constexpr int GR = 256 / L;             // heads at once
    __shared__ float turn[D];               // cosines, then sines, of the rot / 2 pairs
    const PagedKv& kv = a.kv;
    const int tid = threadIdx.x, tok = blockIdx.x;
    int b;
    if (!find_sequence(kv, tok, b)) return;
    int s0, n;
    seq_tokens(kv, b, s0, n);
    const int pos = seq_ctx(kv, b, n) + tok - s0;
    const int half = a.rot >> 1;
    if (tid < half) {
        const double rev = (double)pos * a.freq[tid] * 0.15915494309189535;   // 1 / (2 pi): whole turns drop out
        float s, c;
        sincospif(2.f * (float)(rev - rint(rev)), &s, &c);
        turn[tid] = c;
        turn[half + tid] = s;
    }
    // where the cache holds the token; a token without a place is not written
    int page = -1;
    if (pos >= 0) {
        page = kv.table[(int64_t)b * kv.table_stride + (pos >> kv.page_shift)];
        if ((unsigned)page >= (unsigned)kv.num_pages) {
            if (tid == 0) atomicOr(kv.err, kFlagPage);
            page = -1;
        }
    }
    const int64_t place = (int64_t)page * kv.page_stride + (int64_t)(pos & ((1 << kv.page_shift) - 1)) * D;
    __syncthreads();

    const int e0 = (tid % L) * E;
    const int nq = a.q ? kv.Hq : 0;
    const int units = nq + 2 * kv.Hkv;
    for (int u = tid / L; u < units; u += GR) {
        const bool is_q = u < nq, is_v = u >= nq + kv.Hkv;
        const int h = is_q ? u : (is_v ? u - nq - kv.Hkv : u - nq);
        const int64_t stride = is_q ? a.q_stride : (is_v ? a.v_stride : a.k_stride);
        const void* base = is_q ? a.q : (is_v ? a.v : a.k);
        const char* src = reinterpret_cast<const char*>(base) + ((int64_t)tok * stride + (int64_t)h * D) * SZ;
        Vec16<BF16> y;
        y.load(src + e0 * SZ);
        if (!is_v) {
            const void* weight = is_q ? a.q_norm : a.k_norm;
            const bool pairs = !a.interleaved && e0 < a.rot;
            const int p0 = e0 < half ? e0 + half : e0 - half;      // the partner's elements
            Vec16<BF16> z = y;
            if (pairs) z.load(src + p0 * SZ);
            if (weight) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < E; ++i) ss += y.x[i] * y.x[i];
#pragma unroll
                for (int o = 1; o < L; o <<= 1) ss += __shfl_xor(ss, o);
                const float r = 1.f / sqrtf(ss / (float)D + a.eps);
                Vec16<BF16> g;
                g.load(reinterpret_cast<const char*>(weight) + e0 * SZ);
#pragma unroll
                for (int i = 0; i < E; ++i) y.x[i] = y.x[i] * r * g.x[i];
                if (pairs) {
                    g.load(reinterpret_cast<const char*>(weight) + p0 * SZ);
#pragma unroll
                    for (int i = 0; i < E; ++i) z.x[i] = z.x[i] * r * g.x[i];
                }
            }
            if (pairs) {
                const int f0 = e0 < half ? e0 : p0;
                const float sign = e0 < half ? -1.f : 1.f;
#pragma unroll
                for (int i = 0; i < E; ++i)
                    y.x[i] = y.x[i] * turn[f0 + i] + sign * z.x[i] * turn[half + f0 + i];
            } else if (a.interleaved && e0 < a.rot) {
#pragma unroll
                for (int i = 0; i < E; i += 2) {
                    const float c = turn[(e0 + i) >> 1], s = turn[half + ((e0 + i) >> 1)];
                    const float u0 = y.x[i], u1 = y.x[i + 1];
                    y.x[i] = u0 * c - u1 * s;
                    y.x[i + 1] = u1 * c + u0 * s;
                }
            }
        }
        if (is_q) {
            y.store(reinterpret_cast<char*>(a.out_q) + ((int64_t)tok * a.out_stride + (int64_t)h * D + e0) * SZ);
        } else if (page >= 0) {
            char* cache = reinterpret_cast<char*>(is_v ? a.v_cache : a.k_cache);
            y.store(cache + (place + ((int64_t)h << kv.page_shift) * D + e0) * SZ);
        }
    }
}

}  // namespace df2
