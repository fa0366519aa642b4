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
// Both are one form: with A_i = w_i cos, B_i = -+ w_i' sin (i' the partner of i)
//     y_i = r (x_i A_i + x_i' B_i),    r = 1 / sqrt(mean(x^2) + eps)
// A and B are the same for all query heads of a token and for all its key heads,
// so they are made once a token, in LDS, by all threads, and a head costs two
// products and one scaling an element.  (With the norm's weights and the turn
// applied head by head the kernel was bound by its arithmetic: 120 us for 15
// thousand tokens of 48 heads.)
//
// D * size / 16 lanes hold a head, 16 bytes each; a rotation's partner comes from
// the lane that has it.  A workgroup takes one token, or four neighbouring ones
// where there are enough; with few tokens, several workgroups share one.
//
// Measured: 15 thousand tokens of 32 + 2 * 8 heads of 128 in bf16 85 us for 378 MB,
// 4.4 TB/s, where a large copy reaches 5.1 (eight tokens a workgroup 120 us, one
// 97); a block of 8 tokens 4.4 us, latency of the loads that follow one another:
// sequence, page id, row.
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

// A new token's sequence (the first whose end lies behind it), its first token
// and context; false if the token belongs to none.  The same in the whole
// wave; everything about 64 sequences is loaded at once.
struct TokenSeq {
    int b, s0, ctx;
};
__device__ __forceinline__ bool find_sequence(const PagedKv& kv, int tok, TokenSeq& q) {
    const int lane = lane_id();
    for (int c0 = 0; c0 < kv.B; c0 += 64) {
        const int i = min(c0 + lane, kv.B - 1);
        int s0, n;
        seq_tokens(kv, i, s0, n);
        const int ctx = kv.ctx[i];
        const uint64_t hit = __ballot(c0 + lane < kv.B && s0 + n > tok);
        if (hit) {
            const int f = __builtin_ctzll(hit);
            q.b = c0 + f;
            q.s0 = __builtin_amdgcn_readlane(s0, f);
            q.ctx = __builtin_amdgcn_readlane(ctx, f);
            return q.s0 <= tok;
        }
    }
    return false;
}

// 16 bytes as floats.
template <bool BF16>
struct Vec16 {
    static constexpr int kN = BF16 ? 8 : 4;
    float x[kN];
    __device__ __forceinline__ void load(const void* p) { unpack(*reinterpret_cast<const u32x4_t*>(p)); }
    __device__ __forceinline__ void unpack(u32x4_t w) {
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

template <bool BF16, int D, int T>
__global__ __launch_bounds__(256) void k_append(AppendArgs a) {
    constexpr int E = BF16 ? 8 : 4, SZ = BF16 ? 2 : 4;
    constexpr int L = D / E;                // lanes a head
    constexpr int GR = 256 / L;             // heads at once
    // A and B of the query heads, then of the key heads
    __shared__ __attribute__((aligned(16))) float form[T][2][2][D];
    __shared__ float turn[T][D];            // cosines, then sines, of the rot / 2 pairs
    __shared__ int where[T][3];             // slot of its page, page or -1, sequence or -1
    const PagedKv& kv = a.kv;
    const int tid = threadIdx.x, lane = lane_id(), w = wave_id();
    const int tok0 = blockIdx.x * T;
    const int half = a.rot >> 1;
    const int nq = a.q ? kv.Hq : 0;
    const int units = nq + 2 * kv.Hkv;
    const int u_first = tid / L + GR * blockIdx.y, u_step = GR * gridDim.y;      // this lane's heads
    const int e0 = (tid % L) * E;
    const bool turned = e0 < a.rot, pairs = turned && !a.interleaved;
    const int partner = lane + (pairs ? (e0 < half ? half / E : -(half / E)) : 0);      // whose elements turn with these

    // a head of a token: queries, then keys, then values
    auto source = [&](int tok, int u) {
        const bool is_q = u < nq, is_v = u >= nq + kv.Hkv;
        const int h = is_q ? u : (is_v ? u - nq - kv.Hkv : u - nq);
        const int64_t stride = is_q ? a.q_stride : (is_v ? a.v_stride : a.k_stride);
        const void* base = is_q ? a.q : (is_v ? a.v : a.k);
        return reinterpret_cast<const char*>(base) + ((int64_t)tok * stride + (int64_t)h * D) * SZ;
    };
    // the first heads are on their way while the tokens' places are found
    constexpr int U = 2;
    u32x4_t ahead[U];
    int load_j = 0, load_u = u_first;
    auto load = [&]() {
        u32x4_t x = {0, 0, 0, 0};
        if (load_j < T && tok0 + load_j < kv.N)
            x = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(source(tok0 + load_j, load_u) + e0 * SZ));
        load_u += u_step;
        if (load_u >= units) {
            load_u = u_first;
            ++load_j;
        }
        return x;
    };
#pragma unroll
    for (int i = 0; i < U; ++i) ahead[i] = u_first < units ? load() : u32x4_t{0, 0, 0, 0};

    // the norms' weights for the form's elements that this thread makes
    constexpr int NX = (2 * D + 255) / 256;
    float mine[NX], theirs[NX];
#pragma unroll
    for (int i = 0; i < NX; ++i) {
        const int x = tid + i * 256, e = x % D;
        const void* weight = x < D ? a.q_norm : a.k_norm;
        const int other = a.interleaved ? e ^ 1 : (e < half ? e + half : e - half);
        mine[i] = theirs[i] = 1.f;
        if (weight && x < 2 * D) {
            const int o = e < a.rot ? other : e;
            if constexpr (BF16) {
                mine[i] = bf16_lo(reinterpret_cast<const uint16_t*>(weight)[e]);
                theirs[i] = bf16_lo(reinterpret_cast<const uint16_t*>(weight)[o]);
            } else {
                mine[i] = reinterpret_cast<const float*>(weight)[e];
                theirs[i] = reinterpret_cast<const float*>(weight)[o];
            }
        }
    }

    // a wave a token: its place, and its turns
    for (int j = w; j < T; j += kWaves) {
        TokenSeq q;
        int page = -1, seq = -1;
        int64_t pos = 0;
        bool placed = false, behind = false;
        if (tok0 + j < kv.N && find_sequence(kv, tok0 + j, q)) {
            seq = q.b;
            pos = (int64_t)q.ctx + tok0 + j - q.s0;
            behind = pos >= (int64_t)kv.table_width << kv.page_shift;
            placed = pos >= 0 && !behind;
            if (placed) page = kv.table[(int64_t)q.b * kv.table_stride + (pos >> kv.page_shift)];
        }
        for (int i = lane; i < half; i += 64) {
            const double rev = (double)pos * a.freq[i] * 0.15915494309189535;   // 1 / (2 pi): whole turns drop out
            float s, c;
            sincospif(2.f * (float)(rev - rint(rev)), &s, &c);
            turn[j][i] = c;
            turn[j][half + i] = s;
        }
        // a token without a place in the cache is not written there
        const bool lost = placed && (unsigned)page >= (unsigned)kv.num_pages;
        if (lost) page = -1;
        if (lane == 0) {
            if (lost || behind) atomicOr(kv.err, lost ? kFlagPage : kFlagLength);
            where[j][0] = (int)(pos & ((1 << kv.page_shift) - 1));
            where[j][1] = page;
            where[j][2] = seq;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NX; ++i) {
        const int x = tid + i * 256, kind = x / D, e = x % D;
        if (x >= 2 * D) break;
        const bool first = a.interleaved ? (e & 1) == 0 : e < half;
        const int f = a.interleaved ? e >> 1 : (first ? e : e - half);
#pragma unroll
        for (int j = 0; j < T; ++j) {
            const float c = e < a.rot ? turn[j][f] : 1.f, s = e < a.rot ? turn[j][half + f] : 0.f;
            form[j][kind][0][e] = mine[i] * c;
            form[j][kind][1][e] = first ? -theirs[i] * s : theirs[i] * s;
        }
    }
    __syncthreads();

#pragma unroll 1
    for (int j = 0; j < T; ++j) {
        const int tok = tok0 + j;
        if (tok >= kv.N) return;
        const int page = where[j][1], seq = where[j][2], slot = where[j][0];
        const int64_t place = (int64_t)page * kv.page_stride + (int64_t)slot * D;
#pragma unroll 1
        for (int u = u_first; u < units; u += u_step) {
            const u32x4_t own = ahead[0];
#pragma unroll
            for (int i = 0; i + 1 < U; ++i) ahead[i] = ahead[i + 1];
            ahead[U - 1] = load();
            if (seq < 0) continue;
            Vec16<BF16> y, z;
            y.unpack(own);
            const bool is_q = u < nq, is_v = u >= nq + kv.Hkv;
            const int h = is_q ? u : (is_v ? u - nq - kv.Hkv : u - nq);
            if (!is_v) {
                float r = 1.f;
                if (is_q ? a.q_norm : a.k_norm) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e) ss += y.x[e] * y.x[e];
                    r = 1.f / sqrtf(lanes_sum<L>(ss) * (1.f / D) + a.eps);
                }
                if (a.interleaved) {
#pragma unroll
                    for (int e = 0; e < E; ++e) z.x[e] = y.x[e ^ 1];
                } else {
                    u32x4_t theirs;
#pragma unroll
                    for (int i = 0; i < 4; ++i) theirs[i] = (uint32_t)__shfl((int)own[i], partner);
                    z.unpack(theirs);
                }
                const f32x4_t* fa = reinterpret_cast<const f32x4_t*>(&form[j][is_q ? 0 : 1][0][e0]);
                const f32x4_t* fb = reinterpret_cast<const f32x4_t*>(&form[j][is_q ? 0 : 1][1][e0]);
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                    const f32x4_t x4 = fa[e / 4], y4 = fb[e / 4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y.x[e + i] *= x4[i];
                        if (turned) y.x[e + i] = __builtin_fmaf(z.x[e + i], y4[i], y.x[e + i]);
                        y.x[e + i] *= r;
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
}

}  // namespace df2
