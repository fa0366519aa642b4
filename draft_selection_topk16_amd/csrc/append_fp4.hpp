// New tokens into a paged cache of 4-bit values: norm and rotation as in kvappend.hpp,
// then each block of 32 elements of a key or value head to codes and a scale
// (fp4.hpp), in one pass.
//
// A code is a decision: a key whose fp32 value lies next to a border of two codes
// would fall on one side or the other with the order in which its sum of squares was
// added.  So keys are normed and rotated in fp64 (their share of the arithmetic; the
// chip has half the rate for it, and the pass over queries, keys and values is bound by
// memory) and rounded once, to 4 bits; a cache does not depend on how a batch was
// split.  Queries are fp32 as in kvappend.hpp; values go through as they are, and
// fp32 is exact for them.
//
// D * size / 16 lanes hold a head, 16 bytes each: a block is 4 of them (bf16) or 8, so its
// largest magnitude is two or three register moves away.
//
// Measured: 15 thousand tokens of 32 + 2 * 8 heads of 128 in bf16 97 us for 331 MB (the
// append of bf16 pages 85 for 378), bound by its vector instructions, a third of them the
// keys' fp64.  (With the form's chunks as they lie, in four banks' way, 107; with the library's
// sine of any angle in place of a fraction of a turn 122.)  A batch's 539 tokens in fp32 5 us.
#pragma once

#include "fp4.hpp"
#include "kvappend.hpp"

namespace df2 {

// Where element e of a row of the form lies in LDS: lanes read LANE neighbouring elements
// each, in 16-byte chunks, and the chunks are permuted so that those of one go lie in
// different banks.
template <typename F, int LANE>
__device__ __forceinline__ int form_place(int e) {
    constexpr int PER = 16 / (int)sizeof(F), N = LANE / PER;       // elements of a chunk, chunks of a lane
    const int chunk = e / PER;
    return (chunk ^ ((chunk >> 4) & (N - 1))) * PER + e % PER;
}

template <bool BF16, int D, int T>
__global__ __launch_bounds__(256) void k_append_fp4(AppendArgs a) {
    constexpr int E = BF16 ? 8 : 4, SZ = BF16 ? 2 : 4;
    constexpr int L = D / E;                // lanes a head
    constexpr int GR = 256 / L;             // heads at once
    constexpr int LB = kFp4Block / E;       // lanes a block
    // y_i = r (x_i A_i + x_i' B_i): A and B of the query heads, and of the key heads
    __shared__ __attribute__((aligned(16))) float form_q[T][2][D];
    __shared__ __attribute__((aligned(16))) double form_k[T][2][D];
    __shared__ double turn[T][D];           // cosines, then sines, of the rot / 2 pairs
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
            // whole turns drop out; 1 / (2 pi) in two parts, so that what is left of the angle
            // is as exact as the angle
            constexpr double kTurn = 0.15915494309189535, kTurnLow = -9.839338337591243e-18;
            const double angle = (double)pos * a.freq[i], whole = rint(angle * kTurn);
            double s, c;
            sincospi(2.0 * (__builtin_fma(angle, kTurn, -whole) + angle * kTurnLow), &s, &c);
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
    for (int x = tid; x < 2 * D; x += 256) {
        const bool is_q = x < D;
        const int e = x % D;
        const void* weight = is_q ? a.q_norm : a.k_norm;
        const bool in = e < a.rot, first = a.interleaved ? (e & 1) == 0 : e < half;
        const int other = !in ? e : a.interleaved ? e ^ 1 : (first ? e + half : e - half);
        const int f = a.interleaved ? e >> 1 : (first ? e : e - half);
        float mine = 1.f, theirs = 1.f;
        if (weight) {
            if constexpr (BF16) {
                mine = bf16_lo(reinterpret_cast<const uint16_t*>(weight)[e]);
                theirs = bf16_lo(reinterpret_cast<const uint16_t*>(weight)[other]);
            } else {
                mine = reinterpret_cast<const float*>(weight)[e];
                theirs = reinterpret_cast<const float*>(weight)[other];
            }
        }
#pragma unroll
        for (int j = 0; j < T; ++j) {
            const double c = in ? turn[j][f] : 1.0, s = in ? turn[j][half + f] : 0.0;
            const double fa = mine * c, fb = first ? -(theirs * s) : theirs * s;
            if (is_q) {
                form_q[j][0][form_place<float, E>(e)] = (float)fa;
                form_q[j][1][form_place<float, E>(e)] = (float)fb;
            } else {
                form_k[j][0][form_place<double, E>(e)] = fa;
                form_k[j][1][form_place<double, E>(e)] = fb;
            }
        }
    }
    __syncthreads();

    const int64_t head_bytes = Fp4Page<D>::bytes(kv.page_shift), scales = Fp4Page<D>::scales(kv.page_shift);
#pragma unroll 1
    for (int j = 0; j < T; ++j) {
        const int tok = tok0 + j;
        if (tok >= kv.N) return;
        const int page = where[j][1], seq = where[j][2], slot = where[j][0];
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
                if (a.interleaved) {
#pragma unroll
                    for (int e = 0; e < E; ++e) z.x[e] = y.x[e ^ 1];
                } else {
                    u32x4_t theirs;
#pragma unroll
                    for (int i = 0; i < 4; ++i) theirs[i] = (uint32_t)__shfl((int)own[i], partner);
                    z.unpack(theirs);
                }
            }
            if (is_q) {
                float r = 1.f;
                if (a.q_norm) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e) ss += y.x[e] * y.x[e];
                    r = 1.f / sqrtf(lanes_sum<L>(ss) * (1.f / D) + a.eps);
                }
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                    const int at = form_place<float, E>(e0 + e);
                    const f32x4_t fa = *reinterpret_cast<const f32x4_t*>(&form_q[j][0][at]);
                    const f32x4_t fb = *reinterpret_cast<const f32x4_t*>(&form_q[j][1][at]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y.x[e + i] *= fa[i];
                        if (turned) y.x[e + i] = __builtin_fmaf(z.x[e + i], fb[i], y.x[e + i]);
                        y.x[e + i] *= r;
                    }
                }
                y.store(reinterpret_cast<char*>(a.out_q) + ((int64_t)tok * a.out_stride + (int64_t)h * D + e0) * SZ);
                continue;
            }
            // numbers over the block's scale, ready for the conversion
            float over[E];
            uint64_t top = 0;
            int power;
            const auto larger = [](double x, double m) {
                // as bits, so that a NaN is larger than all
                return (uint64_t)__double_as_longlong(x) > (uint64_t)__double_as_longlong(m) ? x : m;
            };
            if (is_v) {
                uint32_t most = 0;
#pragma unroll
                for (int e = 0; e < E; ++e) most = max(most, __float_as_uint(y.x[e]) & 0x7FFFFFFFu);
                most = lanes_reduce<LB>(most, [](uint32_t x, uint32_t m) { return max(x, m); });
                top = (uint64_t)__double_as_longlong((double)__uint_as_float(most));
                power = fp4_exponent(top);
                const float inv = __uint_as_float((uint32_t)(127 - power) << 23);
#pragma unroll
                for (int e = 0; e < E; ++e) over[e] = y.x[e] * inv;
            } else {
                double r = 1.0, x[E], most = 0.0;
                if (a.k_norm) {
                    double ss = 0.0;
#pragma unroll
                    for (int e = 0; e < E; ++e) ss += (double)y.x[e] * (double)y.x[e];
                    r = 1.0 / sqrt(lanes_sum<L>(ss) * (1.0 / D) + (double)a.eps);
                }
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    typedef double f64x2_t __attribute__((ext_vector_type(2)));
                    const int at = form_place<double, E>(e0 + e);
                    const f64x2_t fa = *reinterpret_cast<const f64x2_t*>(&form_k[j][0][at]);
                    const f64x2_t fb = *reinterpret_cast<const f64x2_t*>(&form_k[j][1][at]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        x[e + i] = (double)y.x[e + i] * fa[i];
                        if (turned) x[e + i] = __builtin_fma((double)z.x[e + i], fb[i], x[e + i]);
                        x[e + i] *= r;
                        most = larger(fabs(x[e + i]), most);
                    }
                }
                most = lanes_reduce<LB>(most, larger);
                top = (uint64_t)__double_as_longlong(most);
                power = fp4_exponent(top);
                const double inv = __longlong_as_double((long long)(1023 - power) << 52);
#pragma unroll
                for (int e = 0; e < E; ++e) over[e] = to_odd(x[e] * inv);
            }
            if (page < 0) continue;
            uint32_t codes = fp4_pair<0>(0u, over[0], over[1]);
            codes = fp4_pair<1>(codes, over[2], over[3]);
            if constexpr (BF16) {
                codes = fp4_pair<2>(codes, over[4], over[5]);
                codes = fp4_pair<3>(codes, over[6], over[7]);
            }
            uint8_t* to = reinterpret_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + (int64_t)page * kv.page_stride +
                          (int64_t)h * head_bytes;
            uint8_t* at = to + slot * Fp4Page<D>::kCodes + e0 / 2;
            if constexpr (BF16) *reinterpret_cast<uint32_t*>(at) = codes;
            else *reinterpret_cast<uint16_t*>(at) = (uint16_t)codes;
            if (e0 % kFp4Block == 0)
                to[scales + slot * Fp4Page<D>::kScales + e0 / kFp4Block] = (uint8_t)fp4_scale_byte(top, power);
        }
    }
}

}  // namespace df2
