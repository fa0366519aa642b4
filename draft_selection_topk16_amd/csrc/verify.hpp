// Verification of drafted tokens against the target's rows, from given
// uniforms ("DFlash 2: Keep Drafting Parallel", section "A Lightweight Path
// Selector": rejection sampling restores the exact target distribution).
//
// Row t of a sequence holds the target's logits after its first t drafted
// tokens.  With weights w(v) = exp((x(v) - max) / temperature), or the given
// probabilities themselves, p(v) = w(v) / Z, Z = sum w:
//   * draft t is accepted while u_t q_t(d_t) < p_t(d_t), q_t(d) the draft's
//     probability of d;
//   * at the first row a where it is not, the next token comes from
//     max(p_a - q_a, 0), which only differs from p_a at the K candidates;
//   * with every draft accepted, from p_a, a = the number of drafts:
//     the first v whose running sum exceeds u_P times the whole sum.
//
// A token is drawn from weights in fp64, because the drawn index must not depend on
// how sums were rounded (151 thousand boundaries stand an fp32 rounding apart from
// a uniform now and then), by chunks of a few hundred elements: the segment of the
// row first, then the chunk, then the element.
//
// Many rows: launch 1 reads every row once, (max, sum) of each segment in fp32, a
// maximum per lane with rescaling, so one pass does.  Launch 2 works on the one row
// that the draw needs, whose place the partial sums decide: each workgroup sums the
// chunks of a segment, the last to finish draws.  Few rows: launch 1 makes every
// row's chunk sums in fp64 at once, launch 2 only decides and draws.
//
// Measured (launch 1 + launch 2, bf16): 64 sequences of 16 rows of 262144 87 + 26 us,
// launch 1 at 6.2 TB/s; 32 of 8 rows of 151936 17 + 17 us for 78 MB; one of 8 rows,
// the second form, 4.8 + 7.3 us (3.6 + 10.8 in the first).  Launch 2 of the first is
// a chain of short steps (2.3 us to the decision, 1.7 for the segment, 1.1 to the last
// arrival, 1.6, 0.8 and 1.9 for segment, chunk and token of one sequence); the fp64
// weights of 32 rows are some 2.5 of its 17 us.
#pragma once

#include "common.hpp"
#include "lanes.hpp"

namespace df2 {

constexpr uint32_t kFlagDraft = 32u;    // a drafted token outside [0, V)
constexpr uint32_t kFlagNoMass = 64u;   // a target row without weight
constexpr int kVerifySegs = 64;         // most segments of a row

enum VerifyKind { kVerifyLogits = 0, kVerifyProbs = 1, kVerifyArgmax = 2 };

struct VerifyArgs {
    const void* target;         // [B, P + 1, V]
    const int32_t* path;        // [B, P]
    const int32_t* cand;        // [B, P, K]
    const float* prob;          // [B, P, K]
    const int32_t* n_draft;     // [B] or NULL
    const float* u;             // [B, P + 1]
    int32_t* out_tok;           // [B, P + 1]
    int32_t* out_len;           // [B]
    float* out_prob;            // [B, P + 1]
    uint64_t* part;             // [B * (P + 1), nseg] (max, sum) or best word of a segment
    double* seg;                // [B, nseg2] fp64 sums of the drawn row's segments
    double* chunk;              // [B, nseg2, 4 * chunks2] and of their chunks
    float* top;                 // few rows: [B * (P + 1), nseg2] maxima of segments, to which
                                // seg and chunk, then of all rows, are relative
    uint32_t* cnt;              // [B] arrivals, zeroed by launch 1
    uint32_t* err;
    int B, P, V, K;
    int nseg_log, per;          // launch 1: segments of a row (2^nseg_log), vectors of each
    int nseg2, per2;            // launch 2: the same
    int chunks2, rounds2;       // chunks of a wave, rounds of 64 vectors in a chunk
    uint32_t k_inv;             // 2^20 / K + 1: x / K for x < 4096
    float c, c_low;             // log2(e) / temperature, and what fp32 leaves of it (Factor)
    float d_min;                // -1000 / c: logits this far under the maximum weigh nothing
    double c64;
};

// Elements of a row split over segments of `per` whole 16-byte vectors where they
// are aligned (the last ones shorter or empty), the elements before the first and
// behind the last vector to the first and last segment.
template <bool BF16>
struct RowCut {
    static constexpr int kE = BF16 ? 8 : 4, kSz = BF16 ? 2 : 4;
    int head, nv, V, per, nseg;
    __device__ __forceinline__ RowCut(const char* row, int V_, int per_, int nseg_) : V(V_), per(per_), nseg(nseg_) {
        const int off = (int)((uintptr_t)row & 15u);
        head = min(V_, off ? (16 - off) / kSz : 0);
        nv = (V_ - head) / kE;
    }
    __device__ __forceinline__ int first_vec(int s) const { return min(s * per, nv); }
    __device__ __forceinline__ int first(int s) const {
        return s == 0 ? 0 : (s == nseg ? V : head + first_vec(s) * kE);
    }
};

template <bool BF16>
__device__ __forceinline__ float row_value(const char* row, int v) {
    if constexpr (BF16) return bf16_lo(reinterpret_cast<const uint16_t*>(row)[v]);
    else return reinterpret_cast<const float*>(row)[v];
}

template <bool BF16>
__device__ __forceinline__ void unpack16(u32x4_t w, float (&x)[BF16 ? 8 : 4]) {
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

// Weights of a row in fp64.  Logits: 2^y, y = (x - m) log2(e) / temperature, as
// 2^e * 2^(j / 32) * 2^(f / 32), |f| <= 1/2: the 32nds from a table in LDS, the rest
// by the series of 2^(f / 32), whose first term left out is below 1.3 10^-12.  That
// is half the fp64 instructions of a series over a whole octave; the pass over a
// row is bound by them.
constexpr int kExpTable = 32;
template <int KIND>
struct Weights {
    const double* table;        // 2^(j / 32)
    double m, c32;              // the row's maximum, 32 log2(e) / temperature
    __device__ __forceinline__ Weights(const double* t, float m_, double c64) : table(t), m(m_), c32(32.0 * c64) {}
    __device__ __forceinline__ double operator()(float x) const {
        const float one[1] = {x};
        double w[1];
        of(one, w);
        return w[0];
    }
    // N of them side by side: one alone waits for each of its steps.
    template <int N>
    __device__ __forceinline__ void of(const float (&x)[N], double (&w)[N]) const {
        if constexpr (KIND == kVerifyProbs) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = fmax((double)x[i], 0.0);
            return;
        }
        double f[N], root[N];
        int n[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            // the difference first: it is exact next to m; stopped where 2^y is 0
            const double y = fmax(((double)x[i] - m) * c32, -2048.0 * kExpTable);
            const double shifted = y + 0x1.8p52;        // its low word is y to the nearest whole
            n[i] = (int)(uint32_t)(uint64_t)__double_as_longlong(shifted);
            f[i] = y - (shifted - 0x1.8p52);
            root[i] = table[n[i] & (kExpTable - 1)];
        }
        __builtin_amdgcn_sched_barrier(0);
        constexpr double k = 0.69314718055994531 / kExpTable;
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = fma(k * k * k * k / 24.0, f[i], k * k * k / 6.0);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = fma(w[i], f[i], k * k / 2.0);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = fma(w[i], f[i], k);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = fma(w[i], f[i], 1.0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = ldexp(w[i] * root[i], n[i] >> 5);
    }
};
__device__ __forceinline__ void fill_exp_table(double* table) {
    if (threadIdx.x < kExpTable) table[threadIdx.x] = exp2((double)threadIdx.x / kExpTable);
}

// log2(e) / temperature as two floats: its rounding to one would move every weight
// the same way.
struct Factor {
    float c, low;
    // 2^(d * factor): the whole octaves apart, so that the argument's rounding is
    // that of a fraction also where d is large
    __device__ __forceinline__ float exp2_of(float d) const {
        const float y = d * c, n = rintf(y);
        if (!(y > -1000.f)) return 0.f;
        return ldexpf(__builtin_amdgcn_exp2f((y - n) + (__builtin_fmaf(d, c, -y) + d * low)), (int)n);
    }
};

// Running (max, sum) of weights.
struct Lse {
    float m, s;
};
template <int KIND>
__device__ __forceinline__ Lse lse_join(Lse a, Lse b, Factor c) {
    if constexpr (KIND == kVerifyProbs) return {0.f, a.s + b.s};
    const float m = fmaxf(a.m, b.m);
    if (m == -INFINITY) return {m, 0.f};
    return {m, a.s * c.exp2_of(a.m - m) + b.s * c.exp2_of(b.m - m)};
}
// The same over groups of N lanes: the maximum first, then the sums at it.
template <int KIND, int N>
__device__ __forceinline__ Lse lse_lanes(Lse a, Factor c) {
    if constexpr (KIND == kVerifyProbs) return {0.f, lanes_sum<N>(a.s)};
    const float m = lanes_max<N>(a.m);
    const float s = m == -INFINITY ? 0.f : a.s * c.exp2_of(a.m - m);
    return {m, lanes_sum<N>(s)};
}

// Launch 1: one workgroup a segment of a row.
template <bool BF16, int KIND>
__global__ __launch_bounds__(kWG) void k_verify_rows(VerifyArgs a) {
    constexpr int E = RowCut<BF16>::kE, SZ = RowCut<BF16>::kSz, U = 4;
    __shared__ uint64_t red[kWaves];
    const int tid = threadIdx.x, lane = lane_id(), w = wave_id();
    const int64_t row = blockIdx.x >> a.nseg_log;
    const int nseg = 1 << a.nseg_log, seg = (int)(blockIdx.x & (nseg - 1));
    if (seg == 0 && tid == 0 && row % (a.P + 1) == 0) a.cnt[row / (a.P + 1)] = 0;
    const char* rp = reinterpret_cast<const char*>(a.target) + (size_t)row * a.V * SZ;
    const RowCut<BF16> cut(rp, a.V, a.per, nseg);
    const int v0 = cut.first_vec(seg), v1 = cut.first_vec(seg + 1);
    const u32x4_t* vp = reinterpret_cast<const u32x4_t*>(rp + (size_t)cut.head * SZ);

    const Factor factor = {a.c, a.c_low};
    Lse acc = {KIND == kVerifyProbs ? 0.f : -INFINITY, 0.f};
    uint64_t best = 0;
    auto take = [&](const float* x, int n, int at) {
        if constexpr (KIND == kVerifyArgmax) {
            for (int i = 0; i < n; ++i) {
                const uint64_t word = cand_word(key_f32(__float_as_uint(x[i])), (uint32_t)(at + i));
                best = word > best ? word : best;
            }
        } else if constexpr (KIND == kVerifyProbs) {
            for (int i = 0; i < n; ++i) acc.s += fmaxf(x[i], 0.f);
        } else {
            float m = x[0];
            for (int i = 1; i < n; ++i) m = fmaxf(m, x[i]);
            if (m > acc.m) {
                acc.s = acc.m == -INFINITY ? 0.f : acc.s * factor.exp2_of(acc.m - m);
                acc.m = m;
            }
            // The difference first: the product's rounding is relative to it.  It stops
            // at d_min: -inf times the factor's two parts would be NaN.
            const float mm = acc.m == -INFINITY ? 0.f : acc.m;
            float y[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                y[i] = 0.f;
                if (i >= n) continue;
                const float d = fmaxf(x[i] - mm, a.d_min);
                y[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(d, a.c, d * a.c_low));
            }
            // pairs first: an eighth of the roundings at the size of the sum
#pragma unroll
            for (int i = E / 2; i > 0; i /= 2)
#pragma unroll
                for (int k = 0; k < i; ++k) y[k] += y[k + i];
            acc.s += y[0];
        }
    };
    for (int v = v0 + tid; v < v1; v += kWG * U) {
        u32x4_t ld[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            ld[i] = __builtin_nontemporal_load(vp + min(v + i * kWG, v1 - 1));
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (v + i * kWG < v1) {
                float x[E];
                unpack16<BF16>(ld[i], x);
                take(x, E, cut.head + (v + i * kWG) * E);
            }
        }
    }
    if (seg == 0 && tid < cut.head) {
        const float x[1] = {row_value<BF16>(rp, tid)};
        take(x, 1, tid);
    }
    const int tail = cut.head + cut.nv * E + tid;
    if (seg == nseg - 1 && tail < a.V) {
        const float x[1] = {row_value<BF16>(rp, tail)};
        take(x, 1, tail);
    }
    if constexpr (KIND == kVerifyArgmax) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const uint64_t y = __shfl_xor((unsigned long long)best, o);
            best = y > best ? y : best;
        }
    } else {
        acc = lse_lanes<KIND, 64>(acc, factor);
        best = ((uint64_t)__float_as_uint(acc.m) << 32) | __float_as_uint(acc.s);
    }
    if (lane == 0) red[w] = best;
    __syncthreads();
    if (tid == 0) {
        uint64_t out = red[0];
        for (int i = 1; i < kWaves; ++i) {
            if constexpr (KIND == kVerifyArgmax) {
                out = red[i] > out ? red[i] : out;
            } else {
                const Lse y = lse_join<KIND>({__uint_as_float((uint32_t)(out >> 32)), __uint_as_float((uint32_t)out)},
                                             {__uint_as_float((uint32_t)(red[i] >> 32)), __uint_as_float((uint32_t)red[i])}, factor);
                out = ((uint64_t)__float_as_uint(y.m) << 32) | __float_as_uint(y.s);
            }
        }
        a.part[row * nseg + seg] = out;
    }
}

struct VerifyLds {
    float m[72];                // maximum and sum of each row (P + 1 <= 65)
    double s[72];
    uint32_t q[72];             // bits of the draft's probability of each drafted token
    float odds[72];             // p of each drafted token
    int cid[64];                // candidates of the drawn row, and what they lose
    double cut[64];
    double sums[kWG];
    double table[kExpTable];
    int taken, nd, pick, seg;
    uint32_t flag;
    double z, target;
};

// One wave finds the first of n <= 256 values whose running sum exceeds
// `target` and takes the sum before it off `target`.  A target that rounding
// put at or past the whole becomes the last bit of it.  Every lane calls; the
// result is the same in all of them.
__device__ __forceinline__ int find_prefix(const double* sum, int n, double& target) {
    const int lane = lane_id();
    double x[4], own = 0.0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[j] = 4 * lane + j < n ? sum[4 * lane + j] : 0.0;
        own += x[j];
    }
    const double incl = lanes_scan(own);
    const double whole = lane_value(incl, 63);
    if (!(target < whole)) target = whole * (1.0 - 0x1p-40);
    const uint64_t some = __ballot(own > 0.0), hit = __ballot(own > 0.0 && target < incl);
    if (!some) return 0;
    const int f = hit ? __builtin_ctzll(hit) : 63 - __builtin_clzll(some);
    double run = f > 0 ? lane_value(incl, f - 1) : 0.0;
    int at = -1, last = 0;
    double before = run;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const double y = lane_value(x[j], f);
        if (at < 0 && y > 0.0) {
            last = 4 * f + j;
            before = run;
            if (target < run + y) at = last;
        }
        run += y;
    }
    target -= before;
    return at >= 0 ? at : last;
}

// First element of chunk i of a segment; the row's ends go to its first and last.
template <bool BF16>
__device__ __forceinline__ int chunk_first(const RowCut<BF16>& cut, int seg, int vectors, int chunks, int i) {
    if (i == 0) return cut.first(seg);
    if (i == chunks) return cut.first(seg + 1);
    return cut.head + min(cut.first_vec(seg) + i * vectors, cut.first_vec(seg + 1)) * RowCut<BF16>::kE;
}

// A wave's chunks of a segment, `chunks` of them, each `rounds` times 64 vectors side
// by side: their weights summed in fp64, left in out, the whole returned (the same
// in every lane).  Four loads at a time, the next four on their way.
template <bool BF16, int KIND>
__device__ __forceinline__ double chunk_sums(const char* rp, const RowCut<BF16>& cut, int seg, int chunks, int rounds,
                                             const Weights<KIND>& weight, double* out) {
    constexpr int E = RowCut<BF16>::kE, SZ = RowCut<BF16>::kSz, U = 4;
    const int lane = lane_id(), w = wave_id();
    const u32x4_t* vp = reinterpret_cast<const u32x4_t*>(rp + (size_t)cut.head * SZ);
    const int v1 = cut.first_vec(seg + 1), v0 = cut.first_vec(seg) + w * chunks * rounds * 64 + lane;
    const int all = chunks * rounds;
    double s = 0.0, whole = 0.0;
    int in_chunk = 0;
    if (w == 0 && seg == 0 && lane < cut.head) s = weight(row_value<BF16>(rp, lane));
    const bool vectors = cut.first_vec(seg) < v1;
    u32x4_t next[U];
    if (vectors) {
#pragma unroll
        for (int u = 0; u < U; ++u) next[u] = vp[min(v0 + u * 64, v1 - 1)];
    }
    for (int i = 0; i < all; i += U) {
        u32x4_t now[U];
        if (vectors) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                now[u] = next[u];
                next[u] = vp[min(v0 + (i + U + u) * 64, v1 - 1)];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + u >= all) break;
            if (v0 + (i + u) * 64 < v1) {
                float x[E];
                unpack16<BF16>(now[u], x);
                double y[E];
                weight.of(x, y);
#pragma unroll
                for (int d = E / 2; d > 0; d /= 2)
#pragma unroll
                    for (int e = 0; e < d; ++e) y[e] += y[e + d];
                s += y[0];
            }
            if (++in_chunk < rounds) continue;
            // the chunk is complete
            const int tail = cut.head + cut.nv * E + lane;
            if (i + u == all - 1 && w == kWaves - 1 && seg == cut.nseg - 1 && tail < cut.V)
                s += weight(row_value<BF16>(rp, tail));
            s = lanes_sum(s);
            if (lane == 0) xstore(out + w * chunks + (i + u) / rounds, s);
            whole += s;
            s = 0.0;
            in_chunk = 0;
        }
    }
    return whole;
}

// What the decision about the drafts needs beside the rows' sums: loaded before
// those are there.
constexpr int kFirst = 2;               // candidates a thread looks at in the first go
struct Drafts {
    int32_t cid[kFirst], cdraft[kFirst];
    float cq[kFirst];
    int32_t draft;                      // wave 0, lane t: draft t
    float at_draft, u_draft;
};
template <bool BF16>
__device__ __forceinline__ Drafts load_drafts(const VerifyArgs& a, VerifyLds& sm, int b, const char* rows) {
    constexpr int SZ = RowCut<BF16>::kSz;
    const int tid = threadIdx.x, lane = lane_id(), w = wave_id(), P = a.P, K = a.K;
    Drafts d;
#pragma unroll
    for (int i = 0; i < kFirst; ++i) {
        const int x = min(tid + i * kWG, P * K - 1);
        d.cid[i] = a.cand[(int64_t)b * P * K + x];
        d.cq[i] = a.prob[(int64_t)b * P * K + x];
        d.cdraft[i] = a.path[(int64_t)b * P + (int)((uint32_t)x * a.k_inv >> 20)];
    }
    d.draft = -1;
    d.at_draft = d.u_draft = 0.f;
    if (w == 0 && lane < P) {
        d.draft = a.path[(int64_t)b * P + lane];
        d.u_draft = a.u[(int64_t)b * (P + 1) + lane];
        if ((unsigned)d.draft < (unsigned)a.V) d.at_draft = row_value<BF16>(rows + (size_t)lane * a.V * SZ, d.draft);
    }
    if (tid < 72) sm.q[tid] = 0;
    fill_exp_table(sm.table);
    return d;
}

// Which drafts are accepted, from the rows' maxima and sums in LDS: sm.taken of
// sm.nd, and p of each.  Every thread calls, after a barrier; ends with one.
template <bool BF16, int KIND>
__device__ __forceinline__ void decide(const VerifyArgs& a, VerifyLds& sm, int b, const Drafts& d) {
    const int tid = threadIdx.x, lane = lane_id(), w = wave_id(), P = a.P, K = a.K;
    // candidates of a row are distinct: one hit at most (the largest otherwise)
    for (int x = tid, i = 0; x < P * K; x += kWG, ++i) {
        const int64_t at = (int64_t)b * P * K + x;
        const int32_t id = i == 0 ? d.cid[0] : i == 1 ? d.cid[1] : a.cand[at];
        const float q = i == 0 ? d.cq[0] : i == 1 ? d.cq[1] : a.prob[at];
        const int t = (int)((uint32_t)x * a.k_inv >> 20);      // x / K
        const int32_t draft = i == 0 ? d.cdraft[0] : i == 1 ? d.cdraft[1] : a.path[(int64_t)b * P + t];
        if (id == draft) atomicMax(&sm.q[t], __float_as_uint(fmaxf(q, 0.f)));
    }
    __syncthreads();
    // lane t of wave 0 takes draft t
    if (w == 0) {
        const int nd = a.n_draft ? min(max(a.n_draft[b], 0), P) : P;
        bool yes = false;
        if (lane < P) {
            double p = 0.0;
            if ((unsigned)d.draft < (unsigned)a.V) {
                if (sm.s[lane] > 0.0) p = Weights<KIND>(sm.table, sm.m[lane], a.c64)(d.at_draft) / sm.s[lane];
            } else if (lane < nd) {
                atomicOr(a.err, kFlagDraft);
            }
            const float u = (d.u_draft >= 0.f) ? fminf(d.u_draft, 0x1.fffffep-1f) : 0.f;
            yes = lane < nd && (double)u * (double)__uint_as_float(sm.q[lane]) < p;
            sm.odds[lane] = (float)p;
        }
        const uint64_t ok = __ballot(yes);
        const int taken = ~ok ? __builtin_ctzll(~ok) : 64;
        if (lane == 0) {
            sm.taken = min(taken, nd);
            sm.nd = nd;
        }
    }
    __syncthreads();
}

// A refused row's candidates, one a lane of wave 1: id (-1: none), value, and the
// draft's probability.
struct Cand {
    int id;
    float value, q;
};
template <bool BF16>
__device__ __forceinline__ Cand load_cand(const VerifyArgs& a, const VerifyLds& sm, int b, const char* rp) {
    const int lane = lane_id(), t = sm.taken;
    Cand c = {-1, 0.f, 0.f};
    if (wave_id() == 1 && lane < a.K && t < sm.nd) {
        const int64_t at = ((int64_t)b * a.P + t) * a.K + lane;
        c.id = a.cand[at];
        c.q = fmaxf(a.prob[at], 0.f);
        if ((unsigned)c.id < (unsigned)a.V) c.value = row_value<BF16>(rp, c.id);
        else atomicOr(a.err, 2u), c.id = -1;
    }
    return c;
}

// One workgroup draws the sequence's next token and writes its outputs.  mine: the
// sum of segment `lane` of row t (waves 0 and 1); chunk_of(g, i): that of chunk i
// of segment g.  What each candidate loses is min(w, q Z).
template <bool BF16, int KIND, typename ChunkOf>
__device__ __forceinline__ void draw_token(const VerifyArgs& a, VerifyLds& sm, int b, const char* rp,
                                           const RowCut<BF16>& cut, const Weights<KIND>& weight, const Cand& cand,
                                           double mine, ChunkOf chunk_of) {
    constexpr int SZ = RowCut<BF16>::kSz, E = RowCut<BF16>::kE;
    const int tid = threadIdx.x, lane = lane_id(), w = wave_id(), P = a.P, R = P + 1, K = a.K, t = sm.taken;
    const int nch = kWaves * a.chunks2, vectors = a.rounds2 * 64;
    const int64_t row0 = (int64_t)b * R;
    const bool mass = sm.s[t] > 0.0;
    const double z = lanes_sum(mine);       // in waves 0 and 1
    if (w == 1) {
        sm.cid[lane] = cand.id;
        sm.cut[lane] = cand.id >= 0 ? fmin(weight(cand.value), (double)cand.q * z) : 0.0;
    }
    __syncthreads();
    // what the candidates among elements e0 .. e1 - 1 lose (places past K are empty)
    auto loss_in = [&](int e0, int e1) {
        double x = 0.0;
        for (int k0 = 0; k0 < K; k0 += 8) {
            int c[8];
            double y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                c[k] = sm.cid[k0 + k];
                y[k] = sm.cut[k0 + k];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) x += (c[k] >= e0 && c[k] < e1) ? y[k] : 0.0;
        }
        return x;
    };
    if (w == 0) {
        double left = 0.0;
        if (lane < a.nseg2) {
            left = mine - loss_in(cut.first(lane), cut.first(lane + 1));
            left = left > 0.0 ? left : 0.0;
            sm.sums[lane] = left;
        }
        float u = a.u[row0 + P];
        u = (u >= 0.f) ? fminf(u, 0x1.fffffep-1f) : 0.f;
        double target = (double)u * lanes_sum(left);
        wave_sync();
        const int at = find_prefix(sm.sums, a.nseg2, target);
        if (lane == 0) {
            sm.seg = at;
            sm.target = target;
            sm.z = z;
        }
    }
    __syncthreads();
    const int g = sm.seg;
    if (tid < nch) {
        const double x = chunk_of(g, tid) -
                         loss_in(chunk_first(cut, g, vectors, nch, tid), chunk_first(cut, g, vectors, nch, tid + 1));
        sm.sums[tid] = x > 0.0 ? x : 0.0;
    }
    __syncthreads();
    if (w == 0) {
        double target = sm.target;
        const int chosen = g * nch + find_prefix(sm.sums, nch, target), chunks = a.nseg2 * nch;
        const int mine_id = lane < K ? sm.cid[lane] : -1;
        int pick = -1, last = -1;
        double run = 0.0, last_odds = 0.0;
        uint64_t inside = 0;
        // `own` elements of a lane from `first` on, the lanes in order
        auto go_through = [&](const float (&x)[E], int first, int own) {
            double full[E], rest[E], sum = 0.0;
            weight.of(x, full);
#pragma unroll
            for (int e = 0; e < E; ++e) rest[e] = full[e] = e < own ? full[e] : 0.0;
            for (uint64_t c = inside; c; c &= c - 1) {
                const int k = __builtin_ctzll(c), d = sm.cid[k] - first;
                const double loss = sm.cut[k];
#pragma unroll
                for (int e = 0; e < E; ++e) rest[e] = d == e ? fmax(rest[e] - loss, 0.0) : rest[e];
            }
#pragma unroll
            for (int e = 0; e < E; ++e) sum += rest[e];
            const double incl = lanes_scan(sum);
            const uint64_t some = __ballot(sum > 0.0), hit = __ballot(sum > 0.0 && target < run + incl);
            if (some) {
                // the lane's element where its running sum passes the target, or its last
                double acc = run + (incl - sum), p = 0.0;
                int found = -1, end = 0;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    acc += rest[e];
                    if (found < 0 && rest[e] > 0.0) {
                        end = e;
                        p = full[e];
                        if (target < acc) found = e;
                    }
                }
                const int f = hit ? __builtin_ctzll(hit) : 63 - __builtin_clzll(some);
                last = __builtin_amdgcn_readlane(first + end, f);
                last_odds = lane_value(p, f);
                if (hit) pick = last;
            }
            run += lane_value(incl, 63);
        };
        auto one = [&](int i, int n) {      // elements i .. i + n - 1, one a lane
            float x[E] = {};
            if (lane < n) x[0] = row_value<BF16>(rp, i + lane);
            go_through(x, i + lane, lane < n ? 1 : 0);
        };
        // What is left of a range is a difference of two sums: where the candidates in it
        // hold all of its weight and lose all of it, rounding may leave something, and
        // where they hold nearly all, nothing.  What is left of an element is exact.  So
        // where the chosen chunk has no element to draw, the target stands at its border:
        // the first element of the next chunk that has one is drawn, or, with none behind
        // it, the last one before it.  visit(j) is the j-th chunk on that way.
        const auto visit = [&](int j) { return chosen + j < chunks ? chosen + j : chunks - 1 - j; };
        for (int j = 0; mass && pick < 0 && j < chunks;) {
            const int at = visit(j), cg = (int)((unsigned)at / (unsigned)nch), ci = at - cg * nch;
            const int e0 = chunk_first(cut, cg, vectors, nch, ci), e1 = chunk_first(cut, cg, vectors, nch, ci + 1);
            inside = __ballot(mine_id >= e0 && mine_id < e1);
            run = 0.0;
            int i = e0;
            if (i < cut.head) {
                one(i, min(cut.head, e1) - i);
                i = cut.head;
            }
            const int vec_end = min(e1, cut.head + cut.nv * E);
            for (; pick < 0 && i < vec_end; i += 64 * E) {
                const int first = i + lane * E;
                float x[E] = {};
                if (first < vec_end) unpack16<BF16>(*reinterpret_cast<const u32x4_t*>(rp + (size_t)first * SZ), x);
                go_through(x, first, first < vec_end ? E : 0);
            }
            if (pick < 0 && vec_end < e1) one(max(vec_end, e0), e1 - max(vec_end, e0));
            pick = pick < 0 ? last : pick;
            if (pick >= 0) break;
            // on to the next chunk with any weight, 64 looked at at once
            uint64_t some = 0;
            for (++j; j < chunks; j += 64) {
                const int c = visit(min(j + lane, chunks - 1)), of = (int)((unsigned)c / (unsigned)nch);
                some = __ballot(j + lane < chunks && chunk_of(of, c - of * nch) > 0.0);
                if (some) break;
            }
            if (some) j += __builtin_ctzll(some);
            target = chosen + j < chunks ? -1.0 : HUGE_VAL;
        }
        const double odds = last_odds;
        const bool ok = mass && pick >= 0 && pick < a.V;
        if (!ok) {
            pick = 0;
            if (lane == 0) atomicOr(a.err, kFlagNoMass);
        }
        if (lane == 0) {
            sm.pick = pick;
            sm.odds[t] = ok ? (float)(odds / sm.z) : 0.f;
            a.out_len[b] = t + 1;
        }
    }
    __syncthreads();
    if (tid < R) {
        a.out_tok[row0 + tid] = tid < t ? a.path[(int64_t)b * P + tid] : (tid == t ? sm.pick : -1);
        a.out_prob[row0 + tid] = tid <= t ? sm.odds[tid] : 0.f;
    }
}

// Launch 2 (sampling, many rows): nseg2 workgroups a sequence sum the row that its
// draw needs; the last one draws.
template <bool BF16, int KIND>
__global__ __launch_bounds__(kWG) void k_verify_draw(VerifyArgs a) {
    constexpr int SZ = RowCut<BF16>::kSz;
    __shared__ VerifyLds sm;
    const int tid = threadIdx.x, lane = lane_id(), w = wave_id();
    const int b = (int)(blockIdx.x / a.nseg2), seg = (int)(blockIdx.x % a.nseg2);
    const int R = a.P + 1;
    const int64_t row0 = (int64_t)b * R;
    const char* rows = reinterpret_cast<const char*>(a.target) + (size_t)row0 * a.V * SZ;

    // Every row's maximum and sum from its segments (a power of two of them: the
    // lanes of a wave take several rows at once).  All loads go out before any is
    // used.
    const Drafts drafts = load_drafts<BF16>(a, sm, b, rows);
    const int parts = R << a.nseg_log;
    const Factor factor = {a.c, a.c_low};
    for (int x0 = w * 64; x0 < parts; x0 += kWG) {
        const int x = x0 + lane;
        Lse acc = {KIND == kVerifyProbs ? 0.f : -INFINITY, 0.f};
        if (x < parts) {
            const uint64_t y = a.part[(row0 << a.nseg_log) + x];
            acc = {__uint_as_float((uint32_t)(y >> 32)), __uint_as_float((uint32_t)y)};
        }
        switch (a.nseg_log) {
            case 0: break;
            case 1: acc = lse_lanes<KIND, 2>(acc, factor); break;
            case 2: acc = lse_lanes<KIND, 4>(acc, factor); break;
            case 3: acc = lse_lanes<KIND, 8>(acc, factor); break;
            case 4: acc = lse_lanes<KIND, 16>(acc, factor); break;
            case 5: acc = lse_lanes<KIND, 32>(acc, factor); break;
            default: acc = lse_lanes<KIND, 64>(acc, factor); break;
        }
        if (x < parts && (x & ((1 << a.nseg_log) - 1)) == 0) {
            sm.m[x >> a.nseg_log] = acc.m;
            sm.s[x >> a.nseg_log] = acc.s;
        }
    }
    __syncthreads();
    decide<BF16, KIND>(a, sm, b, drafts);

    // This segment of row t.  The candidates, for the workgroup that will draw, are
    // on their way meanwhile.
    const int t = sm.taken;
    const Weights<KIND> weight(sm.table, sm.m[t], a.c64);
    const char* rp = rows + (size_t)t * a.V * SZ;
    const RowCut<BF16> cut(rp, a.V, a.per2, a.nseg2);
    const Cand cand = load_cand<BF16>(a, sm, b, rp);
    const int nch = kWaves * a.chunks2;
    double* chunks = a.chunk + (int64_t)b * a.nseg2 * nch;
    const double s = chunk_sums<BF16, KIND>(rp, cut, seg, a.chunks2, a.rounds2, weight, chunks + (int64_t)seg * nch);
    if (lane == 0) sm.sums[w] = s;
    __syncthreads();
    if (tid == 0) xstore(a.seg + (int64_t)b * a.nseg2 + seg, sm.sums[0] + sm.sums[1] + sm.sums[2] + sm.sums[3]);
    if (!block_arrive_last(&a.cnt[b], (uint32_t)a.nseg2, &sm.flag)) return;

    const double mine = w <= 1 && lane < a.nseg2 ? xload(a.seg + (int64_t)b * a.nseg2 + lane) : 0.0;
    draw_token<BF16, KIND>(a, sm, b, rp, cut, weight, cand, mine,
                           [&](int g, int i) { return xload(chunks + (int64_t)g * nch + i); });
}

// Few rows: launch 1 makes the chunk sums of every row in fp64, a segment's
// relative to its own maximum, which the workgroup finds first, the segment in
// registers (at most kHold vectors a lane).
constexpr int kHold = 4;
template <bool BF16, int KIND>
__global__ __launch_bounds__(kWG) void k_verify_sums(VerifyArgs a) {
    constexpr int E = RowCut<BF16>::kE, SZ = RowCut<BF16>::kSz;
    __shared__ double table[kExpTable], sums[kWaves];
    __shared__ float most[kWaves];
    const int tid = threadIdx.x, lane = lane_id(), w = wave_id();
    const int64_t row = blockIdx.x / a.nseg2;
    const int seg = (int)(blockIdx.x % a.nseg2);
    const char* rp = reinterpret_cast<const char*>(a.target) + (size_t)row * a.V * SZ;
    const RowCut<BF16> cut(rp, a.V, a.per2, a.nseg2);
    const u32x4_t* vp = reinterpret_cast<const u32x4_t*>(rp + (size_t)cut.head * SZ);
    const int v1 = cut.first_vec(seg + 1), v0 = cut.first_vec(seg) + w * a.chunks2 * 64 + lane;

    float x[kHold][E], head = -INFINITY, tail = -INFINITY;
    u32x4_t ld[kHold];
#pragma unroll
    for (int i = 0; i < kHold; ++i)
        if (i < a.chunks2 && v0 + i * 64 < v1) ld[i] = __builtin_nontemporal_load(vp + v0 + i * 64);
    if (w == 0 && seg == 0 && lane < cut.head) head = row_value<BF16>(rp, lane);
    const int last = cut.head + cut.nv * E + lane;
    if (w == kWaves - 1 && seg == cut.nseg - 1 && last < a.V) tail = row_value<BF16>(rp, last);
    fill_exp_table(table);
    float m = fmaxf(head, tail);
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        if (i < a.chunks2 && v0 + i * 64 < v1) {
            unpack16<BF16>(ld[i], x[i]);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) x[i][e] = -INFINITY;        // weighs nothing, of either kind
        }
#pragma unroll
        for (int e = 0; e < E; ++e) m = fmaxf(m, x[i][e]);
    }
    m = lanes_max(m);
    if (lane == 0) most[w] = m;
    __syncthreads();
    m = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
    const Weights<KIND> weight(table, m, a.c64);
    const int64_t at = row * a.nseg2 + seg;
    double whole = 0.0;
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        if (i >= a.chunks2) break;
        double y[E];
        weight.of(x[i], y);
#pragma unroll
        for (int d = E / 2; d > 0; d /= 2)
#pragma unroll
            for (int e = 0; e < d; ++e) y[e] += y[e + d];
        double s = y[0];
        if (i == 0 && w == 0 && seg == 0) s += weight(head);
        if (i == a.chunks2 - 1 && w == kWaves - 1 && seg == cut.nseg - 1) s += weight(tail);
        s = lanes_sum(s);
        if (lane == 0) a.chunk[(at * kWaves + w) * a.chunks2 + i] = s;
        whole += s;
    }
    if (lane == 0) sums[w] = whole;
    __syncthreads();
    if (tid == 0) {
        a.top[at] = m;
        a.seg[at] = sums[0] + sums[1] + sums[2] + sums[3];
    }
}

// Launch 2 of few rows: one workgroup a sequence.
template <bool BF16, int KIND>
__global__ __launch_bounds__(kWG) void k_verify_pick(VerifyArgs a) {
    constexpr int SZ = RowCut<BF16>::kSz;
    __shared__ VerifyLds sm;
    __shared__ double scaled[65 * kVerifySegs];     // sums of the rows' segments, relative to the row's maximum
    const int lane = lane_id(), w = wave_id(), b = (int)blockIdx.x, R = a.P + 1;
    const int64_t row0 = (int64_t)b * R;
    const char* rows = reinterpret_cast<const char*>(a.target) + (size_t)row0 * a.V * SZ;
    const Drafts drafts = load_drafts<BF16>(a, sm, b, rows);
    __syncthreads();
    constexpr int U = 4;                            // rows of a wave on their way at once
    for (int r0 = w; r0 < R; r0 += kWaves * U) {
        float m[U];
        double s[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int r = r0 + i * kWaves;
            const bool live = r < R && lane < a.nseg2;
            const int64_t at = (row0 + (live ? r : 0)) * a.nseg2 + (live ? lane : 0);
            m[i] = a.top[at];
            s[i] = a.seg[at];
            if (!live) {
                m[i] = -INFINITY;
                s[i] = 0.0;
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int r = r0 + i * kWaves;
            if (r >= R) break;
            const float most = lanes_max(m[i]);
            double y = s[i];
            if constexpr (KIND != kVerifyProbs) y *= Weights<KIND>(sm.table, most, a.c64)(m[i]);
            scaled[r * kVerifySegs + lane] = y;
            const double z = lanes_sum(y);
            if (lane == 0) {
                sm.m[r] = most;
                sm.s[r] = z;
            }
        }
    }
    __syncthreads();
    decide<BF16, KIND>(a, sm, b, drafts);
    const int t = sm.taken;
    const Weights<KIND> weight(sm.table, sm.m[t], a.c64);
    const char* rp = rows + (size_t)t * a.V * SZ;
    const RowCut<BF16> cut(rp, a.V, a.per2, a.nseg2);
    const Cand cand = load_cand<BF16>(a, sm, b, rp);
    const int64_t at = (row0 + t) * a.nseg2;
    draw_token<BF16, KIND>(a, sm, b, rp, cut, weight, cand, w <= 1 ? scaled[t * kVerifySegs + lane] : 0.0,
                           [&](int g, int i) {
                               const double x = a.chunk[(at + g) * kWaves * a.chunks2 + i];
                               return KIND == kVerifyProbs ? x : x * weight(a.top[at + g]);
                           });
}

// Launch 2 at temperature 0: a draft is accepted while it is its row's best
// token; the next token is the best of the row after the last accepted one.
template <bool BF16>
__global__ __launch_bounds__(kWG) void k_verify_best(VerifyArgs a) {
    __shared__ int best[72];
    const int tid = threadIdx.x, lane = lane_id(), w = wave_id();
    const int b = (int)blockIdx.x, P = a.P, R = P + 1;
    const int64_t row0 = (int64_t)b * R;
    for (int t = w; t < R; t += kWaves) {
        uint64_t x = lane < (1 << a.nseg_log) ? a.part[((row0 + t) << a.nseg_log) + lane] : 0;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const uint64_t y = __shfl_xor((unsigned long long)x, o);
            x = y > x ? y : x;
        }
        if (lane == 0) best[t] = (int)cand_index(x);
    }
    __syncthreads();
    if (w != 0) return;
    const int nd = a.n_draft ? min(max(a.n_draft[b], 0), P) : P;
    bool yes = false;
    if (lane < P) {
        const int32_t d = a.path[(int64_t)b * P + lane];
        if ((unsigned)d >= (unsigned)a.V && lane < nd) atomicOr(a.err, kFlagDraft);
        yes = lane < nd && d == best[lane];
    }
    const uint64_t ok = __ballot(yes);
    const int t = min(~ok ? __builtin_ctzll(~ok) : 64, nd);
    if (lane == 0) a.out_len[b] = t + 1;
    for (int i = lane; i < R; i += 64) {
        a.out_tok[row0 + i] = i <= t ? best[i] : -1;
        a.out_prob[row0 + i] = i <= t ? 1.f : 0.f;
    }
}

}  // namespace df2
