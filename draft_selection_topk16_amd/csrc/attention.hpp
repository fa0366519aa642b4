// Attention of each sequence's new tokens over its paged key/value cache.
//
// For a query row x of token t (position ctx + t) and head h
//     o = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale <x, k_j> - max),
// over the keys j it may see: 0 .. ctx + t (causal) or 0 .. ctx + n - 1 of
// the sequence's n new tokens, and not further back than the window.
//
// The G = Hq / Hkv query heads that share a key/value head are rows of one
// product, so the rows of a sequence are (token, head of the group) pairs,
// n * G of them, and a workgroup takes BM = 32 * WR of them against one
// stretch of the keys.  Keys pass once, in tiles of KT, with the running
// maximum and sum of the softmax in fp32.
//
// Both products run transposed, so that no value crosses lanes between them:
//     S^T [keys x rows] = K Q^T      (a lane holds 16 keys of one row)
//     O^T [D x rows]   += V^T P^T    (the row's P values are where the
//                                     product's operand wants them)
// In the 32x32 output tile, lane l holds column l % 32 (a query row), rows
// 8 * (v / 4) + 4 * (l / 32) + v % 4 for v = 0 .. 15.  The second product
// sums over keys in whatever order both operands agree on: a lane's half
// l / 32 takes just the keys it already holds.  The row statistics are then
// per-lane numbers, met across the two halves once a tile.
//
// K and V tiles go from memory straight to LDS, 16 bytes a lane, two stages;
// the 16-byte chunks of a row are permuted by an exclusive-or with bits of
// the row number, so that the operand reads spread over the banks.  V is read
// transposed (ds_read_b64_tr_b16).
//
// A key past the end of the stretch is replaced by its last key and masked:
// a tile holds nothing but keys that some row of the block may see, so that
// what else stands in the pages (NaN included) never meets the product.
#pragma once

#include "common.hpp"

namespace df2 {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Device flags of the paged operators (see dflash2_device_error).
constexpr uint32_t kFlagPage = 8u;      // a page id outside the cache
constexpr uint32_t kFlagLength = 16u;   // a position outside the page table

// The paged cache and the new tokens, as the kernels read them.
struct PagedKv {
    const int32_t* table;   // [B, table_stride] page ids
    const int32_t* ctx;     // [B] tokens in the cache before the new ones
    const int32_t* start;   // [B + 1] first new token of each sequence
    uint32_t* err;
    int64_t page_stride;    // elements from one page to the next
    int B, N, Hq, Hkv;
    int page_shift, num_pages, table_width;
    int64_t table_stride;
};

struct AttnArgs {
    PagedKv kv;
    const void* q;
    const void* k;
    const void* v;
    void* out;
    float* part;            // [nsplit, N * Hq, D] unnormalised outputs of a split
    float* stat;            // [nsplit, N * Hq, 2] its maximum (log2 units) and sum
    int64_t q_stride, out_stride;
    int G, causal, window;
    int bm;                 // rows of a block
    int split_keys, nsplit; // keys of a split, and the most splits (the last takes what is left)
    float c;                // scale * log2(e)
};

// The new tokens of sequence b, kept inside [0, N).
__device__ __forceinline__ void seq_tokens(const PagedKv& kv, int b, int& s0, int& n) {
    s0 = min(max(kv.start[b], 0), kv.N);
    n = max(min(kv.start[b + 1], kv.N) - s0, 0);
}

// Tokens before the new ones, such that ctx + n stays inside the page table.
// Below -n no position is left that sees a key, so there it stops.
__device__ __forceinline__ int seq_ctx(const PagedKv& kv, int b, int n) {
    const int ctx = max(kv.ctx[b], -n);
    const int64_t cap = (int64_t)kv.table_width << kv.page_shift;
    if ((int64_t)ctx + n > cap) {
        atomicOr(kv.err, kFlagLength);
        return (int)(cap - n);
    }
    return ctx;
}

// The sequence and the block of BM rows that block x of the launch takes: the
// blocks of all sequences stand in a row, and a wave finds the sequence by
// scanning the counts, 64 sequences at a time.  Later blocks of a sequence
// see more keys and come first.
template <int BM>
__device__ __forceinline__ bool find_block(const PagedKv& kv, int G, int x, int& b, int& r0, int& s0,
                                           int& n) {
    const int lane = lane_id();
    int before = 0;
    for (int c0 = 0; c0 < kv.B; c0 += 64) {
        const int i = min(c0 + lane, kv.B - 1);
        int si, ni;
        seq_tokens(kv, i, si, ni);
        const int nb = (c0 + lane < kv.B) ? (ni * G + BM - 1) / BM : 0;
        int incl = nb;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int up = __shfl_up(incl, o);
            incl += lane >= o ? up : 0;
        }
        const uint64_t hit = __ballot(before + incl > x);
        if (hit) {
            const int f = __builtin_ctzll(hit);
            b = c0 + f;
            s0 = __builtin_amdgcn_readlane(si, f);
            n = __builtin_amdgcn_readlane(ni, f);
            const int nbf = __builtin_amdgcn_readlane(nb, f);
            const int at = x - before - (__builtin_amdgcn_readlane(incl, f) - nbf);
            r0 = (nbf - 1 - at) * BM;
            return true;
        }
        before += __builtin_amdgcn_readlane(incl, 63);
    }
    return false;
}

// Splits of a block that sees `keys` keys.
__device__ __forceinline__ int split_count(const AttnArgs& a, int keys) {
    return min(max(1, (keys + a.split_keys - 1) / a.split_keys), a.nsplit);
}

// 16 bytes a lane from memory to LDS: lane l's go to base + 16 l, base the
// same in the wave.  The compiler does not see the write: whoever reads it
// waits for the vector-memory counter and meets a barrier first.
__device__ __forceinline__ void load_to_lds(const void* src, uint32_t lds_base) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %1, off"
        :
        : "s"(lds_base), "v"(src)
        : "memory", "m0");
}

// A value of the lane 32 away.
__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32); }

template <bool BF16, int D>
struct AttnTile {
    static constexpr int kEsz = BF16 ? 2 : 4;
    static constexpr int kRow = D * kEsz;       // bytes of a key
    static constexpr int kChunks = kRow / 16;
    // Permutation of a row's chunks.  K: 16 keys read one chunk each in one go,
    // so they get 16 different places of the 256 bytes that the banks span.
    static __device__ __forceinline__ int swz_k(int row) {
        return kChunks >= 16 ? (row & 15) : ((row >> 1) & 7);
    }
    // V: bf16, four keys of 64 bytes are read in one go; fp32, 128 bytes of
    // two keys that are four apart.
    static __device__ __forceinline__ int swz_v(int row) {
        if constexpr (!BF16) return ((row >> 2) & 1) << 3;
        return kChunks >= 16 ? ((row & 3) << 2) : (((row >> 1) & 1) << 2);
    }
};

// WR waves of 32 rows, WK groups of them on different keys, KS times 32 keys
// a wave in each tile.
template <bool BF16, int D, int WR, int WK, int KS>
struct AttnShape {
    using Tile = AttnTile<BF16, D>;
    static constexpr int kWaves = WR * WK;
    static constexpr int kThreads = 64 * kWaves;
    static constexpr int BM = 32 * WR;
    static constexpr int KT = 32 * WK * KS;
    static constexpr int kTileBytes = KT * Tile::kRow;       // of K, and of V
    static constexpr int kStage = 2 * kTileBytes;
    static constexpr int kLoads = kTileBytes / (1024 * kWaves);
    static constexpr int kMergeBytes = WK > 1 ? kWaves * 32 * D * 4 + kWaves * 256 : 0;
    static constexpr int kLds = 2 * kStage > kMergeBytes ? 2 * kStage : kMergeBytes;
    static_assert(kTileBytes % (1024 * kWaves) == 0, "every wave brings whole loads");
    static_assert(kLds <= 160 * 1024, "LDS of a compute unit");
};

// Four consecutive output values of one row.
template <bool BF16>
__device__ __forceinline__ void store4(void* out, int64_t at, const float (&x)[4]) {
    if constexpr (BF16) {
        // one rounding, to nearest even, of the fp32 result
        bf16x2_t lo = __builtin_convertvector((f32x2_t){x[0], x[1]}, bf16x2_t);
        bf16x2_t hi = __builtin_convertvector((f32x2_t){x[2], x[3]}, bf16x2_t);
        u32x2_t w = {__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
        *reinterpret_cast<u32x2_t*>(reinterpret_cast<uint16_t*>(out) + at) = w;
    } else {
        *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(out) + at) = (f32x4_t){x[0], x[1], x[2], x[3]};
    }
}

template <bool BF16, int D, int WR, int WK, int KS>
__global__ __launch_bounds__(64 * WR * WK) void k_attend(AttnArgs a) {
    using Shape = AttnShape<BF16, D, WR, WK, KS>;
    using Tile = AttnTile<BF16, D>;
    constexpr int RB = Tile::kRow, CH = Tile::kChunks, KT = Shape::KT, BM = Shape::BM;
    constexpr int NL = Shape::kLoads, DB = D / 32;
    extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)lds;

    const PagedKv& kv = a.kv;
    const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
    const int wr = w % WR, wk = w / WR;
    const int half = lane >> 5, col = lane & 31;
    // neighbouring workgroups take different heads: with eight of them, each
    // XCD keeps one head's keys in its L2
    const int lin = blockIdx.x;
    const int h = lin % kv.Hkv, split = (lin / kv.Hkv) % a.nsplit;
    int b, r0, s0, n;
    if (!find_block<BM>(kv, a.G, lin / kv.Hkv / a.nsplit, b, r0, s0, n)) return;
    const int M = n * a.G;
    const int ctx = seq_ctx(kv, b, n);

    // The keys that some row of the block sees, and this split's share of them.
    const int t_lo = r0 / a.G, t_hi = (min(r0 + BM, M) - 1) / a.G;
    const int end = max(a.causal ? ctx + t_hi + 1 : ctx + n, 0);
    const int begin = a.window ? max(ctx + t_lo + 1 - a.window, 0) : 0;
    const int nsplit = split_count(a, end - begin);
    if (split >= nsplit) return;
    const int klo = begin + split * a.split_keys;
    const int khi = split == nsplit - 1 ? end : klo + a.split_keys;

    // This lane's row: row col of the wave's 32 (the last row again past the end).
    const int r = r0 + wr * 32 + col;
    const int rc = min(r, M - 1), t = rc / a.G, head = h * a.G + rc % a.G;
    const int lim = a.causal ? ctx + t + 1 : khi;                 // first key it does not see
    const int low = a.window ? ctx + t + 1 - a.window : 0;        // first key it sees

    // The query rows, as the products want them: half the columns in each lane.
    constexpr int QN = RB / 32;
    u32x4_t qf[QN];
    {
        const char* qp = reinterpret_cast<const char*>(a.q) +
                         ((int64_t)(s0 + t) * a.q_stride + (int64_t)head * D) * Tile::kEsz;
#pragma unroll
        for (int s = 0; s < QN; ++s) qf[s] = *reinterpret_cast<const u32x4_t*>(qp + s * 32 + half * 16);
    }

    f32x16_t o[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int v = 0; v < 16; ++v) o[d][v] = 0.f;
    float m = -INFINITY, l = 0.f;       // l: this lane's half of the row's sum

    // Loads of a tile: load i of wave w covers 1 KB of the K tile and the same
    // of the V tile.
    const int row0 = (w * NL * 64 + lane) / CH;
    const int chunk = lane % CH;
    const int64_t head_off = (int64_t)h << kv.page_shift;
    const int32_t* table = kv.table + (int64_t)b * kv.table_stride;
    auto page_ids = [&](int k0, int (&id)[NL]) {
#pragma unroll
        for (int i = 0; i < NL; ++i) id[i] = table[min(k0 + row0 + i * (64 / CH), khi - 1) >> kv.page_shift];
    };
    uint32_t bad = 0;
    auto load_tile = [&](int k0, int stage, const int (&id)[NL]) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int row = row0 + i * (64 / CH);
            const int key = min(k0 + row, khi - 1);
            const bool ok = (unsigned)id[i] < (unsigned)kv.num_pages;
            bad |= ok ? 0u : 1u;
            const int64_t off = ((int64_t)(ok ? id[i] : 0) * kv.page_stride +
                                 (head_off + (key & ((1 << kv.page_shift) - 1))) * D) * Tile::kEsz;
            const uint32_t at = lds0 + stage * Shape::kStage + (w * NL + i) * 1024;
            load_to_lds(reinterpret_cast<const char*>(a.k) + off + (chunk ^ Tile::swz_k(row)) * 16, at);
            load_to_lds(reinterpret_cast<const char*>(a.v) + off + (chunk ^ Tile::swz_v(row)) * 16,
                        at + Shape::kTileBytes);
        }
    };

    const int ntile = max((khi - klo + KT - 1) / KT, 0);
    if (ntile > 0) {
        int ids[NL];
        page_ids(klo, ids);
        load_tile(klo, 0, ids);
        page_ids(klo + KT, ids);
        for (int it = 0; it < ntile; ++it) {
            const int k0 = klo + it * KT;
            const int stage = it & 1;
            drain_stores();             // vmcnt(0): this wave's part of the tile is in LDS
            __syncthreads();            // everyone's is, and nobody reads the other stage any more
            if (it + 1 < ntile) {
                load_tile(k0 + KT, stage ^ 1, ids);
                page_ids(k0 + 2 * KT, ids);
            }
            const int kw = k0 + wk * KS * 32;          // this wave's first key
            const unsigned char* kt = lds + stage * Shape::kStage;
            const unsigned char* vt = kt + Shape::kTileBytes;

            f32x16_t s[KS];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const int row = (wk * KS + ks) * 32 + col;
                const unsigned char* kp = kt + row * RB;
                const int c0 = (half ^ Tile::swz_k(row)) * 16;
                f32x16_t acc;
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[v] = 0.f;
#pragma unroll
                for (int q = 0; q < QN; ++q) {
                    const u32x4_t kf = *reinterpret_cast<const u32x4_t*>(kp + (c0 ^ (q * 32)));
                    if constexpr (BF16) {
                        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(kf), as_bf16x8(qf[q]), acc, 0, 0, 0);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(kf[e]), __uint_as_float(qf[q][e]),
                                                                      acc, 0, 0, 0);
                    }
                }
                s[ks] = acc;
            }
            // Mask the keys that a row does not see (tiles that every row sees
            // whole need none).
            const int first_lim = a.causal ? ctx + t_lo + 1 : khi;
            const int last_low = a.window ? ctx + t_hi + 1 - a.window : 0;
            if (k0 + KT > min(first_lim, khi) || k0 < last_low) {
                const int top = min(lim, khi);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int v = 0; v < 16; ++v) {
                        const int key = kw + ks * 32 + 8 * (v / 4) + 4 * half + v % 4;
                        s[ks][v] = (key < top && key >= low) ? s[ks][v] : -INFINITY;
                    }
            }
            float mx = s[0][0];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int v = 0; v < 16; ++v) mx = fmaxf(mx, s[ks][v]);
            mx = fmaxf(mx, other_half(mx)) * a.c;
            // The maximum moves only where it grew by more than 2^8, so that most
            // tiles need no rescaling: p stays below 2^8, and p / sum is the same.
            if (__any(mx > m + 8.f)) {
                const float mn = fmaxf(m, mx);
                const float f = m == mn ? 1.f : __builtin_amdgcn_exp2f(m - mn);
                m = mn;
                l *= f;
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int v = 0; v < 16; ++v) o[d][v] *= f;
            }
            const float ms = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                float p[16];
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    p[v] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[ks][v], a.c, -ms));
                    l += p[v];
                }
                const int krow = (wk * KS + ks) * 32;
                if constexpr (BF16) {
                    // P enters the product in bf16 (one rounding, relative 2^-9 at
                    // most a value); the sum keeps the fp32 values
                    const int i = lane & 15, g = lane >> 4;
                    const int tr_key = 4 * (g >> 1) + (i >> 2);
                    const int tr_chunk = 2 * (g & 1) + ((i & 3) >> 1);
                    const unsigned char* vp = vt + (krow + tr_key) * RB + (i & 1) * 8;
                    const int f = Tile::swz_v(krow + tr_key);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        u32x4_t pf;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            pf[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(
                                (f32x2_t){p[8 * j + 2 * e], p[8 * j + 2 * e + 1]}, bf16x2_t));
#pragma unroll
                        for (int d = 0; d < DB; ++d) {
                            typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
                            const unsigned char* at = vp + 16 * j * RB + (((4 * d + tr_chunk) ^ f) * 16);
                            const s16x4_t v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
                            const s16x4_t v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 8 * RB));
                            const s16x8_t vf = __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
                            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, vf), as_bf16x8(pf),
                                                                          o[d], 0, 0, 0);
                        }
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < 16; ++v) {
                        const int row = krow + 8 * (v / 4) + 4 * half + v % 4;
                        const int f = Tile::swz_v(row);
#pragma unroll
                        for (int d = 0; d < DB; ++d) {
                            const float vf = *reinterpret_cast<const float*>(
                                vt + row * RB + ((8 * d + (col >> 2)) ^ f) * 16 + (col & 3) * 4);
                            o[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(vf, p[v], o[d], 0, 0, 0);
                        }
                    }
                }
            }
        }
        if (bad) atomicOr(kv.err, kFlagPage);
    }
    l += other_half(l);

    if constexpr (WK > 1) {
        // The groups' results meet in LDS: statistics first, then each wave's
        // output scaled to the common maximum, summed by group 0.
        float* st = reinterpret_cast<float*>(lds + Shape::kWaves * 32 * D * 4);
        __syncthreads();
        if (half == 0) {
            st[w * 64 + col] = m;
            st[w * 64 + 32 + col] = l;
        }
        __syncthreads();
        float mg = -INFINITY, lg = 0.f;
#pragma unroll
        for (int x = 0; x < WK; ++x) mg = fmaxf(mg, st[(x * WR + wr) * 64 + col]);
#pragma unroll
        for (int x = 0; x < WK; ++x) {
            const float mx = st[(x * WR + wr) * 64 + col];
            lg += mx == -INFINITY ? 0.f : st[(x * WR + wr) * 64 + 32 + col] * __builtin_amdgcn_exp2f(mx - mg);
        }
        const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - mg);
        f32x4_t* mine = reinterpret_cast<f32x4_t*>(lds + w * 32 * D * 4);
        if (wk > 0) {
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    mine[col * (D / 4) + ((8 * d + 2 * v + half) ^ (col & 15))] =
                        (f32x4_t){o[d][4 * v] * f, o[d][4 * v + 1] * f, o[d][4 * v + 2] * f, o[d][4 * v + 3] * f};
        }
        __syncthreads();
        if (wk > 0) return;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
#pragma unroll
                for (int e = 0; e < 4; ++e) o[d][4 * v + e] *= f;
#pragma unroll
                for (int x = 1; x < WK; ++x) {
                    const f32x4_t y = reinterpret_cast<const f32x4_t*>(lds + (x * WR + wr) * 32 * D * 4)
                        [col * (D / 4) + ((8 * d + 2 * v + half) ^ (col & 15))];
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[d][4 * v + e] += y[e];
                }
            }
        m = mg;
        l = lg;
    }
    if (r >= M) return;
    const int64_t grow = (int64_t)(s0 + t) * kv.Hq + head;
    if (nsplit == 1) {
        // a row that sees nothing gives zeros
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        const int64_t at = (int64_t)(s0 + t) * a.out_stride + (int64_t)head * D;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const float y[4] = {o[d][4 * v] * inv, o[d][4 * v + 1] * inv, o[d][4 * v + 2] * inv,
                                    o[d][4 * v + 3] * inv};
                store4<BF16>(a.out, at + 32 * d + 8 * v + 4 * half, y);
            }
    } else {
        const int64_t prow = (int64_t)split * kv.N * kv.Hq + grow;
        if (half == 0) {
            a.stat[2 * prow] = m;
            a.stat[2 * prow + 1] = l;
        }
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const float y[4] = {o[d][4 * v], o[d][4 * v + 1], o[d][4 * v + 2], o[d][4 * v + 3]};
                store4<false>(a.part, prow * D + 32 * d + 8 * v + 4 * half, y);
            }
    }
}

// Joins the splits of each row: sum_s 2^(m_s - m) (o_s, l_s).  A group of D / 4
// lanes takes a row; rows of sequences whose keys made one split are done
// already.
template <bool BF16, int D>
__global__ __launch_bounds__(256) void k_attend_join(AttnArgs a) {
    constexpr int L = D / 4;
    const PagedKv& kv = a.kv;
    const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;
    const int d = (threadIdx.x % L) * 4;
    if (row >= (int64_t)kv.N * kv.Hq) return;
    const int tok = (int)(row / kv.Hq), head = (int)(row % kv.Hq);
    // the token's sequence: the last one that starts at or before it
    int lo = 0, hi = kv.B;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (kv.start[mid + 1] > tok) hi = mid;
        else lo = mid + 1;
    }
    if (lo >= kv.B || tok < kv.start[lo] || tok < 0) return;
    int s0, n;
    seq_tokens(kv, lo, s0, n);
    const int ctx = seq_ctx(kv, lo, n);
    // the block's keys, as k_attend saw them
    const int M = n * a.G, r0 = ((tok - s0) * a.G + head % a.G) / a.bm * a.bm;
    const int t_lo = r0 / a.G, t_hi = (min(r0 + a.bm, M) - 1) / a.G;
    const int end = max(a.causal ? ctx + t_hi + 1 : ctx + n, 0);
    const int begin = a.window ? max(ctx + t_lo + 1 - a.window, 0) : 0;
    const int nsplit = split_count(a, end - begin);
    if (nsplit == 1) return;
    const int64_t rows = (int64_t)kv.N * kv.Hq;
    float m = -INFINITY;
    for (int s = 0; s < nsplit; ++s) m = fmaxf(m, a.stat[2 * (s * rows + row)]);
    float l = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < nsplit; ++s) {
        const int64_t at = s * rows + row;
        const float ms = a.stat[2 * at];
        if (ms == -INFINITY) continue;          // a split of which the row sees nothing
        const float f = __builtin_amdgcn_exp2f(ms - m);
        l += f * a.stat[2 * at + 1];
        const f32x4_t x = *reinterpret_cast<const f32x4_t*>(a.part + at * D + d);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += f * x[e];
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] *= inv;
    store4<BF16>(a.out, (int64_t)tok * a.out_stride + (int64_t)head * D + d, y);
}

}  // namespace df2
