// Attention of few rows over a 4-bit paged cache (fp4.hpp): single tokens and short
// blocks, R = 16 or 32 rows (tokens times heads of a key/value head) a workgroup.
//
// What bounds these is the pass over the cache, a quarter of the bytes of a bf16 one, so
// what is done to a byte on its way has four times the weight: no tile of bf16 in LDS,
// no barrier a tile.  A workgroup's four waves take different keys, 32 at a time, and
// meet at the end.
//
//   S^T [keys x rows] = K Q^T: a lane's share of a key is a stretch of D R / 64
//     neighbouring elements, whole or half blocks with one scale each, so codes go from
//     memory to registers as they lie there and become bf16, scaled, by one conversion
//     for two.  Q has the same share in the same order.
//   O^T [D x rows] += V^T P^T: wants keys side by side where the codes lie by columns,
//     and their scales differ from key to key.  So each wave makes its keys' values
//     bf16, scaled, as they lie, in a part of LDS of its own, and reads them transposed
//     (ds_read_b64_tr_b16): no barrier, a wave's LDS operations stay in order.  (Codes
//     transposed by ds_read_b64_tr_b4, with the scales subtracted from the exponents of P,
//     have a quarter of the LDS traffic but 100 vector instructions more for 16 rows and 64
//     keys: 4 x 131 thousand keys 92 us, and 90 when this one was as new.)
//
// fp32 calls split queries and probabilities into three bf16 numbers each, 24 bits, so that
// three bf16 products stand for each fp32 one (which run at a sixteenth of the rate);
// bf16 calls split the probabilities into two, as k_attend does.
//
// Keys that no row sees (around the stretch's ends) may hold anything: their scores are
// replaced by -inf, their value scales by 1.
//
// Measured (head size 128, bf16, 32 / 8 heads; passes with their join): 4 tokens after 65 to
// 131 thousand 84 us for 428 MB, 6.4 TB/s while keys stream; one after 1003 9.8 us (6.7 and
// 2.8), latency; blocks of 8 (32 rows) after as many 121 us, bound by vector instructions:
// of some 500 for 64 keys and 32 rows the weights take 300.
#pragma once

#include "attention.hpp"
#include "fp4.hpp"

namespace df2 {

typedef int i32x2_t __attribute__((ext_vector_type(2)));

template <bool BF16, int D, int R>
__global__ void k_attend_fp4(AttnArgs a);

template <bool BF16, int D, int R>
struct FewShape {
    static constexpr auto kernel() { return &k_attend_fp4<BF16, D, R>; }
    // keys of a wave at a time (64 would not leave registers for two waves a SIMD)
    static constexpr int kWaves = 4, kThreads = 256, kWaveKeys = 32;
    static constexpr int BM = R, KT = kWaveKeys * kWaves;
    static constexpr int kGroupKeys = 16;               // keys that surely share a page
    static constexpr int NB = D / kFp4Block;
    static constexpr int kWaveLds = kWaveKeys * D * 2;          // a wave's values
    static constexpr int kMergeBytes = kWaves * (R * D * 4 + 2 * R * 4) + R * 8;
    static constexpr int kLds = kWaves * kWaveLds > kMergeBytes ? kWaves * kWaveLds : kMergeBytes;
    static constexpr int kAllLds = kLds + 4 * kPageIds;
    // workgroups resident on a compute unit, and waves of a SIMD: two where the registers
    // of queries and outputs leave room for them
    static constexpr int kResident = D == 256 ? (BF16 && R == 16 ? 2 : 1) : (BF16 || R == 16 ? 2 : 1);
    static_assert(kResident * kAllLds <= 160 * 1024, "LDS of a compute unit");
    static_assert(KT <= kPageIds / 2, "a tile's pages fit the list");
};

// Splits numbers into bf16 parts, largest first, each the nearest to what is left: part i
// of pair j at p[i][j].
template <int PARTS, int N>
__device__ __forceinline__ void split_into_parts(float (&x)[N], uint32_t (&p)[PARTS][N / 2]) {
#pragma unroll
    for (int i = 0; i < PARTS; ++i)
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            p[i][j] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){x[2 * j], x[2 * j + 1]}, bf16x2_t));
            if (i + 1 < PARTS) {
                x[2 * j] -= bf16_lo(p[i][j]);
                x[2 * j + 1] -= bf16_hi(p[i][j]);
            }
        }
}

template <int R>
struct FewTile;
template <>
struct FewTile<16> {
    using Acc = f32x4_t;
    static __device__ __forceinline__ Acc mul(u32x4_t x, u32x4_t y, Acc z) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(x), as_bf16x8(y), z, 0, 0, 0);
    }
};
template <>
struct FewTile<32> {
    using Acc = f32x16_t;
    static __device__ __forceinline__ Acc mul(u32x4_t x, u32x4_t y, Acc z) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(x), as_bf16x8(y), z, 0, 0, 0);
    }
};

template <bool BF16, int D, int R>
__global__ __launch_bounds__(256, (FewShape<BF16, D, R>::kResident)) void k_attend_fp4(AttnArgs a) {
    using Shape = FewShape<BF16, D, R>;
    using Tile = FewTile<R>;
    using Acc = typename Tile::Acc;
    constexpr int NB = Shape::NB, KT = Shape::KT, WK = Shape::kWaves;
    constexpr int LK = 64 / R;              // lanes that share a key: each has D / LK elements
    constexpr int WKEYS = Shape::kWaveKeys, NT = WKEYS / R, NG = WKEYS / 16;     // key tiles of a wave, groups of 16
    constexpr int NV = NB * WKEYS / 64;     // loads of its values
    constexpr int AV = R * R / 64;          // accumulator values a lane: 4 or 16
    constexpr int SH = D / LK;              // elements of a lane's share
    constexpr int KW = SH / 8;              // its words of codes, products over it
    constexpr int OT = D / R;               // output tiles
    constexpr int QP = BF16 ? 1 : 3, PP = BF16 ? 2 : 3;
    extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];

    const PagedKv& kv = a.kv;
    const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
    const int g = lane / R, col = lane % R;

    // its stretch of the line, as in k_attend
    LaneSeq seqs;
    const Cut cut = cut_work<Shape>(a, seqs);
    const bool blocks_whole = cut.whole;
    int wg = blockIdx.x;
    if (!blocks_whole && cut.wgs % 8 == 0 && wg < cut.wgs)
        wg = (int)(blockIdx.x % 8) * (cut.wgs / 8) + (int)(blockIdx.x / 8);
    int32_t* split = a.split + 8 * wg;
    if (a.join && wg < a.wgs && (blocks_whole || wg >= cut.wgs) && threadIdx.x == 0) split[0] = -1;
    if (wg >= cut.wgs) return;
    int line = cut.first(wg), h = 0;
    const int start = line, stop = cut.first(wg + 1);
    Place at;
    at.j = at.blocks = 0;

    unsigned char* const mine = lds + w * Shape::kWaveLds;      // this wave's values
    int32_t* const ids = reinterpret_cast<int32_t*>(lds + Shape::kLds);
    const int64_t head_bytes = Fp4Page<D>::bytes(kv.page_shift), scales_at = Fp4Page<D>::scales(kv.page_shift);
    const int page_mask = (1 << kv.page_shift) - 1;
    // Values in LDS: a key's row of 2 D bytes, its 16-byte chunks permuted so that what 32
    // lanes read in one go, 8 rows of two chunks or 4 of four, lies in all banks.  Writes still
    // meet: eight cycles of conflicts each in 4 contexts of 65 to 131 thousand tokens, 39% of
    // the cycles that the LDS works.
    const auto swz = [](int row) {
        const int far = (row >> 3 & 1) | (row >> 1 & 2);        // bits 2 and 3 of the row, swapped
        return D == 64 ? (row >> 1 & 1) << 2 | far : (row & 3) << 2 | far;
    };
    // the key, of the 32, and the block of load i of the values
    constexpr int KL = 64 / NB;             // keys of a load
    const auto lane_key = [&](int i) {
        const int k = lane / NB;            // of KL
        if constexpr (KL == 16) return i * KL + (k & 3) * 4 + (k >> 2);
        else return i * KL + k;
    };

    while (line < stop) {
        if (blocks_whole) {
            h = line % kv.Hkv;
            if (!find_place<Shape>(a, seqs, blocks_whole, line / kv.Hkv, at)) return;
            at.first = line - h * cut.head_tiles;       // the block is the whole stretch
        } else if (at.j + 1 < at.blocks) {
            at.first += at.k.tiles;         // the next block of the sequence
            ++at.j;
            at.k = block_keys<Shape>(a, at.ctx, at.n, at.j);
        } else {
            h = (int)((unsigned)line / (unsigned)cut.head_tiles);
            if (!find_place<Shape>(a, seqs, blocks_whole, line - h * cut.head_tiles, at)) return;
        }
        // the same in every lane; said so, they live in scalar registers
        const auto uni = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
        const int b = uni(at.b), s0 = uni(at.s0), n = uni(at.n), ctx = uni(at.ctx), r0 = uni(at.j) * R;
        const int M = n * a.G, head_kv = uni(h), tiles = uni(at.k.tiles);
        const int first = uni(h * cut.head_tiles + at.first);
        const int tile0 = blocks_whole ? 0 : uni(line) - first;
        const int tile1 = blocks_whole ? tiles : min(tiles, stop - first);
        const bool whole = tile0 == 0 && tile1 == tiles;
        if (a.join && !blocks_whole && line == start && threadIdx.x == 0) {
            // the first boundary inside a block tells the join about the block
            const bool cuts = tile0 > 0 && cut.first(wg - 1) <= first;
            split[0] = cuts ? cut.owner(first + tiles - 1) : -1;
            split[1] = head_kv;
            split[2] = s0;
            split[3] = r0;
            split[4] = M;
        }
        line += blocks_whole ? 1 : tile1 - tile0;
        const int t_lo = uni(at.k.t_lo), t_hi = uni(at.k.t_hi);
        const int origin = uni(at.k.origin);
        const int klo = max(uni(at.k.begin), origin + tile0 * KT);
        const int khi = min(uni(at.k.end), origin + tile1 * KT);

        // This lane's row (the last row again past the end), and the keys it sees.
        const int r = r0 + col;
        const int rc = min(r, M - 1), t = div_g(a, rc), head = head_kv * a.G + rc - t * a.G;
        const int lim = a.causal || ctx + t < 0 ? ctx + t + 1 : khi;
        const int low = a.window ? ctx + t + 1 - a.window : 0;

        // Its share of the query row.
        u32x4_t qf[QP][KW];
        {
            const char* qp = reinterpret_cast<const char*>(a.q) +
                             ((int64_t)(s0 + t) * a.q_stride + (int64_t)head * D + g * SH) * (BF16 ? 2 : 4);
#pragma unroll
            for (int i = 0; i < KW; ++i) {
                if constexpr (BF16) {
                    qf[0][i] = *reinterpret_cast<const u32x4_t*>(qp + 16 * i);
                } else {
                    float x[8];
                    uint32_t parts[QP][4];
                    *reinterpret_cast<f32x4_t*>(x) = *reinterpret_cast<const f32x4_t*>(qp + 32 * i);
                    *reinterpret_cast<f32x4_t*>(x + 4) = *reinterpret_cast<const f32x4_t*>(qp + 32 * i + 16);
                    split_into_parts<QP, 8>(x, parts);
#pragma unroll
                    for (int p = 0; p < QP; ++p) qf[p][i] = u32x4_t{parts[p][0], parts[p][1], parts[p][2], parts[p][3]};
                }
            }
        }

        Acc o[OT];
#pragma unroll
        for (int d = 0; d < OT; ++d)
#pragma unroll
            for (int v = 0; v < AV; ++v) o[d][v] = 0.f;
        float m = -INFINITY, l = 0.f;           // l: this lane's part of the row's sum
        bool huge = false;                      // some row's maximum is beyond 2^26

        const int64_t head_at = head_kv * head_bytes;
        const uint8_t* const k_head = reinterpret_cast<const uint8_t*>(a.k) + head_at;
        const uint8_t* const v_head = reinterpret_cast<const uint8_t*>(a.v) + head_at;
        const int32_t* table = kv.table + (int64_t)b * kv.table_stride;

        // What a wave holds of its next keys.
        u32x2_t kc2[NT];                        // key codes: KW words a lane and tile
        u32x4_t kc4[NT][KW < 4 ? 1 : KW / 4];
        uint32_t ks[NT];                        // their scales, a byte a block
        u32x4_t vc[NV];
        uint32_t vs[NV];
        // Loads of the wave's keys from k0 on: their groups of 16, each in one page.
        const auto load_next = [&](int k0, int page0) {
            int64_t group[NG];      // where a group's codes begin, in a head's pages
            int64_t group_scale[NG];
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                const int k = min(max(k0 + 16 * i, klo & ~15), (khi - 1) & ~15), slot = k & page_mask;
                const int64_t page = (int64_t)__builtin_amdgcn_readfirstlane(ids[(k >> kv.page_shift) - page0]) * kv.page_stride;
                group[i] = page + slot * (D / 2);
                group_scale[i] = page + scales_at + slot * NB;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int key = lane_key(i) & 15, blk = lane % NB;
                const uint8_t *p, *s;
                if constexpr (NB == 2) {        // a load is two groups
                    p = v_head + (lane < 32 ? group[2 * i] : group[2 * i + 1]);
                    s = v_head + (lane < 32 ? group_scale[2 * i] : group_scale[2 * i + 1]);
                } else {
                    p = v_head + group[i / (NB / 4)];
                    s = v_head + group_scale[i / (NB / 4)];
                }
                vc[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p + (uint32_t)(key * (D / 2) + blk * 16)));
                vs[i] = s[(uint32_t)(key * NB + blk)];
            }
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const uint8_t *p, *s;
                if constexpr (R == 16) {
                    p = k_head + group[i] + (uint32_t)(col * (D / 2) + g * (SH / 2));
                    s = k_head + group_scale[i] + (uint32_t)(col * NB + g * SH / kFp4Block);
                } else {
                    p = k_head + (col < 16 ? group[2 * i] : group[2 * i + 1]) + (uint32_t)((col & 15) * (D / 2) + g * (SH / 2));
                    s = k_head + (col < 16 ? group_scale[2 * i] : group_scale[2 * i + 1]) + (uint32_t)((col & 15) * NB + g * SH / kFp4Block);
                }
                if constexpr (KW == 2) {
                    kc2[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(p));
                    ks[i] = *s;
                } else {
#pragma unroll
                    for (int x = 0; x < KW / 4; ++x) kc4[i][x] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p + 16 * x));
                    if constexpr (KW == 4) ks[i] = *s;
                    else if constexpr (KW == 8) ks[i] = *reinterpret_cast<const uint16_t*>(s);
                    else ks[i] = *reinterpret_cast<const uint32_t*>(s);
                }
            }
        };

        for (int k_win = origin + tile0 * KT; k_win < khi;) {
            // the tiles whose pages fit the list, and their pages
            const int page0 = max(k_win, klo) >> kv.page_shift;
            const int64_t reach = ((int64_t)(page0 + kPageIds) << kv.page_shift) - k_win;
            const int ntile = (int)min(reach / KT, (int64_t)((khi - k_win + KT - 1) / KT));
            const int last_page = min(khi - 1, k_win + ntile * KT - 1) >> kv.page_shift;
            __syncthreads();
            for (int i = threadIdx.x; i <= last_page - page0; i += Shape::kThreads) {
                int id = table[page0 + i];
                if ((unsigned)id >= (unsigned)kv.num_pages) {
                    atomicOr(kv.err, kFlagPage);
                    id = 0;
                }
                ids[i] = id;
            }
            __syncthreads();
            const int k_first = k_win + w * Shape::kWaveKeys, k_end = min(khi, k_win + ntile * KT);
            if (k_first < k_end) {
                load_next(k_first, page0);
            }
            for (int k0 = k_first; k0 < k_end; k0 += KT) {
                // the values to LDS
                if (k0 < klo || k0 + WKEYS > khi) {
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const int key = k0 + lane_key(i);
                        vs[i] = key >= klo && key < khi ? vs[i] : (uint32_t)kFp4Bias;
                    }
                }
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int row = lane_key(i);
                    unsigned char* to = mine + row * (2 * D);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        *reinterpret_cast<u32x4_t*>(to + ((lane % NB * 4 + c) ^ swz(row)) * 16) = fp4_to_bf16(vc[i][c], fp4_scale(vs[i]));
                }
                wave_sync();
                // the next keys are on their way during all of these
                u32x2_t now2[NT];
                u32x4_t now4[NT][KW < 4 ? 1 : KW / 4];
                uint32_t now_s[NT];
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    now2[i] = kc2[i];
                    now_s[i] = ks[i];
#pragma unroll
                    for (int x = 0; x < (KW < 4 ? 1 : KW / 4); ++x) now4[i][x] = kc4[i][x];
                }
                if (k0 + KT < k_end) load_next(k0 + KT, page0);

                // scores
                Acc s[NT];
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int v = 0; v < AV; ++v) s[i][v] = 0.f;
#pragma unroll
                for (int x = 0; x < KW; ++x)
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        u32x4_t kf;
                        if constexpr (KW == 2) kf = fp4_to_bf16(now2[i][x], fp4_scale(now_s[i]));
                        else kf = fp4_to_bf16(now4[i][x / 4][x % 4], fp4_scale(now_s[i] >> (8 * (x / 4)) & 255));
#pragma unroll
                        for (int p = QP - 1; p >= 0; --p) s[i] = Tile::mul(kf, qf[p][x], s[i]);
                    }

                // masks, the row's maximum and the weights
                const int first_lim = a.causal || ctx + t_lo < 0 ? min(ctx + t_lo + 1, khi) : khi;
                const int last_low = max(a.window ? ctx + t_hi + 1 - a.window : 0, klo);
                if (k0 + WKEYS > first_lim || k0 < last_low) {
                    const int top = min(lim, khi), bottom = max(low, klo);
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int v = 0; v < AV; ++v) {
                            const int key = k0 + R * i + (R == 16 ? 4 * g + v : 8 * (v / 4) + 4 * g + v % 4);
                            s[i][v] = (key < top && key >= bottom) ? s[i][v] : -INFINITY;
                        }
                }
                float mx = s[0][0];
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int v = 0; v < AV; ++v) mx = fmaxf(mx, s[i][v]);
                if constexpr (R == 16) {
                    float x, y;
                    pair_of<16>(mx, x, y);
                    mx = fmaxf(x, y);
                }
                {
                    float x, y;
                    pair_of<32>(mx, x, y);
                    mx = fmaxf(x, y) * a.c;
                }
                // the maximum moves only where it grew by more than 2^8, as in k_attend
                if (__any(mx > m + 8.f)) {
                    const float mn = fmaxf(m, mx);
                    const float f = m == mn ? 1.f : __builtin_amdgcn_exp2f(m - mn);
                    m = mn;
                    huge = __any(fabsf(m) > 0x1p26f && m != -INFINITY);
                    l *= f;
#pragma unroll
                    for (int d = 0; d < OT; ++d)
#pragma unroll
                        for (int v = 0; v < AV; ++v) o[d][v] *= f;
                }
                float ms = m == -INFINITY ? 0.f : m, c = a.c;
                if (__builtin_expect(huge, 0)) {        // as in k_attend
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int v = 0; v < AV; ++v) s[i][v] = scaled_minus(s[i][v], a.c, ms);
                    c = 1.f;
                    ms = 0.f;
                }

                // weights, their parts, and the second product: all keys (R 16), or a tile at a time
                constexpr int HT = R == 16 ? 1 : NT, NE = R == 16 ? 4 * NT : 16;
#pragma unroll
                for (int T = 0; T < HT; ++T) {
                    float e[NE];
#pragma unroll
                    for (int i = 0; i < NE; ++i) {
                        const float x = R == 16 ? s[R == 16 ? i / 4 : 0][i % 4] : s[R == 16 ? 0 : T][R == 16 ? 0 : i];
                        e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x, c, -ms));
                        l += e[i];
                    }
                    uint32_t p[PP][NE / 2];
                    split_into_parts<PP, NE>(e, p);
                    // product u takes 8 of a lane's weights: 32 of the wave's keys (R 16), or 16
#pragma unroll
                    for (int u = 0; u < NE / 8; ++u) {
                        const int base = R == 16 ? 32 * u : 32 * T + 16 * u;    // first of its keys
#pragma unroll
                        for (int d = 0; d < OT; ++d) {
                            typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
                            // four rows of 32 bytes for 16 lanes; the second four keys are 16 or 8 rows on
                            const int row = base + 4 * g + ((lane & 15) >> 2);
                            const int chunk = R == 16 ? 2 * d + ((lane & 3) >> 1) : 4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
                            constexpr int NEXT = R == 16 ? 16 : 8;
                            const s16x4_t v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                (lds_s16x4*)(mine + row * (2 * D) + (chunk ^ swz(row)) * 16 + (lane & 1) * 8));
                            const s16x4_t v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                (lds_s16x4*)(mine + (row + NEXT) * (2 * D) + (chunk ^ swz(row + NEXT)) * 16 + (lane & 1) * 8));
                            const u32x4_t vf = __builtin_bit_cast(u32x4_t, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
                            for (int i = PP - 1; i >= 0; --i) {
                                const u32x4_t pf = {p[i][4 * u], p[i][4 * u + 1], p[i][4 * u + 2], p[i][4 * u + 3]};
                                o[d] = Tile::mul(vf, pf, o[d]);
                            }
                        }
                    }
                }
                wave_sync();        // the values have been read before the next ones are written
            }
            k_win += ntile * KT;
        }
        // a row's sum: over the lanes that share it
        if constexpr (R == 16) {
            float x, y;
            pair_of<16>(l, x, y);
            l = x + y;
        }
        {
            float x, y;
            pair_of<32>(l, x, y);
            l = x + y;
        }
        m = stated_max(m, l);

        // The waves' results meet in LDS, scaled to the rows' common maximum, as in k_attend.
        const int part0 = 2 * wg + (tile0 == 0 ? 1 : 0);        // where a part goes
        float* st = reinterpret_cast<float*>(lds + WK * R * D * 4);
        float* joint = st + WK * 2 * R;         // of each row of the block: maximum, sum
        __syncthreads();
        if (g == 0) {
            st[w * 2 * R + col] = m;
            st[w * 2 * R + R + col] = l;
        }
        __syncthreads();
        float mg = -INFINITY, lg = 0.f;
#pragma unroll
        for (int x = 0; x < WK; ++x) mg = fmaxf(mg, st[x * 2 * R + col]);
#pragma unroll
        for (int x = 0; x < WK; ++x) {
            const float mx = st[x * 2 * R + col];
            lg += mx == -INFINITY ? 0.f : st[x * 2 * R + R + col] * __builtin_amdgcn_exp2f(mx - mg);
        }
        const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - mg);
        f32x4_t* to = reinterpret_cast<f32x4_t*>(lds + w * R * D * 4);
#pragma unroll
        for (int d = 0; d < OT; ++d)
#pragma unroll
            for (int v = 0; v < AV / 4; ++v) {
                const int chunk = R == 16 ? 4 * d + g : 8 * d + 2 * v + g;       // four columns
                to[col * (D / 4) + (chunk ^ (col & 15))] =
                    (f32x4_t){o[d][4 * v] * f, o[d][4 * v + 1] * f, o[d][4 * v + 2] * f, o[d][4 * v + 3] * f};
            }
        if (w == 0 && g == 0) {
            joint[2 * col] = mg;
            joint[2 * col + 1] = lg;
        }
        __syncthreads();
        const int live = min(R, M - r0);
#pragma unroll 1
        for (int x = threadIdx.x; x < live * (D / 4); x += Shape::kThreads) {
            const int row = x / (D / 4), c = x % (D / 4);
            f32x4_t y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < WK; ++k)
                y += reinterpret_cast<const f32x4_t*>(lds + k * R * D * 4)[row * (D / 4) + (c ^ (row & 15))];
            const float lr = joint[2 * row + 1];
            if (whole) {
                // a row that sees nothing gives zeros
                const float inv = lr > 0.f ? 1.f / lr : (lr == 0.f ? 0.f : lr);
                const int rr = r0 + row, tt = div_g(a, rr);
                const float out[4] = {y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv};
                store4<BF16>(a.out, (int64_t)(s0 + tt) * a.out_stride + (int64_t)(head_kv * a.G + rr - tt * a.G) * D + 4 * c, out);
            } else {
                const int64_t prow = (int64_t)part0 * R + row;
                const float out[4] = {y[0], y[1], y[2], y[3]};
                store4<false>(a.part, prow * D + 4 * c, out);
                if (c == 0) {
                    a.stat[2 * prow] = joint[2 * row];
                    a.stat[2 * prow + 1] = lr;
                }
            }
        }
    }
}

}  // namespace df2
