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
//
// Measured (head size 128, bf16 unless said; passes back to back):
//   4 contexts of 65 to 131 thousand tokens, 8 new each, 32 / 8 heads: 244 us for 1.61
//     GB, 6.6 TB/s, where a kernel that only reads reaches 7.1;
//   32 contexts of 301 to 12007 tokens, 8 new each, 64 / 8 heads: 161 us for 816 MB
//     (kernel 153, 5.3 TB/s; join 8): some 20 us are the start, the parts (25 MB) and the end;
//   1 new token after 1003, 32 / 8 heads: 11.1 us (7.7 and 3.4), latency: 1.9 us to the
//     cut, 1.5 to the place, 0.8 for page ids, 0.9 for the first tile;
//   3 drafted blocks in fp32 of head size 64, up to 2049 keys: 14.4 us;
//   prompt chunks (739 GFLOP): 694 us, 1060 TFLOP/s, where a large library product
//     reaches 1373 (690 to 757 us on different cards).  Nothing alone bounds it: with its
//     products only, it takes 565 us (the clock falls to 2.05 GHz under them), LDS loads
//     add 40, operand reads 60, exponentials 90.
#pragma once

#include "common.hpp"
#include "fp4.hpp"
#include "lanes.hpp"

namespace df2 {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Device flags of the paged operators (see dflash2_device_error).
constexpr uint32_t kFlagPage = 8u;      // a page id outside the cache
constexpr int kPageIds = 1024;          // page ids that a workgroup holds at a time
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
    float* part;            // [2 * wgs, bm, D] unnormalised outputs of parts of a block
    float* stat;            // [2 * wgs, bm, 2] their maximum (log2 units) and sum
    int32_t* split;         // [wgs, 8] the block that a workgroup's beginning cuts first
    int64_t q_stride, out_stride;
    int G, causal, window;
    int bm;                 // rows of a block
    int wgs, whole;         // workgroups that take stretches; 1: each takes a whole block
    int cus;                // compute units
    int join;               // there may be parts, and a workspace for them
    int choose;             // blocks enough for the kernel to choose whole ones
    double inv_g;           // 1 / G
    float c;                // scale * log2(e)
};

// The new tokens of sequence b, kept inside [0, N).
__device__ __forceinline__ void seq_tokens(const PagedKv& kv, int b, int& s0, int& n) {
    s0 = min(max(kv.start[b], 0), kv.N);
    n = max(min(kv.start[b + 1], kv.N) - s0, 0);
}

// Tokens before the new ones, such that ctx + n stays inside the page table.
// Below -n no position is left that sees a key, so there it stops.
__device__ __forceinline__ int inside_table(const PagedKv& kv, int ctx, int n) {
    ctx = max(ctx, -n);
    const int64_t cap = (int64_t)kv.table_width << kv.page_shift;
    if ((int64_t)ctx + n > cap) {
        atomicOr(kv.err, kFlagLength);
        return (int)(cap - n);
    }
    return ctx;
}

// ----------------------------------------------------------------------------
// How the work is cut.  The blocks of rows of all sequences stand in a row, each
// as many tiles long as its keys make (one at least), once for every key/value
// head; the workgroups, as many as are resident at once, take equal stretches
// of that line.  So every workgroup streams as many keys as the next whatever
// the lengths of the sequences, and starts once.  A block that falls to one
// workgroup is written at once; of one that lies across a boundary, each
// workgroup leaves its part, and k_attend_join adds them up.  A workgroup has at
// most two such parts: where its stretch begins and where it ends.
// Or each workgroup takes one whole block (`whole`: a block counts as one tile of
// the line): there are no parts to leave and join, and blocks of a head run side by
// side and share its keys in the L2.  So it is with many more blocks than
// workgroups (long chunks: the launch has no join then), and where the lengths make
// it the shorter way (Cut).
// Lengths are in device memory, so each wave finds its place itself, a lane to
// a sequence.
// ----------------------------------------------------------------------------
__device__ __forceinline__ int div_g(const AttnArgs& a, int r) {
    int t = (int)((double)r * a.inv_g);
    t -= t * a.G > r;
    return t + ((t + 1) * a.G <= r);
}

// Block j of a sequence: its rows' tokens and the keys that they see.
struct BlockKeys {
    int t_lo, t_hi, begin, end, origin, tiles;
};
template <typename Shape>
__device__ __forceinline__ BlockKeys block_keys(const AttnArgs& a, int ctx, int n, int j) {
    BlockKeys k;
    k.t_lo = div_g(a, j * Shape::BM);
    k.t_hi = div_g(a, min((j + 1) * Shape::BM, n * a.G) - 1);
    k.end = max(a.causal ? ctx + k.t_hi + 1 : ctx + n, 0);
    k.begin = a.window ? max(ctx + k.t_lo + 1 - a.window, 0) : 0;
    k.origin = k.begin & ~(Shape::kGroupKeys - 1);
    k.tiles = max((int)((unsigned)(k.end - k.origin + Shape::KT - 1) / (unsigned)Shape::KT), 1);
    return k;
}

// Sequences of more blocks than this are gone through by the whole wave, a lane to
// a block; others by their lane.
constexpr int kLaneBlocks = 4;

// A lane's sequence: its tokens, blocks and length on the line, and the tiles of its
// longest block.  falls: the next sequence's tokens do not begin behind it.
struct LaneSeq {
    int s0, n, ctx, blocks, tiles, most;
    bool falls;
};
template <typename Shape>
__device__ __forceinline__ LaneSeq lane_seq(const AttnArgs& a, int c0, bool whole) {
    LaneSeq q = {0, 0, 0, 0, 0, 0, false};
    const int lane = lane_id(), i = c0 + lane;
    if (i < a.kv.B) {
        seq_tokens(a.kv, i, q.s0, q.n);
        q.falls = a.kv.start[i + 1] < a.kv.start[i];
        const int ctx = a.kv.ctx[i];
        if (q.n > 0) q.ctx = inside_table(a.kv, ctx, q.n);     // without new tokens, any length is right
        q.blocks = (int)((unsigned)(q.n * a.G + Shape::BM - 1) / (unsigned)Shape::BM);
    }
    if (whole) {
        q.tiles = q.blocks;
        return q;
    }
    if (q.blocks <= kLaneBlocks)
        for (int j = 0; j < q.blocks; ++j) {
            const int tiles = block_keys<Shape>(a, q.ctx, q.n, j).tiles;
            q.tiles += tiles;
            q.most = max(q.most, tiles);
        }
    for (uint64_t big = __ballot(q.blocks > kLaneBlocks); big; big &= big - 1) {
        const int f = __builtin_ctzll(big);
        const int ctx = __builtin_amdgcn_readlane(q.ctx, f), n = __builtin_amdgcn_readlane(q.n, f);
        const int blocks = __builtin_amdgcn_readlane(q.blocks, f);
        int sum = 0, most = 0;
        for (int j = lane; j < blocks; j += 64) {
            const int tiles = block_keys<Shape>(a, ctx, n, j).tiles;
            sum += tiles;
            most = max(most, tiles);
        }
        sum = __builtin_amdgcn_readlane(lanes_scan(sum), 63);
        most = (int)lanes_max((float)most);         // below 2^24, or near enough
        if (lane == f) {
            q.tiles = sum;
            q.most = most;
        }
    }
    return q;
}

// The stretches: `each` tiles and one more in the first `more` of them.
struct Cut {
    int head_tiles, wgs, each, more;
    bool whole;
    __device__ __forceinline__ int first(int i) const { return i * each + min(i, more); }
    // the workgroup that has tile g
    __device__ __forceinline__ int owner(int g) const {
        const int longer = more * (each + 1);
        return g < longer ? (int)((unsigned)g / (unsigned)(each + 1))
                          : more + (int)((unsigned)(g - longer) / (unsigned)each);
    }
};
template <typename Shape>
__device__ __forceinline__ Cut cut_work(const AttnArgs& a, LaneSeq& q) {
    Cut c;
    c.whole = a.whole;
    c.head_tiles = 0;
    int blocks = 0, most = 0;
    bool fell = false, overlap = false;         // starts descended; sequences with tokens follow
    for (int c0 = 0; c0 < a.kv.B; c0 += 64) {
        q = lane_seq<Shape>(a, c0, c.whole);
        const uint64_t falls = __ballot(q.falls), live = __ballot(q.n > 0);
        // 2 << i: the lanes behind i
        overlap |= fell ? live != 0 : falls && (live & -(2ull << __builtin_ctzll(falls)));
        fell |= falls != 0;
        c.head_tiles += __builtin_amdgcn_readlane(lanes_scan(q.tiles), 63);
        if (a.choose) {
            blocks += __builtin_amdgcn_readlane(lanes_scan(q.blocks), 63);
            most = max(most, __builtin_amdgcn_readfirstlane((int)lanes_max((float)q.most)));
        }
    }
    // Sequences that overlap could make a line of any length, beyond what a tile's
    // number holds: no work then, and a flag.  (Starts behind the last sequence may be 0.)
    if (overlap) {
        if (lane_id() == 0) atomicOr(a.kv.err, kFlagLength);
        blocks = c.head_tiles = 0;
    }
    int all = c.head_tiles * a.kv.Hkv;
    c.wgs = min(a.whole ? (int)gridDim.x : a.wgs, all);
    if (a.choose) {
        // Whole blocks where the longest and half of it on top of the average stay
        // within the average and what parts and their join cost, in tiles: 5 for
        // blocks of 32 rows, 16 for larger ones.  (Times with the join, stretches then
        // whole blocks, head size 128: 16 contexts of a thousand tokens and one row
        // 26 us and 26, 8 of them 21 and 23; 32 of 500, 8 new, 64 / 8 heads, 38 and 27;
        // 32 of a thousand 46 and 44; 128 of them 131 and 117; 64 of 500, 32 new, 66 and
        // 42; one chunk of 2048 tokens without context 95 and 58.)
        const int average = (int)((unsigned)all / (unsigned)max(a.wgs, 1));
        if (blocks * a.kv.Hkv <= (int)gridDim.x && max(most, average + most / 2) <= average + (Shape::BM <= 32 ? 5 : 16)) {
            c.whole = true;
            q.tiles = q.blocks;
            c.head_tiles = blocks;
            all = blocks * a.kv.Hkv;
            c.wgs = all;
        }
    }
    // More than one workgroup a compute unit only with eight tiles for each: shorter
    // stretches leave more parts than they save (event times with 512 workgroups and
    // the join, then with 256: 4 contexts of 25 thousand tokens, 8 new, 16 / 2 heads, 6
    // tiles each, 34 + 14.5 and 34 + 9.8 us; 2 of 4000, 32 new, 32 / 8 heads, 2 tiles,
    // 29 + 16.6 and 25 + 12.8; but 16 such, 16 tiles, 68 + 12.1 and 76 + 12.0).  Parts of
    // 16 rows are small: four tiles there (4-bit cache, 8 heads, one token after 64 thousand,
    // 8 tiles each, 31 us with 256 and 28 with 512; 4 after 4000, 2 tiles, 14.4 and 15.7).
    if (!c.whole && c.wgs > a.cus && all < (Shape::BM == 16 ? 4 : 8) * c.wgs) c.wgs = a.cus;
    c.each = c.wgs > 0 ? (int)((unsigned)all / (unsigned)c.wgs) : 0;
    c.more = all - c.each * c.wgs;
    return c;
}

// A block of rows; first: where it begins on the line of its head.
struct Place {
    int b, s0, n, ctx, blocks, j, first;
    BlockKeys k;
};
// The block that has tile g of a head.  q: the lanes' sequences if there are no
// more than 64.
template <typename Shape>
__device__ __forceinline__ bool find_place(const AttnArgs& a, LaneSeq q, bool whole, int g, Place& p) {
    int before = 0;
    for (int c0 = 0; c0 < a.kv.B; c0 += 64) {
        if (a.kv.B > 64) q = lane_seq<Shape>(a, c0, whole);
        const int incl = lanes_scan(q.tiles);
        const uint64_t hit = __ballot(before + incl > g);
        if (hit) {
            const int f = __builtin_ctzll(hit);
            p.b = c0 + f;
            p.s0 = __builtin_amdgcn_readlane(q.s0, f);
            p.n = __builtin_amdgcn_readlane(q.n, f);
            p.ctx = __builtin_amdgcn_readlane(q.ctx, f);
            p.blocks = __builtin_amdgcn_readlane(q.blocks, f);
            p.first = before + __builtin_amdgcn_readlane(incl - q.tiles, f);
            p.j = 0;
            if (whole) {
                // a later block sees more keys: it goes first
                p.j = p.blocks - 1 - (g - p.first);
                p.first = g;
            } else if (p.blocks > 1) {
                for (int j0 = 0; j0 < p.blocks; j0 += 64) {
                    const int j = j0 + lane_id();
                    const int own = j < p.blocks ? block_keys<Shape>(a, p.ctx, p.n, j).tiles : 0;
                    const int sum = lanes_scan(own);
                    const uint64_t here = __ballot(p.first + sum > g);
                    if (here) {
                        const int l = __builtin_ctzll(here);
                        p.j = j0 + l;
                        p.first += __builtin_amdgcn_readlane(sum - own, l);
                        break;
                    }
                    p.first += __builtin_amdgcn_readlane(sum, 63);
                }
            }
            p.k = block_keys<Shape>(a, p.ctx, p.n, p.j);
            return true;
        }
        before += __builtin_amdgcn_readlane(incl, 63);
    }
    return false;
}

// 16 bytes a lane from memory to LDS: lane l's go to base + 16 l, base the
// same in the wave.  The compiler does not see the write: whoever reads it
// waits for the vector-memory counter and meets a barrier first.  (Nothing else
// here uses m0, which the compiler reserves.)  ONCE: bytes that nobody reads
// again (non-temporal): contexts of 131 thousand tokens, 282 us without and 252 us
// with it.
#define DF2_TO_LDS(NT)                             \
    asm volatile(                                  \
        "s_mov_b32 m0, %0\n\t"                     \
        "s_nop 0\n\t"                              \
        "global_load_lds_dwordx4 %1, off" NT       \
        :                                          \
        : "s"(lds_base), "v"(src)                  \
        : "memory")
template <bool ONCE>
__device__ __forceinline__ void load_to_lds(const void* src, uint32_t lds_base) {
    if constexpr (ONCE) DF2_TO_LDS(" nt");
    else DF2_TO_LDS("");
}
#undef DF2_TO_LDS

// Waits until no more than the loads of min(ahead, A) stages, L each, are in
// flight and this wave's LDS reads are done, then meets the workgroup.
template <int A, int L>
__device__ __forceinline__ void wait_and_meet(int ahead) {
    if (A == 0 || ahead >= A)
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(A * L) : "memory");
    else
        wait_and_meet<A == 0 ? 0 : A - 1, L>(ahead);
}

// N products of which each takes one operand from LDS: read(u) brings product u's,
// mul(u, operand) does it.  Operands are read four at a time, a group ahead of the
// products that run meanwhile.  (Left to itself the compiler saves registers:
// it reads each operand just before its product and waits for it.)
template <int N, typename Read, typename Mul>
__device__ __forceinline__ void run_products(Read read, Mul mul) {
    constexpr int G = 4;
    static_assert(N % G == 0, "whole groups");
    u32x4_t f[2][G];
#pragma unroll
    for (int i = 0; i < G; ++i) f[0][i] = read(i);
#pragma unroll
    for (int g = 0; g < N / G; ++g) {
        if (g + 1 < N / G) {
#pragma unroll
            for (int i = 0; i < G; ++i) f[(g + 1) & 1][i] = read((g + 1) * G + i);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < G; ++i) mul(g * G + i, f[g & 1][i]);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// G such loads, 1 KB apart in memory (but for the lanes' offsets) and in LDS, from
// a scalar address: the instruction's offset counts for both.
#define DF2_TO_LDS_1(NT)                                    \
    asm volatile(                                           \
        "s_mov_b32 m0, %0\n\t"                              \
        "s_nop 0\n\t"                                       \
        "global_load_lds_dwordx4 %1, %2" NT                 \
        :                                                   \
        : "s"(lds_base), "v"(off[0]), "s"(base)             \
        : "memory")
#define DF2_TO_LDS_2(NT)                                    \
    asm volatile(                                           \
        "s_mov_b32 m0, %0\n\t"                              \
        "s_nop 0\n\t"                                       \
        "global_load_lds_dwordx4 %1, %3" NT "\n\t"          \
        "global_load_lds_dwordx4 %2, %3 offset:%4" NT       \
        :                                                   \
        : "s"(lds_base), "v"(off[0]), "v"(off[1]), "s"(base), "n"(kLoad) \
        : "memory")
#define DF2_TO_LDS_4(NT)                                    \
    asm volatile(                                           \
        "s_mov_b32 m0, %0\n\t"                              \
        "s_nop 0\n\t"                                       \
        "global_load_lds_dwordx4 %1, %5" NT "\n\t"          \
        "global_load_lds_dwordx4 %2, %5 offset:%6" NT "\n\t" \
        "global_load_lds_dwordx4 %3, %5 offset:%7" NT "\n\t" \
        "global_load_lds_dwordx4 %4, %5 offset:%8" NT       \
        :                                                   \
        : "s"(lds_base), "v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3]), "s"(base), "n"(kLoad), \
          "n"(2 * kLoad), "n"(3 * kLoad)                    \
        : "memory")
template <int G, bool ONCE>
__device__ __forceinline__ void load_to_lds(const void* base, const uint32_t* off, uint32_t lds_base) {
    static_assert(G == 1 || G == 2 || G == 4, "loads in a group");
    constexpr int kLoad = 1024;         // bytes of a wave's load
    // the same in the wave, also where the compiler cannot see it
    const uint64_t addr = (uint64_t)base;
    base = reinterpret_cast<const void*>(
        ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(addr >> 32)) << 32) |
        (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)addr));
    if constexpr (G == 1) {
        if constexpr (ONCE) DF2_TO_LDS_1(" nt");
        else DF2_TO_LDS_1("");
    } else if constexpr (G == 2) {
        if constexpr (ONCE) DF2_TO_LDS_2(" nt");
        else DF2_TO_LDS_2("");
    } else {
        if constexpr (ONCE) DF2_TO_LDS_4(" nt");
        else DF2_TO_LDS_4("");
    }
}
#undef DF2_TO_LDS_1
#undef DF2_TO_LDS_2
#undef DF2_TO_LDS_4

// x * c - m with the product rounded.
__device__ __forceinline__ float scaled_minus(float x, float c, float m) {
#pragma clang fp contract(off)
    const float y = x * c;
    return y - m;
}

// The maximum that a row's part hands to the merges, which take -inf for a part that sees
// nothing.  Scores of NaN raise no maximum: their row's sum is NaN, and shall stay so
// however its keys are divided.
__device__ __forceinline__ float stated_max(float m, float l) { return l != l && m == -INFINITY ? 0.f : m; }

template <bool BF16, int D, bool FP4 = false>
struct AttnTile {
    static constexpr int kEsz = BF16 ? 2 : 4;
    static constexpr int kRow = D * kEsz;       // bytes of a key
    static constexpr int kChunks = kRow / 16;
    // From 4-bit values: both, and 16 lanes write whole blocks of four chunks of rows that
    // are four apart (writes meet all the same, eight cycles each: 32% of the cycles that the LDS
    // works in blocks of 64 rows).
    static __device__ __forceinline__ int swz_fp4(int row) {
        return kChunks >= 16 ? (row & 3) << 2 | ((row >> 2) & 3) : ((row >> 1) & 1) << 2 | ((row >> 2) & 3);
    }
    // Permutation of a row's chunks.  K: 16 keys read one chunk each in one go,
    // so they get 16 different places of the 256 bytes that the banks span.
    static __device__ __forceinline__ int swz_k(int row) {
        if constexpr (FP4 && BF16) return swz_fp4(row);
        return kChunks >= 16 ? (row & 15) : ((row >> 1) & 7);
    }
    // V: bf16, four keys of 64 bytes are read in one go; fp32, 128 bytes of
    // two keys that are four apart.
    static __device__ __forceinline__ int swz_v(int row) {
        if constexpr (FP4 && BF16) return swz_fp4(row);
        if constexpr (!BF16) return ((row >> 2) & 1) << 3;
        return kChunks >= 16 ? ((row & 3) << 2) : (((row >> 1) & 1) << 2);
    }
};

// WR waves of 32 rows, WK groups of them on different keys, KS times 32 keys
// a wave in each tile, NS stages of tiles in LDS.  More than two stages, with as
// many bytes in flight, were slower wherever they were tried (one row block on
// 131 thousand keys: 262 us with three, 349 with five).
// FP4: the cache holds 4-bit values (fp4.hpp), which become BF16's type on their way
// into the tiles.
template <bool BF16, int D, int WR, int WK, int KS, int NS, bool FP4>
__global__ void k_attend(AttnArgs a);

template <bool BF16, int D, int WR, int WK, int KS, int NS, bool FP4 = false>
struct AttnShape {
    using Tile = AttnTile<BF16, D, FP4>;
    static constexpr auto kernel() { return &k_attend<BF16, D, WR, WK, KS, NS, FP4>; }
    static constexpr int kWaves = WR * WK;
    static constexpr int kThreads = 64 * kWaves;
    static constexpr int BM = 32 * WR;
    static constexpr int KT = 32 * WK * KS;
    static constexpr int kTileBytes = KT * Tile::kRow;       // of K, and of V
    static constexpr int kStage = 2 * kTileBytes;
    static constexpr int kLoads = kTileBytes / (1024 * kWaves);     // of a wave for K, and for V
    static constexpr int kRows = KT / kWaves;                       // keys that they bring
    static constexpr int kGroup = kLoads % 4 == 0 && Tile::kRow >= 256 ? 4 : kLoads % 2 == 0 ? 2 : 1;
    static constexpr int kGroupKeys = FP4 ? 16 : kGroup * (64 / Tile::kChunks);
    // loads that may be in flight while the oldest stage is complete
    static constexpr int kAhead = NS > 2 ? (NS - 2) * 2 * kLoads : 0;
    static constexpr int kMergeBytes = WK > 1 ? kWaves * (32 * D * 4 + 256) + BM * 8 : 0;
    static constexpr int kLds = NS * kStage > kMergeBytes ? NS * kStage : kMergeBytes;   // tiles, or the merge
    static constexpr int kAllLds = kLds + 4 * kPageIds;
    // Waves of a SIMD: two where the registers of a row of D values leave room for them.
    // (With two counted everywhere, twice the stretches were cut: blocks of 128 rows,
    // 8 sequences after 6000 tokens, bf16 256 138 us and 116, fp32 128 251 and 239.)
    static constexpr int kSimdWaves = Tile::kRow <= 256 ? 2 : 1;
    // workgroups resident on a compute unit, by LDS and by registers
    static constexpr int kResident = 160 * 1024 / kAllLds < 4 * kSimdWaves / kWaves ? 160 * 1024 / kAllLds
                                                                                    : 4 * kSimdWaves / kWaves;
    static_assert(kResident >= 1, "a workgroup fits a compute unit");
    static_assert(kTileBytes % (1024 * kWaves) == 0, "every wave brings whole loads");
    static_assert(kAhead < 64, "the counter of loads in flight");
    static_assert(kAllLds <= 160 * 1024, "LDS of a compute unit");
    static_assert(KT <= kPageIds / 2, "a tile's pages fit the list");
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

template <bool BF16, int D, int WR, int WK, int KS, int NS, bool FP4>
__global__ __launch_bounds__(64 * WR * WK, (AttnShape<BF16, D, WR, WK, KS, NS, FP4>::kSimdWaves)) void k_attend(AttnArgs a) {
    using Shape = AttnShape<BF16, D, WR, WK, KS, NS, FP4>;
    using Tile = AttnTile<BF16, D, FP4>;
    constexpr int RB = Tile::kRow, CH = Tile::kChunks, KT = Shape::KT, BM = Shape::BM;
    constexpr int NL = Shape::kLoads, DB = D / 32;
    extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)lds;

    const PagedKv& kv = a.kv;
    const int lane = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id());
    const int wr = w % WR, wk = w / WR;
    const int half = lane >> 5, col = lane & 31;
    // A stretch of the line.  Workgroups go to the eight XCDs in turn; those of one
    // XCD take neighbouring stretches.  Whole blocks: neighbouring workgroups take
    // different heads, so that with eight of them an XCD keeps one head's keys.
    LaneSeq seqs;
    const Cut cut = cut_work<Shape>(a, seqs);
    const bool blocks_whole = cut.whole;
    int wg = blockIdx.x;
    if (!blocks_whole && cut.wgs % 8 == 0 && wg < cut.wgs)
        wg = (int)(blockIdx.x % 8) * (cut.wgs / 8) + (int)(blockIdx.x / 8);
    int32_t* split = a.split + 8 * wg;
    if (a.join && wg < a.wgs && (blocks_whole || wg >= cut.wgs) && threadIdx.x == 0) split[0] = -1;
    if (wg >= cut.wgs) return;
    int g = cut.first(wg), h = 0;
    const int start = g, stop = cut.first(wg + 1);
    Place at;
    at.j = at.blocks = 0;
    while (g < stop) {
    if (blocks_whole) {
        h = g % kv.Hkv;
        if (!find_place<Shape>(a, seqs, blocks_whole, g / kv.Hkv, at)) return;
        at.first = g - h * cut.head_tiles;      // the block is the whole stretch
    } else if (at.j + 1 < at.blocks) {
        at.first += at.k.tiles;         // the next block of the sequence
        ++at.j;
        at.k = block_keys<Shape>(a, at.ctx, at.n, at.j);
    } else {
        h = (int)((unsigned)g / (unsigned)cut.head_tiles);
        if (!find_place<Shape>(a, seqs, blocks_whole, g - h * cut.head_tiles, at)) return;
    }
    // the same in every lane; said so, they live in scalar registers
    const auto uni = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
    const int b = uni(at.b), s0 = uni(at.s0), n = uni(at.n), ctx = uni(at.ctx), r0 = uni(at.j) * BM;
    const int M = n * a.G, head_kv = uni(h), tiles = uni(at.k.tiles);
    const int first = uni(h * cut.head_tiles + at.first);
    const int tile0 = blocks_whole ? 0 : uni(g) - first;
    const int tile1 = blocks_whole ? tiles : min(tiles, stop - first);
    const bool whole = tile0 == 0 && tile1 == tiles;
    if (a.join && !blocks_whole && g == start && threadIdx.x == 0) {
        // the first boundary inside a block tells the join about the block
        const bool cuts = tile0 > 0 && cut.first(wg - 1) <= first;
        split[0] = cuts ? cut.owner(first + tiles - 1) : -1;
        split[1] = head_kv;
        split[2] = s0;
        split[3] = r0;
        split[4] = M;
    }
    g += blocks_whole ? 1 : tile1 - tile0;
    const int t_lo = uni(at.k.t_lo), t_hi = uni(at.k.t_hi);
    const int origin = uni(at.k.origin);
    const int klo = max(uni(at.k.begin), origin + tile0 * KT);
    const int khi = min(uni(at.k.end), origin + tile1 * KT);

    // This lane's row: row col of the wave's 32 (the last row again past the end).
    const int r = r0 + wr * 32 + col;
    const int rc = min(r, M - 1), t = div_g(a, rc), head = head_kv * a.G + rc - t * a.G;
    // first key it does not see; a token before position 0 sees none
    const int lim = a.causal || ctx + t < 0 ? ctx + t + 1 : khi;
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
    // of the V tile, RI keys.  Page ids wait in LDS, kPageIds at a time: read
    // from memory tile by tile, each would have to wait for the loads in flight.
    // Loads go in groups of GL, one page each: tiles start at multiples of the
    // group's keys, so in a whole tile (and pages no smaller than a group) a
    // group's address is one scalar, and the lanes' offsets are the same in every
    // tile.  Other tiles (the ends of the stretch, whose keys outside it are
    // replaced by its first or last; small pages) make each lane's address.
    constexpr int RW = Shape::kRows, RI = 64 / CH;      // keys of a wave, of a load
    constexpr bool kOnce = WR <= 4;     // one block has all rows of a sequence, mostly
    constexpr int GL = Shape::kGroup, GK = GL * RI;     // loads and keys of a group
    int32_t* ids = reinterpret_cast<int32_t*>(lds + Shape::kLds);
    const int64_t head_off = (int64_t)head_kv << kv.page_shift;
    const int32_t* table = kv.table + (int64_t)b * kv.table_stride;
    const int page_mask = (1 << kv.page_shift) - 1;
    const bool one_page = page_mask >= GK - 1;
    uint32_t at_k[NL], at_v[NL];        // within RI keys, chunks permuted by row
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int row = w * RW + i * RI + lane / CH;
        at_k[i] = (lane / CH) * RB + ((lane % CH) ^ Tile::swz_k(row)) * 16;
        at_v[i] = (lane / CH) * RB + ((lane % CH) ^ Tile::swz_v(row)) * 16;
    }
    auto load_tile = [&](const void* cache, int k0, uint32_t to, int page0, const uint32_t (&at)[NL]) {
        to += w * NL * 1024;
        // all ids first: the loads are not reordered with LDS reads, which would
        // then wait one by one
        int id[NL];
        if (one_page && k0 >= klo && k0 + KT <= khi) {
#pragma unroll
            for (int i = 0; i < NL; i += GL) id[i] = ids[((k0 + w * RW + i * RI) >> kv.page_shift) - page0];
#pragma unroll
            for (int i = 0; i < NL; i += GL) {
                const int key = k0 + w * RW + i * RI;
                const int64_t off = ((int64_t)__builtin_amdgcn_readfirstlane(id[i]) * kv.page_stride +
                                     (head_off + (key & page_mask)) * D) * Tile::kEsz;
                load_to_lds<GL, kOnce>(reinterpret_cast<const char*>(cache) + off, at + i, to + i * 1024);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NL; ++i)
                id[i] = ids[(min(max(k0 + w * RW + i * RI + lane / CH, klo), khi - 1) >> kv.page_shift) - page0];
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int key = min(max(k0 + w * RW + i * RI + lane / CH, klo), khi - 1);
                const int64_t off = ((int64_t)id[i] * kv.page_stride + (head_off + (key & page_mask)) * D) * Tile::kEsz;
                load_to_lds<kOnce>(reinterpret_cast<const char*>(cache) + off + at[i] % RB, to + i * 1024);
            }
        }
    };
    auto load_k = [&](int k0, int slot, int page0) {
        load_tile(a.k, k0, lds0 + slot * Shape::kTileBytes, page0, at_k);
    };
    auto load_v = [&](int k0, int slot, int page0) {
        load_tile(a.v, k0, lds0 + (NS + slot) * Shape::kTileBytes, page0, at_v);
    };

    // A 4-bit cache: a thread brings whole blocks of 32 codes and their scales into
    // registers, a tile ahead, and puts them into the tile as the products take them.
    // Tiles start at multiples of 16 keys, which share a page, so a wave's load has one
    // address but for its lanes' offsets (head size 64: two).  Keys outside the stretch may
    // hold anything: their scores are masked, the scales of their values made 1.
    constexpr int NB = D / kFp4Block, KL = 64 / NB;     // blocks of a key, keys of a wave's load
    constexpr int FL = KT / KL, NI = (FL + Shape::kWaves - 1) / Shape::kWaves;      // loads of a tile, of a wave
    u32x4_t codes_k[FP4 ? NI : 1], codes_v[FP4 ? NI : 1];
    uint32_t scale_k[FP4 ? NI : 1], scale_v[FP4 ? NI : 1];
    // this lane's key of a load: with 16 keys, four lanes of a row, then rows that are four apart
    const int load_key = KL == 16 && BF16 ? (lane / NB & 3) * 4 + lane / (4 * NB) : lane / NB;
    auto fetch = [&](int k0, int page0) {
        if constexpr (FP4) {
            const int64_t head_at = head_kv * Fp4Page<D>::bytes(kv.page_shift);
            const int64_t scales_at = Fp4Page<D>::scales(kv.page_shift);
            // codes and scales of key k's group of 16, from its page's head on
            const auto group = [&](int k, int64_t& code, int64_t& scale) {
                k = min(max(k, klo & ~15), (khi - 1) & ~15);
                const int64_t at = (int64_t)__builtin_amdgcn_readfirstlane(ids[(k >> kv.page_shift) - page0]) * kv.page_stride + head_at;
                code = at + (k & page_mask) * (D / 2);
                scale = at + scales_at + (k & page_mask) * NB;
            };
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int li = i * Shape::kWaves + w;
                if (FL % Shape::kWaves != 0 && li >= FL) break;
                int64_t code, scale;
                uint32_t key = load_key;        // in the group
                if constexpr (KL == 32) {
                    int64_t code2, scale2;
                    group(k0 + li * KL, code, scale);
                    group(k0 + li * KL + 16, code2, scale2);
                    code = lane < 32 ? code : code2;
                    scale = lane < 32 ? scale : scale2;
                    key &= 15;
                } else {
                    group((k0 + li * KL) & ~15, code, scale);
                    key += li * KL & 15;
                }
                const uint8_t* const ck = reinterpret_cast<const uint8_t*>(a.k) + code;
                const uint8_t* const cv = reinterpret_cast<const uint8_t*>(a.v) + code;
                const uint32_t off = key * (D / 2) + lane % NB * (kFp4Block / 2), off_s = key * NB + lane % NB;
                codes_k[i] = *reinterpret_cast<const u32x4_t*>(ck + off);
                codes_v[i] = *reinterpret_cast<const u32x4_t*>(cv + off);
                scale_k[i] = (reinterpret_cast<const uint8_t*>(a.k) + scale)[off_s];
                scale_v[i] = (reinterpret_cast<const uint8_t*>(a.v) + scale)[off_s];
            }
            if (k0 < klo || k0 + KT > khi) {
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int k = k0 + (i * Shape::kWaves + w) * KL + load_key;
                    scale_v[i] = k >= klo && k < khi ? scale_v[i] : (uint32_t)kFp4Bias;
                }
            }
        }
    };
    auto put = [&](int slot) {
        if constexpr (FP4) {
            constexpr int BC = CH / NB;         // chunks of a block
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int li = i * Shape::kWaves + w;
                if (FL % Shape::kWaves != 0 && li >= FL) break;
                const int row = li * KL + load_key, first = lane % NB * BC;
                unsigned char* to_k = lds + slot * Shape::kTileBytes + row * RB;
                unsigned char* to_v = to_k + NS * Shape::kTileBytes;
                const float sk = fp4_scale(scale_k[i]), sv = fp4_scale(scale_v[i]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if constexpr (BF16) {
                        *reinterpret_cast<u32x4_t*>(to_k + ((first + c) ^ Tile::swz_k(row)) * 16) = fp4_to_bf16(codes_k[i][c], sk);
                        *reinterpret_cast<u32x4_t*>(to_v + ((first + c) ^ Tile::swz_v(row)) * 16) = fp4_to_bf16(codes_v[i][c], sv);
                    } else {
                        f32x4_t lo, hi;
                        fp4_to_f32(codes_k[i][c], sk, lo, hi);
                        *reinterpret_cast<f32x4_t*>(to_k + ((first + 2 * c) ^ Tile::swz_k(row)) * 16) = lo;
                        *reinterpret_cast<f32x4_t*>(to_k + ((first + 2 * c + 1) ^ Tile::swz_k(row)) * 16) = hi;
                        fp4_to_f32(codes_v[i][c], sv, lo, hi);
                        *reinterpret_cast<f32x4_t*>(to_v + ((first + 2 * c) ^ Tile::swz_v(row)) * 16) = lo;
                        *reinterpret_cast<f32x4_t*>(to_v + ((first + 2 * c + 1) ^ Tile::swz_v(row)) * 16) = hi;
                    }
                }
            }
        }
    };

    // The first product of a tile, the scores of its keys for this wave's rows:
    // product u = q * KS + ks takes chunk q of sub-tile ks (neighbouring products
    // add to different sums).
    f32x16_t s[KS];
    constexpr int NQ = KS * QN;
    const int k_row = wk * KS * 32 + col;
    const uint32_t k_at = k_row * RB + (half ^ Tile::swz_k(k_row)) * 16;     // 32 rows on: the same permutation
    auto key_operand = [&](int slot, int u) {
        return *reinterpret_cast<const u32x4_t*>(lds + slot * Shape::kTileBytes + (u % KS) * 32 * RB +
                                                 (k_at ^ (uint32_t)(u / KS * 32)));
    };
    auto scores = [&](int slot, f32x16_t (&x)[KS]) {
        const auto zero = [](f32x16_t& y) {
#pragma unroll
            for (int v = 0; v < 16; ++v) y[v] = 0.f;
        };
        // sums start where their first product stands, which then takes a constant
        if constexpr (BF16) {
            run_products<NQ>([&](int u) { return key_operand(slot, u); },
                             [&](int u, u32x4_t kf) {
                                 if (u < KS) zero(x[u]);
                                 x[u % KS] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                                     as_bf16x8(kf), as_bf16x8(qf[u / KS]), x[u % KS], 0, 0, 0);
                             });
        } else {
            // Each product adds two terms and rounds: a chain of them over all of D puts
            // the roundings of D terms at the score's own size into its exponential.  Four
            // sums of a quarter (two of a half at head size 256, for their registers):
            // outputs at scores of 50 off by 2.5e-7 to 5e-7 instead of 3e-7 to 1e-6, for a
            // twentieth of the time of long chunks (2 of 2000 tokens after 2000, 8 / 2 heads
            // of 128: 504 us, 533).
            static_assert(KS == 1, "one sub-tile");
            constexpr int NA = D <= 128 ? 4 : 2;
            f32x16_t part[NA];
            run_products<NQ>([&](int u) { return key_operand(slot, u); },
                             [&](int u, u32x4_t kf) {
                                 if (u < NA) zero(part[u]);
#pragma unroll
                                 for (int e = 0; e < 4; ++e)
                                     part[u % NA] = __builtin_amdgcn_mfma_f32_32x32x2f32(
                                         __uint_as_float(kf[e]), __uint_as_float(qf[u][e]), part[u % NA], 0, 0, 0);
                             });
#pragma unroll
            for (int i = NA / 2; i > 0; i /= 2)
#pragma unroll
                for (int k = 0; k < i; ++k) part[k] += part[k + i];
            x[0] = part[0];
        }
    };
    // Masks the keys that a row does not see (tiles that every row sees whole need
    // none) and returns the row's maximum in units of log2.
    const int first_lim = a.causal || ctx + t_lo < 0 ? min(ctx + t_lo + 1, khi) : khi;
    const int last_low = max(a.window ? ctx + t_hi + 1 - a.window : 0, klo);
    const int top = min(lim, khi), bottom = max(low, klo);
    auto mask_and_max = [&](int k0, f32x16_t (&x)[KS]) {
        if (k0 + KT > first_lim || k0 < last_low) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    const int key = k0 + (wk * KS + ks) * 32 + 8 * (v / 4) + 4 * half + v % 4;
                    x[ks][v] = (key < top && key >= bottom) ? x[ks][v] : -INFINITY;
                }
        }
        float mx = x[0][0];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int v = 0; v < 16; ++v) mx = fmaxf(mx, x[ks][v]);
        float lower, upper;
        pair_of<32>(mx, lower, upper);
        return fmaxf(lower, upper) * a.c;
    };

    // exp2 of the scores over the row's maximum, into the row's sum and packed for
    // the second product: as they are in fp32; in bf16 as a high part, their rounding
    // (off by 2^-8 of a value at most), and in blocks of up to 64 rows a low part, what
    // the rounding left, rounded likewise: 16 bits in all.  The sum keeps the fp32
    // values.  The low part doubles the second product, which few rows have time for
    // (without and with it: 1 row 10.8 and 10.9 us, 32 contexts of 64 rows 158 and 164,
    // 16 after 1000 23.3 and 23.6, head size 256 61.5 and 64.2); blocks of 128 rows lose a
    // tenth by it (79 and 87) and prompt chunks more (690 and 940), so there the weights
    // are rounded.  Outputs against fp64, relative: 2.1e-3 without it, 1.7e-3, the
    // rounding of the output alone, with it.  Over a 4-bit cache blocks of 64 rows are bound
    // by the products too, and do without (32 contexts of 64 / 8 heads: 126 us with it, 105;
    // of 64 elements 86 and 76, of 256 105 and 98; 2.2e-3).
    constexpr bool kLow = BF16 && WR <= 2 && !FP4;
    constexpr int PN = BF16 ? (kLow ? 16 : 8) : 16;
    bool huge = false;                  // some row's maximum is beyond 2^26
    auto weights = [&](f32x16_t (&x)[KS], uint32_t (&p)[KS][PN]) {
        float ms = m == -INFINITY ? 0.f : m;
        // m is rounded and x * c below is not: from 2^26 on they differ by more than 1, and
        // from 2^31 on the exponential of the difference overflows.  There, both rounded, the
        // differences in x's place and a factor of 1 (scores put back in their own units
        // here cost every tile registers: fp32 of 256 spilled 113 of them, not 78).
        float c = a.c;
        if (__builtin_expect(huge, 0)) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int v = 0; v < 16; ++v) x[ks][v] = scaled_minus(x[ks][v], a.c, ms);
            c = 1.f;
            ms = 0.f;
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            float e[16];
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                e[v] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[ks][v], c, -ms));
                l += e[v];
            }
#pragma unroll
            for (int v = 0; v < (BF16 ? 8 : 16); ++v) {
                if constexpr (BF16) {
                    const auto pack = [](float x0, float x1) {
                        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){x0, x1}, bf16x2_t));
                    };
                    const uint32_t high = pack(e[2 * v], e[2 * v + 1]);
                    p[ks][v] = high;
                    if constexpr (kLow) p[ks][8 + v] = pack(e[2 * v] - bf16_lo(high), e[2 * v + 1] - bf16_hi(high));
                } else {
                    p[ks][v] = __float_as_uint(e[v]);
                }
            }
        }
    };
    // The maximum moves only where it grew by more than 2^8, so that most tiles
    // need no rescaling: p stays below 2^8, and p / sum is the same.
    auto move_max = [&](float mx) {
        if (__any(mx > m + 8.f)) {
            const float mn = fmaxf(m, mx);
            const float f = m == mn ? 1.f : __builtin_amdgcn_exp2f(m - mn);
            m = mn;
            huge = __any(fabsf(m) > 0x1p26f && m != -INFINITY);
            l *= f;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int v = 0; v < 16; ++v) o[d][v] *= f;
        }
    };
    // The second product of a tile.  bf16: product u = (ks * 2 + j) * DB + d takes
    // 16 keys and 32 of the columns.
    constexpr int NV = KS * 2 * DB;
    const int v_row = wk * KS * 32 + 4 * half + ((lane & 15) >> 2);
    const int v_chunk = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    auto value_operand = [&](int slot, int u) {
        typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
        const int d = u % DB, keys = u / DB * 16;       // 16 rows on: the same permutation
        const unsigned char* from = lds + (NS + slot) * Shape::kTileBytes + keys * RB + v_row * RB + (lane & 1) * 8;
        const s16x4_t v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4*)(from + ((4 * d + v_chunk) ^ Tile::swz_v(v_row)) * 16));
        const s16x4_t v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4*)(from + 8 * RB + ((4 * d + v_chunk) ^ Tile::swz_v(v_row + 8)) * 16));
        return __builtin_bit_cast(u32x4_t, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    auto value_product = [&](int u, u32x4_t vf, const uint32_t (&p)[KS][PN]) {
        const int d = u % DB, j = u / DB;
#pragma unroll
        for (int part = 0; part < (kLow ? 2 : 1); ++part) {
            const uint32_t* w4 = &p[j / 2][8 * part + (j & 1) * 4];
            const u32x4_t pf = {w4[0], w4[1], w4[2], w4[3]};
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(vf), as_bf16x8(pf), o[d], 0, 0, 0);
        }
    };
    auto add_values = [&](int slot, const uint32_t (&p)[KS][PN]) {
        if constexpr (BF16) {
            run_products<NV>([&](int u) { return value_operand(slot, u); },
                             [&](int u, u32x4_t f) { value_product(u, f, p); });
        } else {
            const unsigned char* vt = lds + (NS + slot) * Shape::kTileBytes;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    const int row = (wk * KS + ks) * 32 + 8 * (v / 4) + 4 * half + v % 4;
                    const int f = Tile::swz_v(row);
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
                        const float vf = *reinterpret_cast<const float*>(
                            vt + row * RB + ((8 * d + (col >> 2)) ^ f) * 16 + (col & 3) * 4);
                        o[d] = __builtin_amdgcn_mfma_f32_32x32x2f32(vf, __uint_as_float(p[ks][v]), o[d], 0, 0, 0);
                    }
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
        // The query rows have arrived before the first tile's loads go out: a wait
        // for them inside the loop would be one for all loads in flight.
#pragma unroll
        for (int q = 0; q < QN; ++q) asm volatile("" : "+v"(qf[q]));
        uint32_t p[KS][PN];
        if constexpr (FP4) {
            // NS tiles in LDS, one more in registers
            static_assert(NS <= 2, "one stage or two");
            fetch(k_win, page0);
            if constexpr (NS == 2) {
                put(0);
                if (ntile > 1) fetch(k_win + KT, page0);
            }
            for (int it = 0; it < ntile; ++it) {
                const int k0 = k_win + it * KT, slot = it & (NS - 1);
                // two: the tile is whole, and nobody reads the one before it any more
                __syncthreads();
                if (it + NS - 1 < ntile) put((it + NS - 1) & (NS - 1));
                if (it + NS < ntile) fetch(k0 + NS * KT, page0);
                if constexpr (NS == 1) __syncthreads();
                scores(slot, s);
                move_max(mask_and_max(k0, s));
                weights(s, p);
                add_values(slot, p);
            }
        } else {
            // A ring of NS tiles, NS - 1 of them in flight or waiting.
#pragma unroll
            for (int i = 0; i < NS - 1; ++i)
                if (i < ntile) {
                    load_k(k_win + i * KT, i, page0);
                    load_v(k_win + i * KT, i, page0);
                }
            int slot = 0;
            for (int it = 0; it < ntile; ++it) {
                const int k0 = k_win + it * KT;
                // this wave's part of the oldest tile is in LDS; then everyone's is,
                // and nobody reads the tile before it any more
                wait_and_meet<NS - 2, 2 * NL>(ntile - 1 - it);
                if (it + NS - 1 < ntile) {
                    const int free = slot == 0 ? NS - 1 : slot - 1;
                    load_k(k0 + (NS - 1) * KT, free, page0);
                    load_v(k0 + (NS - 1) * KT, free, page0);
                }
                scores(slot, s);
                move_max(mask_and_max(k0, s));
                weights(s, p);
                add_values(slot, p);
                slot = slot == NS - 1 ? 0 : slot + 1;
            }
        }
        k_win += ntile * KT;
    }
    {
        float lower, upper;
        pair_of<32>(l, lower, upper);
        l = lower + upper;
    }
    m = stated_max(m, l);

    const int part0 = 2 * wg + (tile0 == 0 ? 1 : 0);    // where a part goes
    if constexpr (WK > 1) {
        // The groups' results meet in LDS: each wave's output scaled to the rows' common
        // maximum, then summed and written row by row by all threads.  (Short code,
        // not unrolled: code that runs once costs its fetch, 4 us of it here with
        // everything in registers.)
        float* st = reinterpret_cast<float*>(lds + Shape::kWaves * 32 * D * 4);
        float* joint = st + Shape::kWaves * 64;         // of each row of the block: maximum, sum
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
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                mine[col * (D / 4) + ((8 * d + 2 * v + half) ^ (col & 15))] =
                    (f32x4_t){o[d][4 * v] * f, o[d][4 * v + 1] * f, o[d][4 * v + 2] * f, o[d][4 * v + 3] * f};
        if (wk == 0 && half == 0) {
            joint[2 * (wr * 32 + col)] = mg;
            joint[2 * (wr * 32 + col) + 1] = lg;
        }
        __syncthreads();
        const int live = min(BM, M - r0);
#pragma unroll 1
        for (int x = threadIdx.x; x < live * (D / 4); x += Shape::kThreads) {
            const int row = x / (D / 4), c = x % (D / 4), wrow = row / 32, wcol = row % 32;
            f32x4_t y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < WK; ++k)
                y += reinterpret_cast<const f32x4_t*>(lds + (k * WR + wrow) * 32 * D * 4)[wcol * (D / 4) + (c ^ (wcol & 15))];
            const float lr = joint[2 * row + 1];
            if (whole) {
                const float inv = lr > 0.f ? 1.f / lr : (lr == 0.f ? 0.f : lr);
                const int rr = r0 + row, tt = div_g(a, rr);
                const float out[4] = {y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv};
                store4<BF16>(a.out, (int64_t)(s0 + tt) * a.out_stride + (int64_t)(head_kv * a.G + rr - tt * a.G) * D + 4 * c, out);
            } else {
                const int64_t prow = (int64_t)part0 * BM + row;
                const float out[4] = {y[0], y[1], y[2], y[3]};
                store4<false>(a.part, prow * D + 4 * c, out);
                if (c == 0) {
                    a.stat[2 * prow] = joint[2 * row];
                    a.stat[2 * prow + 1] = lr;
                }
            }
        }
    } else {
    if (r >= M) continue;
    if (whole) {
        // a row that sees nothing gives zeros
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        const int64_t to = (int64_t)(s0 + t) * a.out_stride + (int64_t)head * D;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const float y[4] = {o[d][4 * v] * inv, o[d][4 * v + 1] * inv, o[d][4 * v + 2] * inv,
                                    o[d][4 * v + 3] * inv};
                store4<BF16>(a.out, to + 32 * d + 8 * v + 4 * half, y);
            }
    } else {
        const int64_t prow = (int64_t)part0 * BM + wr * 32 + col;
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
    }
}

// Joins the parts of the blocks that lie across workgroups:
//     sum_s 2^(m_s - m) (o_s, l_s)
// over the parts s of a row.  JOIN workgroups for each boundary of stretches, of which the
// first inside a block does the block.  D / 4 lanes take a row, four parts
// at a time; with more parts several such groups share the row and meet in LDS, so
// that a hundred parts of a few rows are a few loads one after another.
constexpr int kJoinThreads = 256;
template <bool BF16, int D, int JOIN>
__global__ __launch_bounds__(kJoinThreads) void k_attend_join(AttnArgs a) {
    constexpr int L = D / 4, NG = kJoinThreads / L;
    __shared__ f32x4_t lds_y[kJoinThreads];
    __shared__ float lds_m[NG], lds_l[NG];
    const int slice = blockIdx.x % JOIN, boundary = 1 + blockIdx.x / JOIN;
    const int32_t* split = a.split + 8 * boundary;
    const int w0 = boundary - 1, w1 = min(split[0], (int)(gridDim.x / JOIN));
    const int h = split[1], s0 = split[2], r0 = split[3], M = split[4];
    if (w1 < 0) return;
    const int group = threadIdx.x / L, d = (threadIdx.x % L) * 4;
    const int live = min(a.bm, M - r0);
    int share = 1;                                      // groups of a row, as long as one go takes all rows
    while (4 * share < w1 - w0 + 1 && share < NG && live * share * 2 <= NG * JOIN) share *= 2;
    const int at_once = NG / share;
    for (int i0 = slice * at_once; i0 < live; i0 += JOIN * at_once) {
        const int i = i0 + group / share, r = r0 + i;
        float m = -INFINITY, l = 0.f;
        f32x4_t y = {0.f, 0.f, 0.f, 0.f};
        if (i < live) {
            for (int w = w0 + group % share; w <= w1; w += 4 * share) {
                float pm[4], pl[4];
                f32x4_t py[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int p = min(w + x * share, w1);
                    const int64_t row = (int64_t)(2 * p + (p == w0 ? 1 : 0)) * a.bm + i;
                    pm[x] = w + x * share <= w1 ? a.stat[2 * row] : -INFINITY;
                    pl[x] = a.stat[2 * row + 1];
                    py[x] = *reinterpret_cast<const f32x4_t*>(a.part + row * D + d);
                }
                float mn = m;
#pragma unroll
                for (int x = 0; x < 4; ++x) mn = fmaxf(mn, pm[x]);
                if (mn == -INFINITY) continue;      // parts of which the row sees nothing
                const float f = __builtin_amdgcn_exp2f(m - mn);
                m = mn;
                l *= f;
                y *= f;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if (pm[x] == -INFINITY) continue;
                    const float e = __builtin_amdgcn_exp2f(pm[x] - mn);
                    l += e * pl[x];
                    y += e * py[x];
                }
            }
        }
        if (share > 1) {
            __syncthreads();
            lds_y[threadIdx.x] = y;
            if (threadIdx.x % L == 0) {
                lds_m[group] = m;
                lds_l[group] = l;
            }
            __syncthreads();
            if (group % share == 0) {
                for (int x = 1; x < share; ++x) {
                    const float mx = lds_m[group + x];
                    if (mx == -INFINITY) continue;
                    const float mn = fmaxf(m, mx);
                    const float f = __builtin_amdgcn_exp2f(m - mn), e = __builtin_amdgcn_exp2f(mx - mn);
                    m = mn;
                    l = f * l + e * lds_l[group + x];
                    y = f * y + e * lds_y[(group + x) * L + threadIdx.x % L];
                }
            }
        }
        if (i >= live || group % share != 0) continue;
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        const int t = div_g(a, r), head = h * a.G + r - t * a.G;
        const float out[4] = {y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv};
        store4<BF16>(a.out, (int64_t)(s0 + t) * a.out_stride + (int64_t)head * D + d, out);
    }
}

}  // namespace df2
