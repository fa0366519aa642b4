// Penalties for repeated tokens, biases and grammar masks on rows of logits.
//
// Row t of sequence b, of token v's value x:
//     y = x;  v seen before the row: y = x > 0 ? x / repetition : x * repetition
//     y = y - frequency * c - presence * [c > 0]      c: how often it was generated
//     y = y + bias(v)
//     v not allowed: -inf
// in fp32, each step rounded once (no contraction), one rounding at the store.  Seen:
// in the history or among the drafts before row t; generated: in the history behind
// the prompt, or such a draft.
//
// A workgroup takes a segment of the vocabulary and some rows of one sequence.  It
// goes through the history once and counts in LDS the tokens that fall into its
// segment (integer sums, so their order does not matter), and lists those that anything
// happens to.  Two passes over the rows follow: all of their vectors are copied, with -inf
// for the forbidden (in place only vectors with forbidden tokens are touched, and one
// that has no others is not read); then the listed tokens are adjusted one by one, a
// thread to a token for all rows.  (With both in one pass nearly every wave went through
// the arithmetic for all eight elements of its vectors, for a token here and there: 512
// rows of 151936 in place, half of them masked, 136 us, now 72, of which the single elements'
// lines are some 40.  8 rows into another tensor: 6.0 us, latency.)  Nothing is kept between
// calls, so a history may be edited at will.
//
// Every load waits for most of a microsecond, so they go out several at a time: four
// vectors of the history, the masks of all rows into LDS at once, four vectors or elements of
// rows.  A token of the history costs one atomic that nothing waits for (with a bitmap read
// and set beside it, 2 sequences of 16 thousand tokens over 1200 words 17 us, now 10).
// Drafts before a workgroup's rows are counted with the history, and a drafted token looks
// through those between its rows only: gone through from the first for each row, they grew
// with the third power of the rows (4096 rows of 4099 14.3 ms, now 140 us).
#pragma once

#include "common.hpp"
#include "lanes.hpp"

#include <type_traits>

namespace df2 {

struct AdjustArgs {
    const void* logits;
    void* out;
    const int32_t* history;     // [B, L], rows history_stride apart; NULL: none
    const int32_t* history_len; // [B]
    const int32_t* prompt_len;  // [B] or NULL: 0
    const int32_t* path;        // [B, R - 1] or NULL
    const float* repetition;    // [B] each, or NULL
    const float* frequency;
    const float* presence;
    const int32_t* bias_token;  // [B, M]
    const float* bias;
    const uint32_t* mask;       // bits of allowed tokens, or NULL
    int64_t seq_stride, row_stride;             // of logits, in elements
    int64_t out_seq_stride, out_row_stride;
    int64_t history_stride, mask_seq_stride, mask_row_stride;
    int B, R, V, L, M;
    int seg, nseg;              // tokens of a segment (a multiple of 32), segments
    int rows, row_groups;       // rows of a workgroup
    int max_words;              // mask words of a segment, all rows of the workgroup; 0: no masks
    int table;                  // biases have a word for each token of the segment; 0: a list of M
};

// What LDS holds of a token: whether the prompt has it, whether a draft is it, whether it
// has a bias, how often it was generated before the workgroup's rows.
constexpr uint32_t kTokenSeen = 1u << 31, kTokenDrafted = 1u << 30, kTokenBiased = 1u << 29, kTokenCount = kTokenBiased - 1;
constexpr int kBiasList = 512;      // biases that are listed: each is looked for in the list of its segment
constexpr int kAdjustThreads = 256;

// `count` bits (up to 8) from bit p of the words on; words behind `last` are not read.
__device__ __forceinline__ uint32_t bits_at(const uint32_t* words, int p, int last) {
    const int w = p >> 5, s = p & 31;
    uint32_t x = words[w] >> s;
    if (s > 24 && w < last) x |= words[w + 1] << (32 - s);
    return x & 0xFFu;
}

template <bool BF16, bool PLACE>
__global__ __launch_bounds__(kAdjustThreads) void k_adjust(AdjustArgs a) {
    using Elem = std::conditional_t<BF16, uint16_t, uint32_t>;
    constexpr int E = BF16 ? 8 : 4;             // elements of 16 bytes
    constexpr uint32_t ALL = (1u << E) - 1;
    constexpr int U = 4;                        // vectors of a thread at a time
    constexpr Elem kLow = BF16 ? 0xFF80u : 0xFF800000u;     // -inf
    extern __shared__ __attribute__((aligned(16))) uint32_t adjust_lds[];
    __shared__ int listed, biased;
    uint32_t* const count = adjust_lds;                     // [seg]
    uint16_t* const list = reinterpret_cast<uint16_t*>(count + a.seg);      // [seg] touched tokens
    uint32_t* const allowed = count + a.seg + a.seg / 2;    // [rows, seg / 32] (with masks)
    // biases: of each token its entry + 1, or (a few) a list of token and entry
    uint32_t* const from = allowed + a.max_words;
    const int tid = threadIdx.x;
    const int s = blockIdx.x % a.nseg, rg = blockIdx.x / a.nseg % a.row_groups, b = blockIdx.x / a.nseg / a.row_groups;
    const int v0 = s * a.seg, len = min(a.seg, a.V - v0);
    const int t0 = rg * a.rows, t1 = min(t0 + a.rows, a.R);

    const bool lists = a.history || a.path || a.M > 0;
    const int seg_words = a.seg >> 5, words = (len + 31) >> 5;      // mask words of the segment
    if (lists) {
        if (tid == 0) listed = biased = 0;
        for (int i = tid; i < a.seg; i += kAdjustThreads) count[i] = 0;
        if (a.table)
            for (int i = tid; i < a.seg; i += kAdjustThreads) from[i] = 0;
    }
    if (a.mask) {
        const uint32_t* row = a.mask + b * a.mask_seq_stride + (v0 >> 5);
        for (int i = tid; i < (t1 - t0) * seg_words; i += kAdjustThreads) {
            const int t = (int)((unsigned)i / (unsigned)seg_words), w = i - t * seg_words;
            if (w < words) allowed[i] = row[(t0 + t) * a.mask_row_stride + w];
        }
    }
    __syncthreads();
    if (a.history) {
        const int n = min(max(a.history_len[b], 0), a.L), prompt = a.prompt_len ? a.prompt_len[b] : 0;
        const int32_t* text = a.history + (int64_t)b * a.history_stride;
        const auto take = [&](int i, int id) {
            const uint32_t v = (uint32_t)id - (uint32_t)v0;
            if (id < 0 || v >= (uint32_t)len) return;
            // nothing is read back, so nothing waits
            if (i >= prompt) atomicAdd(&count[v], 1u);
            else atomicOr(&count[v], kTokenSeen);
        };
        const int head = min((int)((16 - ((uintptr_t)text & 15)) & 15) / 4, n);     // up to the first 16 bytes in line
        if (tid < head) take(tid, text[tid]);
        const int vectors = (n - head) / 4;
        for (int i = tid; i < vectors; i += 4 * kAdjustThreads) {
            u32x4_t ids[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                ids[j] = *reinterpret_cast<const u32x4_t*>(text + head + 4 * min(i + j * kAdjustThreads, vectors - 1));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + j * kAdjustThreads < vectors)
#pragma unroll
                    for (int k = 0; k < 4; ++k) take(head + 4 * (i + j * kAdjustThreads) + k, (int)ids[j][k]);
        }
        for (int i = head + 4 * vectors + tid; i < n; i += kAdjustThreads) take(i, text[i]);
    }
    const int32_t* path = a.path ? a.path + (int64_t)b * (a.R - 1) : nullptr;
    if (path)
        for (int i = tid; i < t1 - 1; i += kAdjustThreads) {
            const uint32_t v = (uint32_t)path[i] - (uint32_t)v0;
            if (path[i] < 0 || v >= (uint32_t)len) continue;
            // before all of these rows, or between them
            if (i < t0) atomicAdd(&count[v], 1u);
            else atomicOr(&count[v], kTokenDrafted);
        }
    for (int i = tid; i < a.M; i += kAdjustThreads) {
        const int id = a.bias_token[(int64_t)b * a.M + i];
        const uint32_t v = (uint32_t)id - (uint32_t)v0;
        if (id < 0 || v >= (uint32_t)len) continue;
        if (a.table) atomicMax(&from[v], (uint32_t)i + 1);      // of a token given twice, the last
        else from[atomicAdd(&biased, 1)] = v << 16 | (uint32_t)(i + 1);
        atomicOr(&count[v], kTokenBiased);
    }
    if (lists) {
        __syncthreads();
        // a thread's neighbouring words, four at a time; one place in the list a wave
        const int each = a.seg / kAdjustThreads;
        uint32_t bits = 0;
        for (int i = 0; i < each; i += 4) {
            const u32x4_t w = *reinterpret_cast<const u32x4_t*>(count + tid * each + i);
#pragma unroll
            for (int k = 0; k < 4; ++k) bits |= (w[k] != 0 ? 1u : 0u) << (i + k);
        }
        const int n = __popc(bits), upto = lanes_scan(n);
        int first = 0;
        if (lane_id() == 63) first = atomicAdd(&listed, upto);
        int to = __builtin_amdgcn_readlane(first, 63) + upto - n;
        for (; bits; bits &= bits - 1) list[to++] = (uint16_t)(tid * each + __builtin_ctz(bits));
    }
    __syncthreads();

    // all vectors of the rows
    const bool in_line = (((uintptr_t)a.out | a.out_seq_stride * sizeof(Elem) | a.out_row_stride * sizeof(Elem)) & 15) == 0 &&
                         (PLACE || (((uintptr_t)a.logits | a.seq_stride * sizeof(Elem) | a.row_stride * sizeof(Elem)) & 15) == 0);
    if ((!PLACE || a.mask) && in_line) {
        // rows begin in line: a vector's mask is a byte of the words, or half of one
        const auto forbidden = [&](int t, int x) {
            if (!a.mask) return 0u;
            const uint8_t* bytes = reinterpret_cast<const uint8_t*>(allowed + (t - t0) * seg_words);
            return E == 8 ? ~bytes[x] & 0xFFu : ~(bytes[x >> 1] >> (4 * (x & 1))) & 0xFu;
        };
        const Elem* in = reinterpret_cast<const Elem*>(a.logits) + b * a.seq_stride + v0;
        Elem* const out = reinterpret_cast<Elem*>(a.out) + b * a.out_seq_stride + v0;
        const int whole = len / E;
        constexpr int RU = 2, XU = 2;                       // rows and vectors of a thread at a time
        for (int t = t0; t < t1; t += RU)
            for (int x0 = tid; x0 < whole; x0 += XU * kAdjustThreads) {
                u32x4_t data[RU][XU];
                uint32_t gone[RU][XU];
#pragma unroll
                for (int j = 0; j < RU * XU; ++j) {
                    const int r = min(t + j / XU, t1 - 1), x = min(x0 + j % XU * kAdjustThreads, whole - 1);
                    gone[j / XU][j % XU] = forbidden(r, x);
                    if (!PLACE || (gone[j / XU][j % XU] && gone[j / XU][j % XU] != ALL))
                        data[j / XU][j % XU] = *reinterpret_cast<const u32x4_t*>(in + r * a.row_stride + x * E);
                }
#pragma unroll
                for (int j = 0; j < RU * XU; ++j) {
                    const int r = t + j / XU, x = x0 + j % XU * kAdjustThreads;
                    const uint32_t bad = gone[j / XU][j % XU];
                    if (r >= t1 || x >= whole || (PLACE && !bad)) continue;
                    u32x4_t y = data[j / XU][j % XU];
                    if (bad) {
                        __attribute__((aligned(16))) Elem e[E];
                        *reinterpret_cast<u32x4_t*>(e) = y;
#pragma unroll
                        for (int k = 0; k < E; ++k) e[k] = bad >> k & 1 ? kLow : e[k];
                        y = *reinterpret_cast<const u32x4_t*>(e);
                    }
                    *reinterpret_cast<u32x4_t*>(out + r * a.out_row_stride + x * E) = y;
                }
            }
        // the elements behind the last whole vector
        const int rest = len - whole * E;
        for (int i = tid; i < (t1 - t0) * rest; i += kAdjustThreads) {
            const int t = t0 + i / rest, k = i % rest;
            const bool bad = forbidden(t, whole) >> k & 1;
            if (!PLACE || bad)
                out[t * a.out_row_stride + whole * E + k] = bad ? kLow : in[t * a.row_stride + whole * E + k];
        }
    } else if (!PLACE || a.mask) {
        const int slots = (a.seg + E - 1) / E + 1;          // vectors of a row that meet the segment
        const int items = (t1 - t0) * slots;
        int t = t0, x = tid;                                // row and vector of this thread's next item
        for (int i0 = 0; i0 < items; i0 += U * kAdjustThreads) {
            // which elements of U vectors are theirs to write, and to forbid
            const Elem* src[U];
            Elem* to[U];
            uint32_t own[U], gone[U];
            u32x4_t data[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                while (x >= slots) {
                    x -= slots;
                    ++t;
                }
                own[j] = gone[j] = 0;
                if (t < t1) {
                    // vectors begin where the row's store address is in line
                    Elem* const out = reinterpret_cast<Elem*>(a.out) + b * a.out_seq_stride + t * a.out_row_stride + v0;
                    const int p = x * E - (int)(((uintptr_t)out & 15) / sizeof(Elem));      // its first token in the segment
                    const int lo = max(p, 0), hi = min(p + E, len);
                    if (lo < hi) {
                        own[j] = (ALL >> (E - (hi - lo))) << (lo - p);
                        gone[j] = a.mask ? ~(bits_at(allowed + (t - t0) * seg_words, lo, words - 1) << (lo - p)) & own[j] : 0u;
                        if (PLACE && !gone[j]) own[j] = 0;
                        src[j] = reinterpret_cast<const Elem*>(a.logits) + b * a.seq_stride + t * a.row_stride + v0 + p;
                        to[j] = out + p;
                        if (own[j] == ALL && gone[j] != ALL && (PLACE || ((uintptr_t)src[j] & 15) == 0))
                            data[j] = *reinterpret_cast<const u32x4_t*>(src[j]);
                    }
                }
                x += kAdjustThreads;
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (own[j] == ALL) {
                    __attribute__((aligned(16))) Elem e[E];
                    if (PLACE || gone[j] == ALL || ((uintptr_t)src[j] & 15) == 0) {
                        *reinterpret_cast<u32x4_t*>(e) = data[j];
                    } else {
#pragma unroll
                        for (int k = 0; k < E; ++k) e[k] = src[j][k];
                    }
#pragma unroll
                    for (int k = 0; k < E; ++k) e[k] = gone[j] >> k & 1 ? kLow : e[k];
                    *reinterpret_cast<u32x4_t*>(to[j]) = *reinterpret_cast<const u32x4_t*>(e);
                } else if (own[j]) {
                    for (int k = 0; k < E; ++k)
                        if (own[j] >> k & 1) to[j][k] = gone[j] >> k & 1 ? kLow : src[j][k];
                }
            }
        }
    }
    if (!lists || listed == 0) return;
    // their stores are done: elements of the same vectors follow
    __syncthreads();

    const float rep = a.repetition ? a.repetition[b] : 1.f;
    const float freq = a.frequency ? a.frequency[b] : 0.f, pres = a.presence ? a.presence[b] : 0.f;
    const auto number = [](Elem e) { return BF16 ? bf16_lo(e) : __uint_as_float(e); };
    const auto element = [](float x) -> Elem {
        if constexpr (BF16) return __builtin_bit_cast(uint16_t, (__bf16)x);
        else return __float_as_uint(x);
    };
    // U rows of a token at a time
    const int quads = (t1 - t0 + U - 1) / U;
    for (int i = tid; i < listed * quads; i += kAdjustThreads) {
        const int quad = (int)((unsigned)i / (unsigned)listed), v = list[i - quad * listed], t = t0 + quad * U;
        const Elem* src = reinterpret_cast<const Elem*>(a.logits) + b * a.seq_stride + v0 + v;
        Elem* to = reinterpret_cast<Elem*>(a.out) + b * a.out_seq_stride + v0 + v;
        Elem e[U];
#pragma unroll
        for (int j = 0; j < U; ++j) e[j] = src[(int64_t)min(t + j, t1 - 1) * a.row_stride];
        const uint32_t w = count[v];
        const bool bias_it = w & kTokenBiased;
        float bias = 0.f;
        if (bias_it) {
            uint32_t entry = a.table ? from[v] : 0u;
            if (!a.table)
                for (int k = 0; k < biased; ++k)
                    if (from[k] >> 16 == (uint32_t)v) entry = max(entry, from[k] & 0xFFFFu);
            bias = a.bias[(int64_t)b * a.M + entry - 1];
        }
        int c = (int)(w & kTokenCount), drafted = t0;       // generated before row t; drafts gone through
        bool seen = (w & kTokenSeen) || c > 0;
#pragma unroll
        for (int j = 0; j < U; ++j) {
#pragma clang fp contract(off)
            if (t + j >= t1) break;
            if (w & kTokenDrafted)
                for (; drafted < t + j; ++drafted)
                    if (path[drafted] == v0 + v) {
                        ++c;
                        seen = true;
                    }
            if (a.mask && !(allowed[(t + j - t0) * seg_words + (v >> 5)] >> (v & 31) & 1)) continue;
            if (!seen && !bias_it) continue;        // a draft of this row or one behind it
            float x = number(e[j]);
            if (seen) x = x > 0.f ? x / rep : x * rep;
            if (c > 0) {
                const float often = freq * (float)c;
                x = x - often;
                x = x - pres;
            }
            if (bias_it) x = x + bias;
            to[(int64_t)(t + j) * a.out_row_stride] = element(x);
        }
    }
}

}  // namespace df2
