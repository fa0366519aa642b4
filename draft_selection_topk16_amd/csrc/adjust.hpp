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
// segment (integer sums, so their order does not matter); a bitmap of the tokens that
// anything happens to lets the rows pass by eight elements at a time, of which most
// are copied (or, in place, not even read: a vector is loaded only if one of its
// tokens is touched, and a vector of forbidden ones is only stored).  Nothing is kept
// between calls, so a sequence's history may be edited at will.
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
};

constexpr uint32_t kTokenSeen = 1u << 31, kTokenDrafted = 1u << 30, kTokenCount = kTokenDrafted - 1;
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
    constexpr Elem kLow = BF16 ? 0xFF80u : 0xFF800000u;     // -inf
    extern __shared__ __attribute__((aligned(16))) uint32_t adjust_lds[];
    uint32_t* const count = adjust_lds;                     // [seg]
    uint32_t* const touched = count + a.seg;                // [seg / 32]
    uint32_t* const from = touched + a.seg / 32;            // [seg] bias entry + 1 (M > 0)
    const int tid = threadIdx.x;
    const int s = blockIdx.x % a.nseg, rg = blockIdx.x / a.nseg % a.row_groups, b = blockIdx.x / a.nseg / a.row_groups;
    const int v0 = s * a.seg, len = min(a.seg, a.V - v0);
    const int t0 = rg * a.rows, t1 = min(t0 + a.rows, a.R);

    const bool lists = a.history || a.path || a.M > 0;
    if (lists) {
        for (int i = tid; i < a.seg + a.seg / 32 + (a.M > 0 ? a.seg : 0); i += kAdjustThreads) adjust_lds[i] = 0;
        __syncthreads();
    }
    const auto touch = [&](uint32_t v) { atomicOr(&touched[v >> 5], 1u << (v & 31)); };
    if (a.history) {
        const int n = min(max(a.history_len[b], 0), a.L), prompt = a.prompt_len ? a.prompt_len[b] : 0;
        const int32_t* text = a.history + (int64_t)b * a.history_stride;
        const auto take = [&](int i, int id) {
            const uint32_t v = (uint32_t)id - (uint32_t)v0;
            if (id < 0 || v >= (uint32_t)len) return;
            if (i >= prompt) atomicAdd(&count[v], 1u);
            atomicOr(&count[v], kTokenSeen);
            touch(v);
        };
        const int head = min((int)((16 - ((uintptr_t)text & 15)) & 15) / 4, n);     // up to the first 16 bytes in line
        if (tid < head) take(tid, text[tid]);
        const int vectors = (n - head) / 4;
        for (int i = tid; i < vectors; i += kAdjustThreads) {
            const u32x4_t ids = *reinterpret_cast<const u32x4_t*>(text + head + 4 * i);
#pragma unroll
            for (int k = 0; k < 4; ++k) take(head + 4 * i + k, (int)ids[k]);
        }
        for (int i = head + 4 * vectors + tid; i < n; i += kAdjustThreads) take(i, text[i]);
    }
    const int32_t* path = a.path ? a.path + (int64_t)b * (a.R - 1) : nullptr;
    if (path)
        for (int i = tid; i < t1 - 1; i += kAdjustThreads) {
            const uint32_t v = (uint32_t)path[i] - (uint32_t)v0;
            if (path[i] < 0 || v >= (uint32_t)len) continue;
            atomicOr(&count[v], kTokenDrafted);
            touch(v);
        }
    for (int i = tid; i < a.M; i += kAdjustThreads) {
        const int id = a.bias_token[(int64_t)b * a.M + i];
        const uint32_t v = (uint32_t)id - (uint32_t)v0;
        if (id < 0 || v >= (uint32_t)len) continue;
        atomicMax(&from[v], (uint32_t)i + 1);       // of a token given twice, the last
        touch(v);
    }
    if (lists) __syncthreads();
    const float rep = a.repetition ? a.repetition[b] : 1.f;
    const float freq = a.frequency ? a.frequency[b] : 0.f, pres = a.presence ? a.presence[b] : 0.f;

    // token v0 + v of row t
    const auto adjusted = [&](float x, int v, int t) {
#pragma clang fp contract(off)
        const uint32_t w = count[v];
        uint32_t c = w & kTokenCount;
        bool seen = w & kTokenSeen;
        if (w & kTokenDrafted)
            for (int j = 0; j < t; ++j)
                if (path[j] == v0 + v) {
                    ++c;
                    seen = true;
                }
        if (seen) x = x > 0.f ? x / rep : x * rep;
        if (c > 0) {
            const float often = freq * (float)c;
            x = x - often;
            x = x - pres;
        }
        if (a.M > 0 && from[v]) x = x + a.bias[(int64_t)b * a.M + from[v] - 1];
        return x;
    };
    const auto number = [](Elem e) { return BF16 ? bf16_lo(e) : __uint_as_float(e); };
    const auto element = [](float x) -> Elem {
        if constexpr (BF16) return __builtin_bit_cast(uint16_t, (__bf16)x);
        else return __float_as_uint(x);
    };

    const int last_word = (a.V - 1) >> 5;
    const int slots = (a.seg + E - 1) / E + 1;              // vectors of a row that meet the segment
    for (int i = tid; i < (t1 - t0) * slots; i += kAdjustThreads) {
        const int t = t0 + i / slots;
        const Elem* row = reinterpret_cast<const Elem*>(a.logits) + b * a.seq_stride + t * a.row_stride;
        Elem* to = reinterpret_cast<Elem*>(a.out) + b * a.out_seq_stride + t * a.out_row_stride;
        const uint32_t* allowed = a.mask ? a.mask + b * a.mask_seq_stride + t * a.mask_row_stride : nullptr;
        // vectors begin where the row's store address is in line
        const int off = (int)(((uintptr_t)(to + v0) & 15) / sizeof(Elem));
        const int p = (i % slots) * E - off;                // first token of the vector in the segment
        const int lo = max(p, 0), hi = min(p + E, len);
        if (lo >= hi) continue;
        const uint32_t own = (ALL >> (E - (hi - lo))) << (lo - p);     // its elements inside the segment
        uint32_t change = lists ? (bits_at(touched, lo, (a.seg >> 5) - 1) << (lo - p)) & own : 0u;
        const uint32_t gone = allowed ? ~(bits_at(allowed, v0 + lo, last_word) << (lo - p)) & own : 0u;
        change &= ~gone;
        if (PLACE && !(change | gone)) continue;
        if (own == ALL) {
            __attribute__((aligned(16))) Elem e[E];
            if (gone == ALL) {
#pragma unroll
                for (int k = 0; k < E; ++k) e[k] = kLow;
            } else {
                const Elem* src = row + v0 + p;
                if (PLACE || ((uintptr_t)src & 15) == 0) {
                    *reinterpret_cast<u32x4_t*>(e) = *reinterpret_cast<const u32x4_t*>(src);
                } else {
#pragma unroll
                    for (int k = 0; k < E; ++k) e[k] = src[k];
                }
                if (change | gone) {
#pragma unroll
                    for (int k = 0; k < E; ++k) {
                        if (change >> k & 1) e[k] = element(adjusted(number(e[k]), p + k, t));
                        if (gone >> k & 1) e[k] = kLow;
                    }
                }
            }
            *reinterpret_cast<u32x4_t*>(to + v0 + p) = *reinterpret_cast<const u32x4_t*>(e);
        } else {
            for (int k = lo - p; k < hi - p; ++k) {
                Elem x = row[v0 + p + k];
                if (change >> k & 1) x = element(adjusted(number(x), p + k, t));
                if (gone >> k & 1) x = kLow;
                to[v0 + p + k] = x;
            }
        }
    }
}

}  // namespace df2
