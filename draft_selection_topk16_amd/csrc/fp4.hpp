// The 4-bit paged cache: the microscaling format of 4-bit floats (sign, two bits of
// exponent, one of mantissa: magnitudes 0, 1/2, 1, 3/2, 2, 3, 4, 6) in blocks of 32
// neighbouring elements of a head with one power of two each.  A page holds, for
// each head, its tokens' codes (D / 2 bytes a token, the first of two in the low half
// of a byte), then their scales (D / 32 bytes a token: the exponent plus 127).
//
// The scale is the smallest power of two, of 2^-120 to 2^120, of which the block's
// largest magnitude is at most 7: then clipping to 6 costs no more than rounding
// between 4 and 6 does.  Codes are the nearest values, ties to the even code.  All
// values are exact in bf16 (two bits of mantissa), so attention multiplies bf16
// numbers and loses nothing over the codes.
#pragma once

#include "common.hpp"
#include "lanes.hpp"

namespace df2 {

constexpr int kFp4Block = 32;
constexpr int kFp4Bias = 127, kFp4Least = -120, kFp4Most = 120;
constexpr uint32_t kFp4NaN = 255;       // scale of a block that holds an infinity or NaN

typedef float f32x2v_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2v_t __attribute__((ext_vector_type(2)));

// Bytes of one head of a page, and where its scales begin.
template <int D>
struct Fp4Page {
    static constexpr int kCodes = D / 2, kScales = D / kFp4Block;     // of a token
    static __host__ __device__ __forceinline__ int64_t bytes(int page_shift) {
        return (int64_t)(kCodes + kScales) << page_shift;
    }
    static __host__ __device__ __forceinline__ int64_t scales(int page_shift) { return (int64_t)kCodes << page_shift; }
};

// Exponent of a block's scale from the bits of its largest magnitude, and the byte
// that stands for it.  1.75 * 2^k is 7 * 2^(k - 2).
__device__ __forceinline__ int fp4_exponent(uint64_t top) {
    const int e = (int)(top >> 52) - 1023 - 2 + ((top & ((1ull << 52) - 1)) > (3ull << 50) ? 1 : 0);
    return min(max(e, kFp4Least), kFp4Most);
}
__device__ __forceinline__ uint32_t fp4_scale_byte(uint64_t top, int e) {
    return (top >> 52) == 0x7FF ? kFp4NaN : (uint32_t)(e + kFp4Bias);
}

// x to fp32 such that rounding the result to 4 bits is rounding x: cut off, and the
// last bit set where anything was lost (a value next to a border of two codes does
// not land on it).
__device__ __forceinline__ float to_odd(double x) {
    const float f = (float)x;
    const double back = (double)f;
    uint32_t w = __float_as_uint(f);
    w -= fabs(back) > fabs(x) ? 1u : 0u;
    w |= back != x ? 1u : 0u;
    return __uint_as_float(w);
}

// Codes of pairs of numbers that are already divided by the scale.
template <int BYTE>
__device__ __forceinline__ uint32_t fp4_pair(uint32_t into, float lo, float hi) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(into, lo, hi, 1.f, BYTE);
}

// The scale as the conversions take it: they use the exponent bits only, so 255 is
// NaN, which makes every value of the block one.
__device__ __forceinline__ float fp4_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight codes as eight bf16, and as eight floats.
__device__ __forceinline__ u32x4_t fp4_to_bf16(uint32_t codes, float scale) {
    u32x4_t w;
    w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
    w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
    w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
    w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
    return w;
}
__device__ __forceinline__ void fp4_to_f32(uint32_t codes, float scale, f32x4_t& lo, f32x4_t& hi) {
    const f32x2v_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 0);
    const f32x2v_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 1);
    const f32x2v_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 2);
    const f32x2v_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 3);
    lo = (f32x4_t){a[0], a[1], b[0], b[1]};
    hi = (f32x4_t){c[0], c[1], d[0], d[1]};
}

// ----------------------------------------------------------------------------
// What a cache holds, as numbers: eight codes a thread, read as four bytes and
// written as 16 (bf16) or 32.  Two caches, 36 million values in all, to bf16: 12 us for 92 MB,
// which the last-level cache helps (14 in an append's pass); to fp32 55 us for 164 MB, 3.0 TB/s.
// ----------------------------------------------------------------------------
struct UnpackArgs {
    const uint8_t* cache[2];    // keys and values
    void* out[2];
    int64_t page_stride, items; // bytes; eights of codes in one cache
    int Hkv, page_shift;
};
constexpr int kUnpackThreads = 256;

template <bool BF16, int D>
__global__ __launch_bounds__(kUnpackThreads) void k_unpack_fp4(UnpackArgs a) {
    const uint8_t* cache = a.cache[blockIdx.y];
    const int64_t i = (int64_t)blockIdx.x * kUnpackThreads + threadIdx.x;
    if (i >= a.items) return;
    constexpr int kEights = D / 8;
    const int in_head = (int)(i & (((int64_t)kEights << a.page_shift) - 1));
    const int64_t head = i / kEights >> a.page_shift;         // page * Hkv + head
    const int64_t page = (int64_t)((uint64_t)head / (uint32_t)a.Hkv);
    const uint8_t* from = cache + page * a.page_stride + (head - page * a.Hkv) * Fp4Page<D>::bytes(a.page_shift);
    const uint32_t codes = *reinterpret_cast<const uint32_t*>(from + 4 * in_head);
    const float scale = fp4_scale(from[Fp4Page<D>::scales(a.page_shift) + in_head / (kFp4Block / 8)]);
    if constexpr (BF16) {
        __builtin_nontemporal_store(fp4_to_bf16(codes, scale), reinterpret_cast<u32x4_t*>(a.out[blockIdx.y]) + i);
    } else {
        f32x4_t lo, hi;
        fp4_to_f32(codes, scale, lo, hi);
        __builtin_nontemporal_store(lo, reinterpret_cast<f32x4_t*>(a.out[blockIdx.y]) + 2 * i);
        __builtin_nontemporal_store(hi, reinterpret_cast<f32x4_t*>(a.out[blockIdx.y]) + 2 * i + 1);
    }
}

}  // namespace df2
