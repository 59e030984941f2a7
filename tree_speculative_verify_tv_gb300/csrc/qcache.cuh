// qcache.cuh -- the paged 4-bit KV cache's format: where a record keeps its codes and
// scales, and the quantiser.
#pragma once

#include "tv_internal.cuh"

namespace tv {
namespace qc {

// Byte offsets inside a record (one page of one KV head).
template <int D>
struct Rec {
    static constexpr uint32_t kGroups = D / kQGroup;
    static constexpr uint32_t kKCodes = 0;                           // [groups][64][16 B]
    static constexpr uint32_t kKScales = kKCodes + qrec_codes(D);    // [64][groups]
    static constexpr uint32_t kVCodes = kKScales + qrec_scales(D);   // [2][D][16 B]
    static constexpr uint32_t kVScales = kVCodes + qrec_codes(D);    // [groups][64]
    static constexpr uint32_t kBytes = kVScales + qrec_scales(D);
};
static_assert(Rec<64>::kBytes == qrec_bytes(64) && Rec<128>::kBytes == qrec_bytes(128), "");

constexpr uint32_t kScaleNaN = 255;

// Bit position of element e (0..7) in its 32-bit word of codes.
__device__ __forceinline__ int code_shift(int e) { return ((e >> 1) + 4 * (e & 1)) * 4; }

// Scale byte of a group whose largest |x| has the bf16 bits `amax` (sign clear): amax / 7
// rounded to four significant bits, ties to even.  The quotient is the reciprocal's product
// corrected by its residual, exact wherever amax is a multiple of 7: a tie (7 times a tie has
// at most 8 significant bits) is exact, and any other quotient is a relative 2^-12 or more
// away from one.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    const float x = __uint_as_float(amax << 16), c = 1.f / 7.f;
    const float q = x * c;
    const uint32_t r = __float_as_uint(fmaf(fmaf(-7.f, q, x), c, q));
    const int b = (int)((r + 0x7FFFFu + ((r >> 20) & 1u)) >> 20) - 840;  // 2^-22 -> 0
    // (an infinity's residual is NaN; its byte is the largest, as any beyond the range)
    return amax > 0x7F80u ? kScaleNaN : amax == 0x7F80u ? 254u : (uint32_t)min(max(b, 0), 254);
}

// With s = (8 + b % 8) 2^(b / 8 - 25), whose fp32 bits are (b + 840) << 20:
// 1 / s, raised by a relative 2^-18: |x| times this, rounded to nearest, is |x| / s
// rounded with halves away from zero.  x has 8 and s 4 significant bits, so a quotient
// that is not a half is a relative 2^-9 or more away from one, far beyond the raise, and
// the raise is far beyond the error of the approximate reciprocal (2^-22).
__device__ __forceinline__ float scale_inverse(uint32_t b) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(__uint_as_float((b + 840u) << 20)));
    return b == kScaleNaN ? 0.f : y * (1.f + 1.f / 262144.f);
}

// Adds code 1..15 of x, times `place` = 2^bit, to a word of eight: 1.5 2^23 + 8 + x / s rounds
// to an integer in the low bits of an fp32, and what the eight exponents add is taken off by
// kNoCodes, where a word starts.  One operation to place a code, on the multiplier's pipe,
// where shift and mask take two on the one that bounds the quantiser.  Only groups with b =
// 254 or 255 could leave 1..15; their values are made to fit before.
constexpr uint32_t kNoCodes = 0u - 0x4B400000u * 0x11111111u;
__device__ __forceinline__ uint32_t put_code(uint32_t word, float x, float inv, uint32_t place) {
    return __float_as_uint(fmaf(x, inv, 12582920.f)) * place + word;
}

// A pair of bf16 within +-6272, what b = 254 reaches (as packed values; a NaN becomes -6272).
__device__ __forceinline__ uint32_t clamp_pair(uint32_t x) {
    asm("min.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(0x45C445C4u));
    asm("max.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(0xC5C4C5C4u));
    return x;
}

// The larger of two packed pairs of bf16 bits without sign (as integers: NaN wins).
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// Codes 2p and 2p + 1 of a word as the bf16 pair (128 + c0, 128 + c1).  The mask and the
// exponent go in by one lop3 (the compiler makes two of the C expression, and these
// operations bound the dequantising: two cycles each per warp).
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int p) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;"
        : "=r"(d)
        : "r"(w >> (4 * p)), "r"(0x000F000Fu), "r"(0x43004300u));
    return d;
}

// Two values (the even one in the low half) s (c - 8) of word w's nibbles p and p + 4: one
// packed fma of 128 + c with s and -136 s, exactly.
__device__ __forceinline__ uint32_t value_pair(uint32_t w, int p, uint32_t s2, uint32_t ms2) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(code_pair(w, p)), "r"(s2), "r"(ms2));
    return d;
}

// bf16 bits of the scale with byte b; in both halves; and -136 times it.
__device__ __forceinline__ uint32_t scale_bf16(uint32_t b) {
    return b == kScaleNaN ? 0x7FC0u : (b << 4) + 0x3480u;
}
__device__ __forceinline__ uint32_t scale_pair(uint32_t b) {
    const uint32_t s = scale_bf16(b);
    return s | (s << 16);
}
__device__ __forceinline__ uint32_t minus_136(uint32_t s2) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(s2), "r"(0xC308C308u));  // exact
    return d;
}

}  // namespace qc
}  // namespace tv
