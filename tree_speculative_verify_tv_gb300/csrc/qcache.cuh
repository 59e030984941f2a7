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
// rounded to four significant bits, ties to even.  amax / 7 needs no more care than one
// correctly rounded fp32 division: 7 times a tie has at most 8 significant bits, so a
// quotient that is a tie is exact, and any other is a relative 2^-12 or more away.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    const uint32_t r = __float_as_uint(__fdiv_rn(__uint_as_float(amax << 16), 7.f));
    const int b = (int)((r + 0x7FFFFu + ((r >> 20) & 1u)) >> 20) - 840;  // 2^-22 -> 0
    return amax > 0x7F80u ? kScaleNaN : (uint32_t)min(max(b, 0), 254);
}

// s = (8 + b % 8) 2^(b / 8 - 25) as fp32; NaN for b = 255.
__device__ __forceinline__ float scale_value(uint32_t b) {
    return b == kScaleNaN ? __uint_as_float(0x7FC00000u) : __uint_as_float((b + 840u) << 20);
}

// 1 / s, raised by a relative 2^-18: |x| times this, rounded to nearest, is |x| / s
// rounded with halves away from zero.  x has 8 and s 4 significant bits, so a quotient
// that is not a half is a relative 2^-9 or more away from one, far beyond the raise.
__device__ __forceinline__ float scale_inverse(uint32_t b) {
    return b == kScaleNaN ? 0.f
                          : __fdiv_rn(1.f + 1.f / 262144.f, __uint_as_float((b + 840u) << 20));
}

// Code 1..15 of the bf16 value with bits `x` (any code for a NaN: its scale says NaN).
__device__ __forceinline__ uint32_t code(uint32_t x, float inv) {
    const float a = fminf(__uint_as_float((x & 0x7FFFu) << 16) * inv, 7.f);
    const int q = __float2int_rn(a);
    return (uint32_t)(8 + ((x & 0x8000u) ? -q : q));
}

}  // namespace qc
}  // namespace tv
