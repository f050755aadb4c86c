// Microscaling formats (OCP Microscaling Formats v1.0) on gfx950's conversion
// instructions, shared by the quantiser and the MX product.
//
// A block is 32 consecutive elements of a row.  Its E8M0 byte is
//   X = max(floor(log2 max|v|) + 127 - emax, 0),   emax = 2 (E2M1), 8 (E4M3),
// that is, the exponent field of the largest magnitude less emax (an all-zero
// block and one whose largest magnitude is subnormal get 0; no finite input
// reaches 255).  X = 255 marks a block that holds a NaN or an infinity.  An
// element's code is v / 2^(X - 127) rounded to the nearest value of the format,
// ties to the even code, magnitudes past the largest value saturated to it.
#pragma once

#include "common.h"

namespace em {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kMxFp4 = 0, kMxFp8 = 1;         // E2M1, E4M3
constexpr int kMxBlock = 32, kMxStep = 128;   // elements of a scale block; of a K step (four blocks)

template <int FMT> constexpr int mx_emax() { return FMT == kMxFp4 ? 2 : 8; }

// 2^(X - 127) as a float (X = 0 is the subnormal 2^-127).
EM_DEV float e8m0_f32(int X) { return __uint_as_float(X ? (uint32_t)X << 23 : 0x00400000u); }

// Maximum over the halves of two words of bf16 magnitudes (sign bits cleared).
EM_DEV uint32_t max_u16x2(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
EM_DEV uint32_t min_u16x2(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// Largest magnitude of eight bf16 values, as bf16 bits in the low half.
EM_DEV uint32_t amax8_bf16(const uint4& v) {
    constexpr uint32_t m = 0x7FFF7FFFu;
    const uint32_t a = max_u16x2(max_u16x2(v.x & m, v.y & m), max_u16x2(v.z & m, v.w & m));
    return max(a & 0xFFFFu, a >> 16);
}

// E8M0 byte of a block from its largest magnitude's bf16 bits (or a float's
// upper 16 bits: the exponent field is the same), 255 for a non-finite one.
template <int FMT>
EM_DEV int e8m0_of(uint32_t amax_hi16) {
    const int e = (int)(amax_hi16 >> 7);
    return e == 255 ? 255 : max(e - mx_emax<FMT>(), 0);
}

// Eight bf16 values (element 2i in the low half of word i) as E2M1 codes,
// element i in nibble i.  The conversion divides by the scale, rounds to
// nearest even and saturates at 6.
EM_DEV uint32_t fp4x8_bf16(const uint4& v, float scale) {
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, v.x), scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, v.y), scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, v.z), scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, v.w), scale, 3);
    return r;
}
// Four float32 values, as 16 bits.
EM_DEV uint16_t fp4x4_f32(const float (&v)[4], float scale) {
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], scale, 1);
    return (uint16_t)r;
}

// Two bf16 values with magnitudes limited to 448 * 2^(X - 127): the E4M3
// conversion turns magnitudes that round past 448 into NaN, the format rule is
// to saturate.  The limit's bf16 bits are exact (exponent field X + 8).
EM_DEV uint32_t clamp_e4m3(uint32_t w, uint32_t lim2) {
    return (w & 0x80008000u) | min_u16x2(w & 0x7FFF7FFFu, lim2);
}
EM_DEV uint32_t e4m3_limit(int X) { return (((uint32_t)(X + 8) << 7) | 0x60u) * 0x00010001u; }

// Four bf16 values as E4M3 codes, element i in byte i.
EM_DEV uint32_t fp8x4_bf16(uint32_t w0, uint32_t w1, float scale, uint32_t lim2) {
    s16x2 r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, clamp_e4m3(w0, lim2)), scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, clamp_e4m3(w1, lim2)), scale, true);
    return __builtin_bit_cast(uint32_t, r);
}
EM_DEV uint32_t fp8x4_f32(const float* v, float scale) {
    const float lim = 448.0f * scale;
    const float a = fminf(fmaxf(v[0], -lim), lim), b = fminf(fmaxf(v[1], -lim), lim);
    const float c = fminf(fmaxf(v[2], -lim), lim), d = fminf(fmaxf(v[3], -lim), lim);
    s16x2 r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, a, b, scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c, d, scale, true);
    return __builtin_bit_cast(uint32_t, r);
}

}  // namespace em
