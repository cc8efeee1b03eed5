// MXFP4 pool rows: the layout, and the conversions of its elements and block scales.
//
// A block is 32 consecutive elements of one head: 32 E2M1 codes (sign, 2 exponent bits, 1
// mantissa bit; magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6) and one E8M0 byte e, the power of two
// 2^(e - 127) that multiplies them (e = 255: NaN), as the OCP microscaling formats define them.
// A slot's row (one for K, one for V) holds its heads in groups of hb = min(Hkv, 8):
//   [hb * D/2 bytes of codes, element 2i in the low nibble | hb * D/32 scale bytes]
// and is padded to a multiple of 16 bytes, so that any run of consecutive slots is one bulk
// copy and a decode CTA's head group is one contiguous piece of a row.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#include "device_utils.cuh"
#endif

namespace pva {
namespace mx {

constexpr int kBlock = 32;
// Block scales that the store writes: 2^-22 .. 2^13.  Every code times such a scale is an f16
// value, which is what the MMAs of the attention kernels take.
constexpr int kScaleLo = 105, kScaleHi = 140, kScaleNan = 255;

#ifdef __CUDACC__
#define PVA_HD __host__ __device__
#else
#define PVA_HD
#endif

// Bytes of one head group's codes and scales in a row.
PVA_HD inline int group_bytes(int num_kv_heads, int D) {
    const int hb = num_kv_heads < 8 ? num_kv_heads : 8;
    return hb * (D / 2 + D / kBlock);
}

PVA_HD inline int row_bytes(int num_kv_heads, int D) {
    const int hb = num_kv_heads < 8 ? num_kv_heads : 8;
    const int raw = num_kv_heads / hb * group_bytes(num_kv_heads, D);
    return (raw + 15) / 16 * 16;
}

// Byte offsets of head h's codes and scales inside a row.  (h / hb is h >> 3: with fewer than
// eight heads there is one group.)
PVA_HD inline int codes_at(int h, int num_kv_heads, int D) {
    return (h >> 3) * group_bytes(num_kv_heads, D) + (h & 7) * (D / 2);
}
PVA_HD inline int scales_at(int h, int num_kv_heads, int D) {
    const int hb = num_kv_heads < 8 ? num_kv_heads : 8;
    return (h >> 3) * group_bytes(num_kv_heads, D) + hb * (D / 2) + (h & 7) * (D / kBlock);
}

#ifdef __CUDACC__

// The two codes of byte I of x -> an f16 pair (low nibble -> low half).  Exact.
template <int I>
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t x) {
    uint32_t r;
    if constexpr (I == 0)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(x));
    else if constexpr (I == 1)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(x));
    else if constexpr (I == 2)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(x));
    else
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Eight fp32 times f -> eight codes (x[0] in the lowest nibble): nearest, ties to even, magnitudes
// above 6 saturate.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float* x, float f) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t.reg .b64 f, p, q, s, t;\n\t.reg .f32 x0, x1, x2, x3, x4, x5, x6, x7;\n\t"
        "mov.b64 f, {%9, %9};\n\t"
        "mov.b64 p, {%1, %2};\n\tmul.rn.f32x2 p, p, f;\n\tmov.b64 {x0, x1}, p;\n\t"
        "mov.b64 q, {%3, %4};\n\tmul.rn.f32x2 q, q, f;\n\tmov.b64 {x2, x3}, q;\n\t"
        "mov.b64 s, {%5, %6};\n\tmul.rn.f32x2 s, s, f;\n\tmov.b64 {x4, x5}, s;\n\t"
        "mov.b64 t, {%7, %8};\n\tmul.rn.f32x2 t, t, f;\n\tmov.b64 {x6, x7}, t;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, x1, x0;\n\tcvt.rn.satfinite.e2m1x2.f32 b, x3, x2;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, x5, x4;\n\tcvt.rn.satfinite.e2m1x2.f32 d, x7, x6;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]), "f"(f));
    return r;
}

// Scale byte -> fp32 (255 -> +inf: a NaN block's codes are stored as zeros, so that its
// elements become 0 * inf = NaN).
__device__ __forceinline__ float scale_f32(uint32_t e) { return __uint_as_float(e << 23); }

// A block scale as an f16 pair (exact for every scale the store writes); a NaN block's becomes f16's
// maximum, which leaves the block's codes zeros.
__device__ __forceinline__ uint32_t scale_f16x2_finite(uint32_t e) {
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %1;" : "=r"(r) : "f"(scale_f32(e)));
    return r;
}

// The NB scale bytes of a head (2 or 4, a row's address) -> fp32; 255 -> NaN.
template <int NB>
__device__ __forceinline__ void scales_f32(const uint8_t* at, float (&f)[NB]) {
    uint32_t w[NB / 2];  // bf16 pairs
    if constexpr (NB == 4) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.bf16x2.ue8m0x2 %0, a;\n\tcvt.rn.bf16x2.ue8m0x2 %1, b;\n\t}"
            : "=r"(w[0]), "=r"(w[1])
            : "r"(*reinterpret_cast<const uint32_t*>(at)));
    } else {
        asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(w[0]) : "h"(*reinterpret_cast<const uint16_t*>(at)));
    }
#pragma unroll
    for (int i = 0; i < NB; i += 2) {
        f[i] = __uint_as_float(w[i / 2] * 65536u);
        f[i + 1] = __uint_as_float(w[i / 2] & 0xFFFF0000u);
    }
}

// Scale byte of a block whose largest magnitude has the fp32 bits `amax` (sign cleared):
// floor(log2 amax) - 2 (the exponent of E2M1's largest binade), held to the range above; a
// block with an infinity or a NaN is a NaN block.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    const int e = (int)(amax >> 23);
    return e == 255 ? kScaleNan : (uint32_t)min(max(e - 2, kScaleLo), kScaleHi);
}

// 1 / scale, the factor that takes an element to its code's range (0 for a NaN block).
__device__ __forceinline__ float inv_scale_f32(uint32_t e) {
    return e == kScaleNan ? 0.f : __uint_as_float((254u - e) << 23);
}

#endif  // __CUDACC__

}  // namespace mx
}  // namespace pva
