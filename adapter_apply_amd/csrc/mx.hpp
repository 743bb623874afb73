// Microscaled storage: blocks of 32 values along a row share a power of two.
// A scale byte e stands for 2^(e - 127), 255 for NaN.  Elements: e2m1 (FP4,
// two codes a byte, the lower nibble first, 16 bytes a block) or two's
// complement / 64 (INT8, 32 bytes a block).  Both kinds are exact in bf16: 2
// and 7 significant bits, and no value is below bf16's smallest, 2^-133.
#pragma once

#include "common.hpp"

namespace aa {

constexpr int kMxBlock = 32;
constexpr int64_t kMxItems = (1 << 27) - 1;   // most groups of 4 blocks in a launch
inline int64_t mx_blocks(int64_t K) { return (K + kMxBlock - 1) / kMxBlock; }

struct MxArgs {
    const void *x;          // quantise: in; dequantise: out
    int64_t ldx;            // elements
    uint8_t *codes;
    int64_t ldc;            // bytes
    uint8_t *scales;
    int64_t lds;
    int64_t M;
    int32_t K;
    int32_t blocks;         // mx_blocks(K)
    uint32_t groups;        // groups of 4 blocks in a row
    uint32_t items;         // M groups
};
hipError_t launch_mx(MxArgs a, bool quantize, int32_t format, int32_t dtype, hipStream_t st);

#ifdef __HIPCC__
// 8 e2m1 codes (element 0 in the lowest nibble) to bf16; scale: the block's
// byte at a float's exponent (0 and 255 there mean 2^-127 and NaN, as in the
// scale byte).  Exact, so there is no rounding.
__device__ __forceinline__ uint4 mx_fp4_bf16(uint32_t c, uint32_t scale_bits) {
    const float s = __uint_as_float(scale_bits);
    return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3)));
}
// The factor of a block's INT8 elements, 2^(e - 127) / 64.
__device__ __forceinline__ float mx_int8_unit(uint32_t e) {
    const float s = __builtin_amdgcn_ldexpf(1.0f, (int)e - 133);
    return e == 255 ? __uint_as_float(0x7fc00000u) : s;
}
// 4 INT8 elements times their unit, to fp32 (exact).
__device__ __forceinline__ void mx_int8_f32(uint32_t c, float unit, float (&v)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)(int8_t)(c >> (8 * e)) * unit;
}
__device__ __forceinline__ uint4 mx_int8_bf16(const uint2 &c, float unit) {
    float a[4], b[4];
    mx_int8_f32(c.x, unit, a);
    mx_int8_f32(c.y, unit, b);
    return make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(b[0], b[1]),
                      pack_bf16x2(b[2], b[3]));
}
#endif

}  // namespace aa
