// Quantisation to microscaled storage and back.
//   e = floor(log2 max |v|) - m        m: 2 for e2m1 (its largest power), 0 for INT8
//   code = nearest element to v / 2^e, ties to the even code, saturating
// A block that holds an infinity or NaN gets scale 255 and reads back as NaN.
//
// The largest magnitude is an integer maximum of the values' bits, whose
// exponent field is the scale byte plus m as it stands (fields below m, and
// fp32's subnormals, give byte 0 = 2^-127).
#include "../../include/adapter_apply.h"
#include "mx.hpp"

namespace aa {

namespace {

// 16 lanes take 4 blocks (one word of scales), a lane 8 values: 16-byte loads of
// bf16, whole lines of codes per wave.  Each thread has U such items' loads in
// flight.  Bound by bytes: bf16 28672 x 4096 to 4 bits 52 us (5.7 TB/s), back 43.5 (6.8
// TB/s); 8192 x 4096 to 8 bits 20.9 us (4.9 TB/s), back 16.0.
constexpr int kMxThreads = 256;

// maximum over 4 neighbouring lanes
__device__ __forceinline__ uint32_t max4(uint32_t v) {
    const uint32_t a = __builtin_amdgcn_update_dpp(0, (int)v, 0xb1, 0xf, 0xf, false);
    v = v > a ? v : a;
    const uint32_t b = __builtin_amdgcn_update_dpp(0, (int)v, 0x4e, 0xf, 0xf, false);
    return v > b ? v : b;
}

template <bool F32>
struct Row8 { uint4 v[F32 ? 2 : 1]; };

template <bool FP4, bool F32, int U>
__global__ __launch_bounds__(kMxThreads) void k_mx_quantize(MxArgs a) {
    const int l16 = threadIdx.x & 15;
    constexpr int E = F32 ? 4 : 2;
    Row8<F32> in[U];
    int64_t row[U];
    int col[U];
    bool live[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = blockIdx.x * (U * kMxThreads / 16) + u * (kMxThreads / 16) + (threadIdx.x >> 4);
        live[u] = i < a.items;
        row[u] = live[u] ? i / a.groups : 0;
        col[u] = live[u] ? (int)(i - (uint32_t)row[u] * a.groups) * 128 + l16 * 8 : 0;
        const bool data = live[u] && col[u] < a.K;
        const char *p = static_cast<const char *>(a.x) + (row[u] * a.ldx + (data ? col[u] : 0)) * E;
#pragma unroll
        for (int h = 0; h < (F32 ? 2 : 1); ++h) {
            in[u].v[h] = ldg_nt(p + 16 * h);
            if (!data) in[u].v[h] = make_uint4(0, 0, 0, 0);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        uint32_t bits[8];                                 // the values as fp32
        const uint4 &q = in[u].v[0];
        if (F32) {
            const uint4 &r = in[u].v[F32 ? 1 : 0];
            bits[0] = q.x; bits[1] = q.y; bits[2] = q.z; bits[3] = q.w;
            bits[4] = r.x; bits[5] = r.y; bits[6] = r.z; bits[7] = r.w;
        } else {
            bits[0] = q.x << 16; bits[1] = q.x & 0xffff0000u;
            bits[2] = q.y << 16; bits[3] = q.y & 0xffff0000u;
            bits[4] = q.z << 16; bits[5] = q.z & 0xffff0000u;
            bits[6] = q.w << 16; bits[7] = q.w & 0xffff0000u;
        }
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t m = bits[e] & 0x7fffffffu;
            top = top > m ? top : m;
        }
        top = max4(top);
        const bool finite = top < 0x7f800000u;
        const uint32_t field = top >> 23, byte = !finite ? 255u : FP4 ? (field > 2 ? field - 2 : 0) : field;
        const bool block = live[u] && col[u] / kMxBlock < a.blocks;
        if (FP4) {
            const float s = __uint_as_float(byte << 23);
            uint32_t c = 0;
#define MX_PK(i) c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(bits[2 * i]), \
                                                              __uint_as_float(bits[2 * i + 1]), s, i)
            MX_PK(0);
            MX_PK(1);
            MX_PK(2);
            MX_PK(3);
#undef MX_PK
            if (block) *reinterpret_cast<uint32_t *>(a.codes + row[u] * a.ldc + col[u] / 2) = finite ? c : 0u;
        } else {
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v = __builtin_amdgcn_ldexpf(__uint_as_float(bits[e]), 133 - (int)byte);
                v = __builtin_amdgcn_fmed3f(__builtin_rintf(v), -127.0f, 127.0f);
                w[e >> 2] |= ((uint32_t)(int)v & 0xffu) << (8 * (e & 3));
            }
            if (block)
                *reinterpret_cast<uint2 *>(a.codes + row[u] * a.ldc + col[u]) =
                    finite ? make_uint2(w[0], w[1]) : make_uint2(0, 0);
        }
        // the word of 4 scales, zero past the row's blocks
        uint32_t word = block ? byte : 0u;
        word |= __shfl_xor((int)word, 4) << 8;            // (right in lanes 0 and 8 of the 16)
        word |= __shfl_xor((int)word, 8) << 16;
        if (l16 == 0 && live[u]) *reinterpret_cast<uint32_t *>(a.scales + row[u] * a.lds + col[u] / 32) = word;
    }
}

template <bool FP4, bool F32, int U>
__global__ __launch_bounds__(kMxThreads) void k_mx_dequantize(MxArgs a) {
    const int l16 = threadIdx.x & 15;
    constexpr int E = F32 ? 4 : 2;
    uint2 code[U];
    uint32_t scale[U];
    int64_t row[U];
    int col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = blockIdx.x * (U * kMxThreads / 16) + u * (kMxThreads / 16) + (threadIdx.x >> 4);
        const bool live = i < a.items;
        row[u] = live ? i / a.groups : 0;
        col[u] = live ? (int)(i - (uint32_t)row[u] * a.groups) * 128 + l16 * 8 : a.K;
        const int c = col[u] < a.K ? col[u] : 0;
        const uint8_t *p = a.codes + row[u] * a.ldc + (FP4 ? c / 2 : c);
        code[u] = FP4 ? make_uint2(ldg<uint32_t>(p), 0) : ldg<uint2>(p);
        scale[u] = a.scales[row[u] * a.lds + c / 32];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (col[u] >= a.K) continue;
        char *o = const_cast<char *>(static_cast<const char *>(a.x)) + (row[u] * a.ldx + col[u]) * E;
        if (!F32) {
            stg_nt(o, FP4 ? mx_fp4_bf16(code[u].x, scale[u] << 23) : mx_int8_bf16(code[u], mx_int8_unit(scale[u])));
            continue;
        }
        float v[8];
        if (FP4) {
            // (bf16 holds every value)
            const uint4 b = mx_fp4_bf16(code[u].x, scale[u] << 23);
            const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = bf16_lo(w[e]);
                v[2 * e + 1] = bf16_hi(w[e]);
            }
        } else {
            const float unit = mx_int8_unit(scale[u]);
            float lo[4], hi[4];
            mx_int8_f32(code[u].x, unit, lo);
            mx_int8_f32(code[u].y, unit, hi);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = lo[e];
                v[4 + e] = hi[e];
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 b = make_uint4(__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                                       __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3]));
            *reinterpret_cast<uint4 *>(o + 16 * h) = b;       // (half lines, which L2 joins)
        }
    }
}

template <bool FP4, bool F32, int U>
void quantize(const MxArgs &a, hipStream_t st) {
    const dim3 grid((a.items + U * kMxThreads / 16 - 1) / (U * kMxThreads / 16));
    hipLaunchKernelGGL((k_mx_quantize<FP4, F32, U>), grid, dim3(kMxThreads), 0, st, a);
}

// Items in flight: few where there are few, or the items' own bytes are many
// (quantise, one and four, us: bf16 1024 x 4096 3.3 and 3.6, 4096 x 4096 9.3 and 8.4,
// 28672 x 4096 56.1 and 52.2; fp32 8192 x 4096 30.8 and 33.9; two back: 43.5, one 43.3,
// four 44.7).
template <bool FP4, bool F32>
hipError_t run(const MxArgs &a, bool q, hipStream_t st) {
    if (q) {
        if (!F32 && a.items >= 1 << 17) quantize<FP4, F32, F32 ? 1 : 4>(a, st);
        else quantize<FP4, F32, 1>(a, st);
        return hipGetLastError();
    }
    constexpr int U = 2;
    const dim3 grid((a.items + U * kMxThreads / 16 - 1) / (U * kMxThreads / 16));
    hipLaunchKernelGGL((k_mx_dequantize<FP4, F32, U>), grid, dim3(kMxThreads), 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx(MxArgs a, bool quantize, int32_t format, int32_t dtype, hipStream_t st) {
    a.blocks = (int32_t)mx_blocks(a.K);
    a.groups = (uint32_t)((a.blocks + 3) / 4);
    const bool f32 = dtype == LORA_DT_F32;
    // (rows of one launch: its threads, at most 16 an item, stay under 2^32; only a projection
    // that is restored has more)
    const int64_t rows = a.M, most = kMxItems / a.groups;
    for (int64_t r = 0; r < rows; r += most) {
        a.M = rows - r < most ? rows - r : most;
        a.items = (uint32_t)(a.M * a.groups);
        hipError_t e;
        if (format == LORA_MX_FP4) e = f32 ? run<true, true>(a, quantize, st) : run<true, false>(a, quantize, st);
        else e = f32 ? run<false, true>(a, quantize, st) : run<false, false>(a, quantize, st);
        if (e != hipSuccess) return e;
        a.x = static_cast<const char *>(a.x) + a.M * a.ldx * (f32 ? 4 : 2);
        a.codes += a.M * a.ldc;
        a.scales += a.M * a.lds;
    }
    return hipSuccess;
}

}  // namespace aa
