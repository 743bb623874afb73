// Gradient kernels of the adapter layer, per slice s and slot i = idx[t]:
//   v[t][j]  = scale sum_n dy[t][n] B[i][n][j]            (k_lin_du)
//   dB[i][n][j] = sum_{t of i} dy[t][n] (scale u[t][j])   (k_lin_wg)
//   dA[i][j][k] = sum_{t of i} v[t][j] x[t][k]            (k_lin_wg, transposed output)
// dx is the tile GEMM of linear.hip.  The contraction index of these products
// is the slow index of lora_b, dy, x and the rank vectors, so those operands
// reach the MFMA through transposed LDS reads.  All sums are fp32, in a fixed
// order (no atomics); splits are summed in order by a kernel of their own.
#include "linear.hpp"

namespace aa {

namespace {

typedef float floatx4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ bf16x8_t frag2(const uint2 &a, const uint2 &b) {
    return __builtin_bit_cast(bf16x8_t, make_uint4(a.x, a.y, b.x, b.y));
}

// Units of a transposed-read row are moved in 32-byte pairs by the row's low
// bits, so that the 4 rows of one transposed read (and 8 rows of two lane
// groups, where the row has 8 pairs) lie in different banks.
template <int CPR>
__device__ __forceinline__ int tr_swz(int row) {
    return CPR == 2 ? 0 : CPR == 4 ? 0 : CPR == 8 ? (row & 3) << 1 : ((row & 3) | ((row >> 3) & 1) << 2) << 1;
}
// Transposed fragment: 8 rows 32 kk + 8 g.. of columns col0..+15.
template <int CPR>
__device__ __forceinline__ bf16x8_t tr_frag(const char *st, int col0, int kk, int lane) {
    const int g = lane >> 4, l16 = lane & 15;
    const int row = kk * 32 + g * 8 + (l16 >> 2), col = col0 + (l16 & 3) * 4;
    const char *p = st + row * (CPR * 16) + ((((col >> 3) ^ tr_swz<CPR>(row)) << 4) | ((col & 4) << 1));
    return frag2(tr_read(p), tr_read(p + 4 * CPR * 16));
}

constexpr int kPadThreads = 256;
struct PadArgs {
    const uint16_t *dy;
    int64_t lddy;
    int32_t T, S;
    PadMap m;
    uint16_t *out;
    int64_t ldo;
};
// dy with every slice padded by zeros to whole 8-element units (widths that
// are multiples of 4 only): 8 bytes per thread.  Bound by its bytes (1501 x 1652:
// 5.3 us); reading the unpadded rows in the kernels would cost each of them the
// 16-byte loads.
__global__ __launch_bounds__(kPadThreads) void k_lin_pad(PadArgs a) {
    const int64_t units = a.ldo / 4, total = units * a.T;
    for (int64_t q = (int64_t)blockIdx.x * kPadThreads + threadIdx.x; q < total;
         q += (int64_t)gridDim.x * kPadThreads) {
        const int64_t t = q / units, c = (q - t * units) * 4;
        uint2 v = make_uint2(0, 0);
        for (int s = 0; s < a.S; ++s) {
            const int64_t d = c - a.m.dst[s];
            if (d >= 0 && d < a.m.n[s]) v = ldg<uint2>(a.dy + t * a.lddy + a.m.src[s] + d);
        }
        *reinterpret_cast<uint2 *>(a.out + t * a.ldo + c) = v;
    }
}

// v: work-group = (tile of at most 64 tokens of one slot, slice, RB ranks,
// split of the slice's columns), 4 waves of 16 tokens.  A stage is 64 columns
// of dy's rows and 64 rows of lora_b, three in flight.  Bound by bytes: 8192 tokens
// of 28672 columns, dy's 470 MB and what lora_b's tiles read again, 680 MB past L2
// in 102 us.
struct DuArgs {
    const uint16_t *dy;
    int64_t lddy;
    int64_t poff[kMaxSlices], n[kMaxSlices];
    const uint16_t *b[kMaxSlices];
    int32_t T, S, L, R, nrb, nsp;
    SegPtrs seg;
    float *part;
};
constexpr int kDuStages = 3;

template <int RB>
__global__ __launch_bounds__(256) void k_lin_du(DuArgs a) {
    constexpr int PB = 64 * 128, QB = 64 * RB * 2, CPR = RB / 8, RPI = 64 / CPR;
    constexpr int QI = QB / 4096, NB = RB / 16;
    static_assert(QI >= 1, "whole DMA instructions per wave");
    __shared__ __attribute__((aligned(16))) char s_stage[kDuStages][PB + QB];
    if ((int)blockIdx.x >= a.seg.header[3]) return;
    const int4 tl = a.seg.tiles_pre[blockIdx.x];
    const int slot = tl.x, p0 = tl.y, ntok = tl.z - tl.y;
    const int s = blockIdx.y / a.nrb, r0 = (blockIdx.y - s * a.nrb) * RB;
    const int64_t n = a.n[s];
    const int nst_all = (int)((n + 63) / 64), per = (nst_all + a.nsp - 1) / a.nsp;
    const int sb = blockIdx.z * per, nst = max(0, min(per, nst_all - sb));
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);

    const void *zero = g_zero16;
    const int plc = (lane & 7) ^ (((w * 8 + (lane >> 3)) >> 1) & 7);
    const uint16_t *pp[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = (i * 4 + w) * 8 + (lane >> 3);
        pp[i] = a.dy + (int64_t)a.seg.perm[p0 + min(row, ntok - 1)] * a.lddy + a.poff[s] + plc * 8;
    }
    auto qrow = [&](int i) { return (i * 4 + w) * RPI + lane / CPR; };
    const uint16_t *qp[QI];
    bool qin[QI];
#pragma unroll
    for (int i = 0; i < QI; ++i) {
        const int j = r0 + ((lane % CPR) ^ tr_swz<CPR>(qrow(i))) * 8;
        qin[i] = j < a.R;
        qp[i] = a.b[s] + ((int64_t)slot * n + qrow(i)) * a.R + (qin[i] ? j : 0);
    }
    auto issue = [&](int v, int stage) {
        const int64_t c = (int64_t)(sb + v) * 64, rem = n - c;
        const uint32_t pl = lds_addr(&s_stage[stage][0]) + w * 1024, ql = pl + PB;
#pragma unroll
        for (int i = 0; i < 2; ++i) dma16(pl + i * 4096, plc * 8 < rem ? (const void *)(pp[i] + c) : zero);
#pragma unroll
        for (int i = 0; i < QI; ++i)
            dma16(ql + i * 4096, qin[i] && qrow(i) < rem ? (const void *)(qp[i] + c * a.R) : zero);
    };
    floatx4_t acc[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) acc[i] = floatx4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kDuStages - 1; ++i)
        if (i < nst) issue(i, i);
    int stage = 0;
    for (int v = 0; v < nst; ++v) {
        if (v + kDuStages - 2 < nst) wait_barrier<(kDuStages - 2) * (2 + QI)>();
        else wait_barrier<0>();
        if (v + kDuStages - 1 < nst) {
            const int ns = stage + kDuStages - 1;
            issue(v + kDuStages - 1, ns >= kDuStages ? ns - kDuStages : ns);
        }
        const char *st = s_stage[stage];
        const int row = w * 16 + l16;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const bf16x8_t p = __builtin_bit_cast(
                bf16x8_t, *reinterpret_cast<const uint4 *>(st + row * 128 + (((kk * 4 + g) ^ ((row >> 1) & 7)) << 4)));
#pragma unroll
            for (int i = 0; i < NB; ++i)
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(tr_frag<CPR>(st + PB, i * 16, kk, lane), p,
                                                                 acc[i], 0, 0, 0);
        }
        if (++stage == kDuStages) stage = 0;
    }
    const int row = w * 16 + l16;
    if (row >= ntok) return;
    float *o = a.part + (((int64_t)s * a.nsp + blockIdx.z) * a.T + p0 + row) * a.R;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int j = r0 + i * 16 + 4 * g;
        if (j < a.R) *reinterpret_cast<floatx4_t *>(o + j) = acc[i];
    }
}

// Weight gradients: work-group = (128 columns of a slice, RB ranks, slot,
// token split), 4 waves of 32 columns, 32 tokens per stage (both operands
// through transposed reads; the rank vectors' three bf16 parts, which hold the
// whole fp32 value, add into the same accumulators).  Slots without tokens
// write zeros.  Bound by its bytes: 8192 tokens, 4096 -> 28672, rank 64, 16 slots,
// 700 MB past L2 in 170 us (median of 24, 164 to 203; 250 with two stages of 64
// tokens); 4096 tokens, 14336 -> 4096, rank 32, 170 MB in 36 us.
constexpr int kWgCols = 128;
constexpr int kWgTokens = 1024;       // token indexes staged at a time
constexpr int kWgStep = 32;           // tokens per stage
constexpr int kWgStages = 3;

template <int RB>
struct WgLds {
    static constexpr int kStage = kWgStep * kWgCols * 2 + kLinPartsBwd * kWgStep * RB * 2;
    __attribute__((aligned(16))) char stage[kWgStages][kStage];
    int tok[kWgTokens];
};

template <int RB, bool TRANSPOSED>
__device__ __forceinline__ void wg_tile(const LinWgArgs &a, int nrb, int bx, WgLds<RB> &sh) {
    constexpr int NP = kLinPartsBwd;
    constexpr int TK = kWgStep, NST = kWgStages;
    constexpr int PB = TK * kWgCols * 2, QB = TK * RB * 2;      // bytes of a stage's p rows and of one part
    constexpr int CPP = kWgCols / 8, CPQ = RB / 8, RPP = 64 / CPP, RPQ = 64 / CPQ;
    constexpr int PI = PB / 4096, QN = NP * QB / 1024, NB = RB / 16;
    auto &s_stage = sh.stage;
    auto &s_tok = sh.tok;
    int s = 0;
    const int mt_all = bx / nrb, r0 = (bx - mt_all * nrb) * RB;
    while (s + 1 < a.S && mt_all >= a.tile_start[s + 1]) ++s;
    const int64_t m0 = (int64_t)(mt_all - a.tile_start[s]) * kWgCols, M = a.m[s];
    const int slot = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    int b = a.seg.slot_start[slot], e = a.seg.slot_start[slot + 1];
    {
        // this split's share, in whole stages
        const int per = ((e - b + a.nsp - 1) / a.nsp + TK - 1) / TK * TK;
        b = min(b + (int)blockIdx.z * per, e);
        e = min(b + per, e);
    }
    const void *zero = g_zero16;
    const int hlr = NP * a.R;
    const uint16_t *hl = a.hl + (int64_t)s * a.T * hlr;

    floatx4_t acc[2][NB];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};

    for (int cb = b; cb < e; cb += kWgTokens) {
        const int cnt = min(kWgTokens, e - cb), nst = (cnt + TK - 1) / TK;
        __syncthreads();
        for (int i = tid; i < cnt; i += 256) s_tok[i] = a.seg.perm[cb + i];
        __syncthreads();
        auto issue = [&](int v, int stage) {
            const uint32_t pl = lds_addr(&s_stage[stage][0]) + w * 1024, ql = pl + PB;
#pragma unroll
            for (int i = 0; i < PI; ++i) {
                const int row = (i * 4 + w) * RPP + lane / CPP, tk = v * TK + row;
                const int64_t c = m0 + ((lane % CPP) ^ tr_swz<CPP>(row)) * 8;
                const bool in = tk < cnt && c < M;
                dma16(pl + i * 4096,
                      in ? (const void *)(a.p + (int64_t)s_tok[in ? tk : 0] * a.ldp + a.poff[s] + c) : zero);
            }
#pragma unroll
            for (int i = 0; i < (QN + 3) / 4; ++i) {
                const int q = i * 4 + w;                       // DMA instruction: part, rows
                if (QN % 4 && q >= QN) break;
                const int part = q / (QB / 1024), row = (q % (QB / 1024)) * RPQ + lane / CPQ, tk = v * TK + row;
                const int j = r0 + ((lane % CPQ) ^ tr_swz<CPQ>(row)) * 8;
                const bool in = tk < cnt && j < a.R;
                dma16(ql + i * 4096,
                      in ? (const void *)(hl + (int64_t)s_tok[in ? tk : 0] * hlr + part * a.R + j) : zero);
            }
        };
        // a wave issues at least kLoads per stage, so waiting for all but
        // NST - 2 times that many leaves no load of the oldest stage open
        constexpr int kLoads = PI + QN / 4;
#pragma unroll
        for (int i = 0; i < NST - 1; ++i)
            if (i < nst) issue(i, i);
        int stage = 0;
        for (int v = 0; v < nst; ++v) {
            if (v + NST - 2 < nst) wait_barrier<(NST - 2) * kLoads>();
            else wait_barrier<0>();
            if (v + NST - 1 < nst) {
                const int ns = stage + NST - 1;
                issue(v + NST - 1, ns >= NST ? ns - NST : ns);
            }
            const char *st = s_stage[stage];
            if (++stage == NST) stage = 0;
#pragma unroll
            for (int kk = 0; kk < TK / 32; ++kk) {
                bf16x8_t p[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) p[i] = tr_frag<CPP>(st, w * 32 + i * 16, kk, lane);
#pragma unroll
                for (int h = 0; h < NP; ++h)
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        const bf16x8_t q = tr_frag<CPQ>(st + PB + h * QB, j * 16, kk, lane);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            acc[i][j] = TRANSPOSED
                                ? __builtin_amdgcn_mfma_f32_16x16x32_bf16(p[i], q, acc[i][j], 0, 0, 0)
                                : __builtin_amdgcn_mfma_f32_16x16x32_bf16(q, p[i], acc[i][j], 0, 0, 0);
                    }
            }
        }
    }

    float *out = a.nsp > 1 ? a.part + (int64_t)blockIdx.z * a.part_stride + a.part_off[s] : a.out[s];
    const bool add = a.accumulate && a.nsp == 1;
    const int rank = a.slot_rank ? a.slot_rank[slot] : a.R;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            // TRANSPOSED: lane holds rank l16, columns 4 g..; else column l16, ranks 4 g..
            const int64_t m = m0 + w * 32 + i * 16 + (TRANSPOSED ? 4 * g : l16);
            const int r = r0 + j * 16 + (TRANSPOSED ? l16 : 4 * g);
            if (m >= M || r >= a.R) continue;
            const int64_t o = TRANSPOSED ? ((int64_t)slot * a.R + r) * M + m : ((int64_t)slot * M + m) * a.R + r;
            floatx4_t *dst = reinterpret_cast<floatx4_t *>(out + o);
            floatx4_t v = acc[i][j];
            // ranks past the slot's own are zero, whatever the rows hold (an
            // infinity times the zero rank vector is NaN)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (r + (TRANSPOSED ? 0 : q) >= rank) v[q] = 0.f;
            if (add) {
                const floatx4_t old = *dst;
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] += old[q];
            }
            *dst = v;
        }
}

struct WgJobs {
    LinWgArgs a, b;      // dA (transposed), dB
    int32_t na, nrb;     // work-groups of a along x
};
template <int RB>
__global__ __launch_bounds__(256) void k_lin_wg(WgJobs j) {
    __shared__ WgLds<RB> sh;
    const int bx = blockIdx.x;
    if (bx < j.na) {
        if ((int)blockIdx.z < j.a.nsp) wg_tile<RB, true>(j.a, j.nrb, bx, sh);
    } else if ((int)blockIdx.z < j.b.nsp) {
        wg_tile<RB, false>(j.b, j.nrb, bx - j.na, sh);
    }
}

// Sum of the token splits, in order (z: dA, dB).
__global__ __launch_bounds__(256) void k_lin_wsum(WgJobs j) {
    const LinWgArgs &a = blockIdx.z ? j.b : j.a;
    const int s = blockIdx.y;
    const int64_t q = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (a.nsp <= 1 || q >= (int64_t)a.L * a.R * a.m[s]) return;
    floatx4_t *dst = reinterpret_cast<floatx4_t *>(a.out[s] + q);
    floatx4_t v = {0.f, 0.f, 0.f, 0.f};
    if (a.accumulate) v = *dst;
#pragma unroll 4
    for (int k = 0; k < a.nsp; ++k) {
        const floatx4_t o = *reinterpret_cast<const floatx4_t *>(a.part + k * a.part_stride + a.part_off[s] + q);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += o[e];
    }
    *dst = v;
}

int du_rb(int32_t R) { return R <= 32 ? 32 : R <= 64 ? 64 : 128; }
int wg_rb(int32_t R) { return R <= 16 ? 16 : R <= 32 ? 32 : 64; }

}  // namespace

hipError_t launch_lin_pad(const void *dy, int64_t lddy, int32_t T, int32_t S, const PadMap &m,
                          uint16_t *out, int64_t ldo, hipStream_t st) {
    PadArgs a{};
    a.dy = static_cast<const uint16_t *>(dy); a.lddy = lddy; a.T = T; a.S = S; a.m = m;
    a.out = out; a.ldo = ldo;
    const int64_t blocks = ((int64_t)T * (ldo / 4) + kPadThreads - 1) / kPadThreads;
    hipLaunchKernelGGL(k_lin_pad, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(kPadThreads), 0,
                       st, a);
    return hipGetLastError();
}

// Splits of the columns: about 1024 work-groups, at most 16 splits of at
// least 4 stages of the widest slice.
int32_t lin_du_splits(int32_t T, int32_t L, const int64_t *N, int32_t S, int32_t R) {
    const int rb = du_rb(R);
    const int64_t base = (int64_t)max_tiles(T, L, kPreTile) * S * ((R + rb - 1) / rb);
    int64_t widest = 0;
    for (int s = 0; s < S; ++s) widest = N[s] > widest ? N[s] : widest;
    int64_t k = 1024 / base;
    if (k > widest / 256) k = widest / 256;
    if (k > 16) k = 16;
    return k < 1 ? 1 : (int32_t)k;
}

hipError_t launch_lin_du(const uint16_t *dy, int64_t lddy, const int64_t *poff, int32_t T,
                         const Slices &sl, int32_t S, int32_t L, int32_t R, const SegPtrs &seg, float *part,
                         int32_t nsp, hipStream_t st) {
    DuArgs a{};
    a.dy = dy; a.lddy = lddy; a.T = T; a.S = S; a.L = L; a.R = R; a.seg = seg; a.part = part;
    a.nsp = nsp;
    for (int s = 0; s < S; ++s) {
        a.poff[s] = poff[s];
        a.n[s] = sl.n[s];
        a.b[s] = static_cast<const uint16_t *>(sl.b[s]);
    }
    const int rb = du_rb(R);
    a.nrb = (R + rb - 1) / rb;
    const dim3 grid((unsigned)seg.max_tiles_pre, (unsigned)(S * a.nrb), (unsigned)nsp);
    switch (rb) {
        case 32: hipLaunchKernelGGL(k_lin_du<32>, grid, dim3(256), 0, st, a); break;
        case 64: hipLaunchKernelGGL(k_lin_du<64>, grid, dim3(256), 0, st, a); break;
        default: hipLaunchKernelGGL(k_lin_du<128>, grid, dim3(256), 0, st, a); break;
    }
    return hipGetLastError();
}

// Token splits while the (column tile, rank block, slot) work-groups of both
// gradients are few: about 1024 work-groups, splits of at least 256 of a slot's
// tokens on average (shorter ones cost their launch more than they save: 1501
// tokens over 7 slots, 1652 x 1352, rank 40: 78 us with three splits, 71
// without), partial sums within kLinWgPartMax elements each.
int32_t lin_wg_splits(int32_t T, int32_t L, const int64_t *MA, const int64_t *MB, int32_t S, int32_t R) {
    int64_t tiles = 0, cols = 0;
    for (const int64_t *M : {MA, MB}) {
        int64_t c = 0;
        for (int s = 0; M && s < S; ++s) {
            tiles += (M[s] + kWgCols - 1) / kWgCols;
            c += M[s];
        }
        if (c > cols) cols = c;
    }
    const int rb = wg_rb(R);
    int64_t k = 1024 / (tiles * L * ((R + rb - 1) / rb));
    if (k > T / L / 256) k = T / L / 256;
    if (k > 16) k = 16;
    while (k > 1 && k * L * R * cols > kLinWgPartMax) --k;
    return k < 1 ? 1 : (int32_t)k;
}

int64_t lin_wg_part(int32_t L, const int64_t *M, int32_t S, int32_t R) {
    int64_t n = 0;
    for (int s = 0; s < S; ++s) n += (int64_t)L * R * M[s];
    return n;
}

hipError_t launch_lin_wg(const LinWgArgs *dA, const LinWgArgs *dB, hipStream_t st) {
    WgJobs j{};
    const LinWgArgs &any = dA ? *dA : *dB;
    const int rb = wg_rb(any.R);
    j.nrb = (any.R + rb - 1) / rb;
    int nx = 0, nsp = 1;
    int64_t widest = 0;
    auto fill = [&](const LinWgArgs &in, LinWgArgs &a) {
        a = in;
        int c = 0;
        int64_t off = 0;
        for (int s = 0; s < a.S; ++s) {
            a.tile_start[s] = c;
            c += (int)((a.m[s] + kWgCols - 1) / kWgCols);
            a.part_off[s] = off;
            off += (int64_t)a.L * a.R * a.m[s];
            if (a.nsp > 1 && a.m[s] > widest) widest = a.m[s];
        }
        for (int s = a.S; s <= kMaxSlices; ++s) a.tile_start[s] = c;
        a.part_stride = off;
        if (a.nsp > nsp) nsp = a.nsp;
        nx += c * j.nrb;
    };
    if (dA) fill(*dA, j.a);
    j.na = nx;
    if (dB) fill(*dB, j.b);
    const dim3 grid((unsigned)nx, (unsigned)any.L, (unsigned)nsp);
    switch (rb) {
        case 16: hipLaunchKernelGGL(k_lin_wg<16>, grid, dim3(256), 0, st, j); break;
        case 32: hipLaunchKernelGGL(k_lin_wg<32>, grid, dim3(256), 0, st, j); break;
        default: hipLaunchKernelGGL(k_lin_wg<64>, grid, dim3(256), 0, st, j); break;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || nsp == 1) return e;
    const int64_t units = (int64_t)any.L * any.R * widest / 4;
    hipLaunchKernelGGL(k_lin_wsum, dim3((unsigned)((units + 255) / 256), (unsigned)any.S, 2), dim3(256), 0, st, j);
    return hipGetLastError();
}

}  // namespace aa
