// A few tokens (decode) beside a 4-bit projection.  k_mx_few, first of two launches:
// fp32 sums of x W^T and of the rank vectors x A^T over K splits, which k_lin_join_rows
// adds up.  k_mx_one, one token: all in one launch.
// Codes go straight from global memory into 16x16x32 MFMA fragments (a lane loads a
// whole block, 16 bytes, and x meets it in that order, 4 fragments a block), x through
// LDS.  A split's codes are in flight together where registers allow, so a call is
// some round trips to memory and its bytes: one token of 4096 x 6144, rank 16, 9.5 us
// (14 MB; 5 us and 2.8 TB/s fit one token's sizes); 16 tokens of 14336 x 4096, 16 slots, 14.8
// us (38 MB, 31 of them codes and scales, those at 2.1 TB/s: the CUs hold 512 work-groups
// at once, the columns' alone, and the 256 of the rank vectors take their places as they
// end) and 5.4 of the join.
#include "linear.hpp"
#include "mx.hpp"

namespace aa {

namespace {

typedef float floatx4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ bf16x8_t frag(const uint4 &u) { return __builtin_bit_cast(bf16x8_t, u); }

// Work-group = 8 waves.  Base: 4 x 16 CT output columns (4 waves side by side, each
// pair's K steps alternating), 16 TB tokens, one K split.  Rank vectors: up to 64 ranks
// of one slice, the y-th different slot among the tokens, one K split; the waves share
// the blocks of 16 ranks and K.
constexpr int kMfWaves = 8;
constexpr int kMfStep = 128;                      // K steps of a lane group's 4 blocks
struct FewArgs {
    LinArgs l;
    int32_t per;              // K steps of kMfStep per split
    int32_t col_tiles;
    int32_t slots;            // different slots that the tokens can name
    int32_t rank_waves;       // blocks of 16 ranks in a work-group: 1, 2 or 4
    int32_t rank_groups;
};

template <int TB, int CT, int CH, bool MULTI>
struct FewLds {
    uint4 x[MULTI ? 2 : 1][CH][TB * 16][16];      // [chunk][step][token][unit ^ token]
    floatx4_t sum[4][CT * TB][64];
};

template <int TB, int CT, int CH, bool MULTI>
__device__ __forceinline__ void few_base(const FewArgs &f, FewLds<TB, CT, CH, MULTI> &sh) {
    const LinArgs &a = f.l;
    constexpr int U = CH / 2, XU = CH * TB * 16 * 16 / (kMfWaves * 64);
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, cw = w & 3, kw = w >> 2;
    const int l16 = lane & 15, g = lane >> 4;
    int sc = 0;
    while (sc + 1 < a.S && (int)blockIdx.x >= a.tile_start[sc + 1]) ++sc;
    const int64_t c0 = (int64_t)(blockIdx.x - a.tile_start[sc]) * (64 * CT) + cw * (16 * CT), cend = a.n[sc];
    const int blocks = (a.K + kMxBlock - 1) / kMxBlock, steps = (blocks + 3) / 4;
    const int first = (int)blockIdx.y * f.per, last = min(first + f.per, steps);

    const uint8_t *wr[CT], *sr[CT];
#pragma unroll
    for (int i = 0; i < CT; ++i) {
        const int64_t n = a.off[sc] + min(c0 + i * 16 + l16, cend - 1);
        wr[i] = reinterpret_cast<const uint8_t *>(a.w) + n * a.ldw;
        sr[i] = a.ws + n * a.ldws;
    }
    floatx4_t acc[CT][TB];
#pragma unroll
    for (int i = 0; i < CT; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};

    // A chunk: the wave's U steps of codes (neighbouring ones, whole lines of 128 bytes a
    // row) and a share of all its x, in registers.
    struct Chunk {
        uint4 code[U][CT];
        u32x4_t x[XU];
        uint32_t scale[U][CT];
    };
    auto load = [&](Chunk &c, int s0) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int st = min(s0 + kw * U + u, steps - 1), b = min(st * 4 + g, blocks - 1);
#pragma unroll
            for (int i = 0; i < CT; ++i) {
                c.code[u][i] = ldg<uint4>(wr[i] + b * 16);
                c.scale[u][i] = *reinterpret_cast<const uint32_t *>(sr[i] + st * 4);
            }
        }
#pragma unroll
        for (int i = 0; i < XU; ++i) {
            const int q = i * kMfWaves * 64 + tid, row = q >> 4 & (TB * 16 - 1), st = q / (TB * 256);
            const int k = (s0 + st) * kMfStep + (q & 15) * 8;
            const uint16_t *x = a.p + (int64_t)min(row, a.T - 1) * a.ldp + k;
            c.x[i] = load_or_zero<u32x4_t>(k < a.K, x);
        }
    };
    auto store_x = [&](const Chunk &c, int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < XU; ++i) {
            const int q = i * kMfWaves * 64 + tid, row = q >> 4 & (TB * 16 - 1), st = q / (TB * 256);
            *reinterpret_cast<u32x4_t *>(&sh.x[buf][st][row][(q ^ row) & 15]) = c.x[i];
        }
    };
    auto compute = [&](const Chunk &c, int s0, int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int st = s0 + kw * U + u;
            if (st >= last) break;
            // (past the last block x is zero, and the scale is no NaN)
            const bool in = st * 4 + g < blocks;
            uint32_t bits[CT];
#pragma unroll
            for (int i = 0; i < CT; ++i) bits[i] = in ? (c.scale[u][i] >> (8 * g) & 0xff) << 23 : 0u;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                bf16x8_t q[CT];
#pragma unroll
                for (int i = 0; i < CT; ++i) {
                    const uint32_t w[4] = {c.code[u][i].x, c.code[u][i].y, c.code[u][i].z, c.code[u][i].w};
                    q[i] = frag(mx_fp4_bf16(w[k], bits[i]));
                }
#pragma unroll
                for (int j = 0; j < TB; ++j) {
                    const bf16x8_t p = frag(sh.x[buf][kw * U + u][j * 16 + l16][(g * 4 + k) ^ l16]);
#pragma unroll
                    for (int i = 0; i < CT; ++i)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(q[i], p, acc[i][j], 0, 0, 0);
                }
            }
        }
    };
    auto use = [&](const Chunk &c, int s0, int buf) __attribute__((always_inline)) {
        store_x(c, buf);
        lds_barrier();
        compute(c, s0, buf);
    };
    // (No chunk ahead of its use: other work-groups of the CU fill the wait, and the
    // registers of a second chunk would cost them their place.)
    Chunk ch;
    if (!MULTI) {
        if (first < last) {
            load(ch, first);
            use(ch, first, 0);
        }
    } else {
        for (int s = first, buf = 0; s < last; s += CH, buf ^= 1) {
            load(ch, s);
            use(ch, s, buf);
        }
    }
    if (kw) {
#pragma unroll
        for (int i = 0; i < CT; ++i)
#pragma unroll
            for (int j = 0; j < TB; ++j) sh.sum[cw][i * TB + j][lane] = acc[i][j];
    }
    __syncthreads();
    if (kw) return;
#pragma unroll
    for (int j = 0; j < TB; ++j) {
        const int t = j * 16 + l16;
        if (t >= a.T) continue;
        float *o = a.part + ((int64_t)blockIdx.y * a.T + t) * a.part_ld + a.off[sc];
#pragma unroll
        for (int i = 0; i < CT; ++i) {
            const int64_t c = c0 + i * 16 + 4 * g;
            const floatx4_t v = sh.sum[cw][i * TB + j][lane];
            floatx4_t r = acc[i][j];
#pragma unroll
            for (int e = 0; e < 4; ++e) r[e] += v[e];
            if (c < cend) *reinterpret_cast<floatx4_t *>(o + c) = r;
        }
    }
}

// u of the y-th different slot's tokens: for each 16 tokens that name it.
template <int TB>
__device__ __forceinline__ void few_ranks(const FewArgs &f, floatx4_t (&s_sum)[kMfWaves][TB][64]) {
    const LinArgs &a = f.l;
    constexpr int U = 4;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int l16 = lane & 15, g = lane >> 4;
    int q = blockIdx.x - f.col_tiles;
    const int y = q % f.slots;
    q /= f.slots;
    const int rw = f.rank_waves, kws = kMfWaves / rw, rb = w % rw, kw = w / rw;
    const int s = q / f.rank_groups, g0 = (q - s * f.rank_groups) * rw * 16, j0 = g0 + rb * 16;
    // the tokens' slots, one token a lane; the first token of each slot leads
    const int mine = lane < a.T ? slot_of_token(a.idx, a.slot_rank, a.L, lane) : -1;
    bool lead = mine >= 0;
    for (int o = 0; o < a.T; ++o) {
        const int other = __shfl(mine, o);
        if (o < lane && other == mine) lead = false;
    }
    unsigned long long leads = __ballot(lead);
    if (y >= __popcll(leads)) return;
    for (int i = 0; i < y; ++i) leads &= leads - 1;
    const int slot = __builtin_amdgcn_readlane(mine, __ffsll(leads) - 1);
    const int rank = a.slot_rank ? min(a.slot_rank[slot], a.R) : a.R;
    if (g0 >= rank) return;
    const unsigned long long own = __ballot(mine == slot);

    const uint16_t *ar = a.other[s] + ((int64_t)slot * a.R + min(j0 + l16, a.R - 1)) * a.K;
    const uint16_t *xr[TB];
    bool any[TB];
    floatx4_t acc[TB];
#pragma unroll
    for (int j = 0; j < TB; ++j) {
        xr[j] = a.p + (int64_t)min(j * 16 + l16, a.T - 1) * a.ldp;
        any[j] = own >> (16 * j) & 0xffff;
        acc[j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    }
    const uint4 z = make_uint4(0, 0, 0, 0);
    const int kb = (int)blockIdx.y * f.per * kMfStep, ke = min(kb + f.per * kMfStep, a.K);
    for (int k0 = kb + kw * 32; k0 < ke && j0 < rank; k0 += U * kws * 32) {
        uint4 av[U], xv[U][TB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = min(k0 + u * kws * 32 + g * 8, a.K - 8);
            av[u] = ldg<uint4>(ar + k);
#pragma unroll
            for (int j = 0; j < TB; ++j) xv[u][j] = ldg<uint4>(xr[j] + k);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = k0 + u * kws * 32 + g * 8 < ke;
            const bf16x8_t q = frag(in ? av[u] : z);
#pragma unroll
            for (int j = 0; j < TB; ++j)
                if (any[j]) acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(q, frag(in ? xv[u][j] : z), acc[j], 0, 0, 0);
        }
    }
#pragma unroll
    for (int j = 0; j < TB; ++j) s_sum[w][j][lane] = acc[j];
    __syncthreads();
    if (w >= TB * rw) return;                     // wave w: rank block w % rw, token block w / rw
    const int tb = w / rw, t = tb * 16 + l16, j = j0 + 4 * g;
    if (!(own >> t & 1) || j >= rank) return;
    floatx4_t r = s_sum[rb][tb][lane];
    for (int i = 1; i < kws; ++i) {
        const floatx4_t o = s_sum[i * rw + rb][tb][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] += o[e];
    }
    *reinterpret_cast<floatx4_t *>(a.part + ((int64_t)blockIdx.y * a.T + t) * a.part_ld + a.cols + s * a.R + j) = r;
}

template <int TB, int CT, int CH, bool MULTI>
__global__ __launch_bounds__(kMfWaves * 64, 4) void k_mx_few(FewArgs f) {
    __shared__ union {
        FewLds<TB, CT, CH, MULTI> base;
        floatx4_t ranks[kMfWaves][TB][64];
    } sh;
    if ((int)blockIdx.x < f.col_tiles) few_base<TB, CT, CH, MULTI>(f, sh.base);
    else few_ranks<TB>(f, sh.ranks);
}

// One token in one launch: work-group = 128 output columns and one K split, 8 waves (4 x
// 32 columns, each pair's steps alternating).  Beside the base sums it finds its split's
// share of the slot's rank vector (the 8 waves along K; the lora_a rows come from L2, as
// every column tile reads them) and adds that share's delta, so that a column tile's
// splits need nothing but adding up.  They go to device-coherent memory, and the
// work-group that completes a tile's count adds them in order, rounds, and leaves the
// count zero for the next call.
struct OneArgs {
    LinArgs l;
    int32_t per, col_tiles;
    int32_t *count;           // [column tiles], zero between calls
};
constexpr int kOneCols = 128;
template <int NRB, int U>
__global__ __launch_bounds__(kMfWaves * 64, 4) void k_mx_one(OneArgs f) {
    constexpr int CT = 2, XU = 2 * U * 16;            // (U steps a wave and round) 16-byte units of x
    __shared__ float s_y[2][kOneCols], s_p[kMfWaves][16 * NRB], s_u[16 * NRB];
    __shared__ uint4 s_x[2][XU];
    __shared__ int s_last;
    const LinArgs &a = f.l;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, cw = w & 3, kw = w >> 2;
    const int l16 = lane & 15, g = lane >> 4;
    int sc = 0;
    while (sc + 1 < a.S && (int)blockIdx.x >= a.tile_start[sc + 1]) ++sc;
    const int tile = blockIdx.x - a.tile_start[sc];
    const int64_t c0 = (int64_t)tile * kOneCols, cend = a.n[sc];
    const int blocks = (a.K + kMxBlock - 1) / kMxBlock, steps = (blocks + 3) / 4;
    const int first = (int)blockIdx.y * f.per, last = min(first + f.per, steps);
    const uint8_t *wr[CT], *sr[CT];
#pragma unroll
    for (int i = 0; i < CT; ++i) {
        const int64_t n = a.off[sc] + min(c0 + cw * 32 + i * 16 + l16, cend - 1);
        wr[i] = reinterpret_cast<const uint8_t *>(a.w) + n * a.ldw;
        sr[i] = a.ws + n * a.ldws;
    }
    floatx4_t acc[CT], au[NRB];
#pragma unroll
    for (int i = 0; i < CT; ++i) acc[i] = floatx4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NRB; ++i) au[i] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    // (its rank, a load later, only masks sums)
    const int named = a.idx[0], slot = named < a.L ? named : -1;
    const int64_t c = c0 + tid;
    const bool col = tid < kOneCols && c < cend;
    uint4 bv[2 * NRB];
    float sc_own = 0.f, y = 0.f;
    int rank = 0;
    // a thread's column of the slot's lora_b: beside the first round's loads, or after
    // the loop where registers are short
    auto load_b = [&]() __attribute__((always_inline)) {
        if (slot < 0) return;
        rank = a.slot_rank ? min(a.slot_rank[slot], a.R) : a.R;
        if (!col) return;
        const uint16_t *b = a.lora[sc] + ((int64_t)slot * cend + c) * a.R;
#pragma unroll
        for (int j = 0; j < 2 * NRB; ++j) bv[j] = ldg<uint4>(b + min(j * 8, a.R - 8));
        sc_own = a.scale[slot];
    };
    int buf = 0;
    for (int s0 = first; s0 < last; s0 += 2 * U, buf ^= 1) {
        uint4 code[U][CT], xv = make_uint4(0, 0, 0, 0);
        uint32_t scale[U][CT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int st = min(s0 + kw * U + u, last - 1), b = min(st * 4 + g, blocks - 1);
#pragma unroll
            for (int i = 0; i < CT; ++i) {
                code[u][i] = ldg<uint4>(wr[i] + b * 16);
                scale[u][i] = *reinterpret_cast<const uint32_t *>(sr[i] + st * 4);
            }
        }
        // x past the split's or the row's end is zero
        const int xk = s0 * kMfStep + tid * 8;
        if (tid < XU && xk < last * kMfStep && xk < a.K) xv = ldg<uint4>(a.p + xk);
        __builtin_amdgcn_sched_barrier(0);
        // the slot's rows of the same steps: a wave's 32 at a time
        constexpr int AU = 2 * U * kMfStep / (32 * kMfWaves);
        uint4 av[AU][NRB];
        if (slot >= 0) {
#pragma unroll
            for (int v = 0; v < AU; ++v) {
                const int k = min(s0 * kMfStep + (v * kMfWaves + w) * 32 + g * 8, min(last * kMfStep, a.K) - 8);
#pragma unroll
                for (int i = 0; i < NRB; ++i)
                    av[v][i] = ldg<uint4>(a.other[sc] + ((int64_t)slot * a.R + min(i * 16 + l16, a.R - 1)) * a.K + k);
            }
        }
        if (NRB == 1 && s0 == first) load_b();
        __builtin_amdgcn_sched_barrier(0);        // every load of the round in flight
        if (tid < XU) s_x[buf][tid] = xv;
        lds_barrier();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // (past the end the scale is no NaN)
            const int st = s0 + kw * U + u;
            const bool in = st < last && st * 4 + g < blocks;
            uint32_t bits[CT];
#pragma unroll
            for (int i = 0; i < CT; ++i) bits[i] = in ? (scale[u][i] >> (8 * g) & 0xff) << 23 : 0u;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bf16x8_t x = frag(s_x[buf][(kw * U + u) * 16 + g * 4 + k]);
#pragma unroll
                for (int i = 0; i < CT; ++i) {
                    const uint32_t c[4] = {code[u][i].x, code[u][i].y, code[u][i].z, code[u][i].w};
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(mx_fp4_bf16(c[k], bits[i])), x, acc[i], 0, 0, 0);
                }
            }
        }
        if (slot >= 0) {
#pragma unroll
            for (int v = 0; v < AU; ++v) {
                // (past the end x is zero, and the row's values there may be anything)
                const int k = s0 * kMfStep + (v * kMfWaves + w) * 32 + g * 8;
                const bool in = k < last * kMfStep && k < a.K;
                const bf16x8_t x = frag(s_x[buf][(v * kMfWaves + w) * 4 + g]);
#pragma unroll
                for (int i = 0; i < NRB; ++i)
                    au[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(in ? av[v][i] : make_uint4(0, 0, 0, 0)), x,
                                                                  au[i], 0, 0, 0);
            }
        }
    }
    if (NRB > 1 || first >= last) load_b();
    // every result column is the token: column 0's lanes give the sums
    if (l16 == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int i = 0; i < CT; ++i) s_y[kw][cw * 32 + i * 16 + 4 * g + e] = acc[i][e];
#pragma unroll
            for (int i = 0; i < NRB; ++i) s_p[w][i * 16 + 4 * g + e] = au[i][e];
        }
    }
    __syncthreads();
    if (tid < 16 * NRB) {
        float u = 0.f;
#pragma unroll
        for (int i = 0; i < kMfWaves; ++i) u += s_p[i][tid];
        s_u[tid] = tid < rank ? u : 0.f;
    }
    __syncthreads();
    if (col) {
        float d = 0.f;
#pragma unroll
        for (int j = 0; j < 2 * NRB; ++j)
            if (j * 8 < rank) {
                const uint32_t bw[4] = {bv[j].x, bv[j].y, bv[j].z, bv[j].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    d += s_u[j * 8 + 2 * q] * bf16_lo(bw[q]);
                    d += s_u[j * 8 + 2 * q + 1] * bf16_hi(bw[q]);
                }
            }
        y = s_y[0][tid] + s_y[1][tid];
        if (rank > 0) y += sc_own * d;            // (an empty slot's scale may be anything)
    }
    // thread's part of the sums: a column's, and of a slice's first tile a rank's
    const bool urow = a.buf && tile == 0 && tid >= kOneCols && tid < kOneCols + a.R;
    const int uj = tid - kOneCols;
    float u = urow ? s_u[uj] : 0.f;
    const int64_t at = col ? a.off[sc] + c : a.cols + sc * a.R + uj;
    if (a.ksp > 1) {
        if (col || urow) {
            __hip_atomic_store(a.part + blockIdx.y * a.part_ld + at, col ? y : u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // stored before it is counted
        }
        __syncthreads();
        if (tid == 0)
            s_last = __hip_atomic_fetch_add(f.count + blockIdx.x, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 == a.ksp;
        __syncthreads();
        if (!s_last) return;
        if (tid == 0) __hip_atomic_store(f.count + blockIdx.x, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (col || urow) {
            float v[kMxFewSplits], sum = 0.f;
#pragma unroll
            for (int k = 0; k < kMxFewSplits; ++k)
                if (k < a.ksp) v[k] = __hip_atomic_load(a.part + k * a.part_ld + at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int k = 0; k < kMxFewSplits; ++k)
                if (k < a.ksp) sum += v[k];
            if (col) y = sum;
            else u = sum;
        }
    }
    if (col) {
        if (a.bias) y += bf16_to_f32(a.bias[a.off[sc] + c]);
        a.out[a.off[sc] + c] = (uint16_t)f32_to_bf16_rne(y);
    } else if (urow) {
        a.buf[(int64_t)sc * a.R + uj] = u;
    }
}

template <int TB, int CT>
hipError_t run(FewArgs f, hipStream_t st) {
    LinArgs &a = f.l;
    int c = 0;
    for (int s = 0; s < a.S; ++s) {
        a.tile_start[s] = c;
        c += (int)((a.n[s] + 64 * CT - 1) / (64 * CT));
    }
    for (int s = a.S; s <= kMaxSlices; ++s) a.tile_start[s] = c;
    f.col_tiles = c;
    const dim3 grid((unsigned)(c + a.S * f.rank_groups * f.slots), (unsigned)a.ksp);
    const dim3 block(kMfWaves * 64);
    if (f.per <= 4) hipLaunchKernelGGL((k_mx_few<TB, CT, 4, false>), grid, block, 0, st, f);
    else if (f.per <= 8 && TB == 1) hipLaunchKernelGGL((k_mx_few<TB, CT, TB == 1 ? 8 : 4, false>), grid, block, 0, st, f);
    else hipLaunchKernelGGL((k_mx_few<TB, CT, 4, true>), grid, block, 0, st, f);
    return hipGetLastError();
}

}  // namespace

// K splits of a few tokens: about 512 work-groups of about four K steps or more (a round
// of a work-group's loads; three of five steps in two).
int32_t mx_few_splits(int32_t K, const int64_t *N, int32_t S) {
    int64_t c = 0;
    for (int s = 0; s < S; ++s) c += (N[s] + 127) / 128;
    const int64_t steps = (K + kMfStep - 1) / kMfStep;
    int64_t k = 512 / c;
    if (k > (steps + 3) / 4) k = (steps + 3) / 4;
    if (k > kMxFewSplits) k = kMxFewSplits;
    if (k < 1) k = 1;
    const int64_t per = (steps + k - 1) / k;      // (whole steps: fewer splits may do)
    return (int32_t)((steps + per - 1) / per);
}

// Up to 16 tokens always (a token's two launches against the tiles', us, 4096 x 6144 of
// rank 16: 4 tokens 12.1 and 16.4, 16 tokens 16.1 and 17.1; rank 128 of 64 slots, 4096 x
// 4096, 16 tokens 21.2 and 35.4).  Up to 32 while the lora_a rows of the slots that they
// can name are few beside the columns, since a slot's rows meet every token's x (32
// tokens, rows and columns: 128 and 4096 14.5 and 15.4 us, 512 and 28672 39.4 and 46.4,
// 256 and 4096 of K 14336 27.7 and 28.0; 384 and 6144 21.1 and 18.0, 6144 and 6144 43
// and 33).
bool mx_few(int32_t T, const int64_t *N, int32_t S, int32_t R, int32_t L) {
    int64_t n = 0;
    for (int s = 0; s < S; ++s) n += N[s];
    if (T > kMxFewTokens || S * R > kLinWideRanks || n > kMxFewCols) return false;
    return T <= 16 || (int64_t)(T < L ? T : L) * S * R <= n / 24;
}

// One token of rank at most 32 takes k_mx_one while the slot's lora_a rows, which each
// of its work-groups reads, are a small part of the work.  Against two launches, us:
// K x N of 4096 x 4096 8.1 and 10.7, x 6144 9.5 and 12.3, x 8192 10.0 and 14.1, x 14336
// 14.6 and 16.9, x 28672 26.4 and 25.4; 14336 x 4096 13.5 and 22.7.
bool mx_one(int32_t T, const int64_t *N, int32_t S, int32_t R) {
    int64_t n = 0;
    for (int s = 0; s < S; ++s) n += N[s];
    return T == 1 && R <= 32 && n <= 16384;
}

static hipError_t launch_one(LinArgs a, int32_t *count, hipStream_t st) {
    OneArgs f{};
    int c = 0;
    for (int s = 0; s < a.S; ++s) {
        a.tile_start[s] = c;
        c += (int)((a.n[s] + kOneCols - 1) / kOneCols);
    }
    for (int s = a.S; s <= kMaxSlices; ++s) a.tile_start[s] = c;
    const int steps = (a.K + kMfStep - 1) / kMfStep;
    a.ksp = mx_few_splits(a.K, a.n, a.S);
    f.l = a;
    f.per = (steps + a.ksp - 1) / a.ksp;
    f.count = count;
    const dim3 grid((unsigned)c, (unsigned)a.ksp);
    const dim3 block(kMfWaves * 64);
    if (a.R > 16) hipLaunchKernelGGL((k_mx_one<2, 2>), grid, block, 0, st, f);
    else if (f.per <= 4) hipLaunchKernelGGL((k_mx_one<1, 2>), grid, block, 0, st, f);
    else hipLaunchKernelGGL((k_mx_one<1, 4>), grid, block, 0, st, f);
    return hipGetLastError();
}

hipError_t launch_mx_few(LinArgs a, int32_t *count, hipStream_t st) {
    a.cols = 0;
    for (int s = 0; s < a.S; ++s) a.cols += a.n[s];
    a.part_ld = a.cols + (int64_t)a.S * a.R;
    if (mx_one(a.T, a.n, a.S, a.R)) return launch_one(a, count, st);
    FewArgs f{};
    a.ksp = mx_few_splits(a.K, a.n, a.S);
    a.wide = 1;
    a.u_slice = a.R;
    a.u_slot = 0;
    f.l = a;
    const int steps = (a.K + kMfStep - 1) / kMfStep;
    f.per = (steps + a.ksp - 1) / a.ksp;
    f.slots = a.T < a.L ? a.T : a.L;
    f.rank_waves = a.R <= 16 ? 1 : a.R <= 32 ? 2 : 4;
    f.rank_groups = (a.R + 16 * f.rank_waves - 1) / (16 * f.rank_waves);
    const hipError_t e = a.T <= 16 ? run<1, 2>(f, st) : run<2, 2>(f, st);
    return e == hipSuccess ? launch_lin_join_rows(a, st) : e;
}

}  // namespace aa
