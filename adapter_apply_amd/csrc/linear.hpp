// Argument blocks and launchers of the adapter layer beside a frozen
// projection: lora_linear and its gradient (linear.hip, linear_bwd.hip), and
// of the per-adapter gradient norm and clip (grad.hip).
#pragma once

#include "common.hpp"

namespace aa {

// The tile GEMM (k_lin_tile).  Forward: out[t][n] = sum_k p[t][k] w[n][k] +
// delta; gradient: out[t][k] = sum_n p[t][n] w[n][k] + delta.
struct LinArgs {
    const uint16_t *p;        // x [T][ldp], or dy (whole 8-element units per slice)
    int64_t ldp;
    const uint16_t *w;        // the projection [sum N][ldw]; null: no base product
    int64_t ldw;              // elements, of a microscaled projection bytes
    const uint8_t *ws;        // its scales (w are LORA_MX_FP4 codes), or null
    int64_t ldws;
    const uint16_t *bias;     // [sum N] or null (forward)
    uint16_t *out;
    int64_t ldo;
    const uint16_t *hl;       // bf16 [S][T][hl_row]: scaled rank vectors' parts (the first two are used)
    int32_t hl_row;           // its row: kLinPartsFwd R or kLinPartsBwd R
    const int32_t *order;     // [T] row -> token, slot-sorted, then [T] the rows' slots; or null (token order)
    const int32_t *idx;
    const int32_t *slot_rank;
    int32_t T, K, S, L, R;
    int32_t accumulate;       // out += delta (no base product); rows without a slot untouched
    int32_t m_tiles, n_tiles;
    int32_t ksp;              // K splits; with part, fp32 sums go to part [ksp][T][part_ld]
    int32_t join_delta;       // the join adds the delta, not the tiles
    const float *u;           // fp32 rank vectors [S][T][R] of the join and of k_lin_few
    const float *scale;
    int32_t wide;             // rank vectors of every slot, x A^T or dy B, as S L R further columns of part
    int32_t base_tiles;       // column tiles before those
    int32_t u_slice, u_slot;  // wide: where a token's ranks are in its row past cols: slice s of
                              // slot i starts at s u_slice + i u_slot
    float *buf;               // where u goes if it is wanted: k_lin_one, join of wide batches; of other
                              // batches the join only clears the rows of tokens without a slot
    const uint16_t *other[kMaxSlices];  // k_lin_one and wide: lora_a [L][R][K]; wide gradient: lora_b
    float *part;
    int64_t part_ld;          // its row: cols, and the further columns of wide batches
    int64_t cols;             // columns of out
    const uint16_t *lora[kMaxSlices];   // forward: lora_b [L][N_s][R]; gradient: lora_a [L][R][K]
    int64_t n[kMaxSlices];              // N_s
    int64_t off[kMaxSlices];            // first row of slice s in w (first column in out)
    int64_t poff[kMaxSlices];           // gradient: first column of slice s in p
    int32_t tile_start[kMaxSlices + 1]; // forward: column tiles by slice
};

hipError_t launch_lin_gemm(LinArgs a, bool gradient, hipStream_t st);
// The sums of a direct batch's splits (a.part, a.ksp), bias and delta, to a.out.
hipError_t launch_lin_join_rows(const LinArgs &a, hipStream_t st);
// A few tokens on a 4-bit projection (mx_few.hip).
constexpr int64_t kMxFewCols = 65536;   // most columns of a token
constexpr int kMxFewTokens = 32;        // most tokens
bool mx_few(int32_t T, const int64_t *N, int32_t S, int32_t R, int32_t L);
bool mx_one(int32_t T, const int64_t *N, int32_t S, int32_t R);     // of those, in one launch
int32_t mx_few_splits(int32_t K, const int64_t *N, int32_t S);
constexpr int kMxFewSplits = 16;        // most K splits
constexpr int kMxCounts = kMxFewCols / 128 + kMaxSlices;   // counts, zero between calls
hipError_t launch_mx_few(LinArgs a, int32_t *count, hipStream_t st);
constexpr int kLinFewTokens = 64;       // most tokens of k_lin_few
constexpr int kLinMaxSplits = 8;
bool lin_one(int32_t T, int32_t K, const int64_t *N, int32_t S, int32_t R);
bool lin_few(int32_t T, int32_t K, const int64_t *N, int32_t S, int32_t R, int32_t L);
bool lin_grouped(int32_t T, int32_t K, int32_t R, int32_t L);
constexpr int kLinSplitTiles = 512;     // work-groups aimed at by K splits
constexpr int kLinEvenTiles = 340;      // most tiles of a joined batch that splits even out
struct LinTilePlan {
    int32_t tile;                       // 64, 128 or 256 rows and columns
    int32_t splits;
};
LinTilePlan lin_tile_plan(int32_t T, int32_t K, const int64_t *N, int32_t S, int32_t R, int32_t L, bool gradient,
                          bool join, bool wide, bool base);
// Whether a gradient's dx through a 4-bit projection reads it restored to bf16.
bool lin_restores(int32_t T, int32_t K, const int64_t *N, int32_t S, int32_t R, int32_t L, bool weights);
// bf16 parts of a rank vector: two where the product is rounded to bf16 (y,
// dx), three where it is an fp32 gradient (split_bf16).
constexpr int kLinPartsFwd = 2;
constexpr int kLinPartsBwd = 3;
// Whether the sizes stay within what one launch's grid takes.
bool lin_grid_fits(int32_t T, int32_t K, const int64_t *N, int32_t S);

// The direct path: no segment build.
constexpr int kLinDirectTokens = 1024;
constexpr int64_t kLinDirectBytesA = 128 << 20;
constexpr int64_t kLinDirectBytesB = 110 << 20;
constexpr int64_t kLinWideBytesB = 176 << 20;
constexpr int64_t kLinWideBytesA = 256 << 20;
// fp32 sums of a call at most: splits times T columns (see lin_tile_plan).
constexpr int64_t kLinJoinMax = 1 << 25;
bool lin_join_delta(int32_t T, int32_t K, const int64_t *N, int32_t S, int32_t R, int32_t L);
bool lin_direct(int32_t T, int32_t K, const int64_t *N, int32_t S, int32_t R, int32_t L);
bool lin_wide(int32_t T, int32_t K, const int64_t *N, int32_t S, int32_t R, int32_t L);
bool lin_wide_gradient(int32_t T, int32_t K, const int64_t *N, int32_t S, int32_t R, int32_t L, bool weights);
constexpr int kLinWideRanks = 1024;     // most S R of a wide batch
hipError_t launch_lin_shrink(const void *x, int64_t ldx, int32_t T, int32_t K, const Slices &sl,
                             int32_t S, int32_t L, int32_t R, const int32_t *idx,
                             const int32_t *slot_rank, float *buf, hipStream_t st);
// Rank vectors of the tokens that have a slot, from partial sums [S][nsp][T][R]
// by slot-sorted position or from a buffer [S][T][R] by token: to hl in `parts`
// bf16 parts of scale * sum, and to buf unscaled (zero for tokens without a
// slot).  hl, buf nullable.
struct LinVectors {
    const float *part;
    int32_t nsp;
    const float *in;        // part null
    uint16_t *hl;
    int32_t parts;
    float *buf;
};
// One or two of them in one launch, with the row order of the tile GEMM (order,
// nullable).
hipError_t launch_lin_vectors(const LinVectors *jobs, int n_jobs, int32_t T, int32_t S, int32_t L, int32_t R,
                              const int32_t *idx, const int32_t *slot_rank, const float *scale,
                              const SegPtrs &seg, int32_t *order, hipStream_t st);

// Gradient side (linear_bwd.hip).
struct PadMap {
    int64_t src[kMaxSlices];   // first column of slice s in dy
    int64_t dst[kMaxSlices];   // first column in the padded copy
    int64_t n[kMaxSlices];     // N_s
};
hipError_t launch_lin_pad(const void *dy, int64_t lddy, int32_t T, int32_t S, const PadMap &m,
                          uint16_t *out, int64_t ldo, hipStream_t st);
// Partial sums [S][nsp][T][R] of dy . lora_b by slot-sorted position.
int32_t lin_du_splits(int32_t T, int32_t L, const int64_t *N, int32_t S, int32_t R);
hipError_t launch_lin_du(const uint16_t *dy, int64_t lddy, const int64_t *poff, int32_t T,
                         const Slices &sl, int32_t S, int32_t L, int32_t R, const SegPtrs &seg, float *part,
                         int32_t nsp, hipStream_t st);
// One weight gradient family: out_s[slot][..] = sum over the slot's tokens of
// rows p (M_s columns at poff[s]) times rank vectors hl.  transposed: out is
// [L][R][M] (lora_a), else [L][M_s][R] (lora_b).
struct LinWgArgs {
    const uint16_t *p;
    int64_t ldp;
    const uint8_t *xs;         // p are LORA_MX_INT8 codes (ldp in bytes) with these scales, or null
    int64_t ldxs;
    const uint16_t *hl;        // bf16 [S][T][3R]
    float *out[kMaxSlices];
    int64_t m[kMaxSlices];
    int64_t poff[kMaxSlices];
    int32_t T, S, L, R;
    int32_t accumulate;
    const int32_t *slot_rank;
    SegPtrs seg;
    float *part;               // fp32 partial sums of the token splits
    int32_t nsp;
    int32_t tile_start[kMaxSlices + 1];
    int64_t part_off[kMaxSlices];   // element offset of slice s inside one split
    int64_t part_stride;            // elements of one split
};
// Partial sums of the token splits stay within this many elements.
constexpr int64_t kLinWgPartMax = 16 << 20;
// MA, MB: the slices' columns of dA and dB (nullable).
int32_t lin_wg_splits(int32_t T, int32_t L, const int64_t *MA, const int64_t *MB, int32_t S, int32_t R);
// Elements of one split's partial sums.
int64_t lin_wg_part(int32_t L, const int64_t *M, int32_t S, int32_t R);
// dA (transposed) and dB in one launch, and the sum of their splits in another;
// either may be null.
hipError_t launch_lin_wg(const LinWgArgs *dA, const LinWgArgs *dB, hipStream_t st);

// Gradient norm and clip (grad.hip).
hipError_t launch_grad_norm(const void *const *g, const int64_t *m, int32_t n, int32_t L, int32_t dtype,
                            int32_t *count, double *part, float *norm, hipStream_t st);
// Bytes of the workspace's counts, before its partial sums.
constexpr size_t kGradCountBytes = sizeof(int32_t) * kMaxSlots;
hipError_t launch_grad_clip(void *const *out, const void *const *g, const int64_t *m, int32_t n,
                            int32_t L, const float *norm, const float *max_norm, int32_t dtype,
                            hipStream_t st);
int64_t grad_items(const int64_t *m, int32_t n, int32_t L);   // partial sums of the norm, or -1

#ifdef __HIPCC__
// 16 zero bytes that masked LDS-DMA lanes read instead of their row.
static __device__ __attribute__((aligned(16))) const uint32_t g_zero16[4] = {0, 0, 0, 0};

// *p, or zeros from g_zero16: the choice is between addresses, since one between
// values would wait for the load where it stands, and between global ones (a choice of
// generic pointers makes a flat load, which the LDS counter waits for too).
template <typename V>
__device__ __forceinline__ V load_or_zero(bool in, const void *p) {
    typedef __attribute__((address_space(1))) const V global_v;
    return *(in ? (global_v *)p : (global_v *)(const void *)g_zero16);
}

// 64 lanes x 16 bytes straight from global memory into LDS at `lds` (uniform)
// + lane * 16.  The load is counted in vmcnt; every reader waits for it with
// wait_barrier.
__device__ __forceinline__ void dma16(uint32_t lds, const void *src) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(src) : "memory", "m0");
}
// The same with 4 bytes a lane.
__device__ __forceinline__ void dma4(uint32_t lds, const void *src) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
                 :: "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(src) : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(N) : "memory");
}
typedef short s16x4_t __attribute__((ext_vector_type(4)));
// Address of an LDS byte as the 32-bit LDS offset DMA and transposed reads use.
__device__ __forceinline__ uint32_t lds_addr(const void *p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}
// Transposed read of a 4-row x 16-column block of 16-bit values per 16 lanes:
// lane i of the group supplies row i / 4, columns 4 (i % 4)..+3 and receives
// column i, rows 0..3.
__device__ __forceinline__ uint2 tr_read(const char *p) {
    typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
    const s16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
    return __builtin_bit_cast(uint2, v);
}
// A token's slot: idx outside [0, L) and slots of rank <= 0 carry no delta.
__device__ __forceinline__ int slot_of_token(const int32_t *idx, const int32_t *slot_rank, int L, int t) {
    const int s = idx[t];
    if (s < 0 || s >= L) return -1;
    return slot_rank && slot_rank[s] <= 0 ? -1 : s;
}
// fp32 as a sum of bf16 parts, each the rounded remainder of those before it:
// a remainder is at most 2^-8 of the part's value, so two parts are within
// 2^-16 of the value and three hold all its 24 bits (2^-24); the MFMA products
// of a part are exact in fp32.  Values past bf16's largest (infinities, NaN,
// and the few fp32 values that round up to infinity) are all in the first part.
__device__ __forceinline__ void split_bf16(float v, uint32_t (&part)[3]) {
    part[0] = f32_to_bf16_rne(v);
    const bool whole = (part[0] & 0x7f80u) == 0x7f80u;
    const float r = whole ? 0.f : v - __uint_as_float(part[0] << 16);
    part[1] = f32_to_bf16_rne(r);
    part[2] = f32_to_bf16_rne(r - __uint_as_float(part[1] << 16));
}
// The parts of 4 ranks j..j+3 of one rank vector row (`parts` of R each).
__device__ __forceinline__ void store_parts(uint16_t *row, int parts, int R, int j, const float (&v)[4]) {
    uint32_t p[4][3];
#pragma unroll
    for (int e = 0; e < 4; ++e) split_bf16(v[e], p[e]);
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (k < parts)
            *reinterpret_cast<uint2 *>(row + k * R + j) = make_uint2(p[0][k] | p[1][k] << 16, p[2][k] | p[3][k] << 16);
}
#endif

}  // namespace aa
