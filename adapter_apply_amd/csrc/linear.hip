// The adapter layer beside a frozen projection:
//   forward   y[t][n]  = sum_k x[t][k] W[n][k] + bias[n] + sum_j (scale u[t][j]) B[i][n][j]
//   gradient  dx[t][k] = sum_n dy[t][n] W[n][k] + sum_s sum_j v_s[t][j] A_s[i][j][k]
// with i = idx[t].  Both are one tile GEMM (k_lin_tile) whose contraction runs
// over the projection's K (or N) and then over the rank vectors of every slot
// that the tile's tokens name, as further K tiles of the same pipeline: the
// delta costs no pass over y and is rounded together with the base product.
//
// A rank vector (fp32) enters the MFMA as two bf16 parts side by side,
// [high | low] against lora rows repeated, so that the product is within 2^-16
// of the fp32 buffer's, well below the bf16 rounding of the output.
#include "linear.hpp"
#include "mx.hpp"

namespace aa {

namespace {

typedef float floatx4_t __attribute__((ext_vector_type(4)));

constexpr int kXcds = 8;

// f(B), .., f(E - 1), each with its index as a constant (loops of this many steps are
// past what the compiler unrolls).
template <int I> struct Index { static constexpr int value = I; };
template <int B, int E, typename F>
__device__ __forceinline__ void each(const F &f) {
    if constexpr (B < E) {
        f(Index<B>());
        each<B + 1, E>(f);
    }
}

__device__ __forceinline__ bf16x8_t frag(const uint4 &u) { return __builtin_bit_cast(bf16x8_t, u); }

// Tile GEMM.  Work-group = BM tokens x BN output columns, WM x WN waves.  A
// K tile is BK contraction steps: P (token rows) and Q (weight rows), DMA'd
// into one of NST LDS stages, NST - 1 tiles ahead.
//
// LDS layout: the 16-byte units of a P row (BK * 2 bytes) are XOR-ed with the
// row's place in the 256-byte bank window, so the 16 rows a quarter wave reads
// together hit 16 different bank groups; the DMA's LDS side is linear, so the
// XOR is applied to the global address.  Gradient (NN): Q rows are contraction
// steps, BN columns wide, and reach the MFMA through transposed reads; the
// XOR moves 32-byte pairs by the row's low bits, so the 4 rows of one
// transposed read hit different banks.
//
// D = Q . P^T (output columns as MFMA rows), so a lane holds 4 consecutive
// output columns of one token.
//
// A tile's 64 steps are two fragment sets of 32.  While the MFMAs of the first
// run, the second is read (the stage is then free, and the DMA of the tile NST
// ahead starts); while those of the second run, the next tile's first set is
// read.  Both barriers of a tile find the MFMA pipe busy.
//
// An infinity or NaN in one slot's lora rows must not reach other slots'
// tokens, and zero times either is NaN, so zeroed rank vectors do not isolate
// them: a 16-token block of one slot takes part in that slot's K tiles only,
// and a block of several goes through a temporary and a select, in the K
// tiles (MIXED) or after them.
//
// Bound by the matrix rate: 8192 tokens, 4096 x 28672, rank 64, 16 slots 1.71 ms
// (median of 24; 1.64 to 2.16); its base product alone 1.48 ms, 1.30 PFLOP/s (1.4 us
// per K tile of 256 x 256, 1.0 at the dense peak of a 2.1 GHz clock).  Small batches
// are bound by L2: 256 tokens, 4096 x 6144 request 280 MB there in 25 us.
//
// kQCodes: the projection's Q rows are 4-bit codes.  Forward: the stage holds the codes
// and their scales, and a wave converts its fragments between the MFMAs (a pair of
// values an instruction).  Gradient, whose transposed reads take 16-bit values and
// whose scales run along the contraction: a thread loads its share of a tile one tile
// ahead of the DMA into registers and writes it to the stage as bf16, in the DMA's
// layout, when the stage is free; everything past the stage is the same.  8192 tokens,
// 4096 x 28672, rank 64: 1.63 to 1.75 ms, by the matrix rate (bf16 rows the same); 256
// tokens of 4096 x 6144 25.0 us, of them 10.7 whatever K is (33 MB of sums) and 1.09 per K
// tile of a CU's two work-groups (bf16 rows 23.3); gradient of 96 tokens of 6144 x 4096
// 25.4 us (bf16 rows 18.4: what the codes save in bytes is less than the conversions and
// the loads one tile ahead cost, so what 4 bits give there is memory).
template <int BM, int BN, int NST, bool SCALES>
struct TileLds {
    __attribute__((aligned(16))) char stage[NST * (BM + BN) * 128];
    __attribute__((aligned(16))) char scales[2][SCALES ? BN * 4 : 16];     // two pairs of tiles' (forward, codes)
    int tok[BM], slot[BM], list[BM + 1], r8[BM + 1], whole[BM / 16], n, nt, any;
    unsigned bits[32];
};
// Work-group i runs on XCD i % 8: each XCD takes a contiguous run of tiles,
// ordered so that 8 token tiles share a column tile before the next.
struct TileAt { int mt, nt; };
__device__ __forceinline__ TileAt tile_at(const LinArgs &a) {
    const int total = a.m_tiles * a.n_tiles;
    const int xcd = blockIdx.x % kXcds, q = total / kXcds, rem = total % kXcds;
    int id = xcd * q + (xcd < rem ? xcd : rem) + blockIdx.x / kXcds;
    const int gm = 8, band = gm * a.n_tiles;
    const int g = id / band, r = id - g * band;
    const int rows = min(gm, a.m_tiles - g * gm);
    const int nt = r / rows;
    return {g * gm + r - nt * rows, nt};
}
// Q operands: bf16 rows of the projection and, past its column tiles, of the
// adapters; its codes only; the adapters' only (the last two apart, so that one's
// registers do not crowd the other's loop: in one body the 128 x 128 tiles spill).
enum { kQRows, kQCodes, kQVectors };

template <int BM, int BN, int WM, int WN, int NST, bool NN, bool MIXED, int Q, bool SCALES>
__device__ __forceinline__ void lin_tile(const LinArgs &a, TileLds<BM, BN, NST, SCALES> &sh, int mt, int nt) {
    constexpr int NW = WM * WN, BK = 64, KK = 2;
    constexpr int MB = BM / WM / 16, NB = BN / WN / 16;
    constexpr int PB = BM * BK * 2, QB = BN * BK * 2;
    constexpr int PI = PB / 1024 / NW, QI = QB / 1024 / NW;
    constexpr int UP = BK / 8;                    // 16-byte units per P row (and Q row, forward)
    constexpr int CPR = NN ? BN / 8 : UP;         // 16-byte units per Q row
    static_assert(PI >= 1 && QI >= 1 && NW % 2 == 0, "whole DMA instructions per wave");
    static_assert(BM * BN * 2 <= NST * (PB + QB), "the output tile fits the stages");
    char *const s_stage = sh.stage;
    auto &s_tok = sh.tok, &s_slot = sh.slot;
    auto &s_list = sh.list, &s_r8 = sh.r8;
    auto &s_whole = sh.whole;
    int &s_n = sh.n, &s_nt = sh.nt, &s_any = sh.any;
    auto &s_bits = sh.bits;

    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = w / WN, wn = w % WN;

    // forward: the tile's slice, whose rows of W start at qb; past those in a wide
    // batch (vec), every slot's lora_a rows of a slice, in the gradient its lora_b
    // columns, whose contraction is the slice's alone
    int sc = 0;
    const uint16_t *qb = a.w;
    int64_t ldq = a.ldw, c0 = (int64_t)nt * BN, cend = a.K, obase = 0;   // columns: first, end, slice's first in out
    const bool vec = Q == kQVectors || (Q == kQRows && MIXED && nt >= a.base_tiles);
    if (vec) {
        const int per = (a.L * a.R + BN - 1) / BN;
        nt -= a.base_tiles;
        sc = nt / per;
        c0 = (int64_t)(nt - sc * per) * BN;
        cend = a.L * a.R;
        qb = a.other[sc];
        ldq = NN ? a.R : a.K;
        obase = a.cols + sc * cend;
    } else if (!NN) {
        while (sc + 1 < a.S && nt >= a.tile_start[sc + 1]) ++sc;
        c0 = (int64_t)(nt - a.tile_start[sc]) * BN;
        cend = a.n[sc];
        qb += a.off[sc] * ldq;
        obase = a.off[sc];
    }
    const int m0 = mt * BM;

    if (tid < 32) s_bits[tid] = 0;
    if (tid == 0) s_any = 0;
    __syncthreads();
    for (int i = tid; i < BM; i += NW * 64) {
        const int m = m0 + i;
        const int pos = min(m, a.T - 1);
        const int t = a.order ? a.order[pos] : pos;
        int sl = -2;
        if (m < a.T)
            sl = MIXED && a.join_delta ? -1 : a.order[a.T + pos];
        s_tok[i] = t;
        s_slot[i] = sl;
        // MIXED: every slot; else the slots that have a 16-token block of their own
        const int first = __shfl(sl, lane & 48);
        const bool whole = !(__ballot(sl != first && sl != -2) >> (lane & 48) & 0xffff);
        if (!MIXED && (lane & 15) == 0) s_whole[i >> 4] = whole;
        if (sl >= 0 && (MIXED || whole)) atomicOr(&s_bits[sl >> 5], 1u << (sl & 31));
        if (sl >= 0) s_any = 1;
    }
    __syncthreads();
    if (tid < 64 && !(MIXED && a.join_delta)) {
        // the tile's slots, ascending
        const unsigned b = tid < 32 ? s_bits[tid] : 0u;
        int c = __popc(b), inc = c;
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up(inc, d);
            if (lane >= d) inc += o;
        }
        if (tid == 31) s_n = inc;
        if (tid < 32) {
            // with each its rank in whole 16-byte units and the K tiles of its
            // [high | low] rank vector
            int nt = 0;
            unsigned bb = b;
            for (int k = inc - c; bb; ++k) {
                const int s = tid * 32 + __ffs(bb) - 1;
                const int r8 = ((a.slot_rank ? min(a.slot_rank[s], a.R) : a.R) + 7) & ~7;
                s_list[k] = s;
                s_r8[k] = r8;
                nt += (2 * r8 + BK - 1) / BK;
                bb &= bb - 1;
            }
            for (int d = 16; d; d >>= 1) nt += __shfl_xor(nt, d, 32);
            if (tid == 0) s_nt = nt;
        }
    }
    __syncthreads();
    if (a.accumulate && !s_any) return;
    // rank-vector K tiles (MIXED: none when the join adds the delta, else this
    // split's share)
    int n_lt = 0, lt0 = 0;
    if (!MIXED || !a.join_delta) {
        n_lt = __builtin_amdgcn_readfirstlane(s_nt) * (NN ? a.S : 1);
        if (MIXED) {
            lt0 = n_lt * (int)blockIdx.y / a.ksp;
            n_lt = n_lt * ((int)blockIdx.y + 1) / a.ksp - lt0;
        }
    }

    // K tiles: the projection's (per slice in the gradient), then per slot
    // (and slice) the [high | low] rank vectors.
    int nk = 0, k0 = 0;
    if (a.w) {
        if (NN && vec)
            nk = (int)((a.n[sc] + BK - 1) / BK);
        else if (NN)
            for (int s = 0; s < a.S; ++s) nk += (int)((a.n[s] + BK - 1) / BK);
        else
            nk = (a.K + BK - 1) / BK;
        // MIXED: this split's share of them
        if (MIXED) {
            const int per = (nk + a.ksp - 1) / a.ksp;
            k0 = min((int)blockIdx.y * per, nk);
            nk = min(per, nk - k0);
        }
    }
    const int nv = nk + n_lt;
    // the rank-vector tile to load or to use next: slot, slice, tile inside it
    struct Cursor { int d, s, c; };
    const int s_first = NN ? 0 : sc, s_last = NN ? a.S - 1 : sc;
    auto step = [&](Cursor &u) {
        if (++u.c < (2 * __builtin_amdgcn_readfirstlane(s_r8[u.d]) + BK - 1) / BK) return;
        u.c = 0;
        if (++u.s <= s_last) return;
        u.s = s_first;
        ++u.d;
    };
    Cursor ld = {0, s_first, 0};
    for (; lt0 > 0; --lt0) step(ld);
    Cursor use = ld;

    // DMA lanes: fixed rows, global units XOR-ed.
    auto pswz = [](int row) { return (row >> 1) & 7; };
    auto qswz = [&](int row) {
        if (!NN) return pswz(row);
        return ((row & 3) | (CPR >= 16 ? ((row >> 3) & 1) << 2 : 0)) << 1;
    };
    const int prow0 = w * (64 / UP) + lane / UP;  // + i * NW * 64 / UP
    const int plc = (lane % UP) ^ pswz(prow0);
    const uint16_t *pptr[PI];
#pragma unroll
    for (int i = 0; i < PI; ++i)
        pptr[i] = a.p + (int64_t)s_tok[prow0 + i * (NW * 64 / UP)] * a.ldp + plc * 8;
    auto qrow = [&](int i) { return (i * NW + w) * (64 / CPR) + lane / CPR; };
    auto qlc = [&](int i) { return (lane % CPR) ^ qswz(qrow(i)); };
    const uint16_t *qptr[QI];
#pragma unroll
    for (int i = 0; i < QI; ++i) {
        qptr[i] = a.w;
        if (a.w) {
            if (NN) {
                int64_t col = c0 + qlc(i) * 8;
                if (col >= cend) col = 0;
                if (vec) {                        // (slot, rank): whole units of one slot
                    const int slot = (int)col / a.R;
                    col += (a.n[sc] - 1) * slot * a.R;
                }
                qptr[i] = qb + qrow(i) * ldq + col;
            } else {
                const int64_t n = min(c0 + qrow(i), cend - 1);
                qptr[i] = qb + n * ldq + qlc(i) * 8;
            }
        }
    }
    const void *zero = g_zero16;
    const uint32_t lds0 = lds_addr(s_stage) + w * 1024;

    constexpr bool codes = Q == kQCodes, staged = codes && NN, direct = codes && !NN;
    // direct: QC instructions of codes (32 bytes a row); and one of 4 blocks' scales a
    // row, a place of their own, before the first of the two tiles that take two each (64
    // lanes there touch as many lines).  Fewer rows than a work-group's instructions
    // cover are loaded twice, to the same place.
    constexpr int QC = BN / 32 / NW > 0 ? BN / 32 / NW : 1;
    static_assert(!direct || QC + 1 <= QI, "a base tile issues no more loads than a rank-vector tile");
    // (a row's two units change places in 8 of 16 rows, so that the 16 rows of a read hit
    // different banks)
    auto code_unit = [](int lane) { return (lane & 1) ^ ((lane >> 4) & 1); };
    const uint8_t *cptr[QC], *sptr = nullptr;
    if (direct) {
        auto row = [&](int r) { return a.off[sc] + min(c0 + r, cend - 1); };
#pragma unroll
        for (int i = 0; i < QC; ++i)
            cptr[i] = reinterpret_cast<const uint8_t *>(a.w) + row((i * NW + w) % (BN / 32) * 32 + lane / 2) * a.ldw +
                      code_unit(lane) * 16;
        sptr = a.ws + row((w * 64 + lane) % BN) * a.ldws;
    }
    int ktile = 0;                                // direct: the next base tile to load
    auto code1 = [&](uint32_t ql0, int i, const void *from) __attribute__((always_inline)) {
        dma16(ql0 + (i * NW + w) % (BN / 32) * 1024, from);
    };
    const uint32_t stage0 = lds_addr(s_stage), scales0 = lds_addr(sh.scales);
    auto scales1 = [&]() __attribute__((always_inline)) {
        dma4(scales0 + (ktile >> 1 & 1) * (BN * 4) + (w * 64) % BN * 4, sptr + (ktile >> 1) * 4);
    };

    // staged: a thread's NQ pieces of a tile, HB code bytes each (a block of 32 or half
    // of one), as rows and blocks such that the 8 lanes of one LDS write hit
    // different banks; pieces past the contraction's end read zeros (code 0, scale 0).
    constexpr int NT = NW * 64, HB = 2 * BN >= NT ? 16 : 8, NQ = BN * 32 / (NT * HB), NL = 2 * NQ;
    struct Pieces { uint4 c[NQ]; uint32_t s[NQ]; };
    const uint8_t *qcode[NQ], *qscale[NQ];
    int qrow_of[NQ], qunit[NQ];                   // the piece's row and first 16-byte unit in the stage
    int q_cs = sc;
    int64_t q_rem = 0, q_at = 0;                  // rows left in the slice, first row
    static_assert(!staged || NL <= QI, "a base tile issues no more loads than a rank-vector tile");
    static_assert(!staged || BN <= 128, "the places of the pieces in a tile");
    if (staged) {
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            const int b = i * NT + tid;
            int row, blk, half = 0;
            if (HB == 16) {
                blk = b % (BN / 32);
                row = b / (BN / 32);
            } else {
                half = b & 1;
                blk = (b >> 1) & 1;
                row = b >> 2;
            }
            qrow_of[i] = row;
            qunit[i] = blk * 4 + half * 2;
            blk = (c0 >> 5) + blk < (a.K + 31) >> 5 ? (int)(c0 >> 5) + blk : 0;
            qcode[i] = reinterpret_cast<const uint8_t *>(a.w) + row * a.ldw + blk * 16 + half * 8;
            qscale[i] = a.ws + row * a.ldws + blk;
        }
    }
    auto load_q = [&](Pieces &r, int i) __attribute__((always_inline)) {
        const bool in = qrow_of[i] < q_rem;
        const uint8_t *c = qcode[i] + q_at * a.ldw;
        if (HB == 16) {
            const u32x4_t v = load_or_zero<u32x4_t>(in, c);
            r.c[i] = make_uint4(v.x, v.y, v.z, v.w);
        } else {
            const uint64_t v = load_or_zero<uint64_t>(in, c);
            r.c[i] = make_uint4((uint32_t)v, (uint32_t)(v >> 32), 0, 0);
        }
        r.s[i] = load_or_zero<uint8_t>(in, qscale[i] + q_at * a.ldws);
    };
    auto begin_q = [&]() {                        // the next tile's slice
        if (q_rem <= 0 && q_cs + 1 < a.S) q_rem = a.n[++q_cs];
    };
    auto end_q = [&]() {
        q_at += q_rem < BK ? (q_rem > 0 ? q_rem : 0) : BK;
        q_rem -= BK;
    };
    auto load_qs = [&](Pieces &r) __attribute__((always_inline)) {
        begin_q();
#pragma unroll
        for (int i = 0; i < NQ; ++i) load_q(r, i);
        end_q();
    };
    // unit u of piece i
    auto store_q = [&](const Pieces &r, int stage, int i, int u) __attribute__((always_inline)) {
        const uint32_t c[4] = {r.c[i].x, r.c[i].y, r.c[i].z, r.c[i].w};
        const int row = qrow_of[i];
        *reinterpret_cast<uint4 *>(s_stage + stage * (PB + QB) + PB + row * (CPR * 16) +
                                   (((qunit[i] + u) ^ qswz(row)) << 4)) = mx_fp4_bf16(c[u], r.s[i] << 23);
    };
    auto store_qs = [&](const Pieces &r, int stage) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int u = 0; u < HB / 4; ++u) store_q(r, stage, i, u);
    };
    Pieces qr;

    // The next base K tile: steps left in its row (forward) or slice, and the
    // offsets into the P and Q rows.
    int cs = NN ? sc : 0;
    int64_t rem = NN ? a.n[cs] : a.K, po = NN ? a.poff[cs] : 0, qo = 0;   // (off[0] is 0)
    const int64_t qstep = NN ? BK * ldq : BK;
    auto next_slice = [&]() {
        if (NN && rem <= 0 && ++cs < a.S) {
            rem = a.n[cs];
            po = a.poff[cs];
            qo = a.off[cs] * a.ldw;
        }
    };
    auto advance = [&]() { rem -= BK; po += BK; qo += qstep; ++ktile; };
    if (MIXED && k0 && nk > 0) {
        if (NN && !vec)
            for (; (int64_t)k0 * BK >= a.n[cs]; ++cs) k0 -= (int)((a.n[cs] + BK - 1) / BK);
        rem = (NN ? a.n[cs] : a.K) - (int64_t)k0 * BK;
        po = (NN ? a.poff[cs] : 0) + (int64_t)k0 * BK;
        qo = NN ? ((vec ? 0 : a.off[cs]) + (int64_t)k0 * BK) * ldq : (int64_t)k0 * BK;
    }
    if (staged) {
        q_cs = cs;
        q_rem = rem;
        q_at = a.off[cs] + (a.n[cs] - rem);
    }
    if (direct) ktile = k0;
    auto issue = [&](int v, int stage) {
        // recomputed here each time: hoisted lane values would crowd the
        // registers of the fast loop
        int lane = tid & 63;
        asm volatile("" : "+v"(lane));
        const int prow0 = w * (64 / UP) + lane / UP, plc = (lane % UP) ^ pswz(prow0);
        auto qrow = [&](int i) { return (i * NW + w) * (64 / CPR) + lane / CPR; };
        auto qlc = [&](int i) { return (lane % CPR) ^ qswz(qrow(i)); };
        const uint32_t pl = lds0 + stage * (PB + QB), ql = pl + PB;
        if (v < nk) {
            next_slice();
            if (staged && v >= NST) {             // (the first NST tiles are written by the prologue)
                store_qs(qr, stage);
                load_qs(qr);
            }
            if (direct && (v == 0 || !(ktile & 1))) scales1();
#pragma unroll
            for (int i = 0; i < PI; ++i)
                dma16(pl + i * NW * 1024, plc * 8 < rem ? (const void *)(pptr[i] + po) : zero);
            if (direct) {
                const uint32_t ql0 = stage0 + stage * (PB + QB) + PB;
#pragma unroll
                for (int i = 0; i < QC; ++i)
                    code1(ql0, i, code_unit(lane) * 32 < rem ? (const void *)(cptr[i] + ktile * 32) : zero);
            }
            if (!codes) {
#pragma unroll
                for (int i = 0; i < QI; ++i)
                    dma16(ql + i * NW * 1024,
                          (NN ? qrow(i) : qlc(i) * 8) < rem ? (const void *)(qptr[i] + qo) : zero);
            }
            advance();
            return;
        }
        const int s = ld.s, c = ld.c, R = a.R;
        const int slot = __builtin_amdgcn_readfirstlane(s_list[ld.d]), r8 = __builtin_amdgcn_readfirstlane(s_r8[ld.d]);
        step(ld);
        const int pj = c * BK + plc * 8;
        const uint16_t *hl = a.hl + (int64_t)s * a.T * a.hl_row + (pj < r8 ? pj : pj - r8 + R);
        const bool pin = pj < 2 * r8;
#pragma unroll
        for (int i = 0; i < PI; ++i) {
            const int row = prow0 + i * (NW * 64 / UP);
            const bool in = s_slot[row] == slot && pin;
            dma16(pl + i * NW * 1024,
                  in ? (const void *)(hl + (uint64_t)(unsigned)s_tok[row] * (unsigned)a.hl_row) : zero);
        }
        // (32-bit lane offsets from scalar bases)
        if (NN) {
            const uint16_t *lo = a.lora[s] + (int64_t)slot * R * a.K + c0;
            const int cmax = (int)min(cend - c0, (int64_t)BN) - 8;
#pragma unroll
            for (int i = 0; i < QI; ++i) {
                const int j2 = c * BK + qrow(i), col = qlc(i) * 8;
                const unsigned j = j2 < r8 ? j2 : j2 - r8;
                dma16(ql + i * NW * 1024,
                      j2 < 2 * r8 ? (const void *)(lo + (uint64_t)j * (unsigned)a.K + (col <= cmax ? col : 0)) : zero);
            }
        } else {
            const uint16_t *lo = a.lora[s] + ((int64_t)slot * cend + c0) * R;
            const int rmax = (int)min(cend - c0, (int64_t)BN) - 1;
            const int j2 = c * BK + qlc(0) * 8;              // the same unit in each of a lane's rows
            lo += j2 < r8 ? j2 : j2 - r8;
#pragma unroll
            for (int i = 0; i < QI; ++i)
                dma16(ql + i * NW * 1024,
                      j2 < 2 * r8 ? (const void *)(lo + min(qrow(i), rmax) * R) : zero);
        }
    };

    floatx4_t acc[NB][MB];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};

    const int g = lane >> 4, l16 = lane & 15;
    // The 8 contraction steps of a lane's fragment kk: direct, the two halves of the 16
    // whose codes it reads at once.
    auto unit = [&](int kk) { return direct ? 2 * g + kk : kk * 4 + g; };
    auto pfrag = [&](const char *st, int mb, int kk) {
        const int row = (wm * MB + mb) * 16 + l16;
        return frag(*reinterpret_cast<const uint4 *>(st + row * (BK * 2) + ((unit(kk) ^ pswz(row)) << 4)));
    };
    const int code_at = (((g >> 1) ^ (l16 >> 3)) << 4) + (g & 1) * 8;     // a row's codes of the lane's 16 steps
    auto qcodes = [&](const char *st, int nb) {
        return *reinterpret_cast<const uint2 *>(st + PB + ((wn * NB + nb) * 16 + l16) * 32 + code_at);
    };
    auto qscale1 = [&](int nb, int kt) {
        return (uint32_t)(uint8_t)sh.scales[kt >> 1 & 1][((wn * NB + nb) * 16 + l16) * 4 + (kt & 1) * 2 + (g >> 1)];
    };
    auto qfrag = [&](const char *st, int nb, int kk) {
        if (NN) {
            const int row = kk * 32 + g * 8 + (l16 >> 2);
            const int col = (wn * NB + nb) * 16 + (l16 & 3) * 4;
            const char *p = st + PB + row * (BN * 2) + ((((col >> 3) ^ qswz(row)) << 4) | ((col & 4) << 1));
            const uint2 x0 = tr_read(p), x1 = tr_read(p + 4 * BN * 2);
            return frag(make_uint4(x0.x, x0.y, x1.x, x1.y));
        }
        const int row = (wn * NB + nb) * 16 + l16;
        return frag(*reinterpret_cast<const uint4 *>(st + PB + row * (BK * 2) + ((unit(kk) ^ pswz(row)) << 4)));
    };
    auto stage_ptr = [&](int v) { return s_stage + (v % NST) * (PB + QB); };
    auto meet_reads = [&]() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };

    auto loads = [&](uint32_t pl, int j, int n) __attribute__((always_inline)) {
        // share j of n of a whole base tile's DMA
#pragma unroll
        for (int i = j * PI / n; i < (j + 1) * PI / n; ++i) dma16(pl + i * NW * 1024, pptr[i] + po);
#pragma unroll
        for (int i = j * QI / n; i < (j + 1) * QI / n; ++i) dma16(pl + PB + i * NW * 1024, qptr[i] + qo);
    };
    // all but the NST - 1 youngest tiles' loads; a base tile of codes has fewer
    auto wait_tile = [&](bool more) __attribute__((always_inline)) {
        if (!more) wait_barrier<0>();
        else if (codes) wait_barrier<(NST - 1) * (PI + (NN ? NL : QC))>();       // (scales come first)
        else wait_barrier<(NST - 1) * (PI + QI)>();
    };
    if (staged) {
        Pieces first[NST];
        for (int i = 0; i < NST; ++i)
            if (i < nv) issue(i, i);
#pragma unroll
        for (int i = 0; i < NST; ++i) load_qs(first[i]);
        load_qs(qr);
#pragma unroll
        for (int i = 0; i < NST; ++i)
            if (i < nk) store_qs(first[i], i);
        wait_barrier<0>();
    } else if (!codes && nk >= NST && rem >= NST * BK) {
        for (int i = 0; i < NST; ++i) {
            loads(lds0 + i * (PB + QB), 0, 1);
            advance();
        }
        wait_tile(true);
    } else {
        for (int i = 0; i < NST; ++i)
            if (i < nv) issue(i, i);
        wait_tile(nv >= NST);
    }
    for (int v = 0; v < nv; ++v) {
        // Fast tiles: tile v's DMA slot takes a whole base tile, v + NST.
        next_slice();
        if (v + NST < nk && rem >= BK) {
            bf16x8_t fq[2][NB], fp[2][MB];
            // One MFMA, then item n of what goes beside the MFMAs: single reads and
            // DMA instructions between single MFMAs, since a clump of them is longer
            // than an MFMA runs.
            auto mfma1 = [&](int set, int n) __attribute__((always_inline)) {
                const int j = n / NB, i = n % NB;
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fq[set][i], fp[set][j], acc[i][j], 0, 0, 0);
            };
            // a fragment set's reads: first the Q fragments, which every MFMA group
            // of the next half needs, then the P fragments
            auto read1 = [&](int set, const char *st, int kk, int i) __attribute__((always_inline)) {
                if (i < NB) fq[set][i] = qfrag(st, i, kk);
                else fp[set][i - NB] = pfrag(st, i - NB, kk);
            };
            constexpr int M = MB * NB, RD = NB + MB, LD = PI + QI;
            constexpr int M1 = M / 4;                     // MFMAs beside the first half's reads
            constexpr int M2 = M - M1;                    // and its DMA
            constexpr int M3 = M * 3 / 4;                 // MFMAs beside the second half's reads
            if (!direct) {
#pragma unroll
                for (int i = 0; i < RD; ++i) read1(0, stage_ptr(v), 0, i);
            }
            // beside the MFMAs once a stage is free: the codes in registers to the
            // stage, the next tile's codes, P's DMA
            constexpr int SU = HB / 4, CI = NQ * SU + NQ + PI;
            auto refill1 = [&](uint32_t pl, int stage, int i) __attribute__((always_inline)) {
                if (i < NQ * SU) {
                    store_q(qr, stage, i / SU, i % SU);
                } else if (i < NQ * SU + NQ) {
                    if (i == NQ * SU) begin_q();
                    load_q(qr, i - NQ * SU);
                    if (i == NQ * SU + NQ - 1) end_q();
                } else {
                    const int p = i - NQ * SU - NQ;
                    dma16(pl + p * NW * 1024, pptr[p] + po);
                }
            };
            // direct: a tile's codes of both sets and their scales
            uint2 qc[NB];
            uint32_t qs[NB];
            constexpr int RC = 2 * NB + MB;
            // one instruction of fragment i / 4's conversion
            uint32_t fu[2][NB][4];
            auto convert1 = [&](int set, int i) __attribute__((always_inline)) {
                const uint32_t c = set ? qc[i / 4].y : qc[i / 4].x;
                const float sc = __uint_as_float(qs[i / 4]);
                bf16x2_t r;
                if (i % 4 == 0) r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 0);
                else if (i % 4 == 1) r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 1);
                else if (i % 4 == 2) r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 2);
                else r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sc, 3);
                fu[set][i / 4][i % 4] = __builtin_bit_cast(uint32_t, r);
                if (i % 4 == 3)
                    fq[set][i / 4] = frag(make_uint4(fu[set][i / 4][0], fu[set][i / 4][1], fu[set][i / 4][2], fu[set][i / 4][3]));
            };
            // the scale of a fragment to a float's exponent, then the first set's conversions
            auto scale1 = [&](int i) __attribute__((always_inline)) {
                if (i % 5 == 0) qs[i / 5] <<= 23;
                else convert1(0, i / 5 * 4 + i % 5 - 1);
            };
            if (direct) {
                // Loop-carried addresses (opaque: else the compiler keeps two sets and
                // advances one at the loop's end, a clump), LDS addresses of a lane's
                // first row.
                const uint16_t *pp[PI];
                const uint8_t *cp[QC];
#pragma unroll
                for (int i = 0; i < PI; ++i) pp[i] = pptr[i] + po;
#pragma unroll
                for (int i = 0; i < QC; ++i) cp[i] = cptr[i] + ktile * 32;
                const int c_row = PB + (wn * NB * 16 + l16) * 32 + code_at;
                const char *const s_row = sh.scales[0] + (wn * NB * 16 + l16) * 4 + (g >> 1);
                const int p_row = (wm * MB * 16 + l16) * (BK * 2);
                int fast = min(nk - NST - v, (int)(rem / BK));
                auto read_p = [&](int set, int st, int i) __attribute__((always_inline)) {
                    fp[set][i] = frag(*reinterpret_cast<const uint4 *>(
                        s_stage + (st + p_row + ((unit(set) ^ pswz(l16)) << 4)) + i * 16 * BK * 2));
                };
                // item i of a tile's first reads: codes and scales in turn, P fragments
                auto read_first = [&](int st, int sst, int i) __attribute__((always_inline)) {
                    if (i >= 2 * NB) read_p(0, st, i - 2 * NB);
                    else if (i % 2) qs[i / 2] = (uint8_t)*(s_row + sst + i / 2 * 64);
                    else qc[i / 2] = *reinterpret_cast<const uint2 *>(s_stage + (st + c_row) + i / 2 * 512);
                };
                // item i of the DMA that a free stage takes
                constexpr int LC = 1 + PI + QC;
                auto dma1 = [&](uint32_t at, int i) __attribute__((always_inline)) {
                    if (i == 0) {
                        if (!(ktile & 1)) scales1();
                    } else if (i <= PI) {
                        dma16(at + w * 1024 + (i - 1) * NW * 1024, pp[i > 0 && i <= PI ? i - 1 : 0]);
                    } else {
                        code1(at + PB, i - 1 - PI, cp[i > PI ? i - 1 - PI : 0]);
                    }
                };
                auto next1 = [&](int i) __attribute__((always_inline)) {
                    if (i > 0 && i <= PI) {
                        const uint16_t *&p = pp[i > 0 && i <= PI ? i - 1 : 0];
                        p += BK;
                        asm volatile("" : "+v"(p));
                    } else if (i > PI) {
                        const uint8_t *&c = cp[i > PI ? i - 1 - PI : 0];
                        c += 32;
                        asm volatile("" : "+v"(c));
                    }
                };
                auto at_of = [&](int v) { return (v % NST) * (PB + QB); };
                auto scales_of = [&](int v) { return ((k0 + v) >> 1 & 1) * (BN * 4) + ((k0 + v) & 1) * 2; };
                // Slots between the MFMAs of a half: about three instructions each.
                constexpr bool WIDE = M >= 64;
                constexpr int MR = WIDE ? M * 3 / 8 : M / 2, MC = WIDE ? MR : M / 2;
#pragma unroll
                for (int i = 0; i < RC; ++i) read_first(at_of(v), scales_of(v), i);
#pragma unroll
                for (int i = 0; i < 5 * NB; ++i) scale1(i);
                do {
                    const int st = at_of(v);
                    const uint32_t at = stage0 + st;
                    // first half: P's second fragments, the codes' from registers, and once
                    // the stage is free its DMA
                    each<0, M>([&](auto slot) __attribute__((always_inline)) {
                        constexpr int n = decltype(slot)::value;
                        if constexpr (n < M1)
                            each<n * MB / M1, (n + 1) * MB / M1>(
                                [&](auto i) __attribute__((always_inline)) { read_p(1, st, i.value); });
                        if constexpr (n == M1) meet_reads();
                        if constexpr (WIDE) {
                            constexpr int D = (n - M1 - 1) / 4;       // DMA in every fourth slot, its next address two on
                            if constexpr (n > M1 && (n - M1 - 1) % 4 == 0 && D < LC) dma1(at, D);
                            if constexpr (n > M1 && (n - M1 - 1) % 4 == 2 && D < LC) next1(D);
                            if constexpr (n < M1 ? n % 2 == 1 : n % 2 == 0) convert1(1, n / 2);
                        } else {
                            if constexpr (n >= M1)
                                each<(n - M1) * LC / M2, (n - M1 + 1) * LC / M2>([&](auto i) __attribute__((always_inline)) {
                                    dma1(at, i.value);
                                    next1(i.value);
                                });
                            each<n * 4 * NB / M, (n + 1) * 4 * NB / M>(
                                [&](auto i) __attribute__((always_inline)) { convert1(1, i.value); });
                        }
                        mfma1(0, n);
                        __builtin_amdgcn_sched_barrier(0);
                    });
                    advance();
                    ++v;
                    wait_tile(true);
                    // second half: the next tile's codes, scales and first P fragments, its
                    // first conversions
                    const int nx = at_of(v), nxs = scales_of(v);
                    each<0, M>([&](auto slot) __attribute__((always_inline)) {
                        constexpr int n = decltype(slot)::value;
                        if constexpr (n < MR)
                            each<n * RC / MR, (n + 1) * RC / MR>(
                                [&](auto i) __attribute__((always_inline)) { read_first(nx, nxs, i.value); });
                        if constexpr (n >= MC)
                            each<(n - MC) * 5 * NB / (M - MC), (n - MC + 1) * 5 * NB / (M - MC)>(
                                [&](auto i) __attribute__((always_inline)) { scale1(i.value); });
                        mfma1(1, n);
                        __builtin_amdgcn_sched_barrier(0);
                    });
                } while (--fast > 0);
            } else if (staged) do {
                const char *st = stage_ptr(v);
                const int stage = v % NST;
                const uint32_t pl = lds0 + stage * (PB + QB);
#pragma unroll
                for (int n = 0; n < M; ++n) {
                    if (n < M1) {
#pragma unroll
                        for (int i = n * RD / M1; i < (n + 1) * RD / M1; ++i) read1(1, st, 1, i);
                    } else {
                        if (n == M1) meet_reads();
#pragma unroll
                        for (int i = (n - M1) * CI / M2; i < (n - M1 + 1) * CI / M2; ++i) refill1(pl, stage, i);
                    }
                    mfma1(0, n);
                    __builtin_amdgcn_sched_barrier(0);
                }
                advance();
                ++v;
                wait_tile(true);
                const char *nx = stage_ptr(v);
#pragma unroll
                for (int n = 0; n < M; ++n) {
                    if (n < M3) {
#pragma unroll
                        for (int i = n * RD / M3; i < (n + 1) * RD / M3; ++i) read1(0, nx, 0, i);
                    }
                    mfma1(1, n);
                    __builtin_amdgcn_sched_barrier(0);
                }
            } while (v + NST < nk && rem >= BK);
            else {
                // Loop-carried addresses, opaque: else the compiler keeps a second set and
                // advances it at the loop's end, a clump (gradient of 8192 tokens, 28672 x 4096, 1860 -> 1837 us).
                const uint16_t *at[LD];
#pragma unroll
                for (int i = 0; i < LD; ++i) at[i] = i < PI ? pptr[i] + po : qptr[i - PI] + qo;
                auto next1 = [&](int i) __attribute__((always_inline)) {
                    at[i] += i < PI ? BK : qstep;
                    asm volatile("" : "+v"(at[i]));
                };
                auto load1 = [&](uint32_t pl, int i) __attribute__((always_inline)) {
                    dma16(i < PI ? pl + i * NW * 1024 : pl + PB + (i - PI) * NW * 1024, at[i]);
                };
                int fast = min(nk - NST - v, (int)min(rem / BK, (int64_t)nk));
                do {
                    const char *st = stage_ptr(v);
                    const uint32_t pl = lds0 + (v % NST) * (PB + QB);
                    // first half: the stage's second fragment set, after which the
                    // stage is free for the tile NST ahead
#pragma unroll
                    for (int n = 0; n < M; ++n) {
                        if (n < M1) {
#pragma unroll
                            for (int i = n * RD / M1; i < (n + 1) * RD / M1; ++i) read1(1, st, 1, i);
                        } else {
                            if (n == M1) meet_reads();
#pragma unroll
                            for (int i = (n - M1) * LD / M2; i < (n - M1 + 1) * LD / M2; ++i) {
                                load1(pl, i);
                                if (M < 64) next1(i);
                            }
                            // (the addresses a slot on)
                            if (M >= 64 && n > M1)
#pragma unroll
                                for (int i = (n - 1 - M1) * LD / M2; i < (n - M1) * LD / M2; ++i) next1(i);
                        }
                        mfma1(0, n);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    advance();
                    ++v;
                    wait_barrier<(NST - 1) * (PI + QI)>();     // tile v has landed
                    // second half: the next tile's first set
                    const char *nx = stage_ptr(v);
#pragma unroll
                    for (int n = 0; n < M; ++n) {
                        if (n == 0 && M >= 64) next1(LD - 1);
                        if (n < M3) {
#pragma unroll
                            for (int i = n * RD / M3; i < (n + 1) * RD / M3; ++i) read1(0, nx, 0, i);
                        }
                        mfma1(1, n);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                } while (--fast > 0);
            }
        }
        // Any other tile, without the pipelined fragments.
        const char *st = stage_ptr(v);
        const bool base = v < nk;
        const int slot = base ? 0 : __builtin_amdgcn_readfirstlane(s_list[use.d]);
        if (!base) step(use);
        bf16x8_t q[KK][NB], p[KK][MB];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                if (direct && base) {
                    // (scales past the row's blocks may be anything)
                    const int kt = k0 + v;
                    const uint32_t s = kt * BK + (g >> 1) * kMxBlock < a.K ? qscale1(i, kt) : 0u;
                    const uint2 c = qcodes(st, i);
                    q[kk][i] = frag(mx_fp4_bf16(kk ? c.y : c.x, s << 23));
                } else {
                    q[kk][i] = qfrag(st, i, kk);
                }
            }
#pragma unroll
            for (int j = 0; j < MB; ++j) p[kk][j] = pfrag(st, j, kk);
        }
        // the stage is free for the tile NST ahead
        if (v + 1 < nv) {
            meet_reads();
            if (v + NST < nv) issue(v + NST, v % NST);
        }
#pragma unroll
        for (int j = 0; j < MB; ++j) {
            const int rs = s_slot[(wm * MB + j) * 16 + (MIXED ? l16 : 0)];
            const bool mine = base || (rs == slot && (MIXED || s_whole[wm * MB + j]));
            if (__ballot(mine) == 0) continue;
            if (!MIXED || __ballot(!mine && rs != -2) == 0) {
#pragma unroll
                for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                    for (int i = 0; i < NB; ++i)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(q[kk][i], p[kk][j], acc[i][j], 0, 0, 0);
            } else {
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    floatx4_t t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk)
                        t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(q[kk][i], p[kk][j], t, 0, 0, 0);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][e] = mine ? acc[i][j][e] + t[e] : acc[i][j][e];
                }
            }
        }
        // tile v + 1 has landed
        wait_tile(v + NST < nv);
    }

    // 16-token blocks that hold several slots: each slot's part from global
    // memory into a temporary, kept for the slot's own tokens.  (At most one
    // block per slot boundary; kept out of the K tiles, where a select on the
    // accumulators made the compiler spill them: 2.45 against 1.75 ms for the
    // forward tiles of 8192 tokens, 4096 x 28672, rank 64.)
    if (!MIXED) {
#pragma unroll
        for (int j = 0; j < MB; ++j) {
            if (s_whole[wm * MB + j]) continue;
            const int row = (wm * MB + j) * 16 + l16, rs = s_slot[row];
            unsigned long long todo = __ballot(rs >= 0) & 0xffff;
            while (todo) {
                const int slot = __builtin_amdgcn_readlane(rs, __ffsll(todo) - 1);
                const bool mine = rs == slot;
                todo &= ~__ballot(mine);
                floatx4_t t[NB];
#pragma unroll
                for (int i = 0; i < NB; ++i) t[i] = floatx4_t{0.f, 0.f, 0.f, 0.f};
                for (int s = NN ? 0 : sc; s < (NN ? a.S : sc + 1); ++s) {
                    const uint16_t *hl = a.hl + ((int64_t)s * a.T + s_tok[row]) * a.hl_row;
                    constexpr int KU = NN ? 1 : 4;            // steps whose loads are in flight together
                    const int r8 = ((a.slot_rank ? min(a.slot_rank[slot], a.R) : a.R) + 7) & ~7;
                    for (int k0 = 0; k0 < 2 * r8; k0 += 32 * KU) {
                        uint4 p[KU], q[KU][NB];
#pragma unroll
                        for (int u = 0; u < KU; ++u) {
                            const int k = k0 + u * 32 + g * 8, kr = k < r8 ? k : k - r8;
                            const bool in = k < 2 * r8;
                            p[u] = mine && in ? ldg<uint4>(hl + (k < r8 ? k : kr + a.R)) : make_uint4(0, 0, 0, 0);
#pragma unroll
                            for (int i = 0; i < NB; ++i) {
                                const int64_t n = min(c0 + (wn * NB + i) * 16 + l16, cend - 1);
                                q[u][i] = make_uint4(0, 0, 0, 0);
                                if (!in) continue;
                                if (NN) {
                                    const uint16_t *c = a.lora[s] + ((int64_t)slot * a.R + kr) * a.K + n;
                                    uint32_t v[8];
#pragma unroll
                                    for (int e = 0; e < 8; ++e) v[e] = c[(int64_t)e * a.K];
                                    q[u][i] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16,
                                                         v[6] | v[7] << 16);
                                } else {
                                    q[u][i] = ldg<uint4>(a.lora[s] + ((int64_t)slot * cend + n) * a.R + kr);
                                }
                            }
                        }
#pragma unroll
                        for (int u = 0; u < KU; ++u)
#pragma unroll
                            for (int i = 0; i < NB; ++i)
                                t[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(q[u][i]), frag(p[u]), t[i], 0, 0, 0);
                    }
                }
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][e] += mine ? t[i][e] : 0.f;
            }
        }
    }

    // One rounding per output element; a split leaves its fp32 sums by row.
    if (MIXED && a.part) {
#pragma unroll
        for (int j = 0; j < MB; ++j) {
            const int row = (wm * MB + j) * 16 + l16;
            if (m0 + row >= a.T) continue;
            float *o = a.part + ((int64_t)blockIdx.y * a.T + m0 + row) * a.part_ld + obase;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int64_t c = c0 + (wn * NB + i) * 16 + 4 * g;
                if (c < cend) *reinterpret_cast<floatx4_t *>(o + c) = acc[i][j];
            }
        }
        return;
    }
    if (NN && a.accumulate) {
#pragma unroll
        for (int j = 0; j < MB; ++j) {
            const int row = (wm * MB + j) * 16 + l16;
            if (s_slot[row] < 0) continue;
            uint16_t *o = a.out + (int64_t)s_tok[row] * a.ldo;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int64_t c = c0 + (wn * NB + i) * 16 + 4 * g;
                if (c >= cend) continue;
                const floatx4_t r = acc[i][j];
                uint2 *dst = reinterpret_cast<uint2 *>(o + c);
                const uint2 old = *dst;
                *dst = make_uint2(pack_bf16x2(r[0] + bf16_lo(old.x), r[1] + bf16_hi(old.x)),
                                  pack_bf16x2(r[2] + bf16_lo(old.y), r[3] + bf16_hi(old.y)));
            }
        }
        return;
    }
    // Through LDS (the stages are free), so that a wave writes whole rows: 8
    // bytes per lane, the 16-byte units of a row XOR-ed with the row.
    constexpr int UO = BN / 8;
    wait_barrier<0>();
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int cl = (wn * NB + i) * 16 + 4 * g;
        floatx4_t bias = {0.f, 0.f, 0.f, 0.f};
        if (!NN && a.bias && c0 + cl < cend) {
            const uint16_t *b = a.bias + obase + c0 + cl;
#pragma unroll
            for (int e = 0; e < 4; ++e) bias[e] = bf16_to_f32(b[e]);
        }
#pragma unroll
        for (int j = 0; j < MB; ++j) {
            const int row = (wm * MB + j) * 16 + l16;
            const floatx4_t r = acc[i][j];
            *reinterpret_cast<uint2 *>(s_stage + row * (BN * 2) + (((cl >> 3) ^ (row & (UO - 1))) << 4) +
                                       ((cl & 4) << 1)) =
                make_uint2(pack_bf16x2(r[0] + bias[0], r[1] + bias[1]), pack_bf16x2(r[2] + bias[2], r[3] + bias[3]));
        }
    }
    __syncthreads();
    constexpr int LPR = BN / 4, RPW = 64 / LPR > 0 ? 64 / LPR : 1;   // lanes per row, rows per wave store
    constexpr int EU = BM / (NW * RPW) < 16 ? BM / (NW * RPW) : 16;  // stores in flight
    const int cl = (lane % LPR) * 4;
    if (c0 + cl >= cend) return;
    for (int r0 = w * RPW + lane / LPR; r0 < BM; r0 += NW * RPW * EU) {
        uint2 v[EU];
        int tok[EU], sl[EU];
#pragma unroll
        for (int i = 0; i < EU; ++i) {
            const int row = r0 + i * NW * RPW;
            v[i] = *reinterpret_cast<const uint2 *>(
                s_stage + row * (BN * 2) + (((cl >> 3) ^ (row & (UO - 1))) << 4) + ((cl & 4) << 1));
            tok[i] = s_tok[row];
            sl[i] = s_slot[row];
        }
#pragma unroll
        for (int i = 0; i < EU; ++i)
            if (sl[i] != -2)
                __builtin_nontemporal_store(
                    __builtin_bit_cast(unsigned long, v[i]),
                    reinterpret_cast<unsigned long *>(a.out + (int64_t)tok[i] * a.ldo + obase + c0 + cl));
    }
}

template <int BM, int BN, int WM, int WN, int NST, bool NN, bool MIXED, bool MX>
__global__ __launch_bounds__(WM * WN * 64, BM < 256 ? 2 : 1) void k_lin_tile(LinArgs a) {
    __shared__ TileLds<BM, BN, NST, MX && !NN> sh;
    const TileAt at = tile_at(a);
    if constexpr (!MX) {
        lin_tile<BM, BN, WM, WN, NST, NN, MIXED, kQRows, false>(a, sh, at.mt, at.nt);
    } else {
        if (MIXED && at.nt >= a.base_tiles) lin_tile<BM, BN, WM, WN, NST, NN, MIXED, kQVectors, !NN>(a, sh, at.mt, at.nt);
        else lin_tile<BM, BN, WM, WN, NST, NN, MIXED, kQCodes, !NN>(a, sh, at.mt, at.nt);
    }
}

// Rank vectors of a small batch: u[t][j] = sum_k x[t][k] A[i][j][k] with no
// segment build.  Work-group = (16 tokens, the y-th different slot among them,
// 16 ranks of a slice), 8 waves each taking every eighth 64-column step of K
// straight from global memory into 16x16x32 MFMA fragments; the waves' sums
// are added in order.  Work-groups of y past the block's slots end at once;
// y = 0 clears buf for the tokens without a slot.  Latency: 9.4 us for 4 tokens of K
// 4096, rank 16; past some tokens the lora_a reads per block of 16 (500 tokens, K
// 2056, rank 8, 520 slots: 8.5 us).
constexpr int kShWaves = 8;
struct LinShrinkArgs {
    const uint16_t *x;
    int64_t ldx;
    int32_t T, K, S, L, R;
    const uint16_t *a[kMaxSlices];
    const int32_t *idx, *slot_rank;
    float *buf;
};

__global__ __launch_bounds__(kShWaves * 64) void k_lin_shrink(LinShrinkArgs a) {
    constexpr int U = 4;                          // steps in flight
    __shared__ floatx4_t s_sum[kShWaves][64];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int l16 = lane & 15, g = lane >> 4;
    const int t0 = blockIdx.x * 16, nrb = (a.R + 15) / 16;
    const int s = blockIdx.z / nrb, j0 = (blockIdx.z - s * nrb) * 16;
    const int t = t0 + l16;
    const int mine = t < a.T ? slot_of_token(a.idx, a.slot_rank, a.L, t) : -2;
    // lanes 0..15 that name a slot first; the y-th of them is this group's slot
    bool lead = mine >= 0 && lane < 16;
#pragma unroll
    for (int o = 0; o < 15; ++o) {
        const int other = __builtin_amdgcn_readlane(mine, o);
        if (o < lane && other == mine) lead = false;
    }
    unsigned long long leads = __ballot(lead);
    if (blockIdx.y == 0 && tid < 256) {
        const int tt = tid >> 4, jj = j0 + (tid & 15);
        const int sl = __shfl(mine, tt);
        if (sl == -1 && jj < a.R) a.buf[((int64_t)s * a.T + t0 + tt) * a.R + jj] = 0.f;
    }
    if ((int)blockIdx.y >= __popcll(leads)) return;
    for (unsigned y = 0; y < blockIdx.y; ++y) leads &= leads - 1;
    const int slot = __builtin_amdgcn_readlane(mine, __ffsll(leads) - 1);

    const uint16_t *xr = a.x + (int64_t)min(t, a.T - 1) * a.ldx;
    const uint16_t *ar = a.a[s] + ((int64_t)slot * a.R + min(j0 + l16, a.R - 1)) * a.K;
    const int r = a.slot_rank ? min(a.slot_rank[slot], a.R) : a.R;
    floatx4_t acc = {0.f, 0.f, 0.f, 0.f};
    const uint4 z = make_uint4(0, 0, 0, 0);
    for (int kb = w * 64; kb < a.K; kb += U * kShWaves * 64) {
        uint4 xv[U][2], av[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = kb + u * kShWaves * 64 + h * 32 + g * 8, kc = k < a.K ? k : 0;
                xv[u][h] = ldg<uint4>(xr + kc);
                av[u][h] = ldg<uint4>(ar + kc);
            }
        __builtin_amdgcn_sched_barrier(0);        // every load of the round in flight
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = kb + u * kShWaves * 64 + h * 32 + g * 8 < a.K;
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(in ? av[u][h] : z), frag(in ? xv[u][h] : z), acc,
                                                             0, 0, 0);
            }
    }
    s_sum[w][lane] = acc;
    __syncthreads();
    if (w) return;
    floatx4_t sum = s_sum[0][lane];
    for (int i = 1; i < kShWaves; ++i) {
        const floatx4_t o = s_sum[i][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += o[e];
    }
    const int j = j0 + 4 * g;
    if (mine != slot || j >= a.R) return;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (j + e >= r) sum[e] = 0.f;
    *reinterpret_cast<floatx4_t *>(a.buf + ((int64_t)s * a.T + t) * a.R + j) = sum;
}

// r += the delta of one token's 4 columns of slice s, whose lora_b rows start at
// b: fp32 FMAs with the rank vector (a slot's rows meet its own tokens only).
__device__ __forceinline__ void add_delta(floatx4_t &r, const LinArgs &a, const uint16_t *b, int s, int t, int slot) {
    const float *u = a.u + ((int64_t)s * a.T + t) * a.R;
    const int rank = a.slot_rank ? min(a.slot_rank[slot], a.R) : a.R;
    const float sc = a.scale[slot];
    floatx4_t d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
    for (int j = 0; j < rank; j += 8) {
        const floatx4_t u0 = ldg<floatx4_t>(u + j), u1 = ldg<floatx4_t>(u + j + 4);
        const float v[8] = {u0[0], u0[1], u0[2], u0[3], u1[0], u1[1], u1[2], u1[3]};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint4 w = ldg<uint4>(b + (int64_t)e * a.R + j);
            const uint32_t bw[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                d[e] += v[2 * q] * bf16_lo(bw[q]);
                d[e] += v[2 * q + 1] * bf16_hi(bw[q]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] += sc * d[e];
}

// A few tokens (decode): work-group = 16 * CT output columns, 16 * TB tokens
// (all of them), 8 waves each taking every eighth 64-column step of K straight
// from global memory into 16x16x32 MFMA fragments -- W is read once, 64 bytes
// of 16 rows per load, with U steps in flight.  The waves' sums are added in
// order through LDS; then each thread adds the delta of one token and 4
// columns.  4096 x 6144: 14.9 us for 4 tokens, 3.4 TB/s of W.
constexpr int kFewWaves = 8;
template <int TB, int CT, int U>
__global__ __launch_bounds__(kFewWaves * 64) void k_lin_few(LinArgs a) {
    __shared__ floatx4_t s_sum[kFewWaves][CT * TB][64];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int l16 = lane & 15, g = lane >> 4;
    int sc = 0;
    while (sc + 1 < a.S && (int)blockIdx.x >= a.tile_start[sc + 1]) ++sc;
    const int64_t c0 = (int64_t)(blockIdx.x - a.tile_start[sc]) * (16 * CT), cend = a.n[sc];

    const uint16_t *xr[TB], *wr[CT];
#pragma unroll
    for (int i = 0; i < TB; ++i) xr[i] = a.p + (int64_t)min(i * 16 + l16, a.T - 1) * a.ldp;
#pragma unroll
    for (int i = 0; i < CT; ++i) wr[i] = a.w + (a.off[sc] + min(c0 + i * 16 + l16, cend - 1)) * a.ldw;
    floatx4_t acc[CT][TB];
#pragma unroll
    for (int i = 0; i < CT; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    const uint4 z = make_uint4(0, 0, 0, 0);
    for (int kb = w * 64; kb < a.K; kb += U * kFewWaves * 64) {
        uint4 wv[U][2][CT], xv[U][2][TB];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = kb + u * kFewWaves * 64 + h * 32 + g * 8, kc = k < a.K ? k : 0;
#pragma unroll
                for (int i = 0; i < CT; ++i) wv[u][h][i] = ldg<uint4>(wr[i] + kc);
#pragma unroll
                for (int j = 0; j < TB; ++j) xv[u][h][j] = ldg<uint4>(xr[j] + kc);
            }
        __builtin_amdgcn_sched_barrier(0);        // every load of the round in flight
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = kb + u * kFewWaves * 64 + h * 32 + g * 8 < a.K;
#pragma unroll
                for (int i = 0; i < CT; ++i)
#pragma unroll
                    for (int j = 0; j < TB; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            frag(in ? wv[u][h][i] : z), frag(in ? xv[u][h][j] : z), acc[i][j], 0, 0, 0);
            }
    }
#pragma unroll
    for (int i = 0; i < CT; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) s_sum[w][i * TB + j][lane] = acc[i][j];
    __syncthreads();
    if (w >= CT * TB) return;                     // wave w: column block w / TB, token block w % TB
    floatx4_t r = s_sum[0][w][lane];
#pragma unroll
    for (int i = 1; i < kFewWaves; ++i) {
        const floatx4_t o = s_sum[i][w][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] += o[e];
    }
    const int t = (w % TB) * 16 + l16;
    const int64_t c = c0 + (w / TB) * 16 + 4 * g;
    if (t >= a.T || c >= cend) return;
    const int64_t col = a.off[sc] + c;
    if (a.bias) {
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] += bf16_to_f32(a.bias[col + e]);
    }
    const int slot = slot_of_token(a.idx, a.slot_rank, a.L, t);
    if (slot >= 0) add_delta(r, a, a.lora[sc] + ((int64_t)slot * cend + c) * a.R, sc, t, slot);
    *reinterpret_cast<uint2 *>(a.out + (int64_t)t * a.ldo + col) =
        make_uint2(pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3]));
}

// One token: one launch.  Work-group = 16 CT output columns, as k_lin_few, and
// the rank vector of the token's slot beside them (16 NRB lora_a rows of the
// slice, the same for every work-group and so read from L2): W and lora_a rows
// meet the same x fragments.  QKV of 4096, rank 16: 18.0 us against 22 of
// k_lin_shrink and k_lin_few; two column blocks halve the lora_a reads (one:
// 20.2, four leave CUs idle: 23.2).
template <int CT, int NRB, int U>
__global__ __launch_bounds__(kFewWaves * 64) void k_lin_one(LinArgs a) {
    __shared__ float s_sum[kFewWaves][CT + NRB][16];
    __shared__ float s_u[16 * NRB];
    __shared__ int s_own;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int l16 = lane & 15, g = lane >> 4;
    int sc = 0;
    while (sc + 1 < a.S && (int)blockIdx.x >= a.tile_start[sc + 1]) ++sc;
    const int tile = blockIdx.x - a.tile_start[sc];
    const int64_t c0 = (int64_t)tile * (16 * CT), cend = a.n[sc];
    const uint16_t *wr[CT], *ar[NRB];
#pragma unroll
    for (int i = 0; i < CT; ++i) wr[i] = a.w + (a.off[sc] + min(c0 + i * 16 + l16, cend - 1)) * a.ldw;
    uint4 bv[CT][(NRB + 1) / 2];
    int slot = -1, rank = 0;
    float sc_own = 0.f;
    floatx4_t acc[CT], au[NRB];
#pragma unroll
    for (int i = 0; i < CT; ++i) acc[i] = floatx4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NRB; ++i) au[i] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    const uint4 z = make_uint4(0, 0, 0, 0);
    for (int kb = w * 64; kb < a.K; kb += U * kFewWaves * 64) {
        uint4 wv[U][2][CT], xv[U][2], av[U][2][NRB];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = kb + u * kFewWaves * 64 + h * 32 + g * 8, kc = k < a.K ? k : 0;
#pragma unroll
                for (int i = 0; i < CT; ++i) wv[u][h][i] = ldg<uint4>(wr[i] + kc);
                xv[u][h] = ldg<uint4>(a.p + kc);
            }
        __builtin_amdgcn_sched_barrier(0);
        if (kb == w * 64) {
            // the slot's loads, one after the other, behind those of W
            slot = slot_of_token(a.idx, a.slot_rank, a.L, 0);
            const int so = max(slot, 0);
            rank = slot < 0 ? 0 : a.slot_rank ? min(a.slot_rank[so], a.R) : a.R;
            sc_own = a.scale[so];
#pragma unroll
            for (int i = 0; i < NRB; ++i)
                ar[i] = a.other[sc] + ((int64_t)so * a.R + min(i * 16 + l16, a.R - 1)) * a.K;
#pragma unroll
            for (int i = 0; i < CT; ++i) {
                const uint16_t *b = a.lora[sc] + ((int64_t)so * cend + min(c0 + i * 16 + l16, cend - 1)) * a.R;
#pragma unroll
                for (int j = 0; j < (NRB + 1) / 2; ++j) bv[i][j] = ldg<uint4>(b + min(j * 32 + g * 8, a.R - 8));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = kb + u * kFewWaves * 64 + h * 32 + g * 8, kc = k < a.K ? k : 0;
#pragma unroll
                for (int i = 0; i < NRB; ++i) av[u][h][i] = ldg<uint4>(ar[i] + kc);
            }
        __builtin_amdgcn_sched_barrier(0);        // every load of the round in flight
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = kb + u * kFewWaves * 64 + h * 32 + g * 8 < a.K;
                const bf16x8_t x = frag(in ? xv[u][h] : z);
#pragma unroll
                for (int i = 0; i < CT; ++i)
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(in ? wv[u][h][i] : z), x, acc[i], 0, 0, 0);
#pragma unroll
                for (int i = 0; i < NRB; ++i)
                    au[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(in ? av[u][h][i] : z), x, au[i], 0, 0, 0);
            }
    }
    // every result column is the token: column 0's lanes give the sums
    if (l16 == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int i = 0; i < CT; ++i) s_sum[w][i][4 * g + e] = acc[i][e];
#pragma unroll
            for (int i = 0; i < NRB; ++i) s_sum[w][CT + i][4 * g + e] = au[i][e];
        }
    }
    if (tid == 0) s_own = rank;                   // (a wave without a K step knows no slot)
    __syncthreads();
    rank = s_own;
    if (tid < 16 * NRB) {
        float u = 0.f;
#pragma unroll
        for (int i = 0; i < kFewWaves; ++i) u += s_sum[i][CT + (tid >> 4)][tid & 15];
        if (tid >= rank) u = 0.f;
        s_u[tid] = u;
        if (a.buf && tile == 0 && tid < a.R) a.buf[(int64_t)sc * a.R + tid] = u;
    }
    __syncthreads();
    if (w) return;
#pragma unroll
    for (int i = 0; i < CT; ++i) {
        const int64_t c = c0 + i * 16 + l16;
        float d = 0.f, y = 0.f;
        if (slot >= 0) {
#pragma unroll
            for (int jb = 0; jb < (NRB + 1) / 2; ++jb) {
                const int j = jb * 32 + g * 8;
                if (j < rank) {
                    const uint32_t bw[4] = {bv[i][jb].x, bv[i][jb].y, bv[i][jb].z, bv[i][jb].w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        d += s_u[j + 2 * q] * bf16_lo(bw[q]);
                        d += s_u[j + 2 * q + 1] * bf16_hi(bw[q]);
                    }
                }
            }
            d += __shfl_xor(d, 16);
            d += __shfl_xor(d, 32);
            d *= sc_own;
        }
#pragma unroll
        for (int k = 0; k < kFewWaves; ++k) y += s_sum[k][i][l16];
        if (g == 0 && c < cend) {
            if (a.bias) y += bf16_to_f32(a.bias[a.off[sc] + c]);
            a.out[a.off[sc] + c] = (uint16_t)f32_to_bf16_rne(y + d);
        }
    }
}

// The K splits of a tile GEMM, summed in order, bias (and with join_delta the
// forward's delta) added, rounded once.  Wave = 16 rows x 64 columns in the
// layout of a 16x16 MFMA result (row lane % 16, 4 columns).  The delta: for each
// slot among the 16 rows, its lora_b rows straight from global memory into
// fragments (the next step's loads in flight), times the rows' scaled rank
// vectors split into two bf16 parts, kept by the slot's own rows only.  Bound by
// those rows: 1024 tokens of 128 slots, 8192 columns, ranks to 128: 60 us; with
// no delta 4.2 us for 96 x 4096 in four splits.
// (Three waves per SIMD: without a bound the compiler takes registers for two, 73
// us; bounded to four it spills, 99.)
constexpr int kJoinRows = 16;
constexpr int kJoinCols = 256;
__global__ __launch_bounds__(256, 3) void k_lin_join(LinArgs a) {
    constexpr int NB = 4;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, l16 = lane & 15, g = lane >> 4;
    const int m = blockIdx.y * kJoinRows + l16;
    const bool real = m < a.T;
    const int mc = min(m, a.T - 1);
    const int t = a.order[mc];
    const int slot = a.join_delta && real ? a.order[a.T + mc] : -1;
    const int64_t c0 = (int64_t)blockIdx.x * kJoinCols + w * (NB * 16);
    if (c0 >= a.part_ld) return;
    floatx4_t v[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) v[i] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < a.ksp; ++k) {
        const float *p = a.part + ((int64_t)k * a.T + mc) * a.part_ld;
        floatx4_t o[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) o[i] = ldg<floatx4_t>(p + min(c0 + i * 16 + 4 * g, a.part_ld - 4));
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i][e] += o[i][e];
    }
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i][e] += bf16_to_f32(a.bias[min(c0 + i * 16 + 4 * g, a.part_ld - 4) + e]);
    }
    if (a.join_delta) {
        // a lane's lora_b row of each 16-column block and its slice, by selects
        // (an index that differs between lanes would load the arguments from
        // memory one after the other).  A block may straddle slices: columns
        // 4 g..+3 of a result lane are of one slice, found the same way.
        const uint16_t *row[NB];
        int64_t n[NB];
        int sb[NB], first = 0, last = 0;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int64_t c = min(c0 + i * 16 + l16, a.part_ld - 1), cv = min(c0 + i * 16 + 4 * g, a.part_ld - 4);
            int64_t o = 0;
            n[i] = a.n[0];
            row[i] = a.lora[0];
            sb[i] = 0;
#pragma unroll
            for (int s = 1; s < kMaxSlices; ++s)
                if (s < a.S) {
                    if (c >= a.off[s]) { o = a.off[s]; n[i] = a.n[s]; row[i] = a.lora[s]; }
                    if (cv >= a.off[s]) sb[i] = s;
                }
            row[i] += (c - o) * a.R;
        }
        for (int s = 1; s < a.S; ++s) {
            if (c0 >= a.off[s]) first = s;
            if (min(c0 + NB * 16, a.part_ld) - 1 >= a.off[s]) last = s;
        }
        const int rank_own = slot < 0 ? 0 : a.slot_rank ? min(a.slot_rank[slot], a.R) : a.R;
        const float sc = slot < 0 ? 0.f : a.scale[slot];
        unsigned long long todo = __ballot(slot >= 0) & 0xffff;
        int cur = -1, rank = 0, k0 = 0;
        auto pop = [&]() {
            const int l = __ffsll(todo) - 1;
            cur = __builtin_amdgcn_readlane(slot, l);
            rank = __builtin_amdgcn_readlane(rank_own, l);
            todo &= ~__ballot(slot == cur);
            k0 = 0;
        };
        auto fetch = [&](uint4 (&q)[NB]) {
            const int k = k0 + g * 8;
#pragma unroll
            for (int i = 0; i < NB; ++i)
                q[i] = k < rank ? ldg<uint4>(row[i] + (int64_t)cur * n[i] * a.R + k) : make_uint4(0, 0, 0, 0);
        };
        uint4 q[NB], qn[NB];
        floatx4_t d[NB];
        if (todo) {
            pop();
            fetch(q);
        }
        while (cur >= 0) {
            const int at = cur, kb = k0;
            const bool mine = slot == at;
            if (kb == 0) {
#pragma unroll
                for (int i = 0; i < NB; ++i) d[i] = floatx4_t{0.f, 0.f, 0.f, 0.f};
            }
            k0 += 32;
            if (k0 >= rank) {
                if (todo) pop();
                else cur = -1;
            }
            if (cur >= 0) fetch(qn);
            const int k = kb + g * 8;
            for (int s = first; s <= last; ++s) {
                uint32_t part[8][3];
#pragma unroll
                for (int e = 0; e < 8; ++e) part[e][0] = part[e][1] = 0;
                if (mine && k < rank_own) {
                    const float *u = a.u + ((int64_t)s * a.T + t) * a.R + k;
                    const floatx4_t u0 = ldg<floatx4_t>(u), u1 = ldg<floatx4_t>(u + 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        split_bf16(sc * u0[e], part[e]);
                        split_bf16(sc * u1[e], part[4 + e]);
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bf16x8_t p = frag(make_uint4(part[0][h] | part[1][h] << 16, part[2][h] | part[3][h] << 16,
                                                       part[4][h] | part[5][h] << 16, part[6][h] | part[7][h] << 16));
#pragma unroll
                    for (int i = 0; i < NB; ++i) {
                        const floatx4_t r = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(q[i]), p, d[i], 0, 0, 0);
                        if (first == last) d[i] = r;
                        else if (sb[i] == s) d[i] = r;
                    }
                }
            }
            if (cur != at) {
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[i][e] = mine ? v[i][e] + d[i][e] : v[i][e];
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) q[i] = qn[i];
        }
    }
    if (!real) return;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int64_t c = c0 + i * 16 + 4 * g;
        if (c < a.part_ld)
            *reinterpret_cast<uint2 *>(a.out + (int64_t)t * a.ldo + c) =
                make_uint2(pack_bf16x2(v[i][0], v[i][1]), pack_bf16x2(v[i][2], v[i][3]));
    }
}

// Two columns c, c + 1 of one token: the sum of the splits o, bias, delta (the
// rank vector from u), rounded once.
struct JoinB {                // a thread's two lora_b rows (forward), and their first 16 ranks
    const uint16_t *p;
    int s;
    uint4 b0[2], b1[2];
};
template <bool NN, int MK>
__device__ __forceinline__ void join_row(const LinArgs &a, int t, int64_t c, int slot, int rank,
                                         const float2 (&o)[MK], const JoinB &jb, const float *u, int64_t ldu) {
    if (c >= a.cols) return;
    float v0 = 0.f, v1 = 0.f;
#pragma unroll
    for (int k = 0; k < MK; ++k)
        if (k < a.ksp) {
            v0 += o[k].x;
            v1 += o[k].y;
        }
    if (a.bias) {
        v0 += bf16_to_f32(a.bias[c]);
        v1 += bf16_to_f32(a.bias[c + 1]);
    }
    if (NN && slot >= 0) {
        float d0 = 0.f, d1 = 0.f;
        for (int s = 0; s < a.S; ++s) {
            const uint16_t *b = a.lora[s] + (int64_t)slot * a.R * a.K + c;
            const float *us = u + s * ldu;
            for (int j = 0; j < rank; j += 8) {   // (vectors are zero past the rank)
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = ldg<uint32_t>(b + (int64_t)(j + e) * a.K);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    d0 += us[j + e] * bf16_lo(w[e]);
                    d1 += us[j + e] * bf16_hi(w[e]);
                }
            }
        }
        const float sc = a.scale[slot];
        v0 += sc * d0;
        v1 += sc * d1;
    }
    if (!NN && slot >= 0) {
        float d0 = 0.f, d1 = 0.f;
        const float *us = u + jb.s * ldu;
        auto add8 = [&](const uint4 &b0, const uint4 &b1, int j) __attribute__((always_inline)) {
            const floatx4_t u0 = *reinterpret_cast<const floatx4_t *>(us + j);
            const floatx4_t u1 = *reinterpret_cast<const floatx4_t *>(us + j + 4);
            const float uv[8] = {u0[0], u0[1], u0[2], u0[3], u1[0], u1[1], u1[2], u1[3]};
            const uint32_t w0[4] = {b0.x, b0.y, b0.z, b0.w}, w1[4] = {b1.x, b1.y, b1.z, b1.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                d0 += uv[2 * q] * bf16_lo(w0[q]);
                d0 += uv[2 * q + 1] * bf16_hi(w0[q]);
                d1 += uv[2 * q] * bf16_lo(w1[q]);
                d1 += uv[2 * q + 1] * bf16_hi(w1[q]);
            }
        };
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (i * 8 < rank) add8(jb.b0[i], jb.b1[i], i * 8);
#pragma unroll 2
        for (int j = 16; j < rank; j += 8) add8(ldg<uint4>(jb.p + j), ldg<uint4>(jb.p + a.R + j), j);
        const float sc = a.scale[slot];
        v0 += sc * d0;
        v1 += sc * d1;
    }
    *reinterpret_cast<uint32_t *>(a.out + (int64_t)t * a.ldo + c) = pack_bf16x2(v0, v1);
}
// The same for a direct batch, whose rows are in token order: 16 rows then name
// up to 16 slots, and one after the other they cost the MFMA form above more
// than it saves (256 tokens of 8 slots, 6144 columns, rank 16: 22.8 against
// 12.6 us).  Work-group = one token x 512 columns, 2 per thread, so that a
// wave's lora_b loads cover whole lines: fp32 FMAs with the token's rank vector.
// In a wide batch every work-group first sums the splits of its token's rank
// vector.  Gradient (NN, wide only): v against the slot's lora_a rows.
template <bool NN, int MK>
__global__ __launch_bounds__(256) void k_lin_join_rows(LinArgs a) {
    const int t = blockIdx.y;
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 2;
    const int slot = slot_of_token(a.idx, a.slot_rank, a.L, t);
    const float *pt = a.part + (int64_t)t * a.part_ld;
    const int64_t split = (int64_t)a.T * a.part_ld;
    float2 o[MK];
#pragma unroll
    for (int k = 0; k < MK; ++k)
        if (k < a.ksp) o[k] = *reinterpret_cast<const float2 *>(pt + k * split + min(c, a.cols - 2));
    JoinB jb;
    if (!NN && slot >= 0) {
        // the column's slice by selects (an index that differs between lanes
        // would load the arguments from memory, one after the other); the rows' loads run
        // beside those of the rank vector's sums
        const int64_t cc = min(c, a.cols - 2);
        int64_t off = 0, n = a.n[0];
        jb.s = 0;
        jb.p = a.lora[0];
#pragma unroll
        for (int i = 1; i < kMaxSlices; ++i)
            if (i < a.S && cc >= a.off[i]) { jb.s = i; off = a.off[i]; n = a.n[i]; jb.p = a.lora[i]; }
        jb.p += ((int64_t)slot * n + cc - off) * a.R;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            jb.b0[i] = ldg<uint4>(jb.p + min(i * 8, a.R - 8));
            jb.b1[i] = ldg<uint4>(jb.p + a.R + min(i * 8, a.R - 8));
        }
    }
    const int rank = slot < 0 ? 0 : a.slot_rank ? min(a.slot_rank[slot], a.R) : a.R;
    if (NN || a.wide) {
        __shared__ __attribute__((aligned(16))) float s_u[kLinWideRanks];
        for (int q = threadIdx.x; q < a.S * a.R; q += 256) {
            const int s = q / a.R, j = q - s * a.R;
            float u = 0.f;
            if (j < rank) {
                const float *p = pt + a.cols + s * a.u_slice + slot * a.u_slot + j;
                float w[MK];
#pragma unroll
                for (int k = 0; k < MK; ++k)
                    if (k < a.ksp) w[k] = p[k * split];
#pragma unroll
                for (int k = 0; k < MK; ++k)
                    if (k < a.ksp) u += w[k];
            }
            s_u[q] = u;
            if (a.buf && blockIdx.x == 0) a.buf[((int64_t)s * a.T + t) * a.R + j] = u;
        }
        __syncthreads();
        join_row<NN>(a, t, c, slot, rank, o, jb, s_u, a.R);
        return;
    }
    if (a.buf && slot < 0 && blockIdx.x == 0) {
        // the rank vectors of a token without a slot, which the grouped shrink leaves
        for (int s = 0; s < a.S; ++s)
            for (int j = threadIdx.x; j < a.R; j += 256) a.buf[((int64_t)s * a.T + t) * a.R + j] = 0.f;
    }
    join_row<NN>(a, t, c, slot, rank, o, jb, a.u + (int64_t)t * a.R, (int64_t)a.T * a.R);
}
// Rank vectors from partial sums (by slot-sorted position) or from a caller's
// buffer (by token): sums the splits in order, zeroes ranks past the slot's
// own, scales, splits into bf16 parts, and clears buf for tokens without a
// slot.  Latency bound: 9.7 us for 8192 tokens of 2 x 64 ranks with the row order,
// 5.6 for 1024 of 128.
constexpr int kRedThreads = 256;
struct LinReduceArgs {
    LinVectors job[2];
    int32_t n_jobs, T, S, L, R;
    const int32_t *idx, *slot_rank;
    const float *scale;
    SegPtrs seg;
    int32_t *order;
};

// The row order of the tile GEMM: each slot's tokens, slots ascending, then
// the tokens without a slot in token order; and each row's slot (or -1) after
// it.  A work-group writes 256 positions of the slots' runs and places its 256
// tokens without a slot, whose number before it is counted from idx (a bitmap
// of the slots in use in LDS), or past kOrderScan tokens from the slots' runs,
// since the counting grows with the square of the tokens (all of k_lin_vectors,
// rank 8, us: 4096 tokens, 8 slots 5.7 and by the runs 4.9, 1024 slots 5.3 and 7.9;
// 8192 tokens 8.0 and 5.6; 2^20 tokens 1180 and 37, of 1024 slots 1190 and 203).
constexpr int kOrderScan = 4096;
__device__ __forceinline__ void row_order(const LinReduceArgs &a) {
    constexpr int NW = kRedThreads / 64;
    __shared__ unsigned s_act[kMaxSlots / 32];
    __shared__ int s_cnt[NW], s_before[NW];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int base = blockIdx.x * kRedThreads, t = base + tid;
    for (int i = tid; i < kMaxSlots; i += kRedThreads) {
        const unsigned long long b = __ballot(i < a.L && (!a.slot_rank || a.slot_rank[i] > 0));
        if (lane == 0) {
            s_act[i >> 5] = (unsigned)b;
            s_act[(i >> 5) + 1] = (unsigned)(b >> 32);
        }
    }
    __syncthreads();
    auto none = [&](int s) { return s < 0 || s >= a.L || !(s_act[s >> 5] >> (s & 31) & 1); };
    int before = 0;
    if (base <= kOrderScan) {
#pragma unroll 8
        for (int i = tid; i < base; i += kRedThreads) before += none(a.idx[i]);
    } else {
        // all tokens before the block but the slots' own (a run ascends)
        before = tid == 0 ? base : 0;
        for (int s = tid; s < a.L; s += kRedThreads) {
            const int start = a.seg.slot_start[s];
            int lo = start, hi = a.seg.slot_start[s + 1];
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (a.seg.perm[mid] < base) lo = mid + 1;
                else hi = mid;
            }
            before -= lo - start;
        }
    }
    for (int d = 32; d; d >>= 1) before += __shfl_xor(before, d);
    const bool mine = t < a.T && none(a.idx[t]);
    const unsigned long long b = __ballot(mine);
    if (lane == 0) {
        s_before[w] = before;
        s_cnt[w] = __popcll(b);
    }
    __syncthreads();
    const int run_end = a.seg.header[0];
    if (mine) {
        int pos = run_end + __popcll(b & ((1ull << lane) - 1));
        for (int i = 0; i < NW; ++i) pos += s_before[i];
        for (int i = 0; i < w; ++i) pos += s_cnt[i];
        a.order[pos] = t;
        a.order[a.T + pos] = -1;
    }
    if (t < run_end) {
        const int tok = a.seg.perm[t];
        a.order[t] = tok;
        a.order[a.T + t] = a.idx[tok];
    }
}

// grid.y: a slice of a job, then the row order.
__global__ __launch_bounds__(kRedThreads) void k_lin_vectors(LinReduceArgs a) {
    if ((int)blockIdx.y == a.S * a.n_jobs) {
        if ((int)blockIdx.x * kRedThreads < a.T) row_order(a);
        return;
    }
    const LinVectors &v = a.job[blockIdx.y / a.S];
    const int s = blockIdx.y % a.S;
    const unsigned rq = a.R / 4;                              // 4 ranks per thread
    const int64_t q = (int64_t)blockIdx.x * kRedThreads + threadIdx.x;
    const int64_t i = q < UINT32_MAX ? (int64_t)((unsigned)q / rq) : q / rq;
    const int j = (int)(q - i * rq) * 4;
    if (i >= a.T) return;
    // as a token: buf of tokens without a slot
    if (v.buf && slot_of_token(a.idx, a.slot_rank, a.L, (int)i) < 0)
        *reinterpret_cast<floatx4_t *>(v.buf + ((int64_t)s * a.T + i) * a.R + j) = floatx4_t{0.f, 0.f, 0.f, 0.f};
    // as a slot-sorted position
    if (i >= a.seg.header[0]) return;
    const int t = a.seg.perm[i];
    const int slot = a.idx[t];
    const int r = a.slot_rank ? min(a.slot_rank[slot], a.R) : a.R;
    floatx4_t sum = {0.f, 0.f, 0.f, 0.f};
    if (v.part) {
#pragma unroll 4
        for (int k = 0; k < v.nsp; ++k) {
            const floatx4_t o = *reinterpret_cast<const floatx4_t *>(
                v.part + (((int64_t)s * v.nsp + k) * a.T + i) * a.R + j);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] += o[e];
        }
    } else {
        sum = *reinterpret_cast<const floatx4_t *>(v.in + ((int64_t)s * a.T + t) * a.R + j);
    }
    const float sc = a.scale[slot];
    const int64_t row = (int64_t)s * a.T + t;
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (j + e >= r) sum[e] = 0.f;
        x[e] = j + e < r ? sc * sum[e] : 0.f;
    }
    if (v.hl) store_parts(v.hl + row * v.parts * a.R, v.parts, a.R, j, x);
    if (v.buf) *reinterpret_cast<floatx4_t *>(v.buf + row * a.R + j) = sum;
}

// Column tiles of width b by slice; returns their number.
int column_tiles(LinArgs &a, int b) {
    int c = 0;
    for (int s = 0; s < a.S; ++s) {
        a.tile_start[s] = c;
        c += (int)((a.n[s] + b - 1) / b);
    }
    for (int s = a.S; s <= kMaxSlices; ++s) a.tile_start[s] = c;
    return c;
}

template <int BM, int BN, int WM, int WN, int NST, bool MIXED, bool MX>
hipError_t run_tile_of(LinArgs a, bool gradient, int ksp, hipStream_t st) {
    a.m_tiles = (a.T + BM - 1) / BM;
    a.base_tiles = a.n_tiles = gradient ? (a.K + BN - 1) / BN : column_tiles(a, BN);
    a.ksp = ksp;
    int64_t cols = a.K;
    if (!gradient) {
        cols = 0;
        for (int s = 0; s < a.S; ++s) cols += a.n[s];
    }
    a.cols = a.part_ld = cols;
    if (a.wide) {
        a.part_ld += (int64_t)a.S * a.L * a.R;
        a.u_slice = a.L * a.R;
        a.u_slot = a.R;
        a.n_tiles += a.S * ((a.L * a.R + BN - 1) / BN);
    }
    if (ksp == 1 && !a.join_delta) a.part = nullptr;
    const dim3 grid((unsigned)(a.m_tiles * a.n_tiles), (unsigned)ksp), block(WM * WN * 64);
    if (gradient) hipLaunchKernelGGL((k_lin_tile<BM, BN, WM, WN, NST, true, MIXED, MX && MIXED>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_lin_tile<BM, BN, WM, WN, NST, false, MIXED, MX>), grid, block, 0, st, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.part) return e;
    if (a.join_delta && !gradient && !a.order) return launch_lin_join_rows(a, st);
    if (a.join_delta && gradient)
        hipLaunchKernelGGL((k_lin_join_rows<true, kLinMaxSplits>), dim3((unsigned)((cols + 511) / 512), (unsigned)a.T), dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL(k_lin_join, dim3((unsigned)((cols + kJoinCols - 1) / kJoinCols),
                                            (unsigned)((a.T + kJoinRows - 1) / kJoinRows)), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int NST, bool MIXED>
hipError_t run_tile(const LinArgs &a, bool gradient, int ksp, hipStream_t st) {
    return a.ws ? run_tile_of<BM, BN, WM, WN, NST, MIXED, true>(a, gradient, ksp, st)
                : run_tile_of<BM, BN, WM, WN, NST, MIXED, false>(a, gradient, ksp, st);
}

template <int CT, int NRB, int U>
hipError_t run_one(LinArgs a, hipStream_t st) {
    const int n = column_tiles(a, 16 * CT);
    hipLaunchKernelGGL((k_lin_one<CT, NRB, U>), dim3((unsigned)n), dim3(kFewWaves * 64), 0, st, a);
    return hipGetLastError();
}

template <int TB, int CT, int U>
hipError_t run_few(LinArgs a, hipStream_t st) {
    const int n = column_tiles(a, 16 * CT);
    hipLaunchKernelGGL((k_lin_few<TB, CT, U>), dim3((unsigned)n), dim3(kFewWaves * 64), 0, st, a);
    return hipGetLastError();
}

int64_t tiles(int32_t T, int32_t K, const int64_t *N, int32_t S, bool gradient, int b) {
    int64_t c = 0;
    if (gradient) c = (K + b - 1) / b;
    else
        for (int s = 0; s < S; ++s) c += (N[s] + b - 1) / b;
    return c * ((T + b - 1) / b);
}

}  // namespace

// A launch's threads stay under 2^32: tile work-groups of 256 threads, and
// column tiles times rank blocks of the weight gradients.
bool lin_grid_fits(int32_t T, int32_t K, const int64_t *N, int32_t S) {
    for (int s = 0; s < S; ++s)
        if (N[s] > (1 << 24)) return false;
    return K <= (1 << 24) && tiles(T, K, N, S, false, 256) <= (1 << 22) &&
           tiles(T, K, N, S, true, 256) <= (1 << 22);
}

// The tiles of a batch and their K splits.  join, wide: LinArgs' join_delta and
// wide; base: there is a base product.  (Times at this rule and the next ones: us of
// whole calls in graph replays.  They repeat within 2 %, so figures nearer than
// that are ties.)
LinTilePlan lin_tile_plan(int32_t T, int32_t K, const int64_t *N, int32_t S, int32_t R, int32_t L, bool gradient,
                          bool join, bool wide, bool base) {
    // 256 x 256 from 192 tiles on, most of a tile per CU (4096 tokens, 4096 x 4096, 256
    // tiles: 143 us, 163 with 128 x 128; 2048 tokens, 4096 x 6144, 192 tiles: 132 and
    // 128; 128 tiles: 132 and 97).
    if (!join && tiles(T, K, N, S, gradient, 256) >= 192) return {256, 1};
    int64_t nk = (K + 63) / 64;
    if (gradient) {
        nk = 0;
        for (int s = 0; s < S; ++s) nk += (N[s] + 63) / 64;
    }
    if (!base) nk = 0;
    // K splits, about kLinSplitTiles work-groups of at least 8 K tiles each; 4 of a
    // few tokens that are joined anyway, whose sums are small (4 tokens of 1352 x
    // 1652 9.5 us, 11.5 with 8; 64 tokens 11.7 and 12.5, of 512 x 4096 10.6 and 11.0,
    // of 2048 x 2048 12.3 and 11.8; 128 tokens 14.7 and 13.6)
    const int least = join && T <= 64 ? 4 : 8;
    auto splits = [&](int64_t t) {
        int64_t k = kLinSplitTiles / t;
        if (k > nk / least) k = nk / least;
        if (k > kLinMaxSplits) k = kLinMaxSplits;
        return (int32_t)(k < 1 ? 1 : k);
    };
    int64_t t128 = tiles(T, K, N, S, gradient, 128), t64 = tiles(T, K, N, S, gradient, 64);
    if (wide) {
        t128 += (int64_t)S * ((L * R + 127) / 128) * ((T + 127) / 128);
        t64 += (int64_t)S * ((L * R + 63) / 64) * ((T + 63) / 64);
    }
    // From 192 tiles of 128 x 128 on a join costs more than even work-groups give
    // (2048 tokens, 4096 x 4096: 97 us; 132 with 256 x 256, 147 with 64 x 64), but
    // for one tile per CU of many K tiles, which two splits overlap (the gradient of
    // 1024 tokens, 28672 x 4096, 448 K tiles: 303 and 277; 6144 x 4096, 96 K tiles:
    // 94.7 and 96.2).  Where a join runs anyway, two or three splits even the
    // work-groups out up to 340 tiles (512 tokens, 4096 x 6144, 204 tiles: 58.5,
    // two splits 54.9; 1024 tokens, 14336 x 4096, 264 tiles: 198, 172 and 156; 452
    // tiles: 117 and 126 with two).
    if (t128 >= 192) {
        int32_t k = t128 <= 256 && nk >= 192 ? 2 : 1;
        if (join && t128 <= kLinEvenTiles && nk >= 24) k = t128 > 256 ? 3 : 2;
        return {128, k};
    }
    // Fewer tiles: K splits, joined by a second launch.  Tiles of 64 x 64 read each
    // operand twice as often, which shows once all their K tiles together pass some
    // 16000 (256 tokens, K x N, with them and with 128 x 128: 2048 x 2048 16.1 and
    // 20.0 us, 4096 x 4096 41.0 and 36.9, 14336 x 4096 89.4 and 52.1; 128 tokens,
    // 4096 x 6144 26.3 and 31.0), or once they no longer run at the same time (the
    // gradient of 1501 tokens, 1652 x 1352, 528 of them: 61.4 and 53.1).
    if (t128 * splits(t128) >= kLinSplitTiles / 2 && (t64 > kLinSplitTiles || t64 * nk > 16384))
        return {128, splits(t128)};
    // (two stages: a work-group has few K tiles, and more stages fill for longer;
    // 16 tokens of 14336 x 4096: 26.3 us, with four 28.2)
    return {64, splits(t64)};
}

// The fp32 sums of any batch stay within kLinJoinMax elements, which the
// workspace holds: splits times the tiles' elements; unsplit, lin_join_delta
// tests them itself, and a direct batch or a wide gradient, whose further columns
// are no more than the layer's own, is bounded by its bytes at rank 8 and up.
static_assert(kLinSplitTiles * 128 * 128 <= kLinJoinMax, "sums of split tiles");
static_assert(2 * 256 * 128 * 128 <= kLinJoinMax && 3 * kLinEvenTiles * 128 * 128 <= kLinJoinMax, "sums of even tiles");
static_assert(2 * (kLinWideBytesB / 32) <= kLinJoinMax && 2 * (kLinWideBytesA / 32) <= kLinJoinMax &&
              kLinDirectBytesB / 32 <= kLinJoinMax, "unsplit sums");

hipError_t launch_lin_join_rows(const LinArgs &a, hipStream_t st) {
    const dim3 rows((unsigned)((a.cols + 511) / 512), (unsigned)a.T);
    if (a.ksp <= kLinMaxSplits) hipLaunchKernelGGL((k_lin_join_rows<false, kLinMaxSplits>), rows, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_lin_join_rows<false, kMxFewSplits>), rows, dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_lin_gemm(LinArgs a, bool gradient, hipStream_t st) {
    // (4-bit batches that lin_few would take: mx_few, or the tiles)
    if (!gradient && !a.ws && lin_one(a.T, a.K, a.n, a.S, a.R)) return a.R <= 16 ? run_one<2, 1, 2>(a, st) : run_one<2, 2, 2>(a, st);
    if (!gradient && !a.ws && lin_few(a.T, a.K, a.n, a.S, a.R, a.L)) {
        if (a.T <= 16) return run_few<1, 1, 4>(a, st);
        if (a.T <= 32) return run_few<2, 2, 4>(a, st);
        return run_few<4, 2, 2>(a, st);
    }
    const LinTilePlan p = lin_tile_plan(a.T, a.K, a.n, a.S, a.R, a.L, gradient, a.join_delta, a.wide, a.w != nullptr);
    // (a gradient's 4-bit projection is restored for these: its codes are no bf16 rows)
    if (p.tile == 256 && gradient && a.ws) return hipErrorInvalidValue;
    if (p.tile == 256) return gradient ? run_tile_of<256, 256, 2, 2, 2, false, false>(a, true, 1, st)
                                       : run_tile<256, 256, 2, 2, 2, false>(a, false, 1, st);
    if (p.tile == 128) return run_tile<128, 128, 2, 2, 2, true>(a, gradient, p.splits, st);
    return run_tile<64, 64, 2, 2, 2, true>(a, gradient, p.splits, st);
}

// Whether a sorted forward batch leaves the delta to the join: when the
// rank-vector K tiles that a 128-token tile is expected to meet (its share of
// the slots, and one for a slot that continues) pass a share of its base K
// tiles, and the fp32 sums stay within kLinJoinMax.  The share is larger where
// writing and reading the sums weighs more than a few tiles' tail.  With the
// delta in the tiles against the join, K 4096, share in brackets: 512 tokens,
// 6144 columns, rank 64, 32 slots [.28] 99.8 against 82.3 us, rank 128, 16
// slots [.31] 99.8 against 85.3; 1024 tokens, 4096 columns, rank 128, 16 slots
// [.19] 89.6 against 94.2; 2048 tokens, 4096 columns, rank 128, 64 slots [.31]
// 148 against 154; K 8192, 1024 tokens, 8192 columns, rank 128, 128 slots
// [.53] 343 against 309.
bool lin_join_delta(int32_t T, int32_t K, const int64_t *N, int32_t S, int32_t R, int32_t L) {
    int64_t n = 0;
    for (int s = 0; s < S; ++s) n += N[s];
    if ((int64_t)T * n > kLinJoinMax || (T + kJoinRows - 1) / kJoinRows > 65535) return false;
    const double slots = 128.0 * (T < L ? T : L) / T + 1.0;
    return slots * ((2 * R + 63) / 64) > K / 64 * ((int64_t)T * n <= 1 << 22 ? 0.25 : 0.4);
}

// The further columns of a wide batch, x A^T of every slot, in whole 64-column
// tiles; 0 when they would be more than the layer's own (or their vectors more
// than the join holds).
static int64_t wide_cols(int64_t n, int32_t S, int32_t R, int32_t L) {
    const int64_t c = (int64_t)S * ((L * R + 63) / 64) * 64;
    return c <= n && S * R <= kLinWideRanks ? c : 0;
}
static int64_t columns(const int64_t *N, int32_t S) {
    int64_t n = 0;
    for (int s = 0; s < S; ++s) n += N[s];
    return n;
}

// One token of rank at most 32 takes the one launch of k_lin_one while K is at
// most two rounds of its loads and its work-groups (32 columns, each reading the
// slot's lora_a rows) fit the CUs once, or K and the rank are small.  Against the
// wide tiles (two launches), us, medians of graph replays that repeat within 2 %:
// K x N of 2048 x 2048 8.6 and 9.5, 1024 x 16384 9.6 and 14.9, 2048 x 16384 18.1 and
// 20.8 (rank 32 22.0 and 21.6, 1536 x 12288 19.1 and 15.4); 4096 x 4096 15.0 and
// 13.8, x 5120 15.9 and 15.5, x 5632 15.9 and 16.1, x 6144 15.8 and 16.8, x 8192
// 17.7 and 18.8, x 8448 28.6 and 19.3; 3200 x 8192 13.9 and 17.1, x 8448 22.8 and
// 17.2.  Longer K: 5120 x 5120 18.5 and 16.9; 8192 x 1024 25.3 and 12.2.
bool lin_one(int32_t T, int32_t K, const int64_t *N, int32_t S, int32_t R) {
    const int64_t n = columns(N, S);
    if (T != 1 || R > 32) return false;
    if (n > 8192) return n <= 16384 && K <= 2048 && R <= 16;
    return K <= 2048 || (K <= 4096 && R <= 16 && n > 5120);
}

// Whether k_lin_few (or k_lin_one) takes a forward batch.  Its work-groups read
// x over and over, so the tiles overtake it as tokens times W grow.  Against the wide tiles, us: 2048 x 1024,
// 4 tokens 11.3 and 9.2; with as many further columns as the layer's (4096 x 6144,
// rank 16, 128 slots) one token 20.9 and 23.2, 4 tokens 23.4 and 23.2.  Where lora_a
// is too large for those, against k_lin_shrink and the tiles (rank 16, medians that
// repeat within 2 %): 4096 x 6144, 4 tokens 23.5 and 24.4, 8 tokens 25.7 and 25.4,
// 16 tokens 29.1 and 26.8, 64 tokens 39.3 and 31.5; 4096 x 4096, 16 tokens 22.6 and
// 24.8; 8192 x 8192, 2 tokens 38.1 and 38.3, 4 tokens 40.6 and 39.9, 8 tokens 46.3
// and 41.3; 2048 x 8192, 16 tokens 19.1 and 21.2.  Past 16 tokens: 1032 x 2056, 48
// tokens 13.2 and 14.4; 1032 x 8200, 17 tokens 15.2 and 16.6, 48 tokens 20.2 and
// 20.0; 2048 x 2048, 20 tokens 16.9 and 15.4.
bool lin_few(int32_t T, int32_t K, const int64_t *N, int32_t S, int32_t R, int32_t L) {
    if (lin_one(T, K, N, S, R)) return true;
    const int64_t n = columns(N, S), wide = wide_cols(n, S, R, L);
    if (T > kLinFewTokens || n > 32768) return false;
    if (wide) return T <= 2 && 2 * wide > n;
    return T * n * K <= (T > 16 ? 1 << 27 : 1 << 28);
}

// Direct batches whose rank vectors come out of the tiles as further columns: a
// launch less (256 tokens, rank 16, 4096 x 6144, us, on bf16 and on codes: 8 slots
// 37.2 and 37.1 against 46.4 and 46.2 of the slot-grouped kernels, 64 slots 41.0 and
// 41.2 against 45.7 and 46.3, 128 slots 47.4 and 48.6 against 52.4 and 52.7).
bool lin_wide(int32_t T, int32_t K, const int64_t *N, int32_t S, int32_t R, int32_t L) {
    return !lin_few(T, K, N, S, R, L) && wide_cols(columns(N, S), S, R, L) > 0;
}

// The same for dx: v = dy B of every slot as further columns, added by the join,
// which reads S R lora_a rows per token.  weights: dA or dB are wanted too, which
// need the segments and the vectors in parts either way.  Against the sorted form
// (us; MB (2^20) of lora_a and sums): dx alone, rank 16, 8 slots, 6144 x 4096: 16
// tokens 20.3 and 40.9, 512 (224 MB) 56.0 and 69.9, 640 (280 MB) 70.1 and 76.6, 896
// (392 MB) 83.6 and 94.6, 1024 (448 MB) 106 and 100; 8192 x 8192, 512 tokens (192
// MB) 110 and 104, 640 (240 MB) 122 and 140, 768 (288 MB) 141 and 140, 1024 (384 MB)
// 214 and 154; 4096 x 4096, 768 tokens (144 MB) 52.1 and 62.6, 1024 (192 MB) 73.8 and
// 65.6; 4096 x 14336, 512 tokens (336 MB) 95.7 and 91.0: no one number of bytes parts
// them, and past 256 MB what is lost grows larger than what is won.  With weights 96
// tokens 45.4 and 55.3, 256 55.9 and 62.0; rank 64, 96 tokens (150 MB) 67.7 and 72.5,
// 256 (400 MB) 81.8 and 78.0.  A contraction many times K keeps the further columns'
// few tiles long: 28672 x 4096, 96 tokens, with weights 119 and 108.  Through 4 bits: dx
// alone, 6144 x 4096, 512 tokens 57.1 and 67.2, 640 74.2 and 73.2, 896 85.1 and 103.9, 1024
// 107 and 104; 4096 x 4096, 768 tokens 54.8 and 69.4, 1024 73.4 and 69.6; with weights 96
// tokens of rank 16, 4 slots 47.9 and 49.8, 256 of 8 slots 56.9 and 59.1; rank 64, 96
// tokens 60.5 and 58.8, 256 78.1 and 66.3.
bool lin_wide_gradient(int32_t T, int32_t K, const int64_t *N, int32_t S, int32_t R, int32_t L, bool weights) {
    if (T > (weights ? 512 : kLinDirectTokens) || wide_cols(K, S, R, L) == 0) return false;
    if (weights && columns(N, S) > 4 * (int64_t)K) return false;
    return (int64_t)T * K * (2 * S * R + 16) <= (weights ? kLinWideBytesB : kLinWideBytesA);
}

// The 256 x 256 gradient tiles (of a call that is not wide: their plan is the one that
// launch_lin_gemm makes) read a restored projection; they have no form on codes.  Against
// 128 x 128 tiles on codes, us for dx (N x K; number of 256 x 256 tiles): 769 and 1024
// tokens, 4096 x 14336 (224) 146 and 158, 141 and 160; 1536 and 1792 tokens, 8192 x 8192
// (192, 224) 220 and 241, 226 and 288; 3200 and 4096 tokens, 6144 x 4096 (208, 256) 207
// and 249, 212 and 261, 28672 x 4096 765 and 941, 807 and 994; 8192 tokens of those 1642
// and 2069.  Just past 256 tiles, where some CUs take two of them, it is the other way:
// 1280 tokens, 4096 x 14336 (280) 234 and 203, 2560 tokens, 8192 x 8192 (320) 397 and
// 362, 5120 tokens, 6144 x 4096 (320) 364 and 330.
bool lin_restores(int32_t T, int32_t K, const int64_t *N, int32_t S, int32_t R, int32_t L, bool weights) {
    return T > 0 && !lin_wide_gradient(T, K, N, S, R, L, weights) &&
           lin_tile_plan(T, K, N, S, R, L, true, false, false, true).tile == 256;
}

// Direct batches whose rank vectors the slot-grouped kernels find (whole
// 64-column steps, in-kernel discovery).
bool lin_grouped(int32_t T, int32_t K, int32_t R, int32_t L) {
    return T > 8 && grp_discovers(T, L) && R % 16 == 0 && R <= kGrpMaxPartialRank && K % 64 == 0 &&
           grp_kchunks(K) <= kMaxKcGrp;
}

// Whether a forward batch takes the direct path: rank vectors without a segment
// build, and the delta in k_lin_few or k_lin_join_rows.  k_lin_join_rows reads
// lora_b rows once per token, and k_lin_shrink lora_a rows once per block of 16
// tokens, so their bytes bound it, with some 16 of sums per output.  Wide against
// sorted (us; MB of lora_b and sums; 8 slots), bf16 and in brackets 4-bit projections,
// K 4096, 6144 columns: 512 tokens of rank 16 (151 MB) 54.5 and 60.1 (55.7 and 64.2),
// 777 tokens (229 MB) 82.5 and 82.3 (82.6 and 82.5), 1024 (302 MB) 92.1 and 84.5 (93.1
// and 85.2); rank 64, 128 tokens (113 MB) 37.4 and 43.9 (41.1 and 47.6), 192 (170 MB)
// 54.6 and 55.0 (53.5 and 56.0), 256 (226 MB) 62.9 and 56.6 (61.4 and 57.5); 28672
// columns, 128 tokens of rank 16 (176 MB) 72.8 and 64.5, the only one the other way
// (59.1 and 64.7), 256 of rank 8 (235 MB) 113 and 83 (95 and 82); 14336 x 4096, 777 tokens
// of rank 16 (153 MB) 122 and 150 (123 and 150).
// With the slot-grouped kernels, 4096 x 6144, rank 48, 64 slots: 96 tokens (66 MB) 42.0
// and 45.0 (46.1 and 48.7), 128 (88 MB) 45.5 and 43.9 (50.2 and 48.3), 160 (110 MB) 55.9
// and 51.7 (54.9 and 52.1), 256 (176 MB) 65.8 and 54.7 (65.3 and 54.9): the bound is
// some 5 % late for them.  With k_lin_shrink, rank 40, 64 slots (MB of lora_a): 32 tokens
// (75 MB) 34.5 and 41.9 (34.4 and 41.8), 48 (113 MB) 30.7 and 42.5 (30.6 and 42.9), 96
// (226 MB) 43.8 and 45.1 (47.6 and 49.3).
bool lin_direct(int32_t T, int32_t K, const int64_t *N, int32_t S, int32_t R, int32_t L) {
    if (lin_few(T, K, N, S, R, L)) return true;
    const bool wide = lin_wide(T, K, N, S, R, L);
    if (T > kLinDirectTokens ||
        T * columns(N, S) * (2 * R + 16) > (wide ? kLinWideBytesB : kLinDirectBytesB)) return false;
    if (wide || lin_grouped(T, K, R, L)) return true;
    const int64_t slots = L < 16 ? L : 16, blocks = (T + 15) / 16, ranks = (int64_t)S * ((R + 15) / 16);
    return blocks * slots * ranks * K * 64 <= kLinDirectBytesA;
}

hipError_t launch_lin_shrink(const void *x, int64_t ldx, int32_t T, int32_t K, const Slices &sl,
                             int32_t S, int32_t L, int32_t R, const int32_t *idx,
                             const int32_t *slot_rank, float *buf, hipStream_t st) {
    LinShrinkArgs a{};
    a.x = static_cast<const uint16_t *>(x); a.ldx = ldx; a.T = T; a.K = K; a.S = S; a.L = L; a.R = R;
    for (int s = 0; s < S; ++s) a.a[s] = static_cast<const uint16_t *>(sl.a[s]);
    a.idx = idx; a.slot_rank = slot_rank; a.buf = buf;
    int y = L < 16 ? L : 16;
    if (y > T) y = T;
    const dim3 grid((unsigned)((T + 15) / 16), (unsigned)y, (unsigned)(S * ((R + 15) / 16)));
    hipLaunchKernelGGL(k_lin_shrink, grid, dim3(kShWaves * 64), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_lin_vectors(const LinVectors *jobs, int n_jobs, int32_t T, int32_t S, int32_t L, int32_t R,
                              const int32_t *idx, const int32_t *slot_rank, const float *scale,
                              const SegPtrs &seg, int32_t *order, hipStream_t st) {
    LinReduceArgs a{};
    for (int i = 0; i < n_jobs; ++i) a.job[i] = jobs[i];
    a.n_jobs = n_jobs; a.T = T; a.S = S; a.L = L; a.R = R;
    a.idx = idx; a.slot_rank = slot_rank; a.scale = scale; a.seg = seg; a.order = order;
    const int64_t items = (int64_t)T * (R / 4);              // R >= 8: at least T threads
    const dim3 grid((unsigned)((items + kRedThreads - 1) / kRedThreads), (unsigned)(S * n_jobs + (order ? 1 : 0)));
    hipLaunchKernelGGL(k_lin_vectors, grid, dim3(kRedThreads), 0, st, a);
    return hipGetLastError();
}

}  // namespace aa
