// C-ABI entry points of the adapter layer beside a frozen projection and its
// gradient, and of the per-adapter gradient norm and clip: argument checks (all
// before any launch), workspace carving and launches.  Declarations and
// contracts: include/adapter_apply.h.
#include <string.h>

#include "checks.hpp"
#include "linear.hpp"

using namespace aa;

namespace {

inline int64_t round8(int64_t v) { return (v + 7) / 8 * 8; }

// Workspace of lora_linear and lora_linear_backward.  Behind the call's own
// regions stands room for the largest exchange region that a one-launch segment
// build of any T and L takes below the last line: those bytes need to be zero and
// are left zero, and no layer that shares the workspace writes there, whatever
// its sizes (the region ends where the buffer does, so it is not at one place of
// the layout).
struct LinWs {
    SegLayout seg;
    size_t order;       // int32 [2][T]: row order of the tile GEMM and the rows' slots
    size_t hl_u;        // bf16 [S][T][kLinPartsBwd R]: scale * u in parts
    size_t hl_v;        // the same of v
    size_t v;           // fp32 [S][T][R]: v by token (wide gradients)
    size_t part;        // fp32 partial sums
    size_t pad;         // bf16 [T][pad_cols]: dy with slices of whole 8-element units
    size_t data;        // end of the call's own regions
    size_t end;
    bool padded;        // some N_s % 8: dy goes through pad
    int64_t pad_cols;
};

LinWs lin_ws(int32_t T, int32_t K, const int64_t *N, int32_t S, int32_t R, int32_t L) {
    LinWs w{};
    w.seg = seg_layout(T, L);
    size_t o = w.seg.end;
    const size_t tsr = (size_t)T * S * R;
    w.order = o; o = align256(o + 2 * sizeof(int32_t) * (size_t)T);
    w.hl_u = o;  o = align256(o + 2 * kLinPartsBwd * tsr);
    w.hl_v = o;  o = align256(o + 2 * kLinPartsBwd * tsr);
    w.v = o;     o = align256(o + 4 * tsr);
    w.part = o;
    // the shrink's K splits: either one, or within an eighth of its input
    // bytes (pre_kspl: 8 k T S R <= in_bytes / 8)
    size_t part = 4 * tsr;
    const size_t split = (size_t)K * ((size_t)T + (size_t)(T < L ? T : L) * S * R) / 8;
    if (split > part) part = split;
    // the grouped shrink's chunks of 512 columns (direct batches)
    size_t kc = ((size_t)K + 511) / 512;
    if (kc > (size_t)kMaxKcGrp) kc = (size_t)kMaxKcGrp;
    const size_t gt = T < kLinDirectTokens ? T : kLinDirectTokens;
    if (4 * gt * S * R * kc > part) part = 4 * gt * S * R * kc;
    // the gradient's column splits: k tiles S <= 1024 with at least T / 64
    // tiles, and at most 16, so k T <= min(16 T, T + 65536)
    size_t kt = (size_t)T + 65536;
    if (kt > 16 * (size_t)T) kt = 16 * (size_t)T;
    if (4 * (size_t)S * R * kt > part) part = 4 * (size_t)S * R * kt;
    // the token splits of both weight gradients (none up to 511 tokens)
    if (T > 256) {
        size_t wg = (size_t)131072 * R;
        if (wg > (size_t)kLinWgPartMax) wg = (size_t)kLinWgPartMax;
        if (2 * 4 * wg > part) part = 2 * 4 * wg;
    }
    // the tile GEMM's sums: at most kLinMaxSplits of them, at most kLinJoinMax
    size_t cols = 0;
    for (int s = 0; s < S; ++s) cols += (size_t)N[s];
    if (cols < (size_t)K) cols = (size_t)K;
    size_t sums = kLinMaxSplits * (size_t)T * 2 * cols;     // (wide batches: up to as many columns more)
    if (sums > (size_t)kLinJoinMax) sums = (size_t)kLinJoinMax;
    if (4 * sums > part) part = 4 * sums;
    o = align256(o + part);
    w.pad = o;
    for (int s = 0; s < S; ++s) {
        w.padded = w.padded || N[s] % 8;
        w.pad_cols += round8(N[s]);
    }
    if (w.padded) o = align256(o + sizeof(uint16_t) * (size_t)T * w.pad_cols);
    w.data = o;
    w.end = o + seg_x_bytes(kSegOneMaxWg * kSegThreads, kMaxSlots) + 256;
    return w;
}

lora_status_t check_layer(int32_t T, int32_t K, int64_t ldx, const int64_t *N, int32_t S, int32_t L,
                          int32_t R, int64_t ldy, int32_t dtype) {
    CHECK(check_sizes(T, S, L, R, dtype));
    if (dtype != LORA_DT_BF16) return LORA_E_DTYPE;
    CHECK(check_k(K, ldx));
    int64_t total = 0;
    CHECK(check_n(N, S, ldy, 0, &total));
    if (!lin_grid_fits(T, K, N, S)) return LORA_E_SHAPE;
    return LORA_OK;
}

SegPtrs lin_seg(void *ws, size_t ws_bytes, const LinWs &w, int32_t T, int32_t L) {
    SegPtrs seg = seg_ptrs(ws, w.seg);
    attach_seg_x(seg, ws, ws_bytes, T, L, 0, w.data);
    return seg;
}

// x A^T by slot-sorted position in the workspace's partial sums; returns the
// number of K splits.
lora_status_t sorted_shrink(const void *x, int64_t ldx, int32_t T, int32_t K, const Slices &sl, int32_t S,
                            int32_t L, int32_t R, const int32_t *slot_rank, const SegPtrs &seg, float *part,
                            int32_t *nsp, hipStream_t st) {
    *nsp = pre_kspl(T, K, S, R, L, seg.max_tiles_pre, kMaxKcGrp);
    return launched(launch_pre_shrink(x, ldx, T, K, sl, S, L, R, slot_rank, seg, nullptr, st, GroupMap(), part, nsp));
}

}  // namespace

extern "C" {

lora_status_t lora_linear_workspace_size(int32_t T, int32_t K, const int64_t *N, int32_t S, int32_t R,
                                         int32_t L, size_t *bytes) {
    if (!bytes || !N) return LORA_E_NULL;
    int64_t total = 0;
    CHECK(check_sizes(T, S, L, R, LORA_DT_BF16));
    if (K < 1) return LORA_E_SHAPE;
    CHECK(check_n(N, S, INT64_MAX / 8 * 4, 0, &total));
    if (!lin_grid_fits(T, K, N, S)) return LORA_E_SHAPE;
    *bytes = lin_ws(T, K, N, S, R, L).end;
    return LORA_OK;
}

lora_status_t lora_linear(void *y, int64_t ldy, const void *x, int64_t ldx, int32_t T, int32_t K,
                          const void *W, int64_t ldw, const void *bias, const void *const *A,
                          const void *const *B, const int64_t *N, int32_t S, int32_t L, int32_t R,
                          const int32_t *idx, const int32_t *slot_rank, const float *scale, float *buf,
                          int32_t dtype, uint32_t flags, void *ws, size_t ws_bytes, void *stream) {
    CHECK(check_layer(T, K, ldx, N, S, L, R, ldy, dtype));
    CHECK(check_k(K, ldw));
    if (T == 0) return LORA_OK;
    if (!y || !x || !W || !idx || !scale) return LORA_E_NULL;
    CHECK(check_ptrs(A, S));
    CHECK(check_ptrs(B, S));
    if (!al(y, 16) || !al(x, 16) || !al(W, 16) || !al(buf, 16) || !al(bias, 2)) return LORA_E_ALIGN;
    const LinWs wl = lin_ws(T, K, N, S, R, L);
    CHECK(check_ws(ws, ws_bytes, wl.end));

    hipStream_t st = static_cast<hipStream_t>(stream);
    char *wp = static_cast<char *>(ws);
    const Slices sl = make_slices(A, B, N, S, 0);
    uint16_t *hl = reinterpret_cast<uint16_t *>(wp + wl.hl_u);
    int32_t *order = nullptr;
    const bool direct = lin_direct(T, K, N, S, R, L);
    const bool join = direct || lin_join_delta(T, K, N, S, R, L);
    const bool wide = direct && lin_wide(T, K, N, S, R, L);
    float *u = buf, *u_out = nullptr;
    // fp32 rank vectors by token, in buf if it is wanted
    if (join && !u) u = reinterpret_cast<float *>(wp + wl.hl_u);
    if (lin_one(T, K, N, S, R) || wide) {
        u_out = buf;
    } else if (direct) {
        if (!lin_few(T, K, N, S, R, L) && lin_grouped(T, K, R, L)) {
            float *part = reinterpret_cast<float *>(wp + wl.part);
            CHECK(launched(launch_grp_shrink(x, ldx, T, K, sl, S, L, R, idx, slot_rank, part, nullptr, nullptr, st)));
            CHECK(launched(launch_grp_reduce(T, S, L, R, idx, slot_rank, part, grp_kchunks(K), u, nullptr, st)));
            u_out = buf;
        } else {
            CHECK(launched(launch_lin_shrink(x, ldx, T, K, sl, S, L, R, idx, slot_rank, u, st)));
        }
    } else {
        const SegPtrs seg = lin_seg(ws, ws_bytes, wl, T, L);
        float *part = reinterpret_cast<float *>(wp + wl.part);
        order = reinterpret_cast<int32_t *>(wp + wl.order);
        int32_t nsp = 1;
        if (!(flags & LORA_FLAG_SEGMENTS_READY))
            CHECK(launched(launch_segments(idx, slot_rank, T, L, R, seg, st)));
        CHECK(sorted_shrink(x, ldx, T, K, sl, S, L, R, slot_rank, seg, part, &nsp, st));
        const LinVectors v{part, nsp, nullptr, join ? nullptr : hl, kLinPartsFwd, join ? u : buf};
        CHECK(launched(launch_lin_vectors(&v, 1, T, S, L, R, idx, slot_rank, scale, seg, order, st)));
    }
    LinArgs a{};
    a.p = static_cast<const uint16_t *>(x); a.ldp = ldx;
    a.w = static_cast<const uint16_t *>(W); a.ldw = ldw;
    a.bias = static_cast<const uint16_t *>(bias);
    a.out = static_cast<uint16_t *>(y); a.ldo = ldy;
    a.part = reinterpret_cast<float *>(wp + wl.part);
    a.join_delta = join;
    a.wide = wide; a.u = u; a.scale = scale; a.buf = u_out;
    a.hl = hl; a.hl_row = kLinPartsFwd * R; a.order = order; a.idx = idx; a.slot_rank = slot_rank;
    a.T = T; a.K = K; a.S = S; a.L = L; a.R = R;
    for (int s = 0; s < S; ++s) {
        a.lora[s] = static_cast<const uint16_t *>(B[s]);
        a.other[s] = static_cast<const uint16_t *>(A[s]);
        a.n[s] = N[s];
        a.off[s] = sl.off[s];
    }
    return launched(launch_lin_gemm(a, false, st));
}

lora_status_t lora_linear_backward(void *dx, int64_t lddx, float *const *dA, float *const *dB,
                                   const void *dy, int64_t lddy, const void *x, int64_t ldx, int32_t T,
                                   int32_t K, const void *W, int64_t ldw, const void *const *A,
                                   const void *const *B, const int64_t *N, int32_t S, int32_t L, int32_t R,
                                   const int32_t *idx, const int32_t *slot_rank, const float *scale,
                                   const float *buf, int32_t dtype, uint32_t flags, void *ws,
                                   size_t ws_bytes, void *stream) {
    CHECK(check_layer(T, K, x ? ldx : K, N, S, L, R, lddy, dtype));
    if (dx) CHECK(check_k(K, lddx));
    if (dx && W) CHECK(check_k(K, ldw));
    if (!dx && !dA && !dB) return LORA_E_NULL;
    for (int s = 0; s < S; ++s) {
        if ((dA && !dA[s]) || (dB && !dB[s])) return LORA_E_NULL;
        if ((dA && !al(dA[s], 16)) || (dB && !al(dB[s], 16))) return LORA_E_ALIGN;
    }
    const LinWs wl = lin_ws(T, K, N, S, R, L);
    if (!wl.padded && lddy % 8) return LORA_E_ALIGN;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (T == 0) {
        if (flags & LORA_FLAG_ACCUMULATE) return LORA_OK;
        for (int s = 0; s < S; ++s) {
            if (dA) CHECK(launched(launch_fill_zero(dA[s], sizeof(float) * (size_t)L * R * K, st)));
            if (dB) CHECK(launched(launch_fill_zero(dB[s], sizeof(float) * (size_t)L * R * N[s], st)));
        }
        return LORA_OK;
    }
    if (!dy || !idx || !scale) return LORA_E_NULL;
    if (!x && (dA || (dB && !buf))) return LORA_E_NULL;
    CHECK(check_ptrs(A, S));
    CHECK(check_ptrs(B, S));
    if (!al(dx, 16) || !al(dy, 16) || !al(x, 16) || !al(W, 16) || !al(buf, 16)) return LORA_E_ALIGN;
    CHECK(check_ws(ws, ws_bytes, wl.end));
    const void *outs[2 * kMaxSlices + 1];
    int n_out = 0;
    if (dx) outs[n_out++] = dx;
    for (int s = 0; s < S; ++s) {
        if (dA) outs[n_out++] = dA[s];
        if (dB) outs[n_out++] = dB[s];
    }
    for (int i = 1; i < n_out; ++i)
        for (int j = 0; j < i; ++j)
            if (outs[i] == outs[j]) return LORA_E_SHAPE;

    char *wp = static_cast<char *>(ws);
    const Slices sl = make_slices(A, B, N, S, 0);
    const SegPtrs seg = lin_seg(ws, ws_bytes, wl, T, L);
    uint16_t *hl_u = reinterpret_cast<uint16_t *>(wp + wl.hl_u);
    uint16_t *hl_v = reinterpret_cast<uint16_t *>(wp + wl.hl_v);
    float *part = reinterpret_cast<float *>(wp + wl.part);
    int32_t *order = reinterpret_cast<int32_t *>(wp + wl.order);
    const bool wide = dx && W && lin_wide_gradient(T, K, N, S, R, L, dA || dB);
    if (!(flags & LORA_FLAG_SEGMENTS_READY) && (dA || dB || !wide))
        CHECK(launched(launch_segments(idx, slot_rank, T, L, R, seg, st)));

    // dy with whole 8-element units per slice
    const uint16_t *p = static_cast<const uint16_t *>(dy);
    int64_t ldp = lddy, poff[kMaxSlices];
    for (int s = 0; s < S; ++s) poff[s] = sl.off[s];
    if (wl.padded) {
        PadMap m{};
        int64_t c = 0;
        for (int s = 0; s < S; ++s) {
            m.src[s] = sl.off[s];
            m.dst[s] = poff[s] = c;
            m.n[s] = N[s];
            c += round8(N[s]);
        }
        uint16_t *pad = reinterpret_cast<uint16_t *>(wp + wl.pad);
        ldp = wl.pad_cols;
        CHECK(launched(launch_lin_pad(dy, lddy, T, S, m, pad, ldp, st)));
        p = pad;
    }
    // rank vectors in parts: scale * u for dB, v for dx and dA
    LinVectors job[2];
    int n_jobs = 0;
    if (dB) {
        LinVectors v{nullptr, 0, buf, hl_u, kLinPartsBwd, nullptr};
        if (!buf) {
            v.part = part;
            CHECK(sorted_shrink(x, ldx, T, K, sl, S, L, R, slot_rank, seg, part, &v.nsp, st));
            // (before the partial sums of v take their place)
            CHECK(launched(launch_lin_vectors(&v, 1, T, S, L, R, idx, slot_rank, scale, seg, nullptr, st)));
        } else {
            job[n_jobs++] = v;
        }
    }
    LinArgs a{};
    a.p = p; a.ldp = ldp;
    a.w = static_cast<const uint16_t *>(W); a.ldw = ldw;
    a.out = static_cast<uint16_t *>(dx); a.ldo = lddx;
    a.part = part;
    a.idx = idx; a.slot_rank = slot_rank; a.scale = scale;
    a.T = T; a.K = K; a.S = S; a.L = L; a.R = R;
    for (int s = 0; s < S; ++s) {
        a.lora[s] = static_cast<const uint16_t *>(A[s]);
        a.other[s] = static_cast<const uint16_t *>(B[s]);
        a.n[s] = N[s];
        a.off[s] = sl.off[s];
        a.poff[s] = poff[s];
    }
    if (wide) {
        float *v = reinterpret_cast<float *>(wp + wl.v);
        a.wide = a.join_delta = 1;
        a.buf = dA ? v : nullptr;
        CHECK(launched(launch_lin_gemm(a, true, st)));
        if (dA) job[n_jobs++] = LinVectors{nullptr, 0, v, hl_v, kLinPartsBwd, nullptr};
    } else if (dx || dA) {
        const int32_t nsp = lin_du_splits(T, L, N, S, R);
        CHECK(launched(launch_lin_du(p, ldp, poff, T, sl, S, L, R, seg, part, nsp, st)));
        job[n_jobs++] = LinVectors{part, nsp, nullptr, hl_v, kLinPartsBwd, nullptr};
    }
    if (n_jobs)
        CHECK(launched(launch_lin_vectors(job, n_jobs, T, S, L, R, idx, slot_rank, scale, seg,
                                          dx && !wide ? order : nullptr, st)));
    if (dA || dB) {
        LinWgArgs wa{}, wb{};
        wa.T = T; wa.S = S; wa.L = L; wa.R = R; wa.slot_rank = slot_rank; wa.seg = seg;
        wa.accumulate = (flags & LORA_FLAG_ACCUMULATE) != 0;
        wb = wa;
        wa.p = static_cast<const uint16_t *>(x); wa.ldp = ldx; wa.hl = hl_v;
        wb.p = p; wb.ldp = ldp; wb.hl = hl_u;
        for (int s = 0; s < S; ++s) {
            wa.out[s] = dA ? dA[s] : nullptr;
            wa.m[s] = K;
            wb.out[s] = dB ? dB[s] : nullptr;
            wb.m[s] = N[s];
            wb.poff[s] = poff[s];
        }
        wa.nsp = wb.nsp = lin_wg_splits(T, L, dA ? wa.m : nullptr, dB ? N : nullptr, S, R);
        wa.part = part;
        wb.part = part + (dA && wa.nsp > 1 ? wa.nsp * lin_wg_part(L, wa.m, S, R) : 0);
        CHECK(launched(launch_lin_wg(dA ? &wa : nullptr, dB ? &wb : nullptr, st)));
    }
    if (dx && !wide) {
        a.hl = hl_v; a.hl_row = kLinPartsBwd * R; a.order = order;
        a.accumulate = W == nullptr;
        CHECK(launched(launch_lin_gemm(a, true, st)));
    }
    return LORA_OK;
}

static lora_status_t check_grads(const void *const *g, const int64_t *m, int32_t n, int32_t L, int32_t dtype) {
    if (dtype != LORA_DT_F32 && dtype != LORA_DT_BF16) return LORA_E_DTYPE;
    if (n < 0 || L < 1 || L > LORA_MAX_SLOTS) return LORA_E_SHAPE;
    if (n > 0 && (!g || !m)) return LORA_E_NULL;
    if (grad_items(m, n, L) < 0) return LORA_E_SHAPE;
    for (int32_t i = 0; i < n; ++i) {
        if (m[i] == 0) continue;
        if (!g[i]) return LORA_E_NULL;
        if (!al(g[i], dtype == LORA_DT_BF16 ? 2 : 4)) return LORA_E_ALIGN;
    }
    return LORA_OK;
}

// Every output at an address of its own, and at a gradient's only if it is that
// tensor's: else work-groups of two tensors would scale the same elements.  The
// outputs go through a hash table on the stack, kOutBlock at a time, each block
// against every later output and every gradient (no memory is allocated).
constexpr int32_t kOutBlock = 2048;
static lora_status_t check_outputs(const void *const *out, const void *const *g, const int64_t *m, int32_t n) {
    int32_t table[2 * kOutBlock];                 // 1 + the index of an output, or 0
    for (int32_t b = 0; b < n;) {
        const int32_t e = n - b < kOutBlock ? n : b + kOutBlock;
        size_t size = 16;
        while (size < 2 * (size_t)(e - b)) size *= 2;
        memset(table, 0, size * sizeof(table[0]));
        // the entry of address p, or the empty one where it belongs
        auto find = [&](const void *p) -> int32_t & {
            size_t h = (size_t)((reinterpret_cast<uintptr_t>(p) >> 1) * 0x9E3779B97F4A7C15ull >> 20) & (size - 1);
            while (table[h] && out[table[h] - 1] != p) h = (h + 1) & (size - 1);
            return table[h];
        };
        for (int32_t i = b; i < n; ++i) {
            if (m[i] == 0) continue;
            int32_t &at = find(out[i]);
            if (at) return LORA_E_SHAPE;
            if (i < e) at = i + 1;
        }
        for (int32_t i = 0; i < n; ++i) {
            if (m[i] == 0) continue;
            const int32_t at = find(g[i]);
            if (at && at != i + 1) return LORA_E_SHAPE;
        }
        b = e;
    }
    return LORA_OK;
}

lora_status_t lora_grad_workspace_size(const int64_t *m, int32_t n, int32_t L, size_t *bytes) {
    if (!bytes || (n > 0 && !m)) return LORA_E_NULL;
    if (n < 0 || L < 1 || L > LORA_MAX_SLOTS) return LORA_E_SHAPE;
    const int64_t items = grad_items(m, n, L);
    if (items < 0) return LORA_E_SHAPE;
    *bytes = kGradCountBytes + align256(sizeof(double) * (size_t)items);
    return LORA_OK;
}

lora_status_t lora_grad_norm(float *norm, const void *const *g, const int64_t *m, int32_t n, int32_t L,
                             int32_t dtype, void *ws, size_t ws_bytes, void *stream) {
    CHECK(check_grads(g, m, n, L, dtype));
    if (!norm) return LORA_E_NULL;
    if (!al(norm, 4)) return LORA_E_ALIGN;
    size_t need = 0;
    CHECK(lora_grad_workspace_size(m, n, L, &need));
    CHECK(check_ws(ws, ws_bytes, need));
    double *part = reinterpret_cast<double *>(static_cast<char *>(ws) + kGradCountBytes);
    return launched(launch_grad_norm(g, m, n, L, dtype, static_cast<int32_t *>(ws), part, norm,
                                     static_cast<hipStream_t>(stream)));
}

lora_status_t lora_grad_clip(void *const *out, const void *const *g, const int64_t *m, int32_t n, int32_t L,
                             const float *norm, const float *max_norm, int32_t dtype, void *stream) {
    CHECK(check_grads(g, m, n, L, dtype));
    CHECK(check_grads(const_cast<const void *const *>(out), m, n, L, dtype));
    if (!norm || !max_norm) return LORA_E_NULL;
    if (!al(norm, 4) || !al(max_norm, 4)) return LORA_E_ALIGN;
    CHECK(check_outputs(const_cast<const void *const *>(out), g, m, n));
    return launched(launch_grad_clip(out, g, m, n, L, norm, max_norm, dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
