// Host-side argument checks and slice packing shared by the entry points of the
// C ABI (abi.hip, abi_linear.hip).  Every check runs before anything is enqueued.
#pragma once

#include "../../include/adapter_apply.h"
#include "common.hpp"

namespace aa {
namespace {

inline bool al(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline lora_status_t launched(hipError_t e) { return e == hipSuccess ? LORA_OK : LORA_E_LAUNCH; }

lora_status_t check_sizes(int32_t T, int32_t S, int32_t L, int32_t R, int32_t dtype) {
    if (dtype != LORA_DT_F32 && dtype != LORA_DT_BF16) return LORA_E_DTYPE;
    if (T < 0 || L < 1 || L > LORA_MAX_SLOTS) return LORA_E_SHAPE;
    if (R < 1 || R > LORA_MAX_RANK) return LORA_E_RANK;
    if (S < 1 || S > LORA_MAX_SLICES) return LORA_E_SLICES;
    if (R % (dtype == LORA_DT_BF16 ? 8 : 4)) return LORA_E_ALIGN;
    // decode tiles index grid.y / grid.z
    if (max_tiles(T, L, kDecTile) > 65535) return LORA_E_SHAPE;
    return LORA_OK;
}

lora_status_t check_k(int32_t K, int64_t ldx) {
    if (K < 1 || ldx < K) return LORA_E_SHAPE;
    if (K % 8 || ldx % 8) return LORA_E_ALIGN;
    return LORA_OK;
}

lora_status_t check_n(const int64_t *N, int32_t S, int64_t ldy, int64_t y_col_offset,
                      int64_t *total) {
    if (!N) return LORA_E_NULL;
    int64_t t = 0;
    for (int s = 0; s < S; ++s) {
        if (N[s] < 1) return LORA_E_SHAPE;
        if (N[s] % 4) return LORA_E_ALIGN;
        t += N[s];
    }
    if (y_col_offset < 0 || ldy < y_col_offset + t) return LORA_E_SHAPE;
    if (ldy % 4 || y_col_offset % 4) return LORA_E_ALIGN;
    *total = t;
    return LORA_OK;
}

lora_status_t check_ptrs(const void *const *P, int32_t S) {
    if (!P) return LORA_E_NULL;
    for (int s = 0; s < S; ++s) {
        if (!P[s]) return LORA_E_NULL;
        if (!al(P[s], 16)) return LORA_E_ALIGN;
    }
    return LORA_OK;
}

#define CHECK(expr)                          \
    do {                                     \
        lora_status_t _st = (expr);          \
        if (_st != LORA_OK) return _st;      \
    } while (0)

lora_status_t check_ws(const void *ws, size_t ws_bytes, size_t need) {
    if (!ws) return LORA_E_NULL;
    if (!al(ws, 256)) return LORA_E_ALIGN;
    if (ws_bytes < need) return LORA_E_WORKSPACE;
    return LORA_OK;
}

Slices make_slices(const void *const *A, const void *const *B, const int64_t *N, int32_t S,
                   int64_t y_col_offset) {
    Slices sl{};
    int64_t off = y_col_offset;
    for (int s = 0; s < S; ++s) {
        sl.a[s] = A ? A[s] : nullptr;
        sl.b[s] = B ? B[s] : nullptr;
        sl.n[s] = N ? N[s] : 0;
        sl.off[s] = off;
        off += sl.n[s];
    }
    for (int s = S; s <= kMaxSlices; ++s) sl.off[s] = off;
    return sl;
}

}  // namespace
}  // namespace aa
