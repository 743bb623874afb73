"""The forms that the layer's calls take, by the library's own rules (host
functions of libadapter_apply.so, called by their C++ names), so that tests can
state which form a shape reaches without a GPU."""
import ctypes as C

import adapter_apply_amd as aa

WS_SUMS = 1 << 25        # fp32 sums that a workspace holds at most


class Plan(C.Structure):
    _fields_ = [("tile", C.c_int32), ("splits", C.c_int32)]


_i, _b, _n = C.c_int32, C.c_bool, C.POINTER(C.c_int64)
RULES = {
    "lin_one": ("_ZN2aa7lin_oneEiiPKlii", _b, [_i, _i, _n, _i, _i]),
    "lin_few": ("_ZN2aa7lin_fewEiiPKliii", _b, [_i, _i, _n, _i, _i, _i]),
    "lin_wide": ("_ZN2aa8lin_wideEiiPKliii", _b, [_i, _i, _n, _i, _i, _i]),
    "lin_direct": ("_ZN2aa10lin_directEiiPKliii", _b, [_i, _i, _n, _i, _i, _i]),
    "lin_grouped": ("_ZN2aa11lin_groupedEiiii", _b, [_i, _i, _i, _i]),
    "lin_join_delta": ("_ZN2aa14lin_join_deltaEiiPKliii", _b, [_i, _i, _n, _i, _i, _i]),
    "lin_wide_gradient": ("_ZN2aa17lin_wide_gradientEiiPKliiib", _b, [_i, _i, _n, _i, _i, _i, _b]),
    "lin_tile_plan": ("_ZN2aa13lin_tile_planEiiPKliiibbbb", Plan, [_i, _i, _n, _i, _i, _i, _b, _b, _b, _b]),
    "lin_wg_splits": ("_ZN2aa13lin_wg_splitsEiiPKlS1_ii", _i, [_i, _i, _n, _n, _i, _i]),
    "lin_du_splits": ("_ZN2aa13lin_du_splitsEiiPKlii", _i, [_i, _i, _n, _i, _i]),
}
_fn = {}


def rule(name, *args):
    if name not in _fn:
        symbol, res, types = RULES[name]
        f = getattr(aa.lib(), symbol)
        f.restype, f.argtypes = res, types
        _fn[name] = f
    return _fn[name](*args)


def _widths(N):
    return (C.c_int64 * len(N))(*N)


def _sums(T, cols, further, plan, join):
    """Elements of fp32 sums the tiles leave for a join (none: 0)."""
    return plan.splits * T * (cols + further) if join or plan.splits > 1 else 0


def forward(T, K, N, R, L):
    """(form, tile, split or not) of lora_linear, and its fp32 sums."""
    S, n = len(N), _widths(N)
    if rule("lin_one", T, K, n, S, R):
        return ("one", 16 if R <= 16 else 32, False), 0
    if rule("lin_few", T, K, n, S, R, L):
        return ("few", 16 if T <= 16 else 32 if T <= 32 else 64, False), 0
    wide, direct = rule("lin_wide", T, K, n, S, R, L), rule("lin_direct", T, K, n, S, R, L)
    wide = wide and direct
    join = direct or rule("lin_join_delta", T, K, n, S, R, L)
    p = rule("lin_tile_plan", T, K, n, S, R, L, False, join, wide, True)
    name = ("wide" if wide else ("grouped" if rule("lin_grouped", T, K, R, L) else "direct") if direct
            else "join" if join else "tiles")
    return (name, p.tile, p.splits > 1), _sums(T, sum(N), S * L * R if wide else 0, p, join)


def gradient(T, K, N, R, L, weights=True, base=True):
    """The same of lora_linear_backward's dx; base: with W."""
    S, n = len(N), _widths(N)
    wide = base and rule("lin_wide_gradient", T, K, n, S, R, L, weights)
    p = rule("lin_tile_plan", T, K, n, S, R, L, True, wide, wide, base)
    name = "wide" if wide else "tiles" if base else "in place"
    return (name, p.tile, p.splits > 1), _sums(T, K, S * L * R if wide else 0, p, wide)


def weight_splits(T, K, N, R, L):
    n = _widths(N)
    return rule("lin_wg_splits", T, L, _widths([K] * len(N)), n, len(N), R)
