"""The forms that the layer's calls on a 4-bit projection take, by the library's own
rules (see tests/layer_rules.py)."""
from tests import layer_rules
from tests.layer_rules import _b, _i, _n, _widths, rule

layer_rules.RULES.update({
    "lin_restores": ("_ZN2aa12lin_restoresEiiPKliiib", _b, [_i, _i, _n, _i, _i, _i, _b]),
    "mx_few": ("_ZN2aa6mx_fewEiPKliii", _b, [_i, _n, _i, _i, _i]),
    "mx_one": ("_ZN2aa6mx_oneEiPKlii", _b, [_i, _n, _i, _i]),
    "mx_few_splits": ("_ZN2aa13mx_few_splitsEiPKli", _i, [_i, _n, _i]),
})


def restores(T, K, N, R, L, weights=True):
    return rule("lin_restores", T, K, _widths(N), len(N), R, L, weights)


def forward(T, K, N, R, L):
    """The form of lora_linear_mx: of one token, its blocks of ranks and rounds of loads; of
    a few, blocks of tokens, K steps in flight together, whether a split takes several such
    rounds, and whether the join adds more than 8 splits; else as layer_rules.forward."""
    S, n = len(N), _widths(N)
    if rule("mx_few", T, n, S, R, L):
        splits, steps = rule("mx_few_splits", K, n, S), (K + 127) // 128
        per = (steps + splits - 1) // splits
        if rule("mx_one", T, n, S, R):
            u = 2 if R > 16 or per <= 4 else 4
            return "one", 1 if R <= 16 else 2, u, per > 2 * u, splits > 1
        blocks = 1 if T <= 16 else 2
        chunk = 8 if 4 < per <= 8 and blocks == 1 else 4
        return "few", blocks, chunk, per > chunk, splits > 8
    wide, direct = rule("lin_wide", T, K, n, S, R, L), rule("lin_direct", T, K, n, S, R, L)
    wide = wide and direct
    join = direct or rule("lin_join_delta", T, K, n, S, R, L)
    p = rule("lin_tile_plan", T, K, n, S, R, L, False, join, wide, True)
    name = ("wide" if wide else ("grouped" if rule("lin_grouped", T, K, R, L) else "direct") if direct
            else "join" if join else "tiles")
    return name, p.tile, p.splits > 1


def sums(T, K, N, R, L):
    """fp32 sums that lora_linear_mx leaves for a join."""
    S, n = len(N), _widths(N)
    if rule("mx_few", T, n, S, R, L):
        return rule("mx_few_splits", K, n, S) * T * (sum(N) + S * R)
    name = forward(T, K, N, R, L)[0]
    p = rule("lin_tile_plan", T, K, n, S, R, L, False, name != "tiles", name == "wide", True)
    return layer_rules._sums(T, sum(N), S * L * R if name == "wide" else 0, p, name != "tiles")


def gradient(T, K, N, R, L, weights=True):
    """The form of dx through 4 bits."""
    form = layer_rules.gradient(T, K, N, R, L, weights=weights)[0]
    return ("restored", *form[1:]) if restores(T, K, N, R, L, weights) else form


def drawn_forms(shapes):
    """Form -> a shape that takes it."""
    forms = {}
    for c in shapes:
        forms.setdefault(("y", *forward(*c)), c)
        for w in (True, False):
            forms.setdefault(("dx", *gradient(*c, weights=w)), c)
    return forms
