"""The forms that the layer's calls on a 4-bit projection take, by the library's own
rules (see tests/layer_rules.py)."""
from tests import layer_rules
from tests.layer_rules import _b, _i, _n, _widths, rule

layer_rules.RULES["lin_restores"] = ("_ZN2aa12lin_restoresEiiPKliiib", _b, [_i, _i, _n, _i, _i, _i, _b])


def restores(T, K, N, R, L, weights=True):
    return rule("lin_restores", T, K, _widths(N), len(N), R, L, weights)
