"""Rules that the calls on a 4-bit projection rest on, without a GPU."""
from tests import layer_rules, mx_rules
from tests.test_layer_rules_cpu import drawn

EDGES = [(T, K, N, R, L) for T in (0, 1, 8, 257, 1024, 1536, 8192) for K in (8, 4096, 14336, 1 << 16)
         for N in ((4,), (14336, 14336), (1 << 20,)) for R in (8, 512) for L in (1, 1024)]


def test_the_tiles_that_read_bf16_rows_get_them():
    """256 x 256 gradient tiles have no form on codes: a projection is restored exactly
    where the gradient's plan is of them."""
    seen = set()
    for c in [*EDGES, *drawn(20000, 21)]:
        for w in (True, False):
            want = c[0] > 0 and layer_rules.gradient(*c, weights=w)[0][1] == 256
            assert mx_rules.restores(*c, weights=w) == want, (c, w)
            seen.add(want)
    assert seen == {True, False}
