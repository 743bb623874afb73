"""Rules that the calls on a 4-bit projection rest on, without a GPU."""
import random

import pytest

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


def test_every_form_is_tested():
    """Each form that the rules choose for a drawn shape is one that the GPU tests reach
    (tests/test_gpu_mx.py, tests/test_gpu_mx_forms.py)."""
    from tests.test_gpu_mx import FEW_SHAPES, SHAPES
    from tests.test_gpu_mx_forms import FORMS
    tested = set()
    for s in SHAPES + FEW_SHAPES + FORMS:
        tested.add(("y", *mx_rules.forward(*s[:5])))
        if s in FEW_SHAPES:
            continue
        tested.add(("dx", *mx_rules.gradient(*s[:5])))
        if s in FORMS or s[0] < 1100:
            tested.add(("dx", *mx_rules.gradient(*s[:5], weights=False)))
    rng = random.Random(25)
    pick = lambda lo, hi: int(2 ** rng.uniform(lo, hi))
    few = [(rng.choice((1, 1, 2, 9, 16, 17, 32)), 8 * pick(0, 11), tuple(4 * pick(0, 13.9) for _ in range(rng.choice((1, 1, 2, 3)))),
            8 * rng.choice((1, 2, 3, 4, 8, 16)), pick(0, 6)) for _ in range(20000)]
    forms = mx_rules.drawn_forms([*drawn(40000, 22), *few])
    assert len(forms) > 30
    missing = {f: c for f, c in forms.items() if f not in tested}
    assert not missing, missing


@pytest.mark.parametrize("T,K,N,R,form", [
    (1, 4096, (4096, 1024, 1024), 16, "one"), (1, 4096, (14336,), 32, "one"), (1, 4096, (28672,), 16, "few"),
    (1, 4096, (4096,), 64, "few"), (16, 4096, (4096,), 128, "few"), (32, 4096, (28672,), 16, "few"),
    (32, 4096, (4096, 1024, 1024), 16, "wide")])
def test_few_tokens_take_the_form_that_measured_faster(T, K, N, R, form):
    assert mx_rules.forward(T, K, N, R, 8)[0] == form


def test_sums_stay_within_the_workspace():
    """The fp32 sums of a forward call: what its workspace holds for them (those of a few
    tokens have 16 splits of the columns and ranks of up to 32)."""
    edges = [(T, K, N, R, L) for T in (1, 16, 17, 32, 33, 64, 1024, 8192) for K in (8, 1536, 16384)
             for N in ((4,), (32768,), (65536,), (65540,), (4096,) * 8) for R in (8, 128, 512) for L in (1, 64, 1024)]
    for c in [*edges, *drawn(20000, 24)]:
        T, K, N, R, L = c
        tiles = min(layer_rules.WS_SUMS, 8 * T * 2 * max(K, sum(N)))
        few = 16 * min(T, 32) * (sum(N) + len(N) * R) if sum(N) <= 65536 else 0
        assert mx_rules.sums(*c) <= max(tiles, few), c
        assert mx_rules.forward(*c)[0] in ("one", "few") or mx_rules.sums(*c) <= tiles, c
