"""Sizes and rules of the layer entry points that their calls rest on, without a
GPU: the workspace of layers that share one, the forms and their sums."""
import random

import pytest

import adapter_apply_amd as aa
from tests import layer_rules


def seg_exchange_bytes(T, L):
    """The region of the one-launch segment build, zero between calls: int32
    counts of each of its work-groups (1024 tokens, at most 16) over L + 1 keys,
    and a 256-byte line; it ends where the workspace's last line begins."""
    groups = min(max((T + 1023) // 1024, 1), 16)
    return (4 * groups * (L + 1) + 255) // 256 * 256 + 256


def size(T, K, N, R, L):
    return aa.lora_linear_workspace_size(T, K, N, R, L)


def data_end(T, K, N, R, L):
    """Where a call's own regions end: room for the largest exchange region and
    the last line are the end of its size."""
    return size(T, K, N, R, L) - 256 - seg_exchange_bytes(1 << 20, 1024)


def shares(a, b):
    """a and b on a workspace as large as the larger one's size (and larger)."""
    for ws in (max(size(*a), size(*b)), max(size(*a), size(*b)) + 4096):
        for p, q in ((a, b), (b, a)):
            assert data_end(*p) <= ws - 256 - seg_exchange_bytes(q[0], q[4]), (p, q)


@pytest.mark.parametrize("a,b", [
    ((8192, 1024, (4096,), 16, 64), (4096, 1024, (4092,), 16, 64)),
    ((7168, 64, (1024,), 8, 64), (4096, 64, (1020,), 8, 64)),
    ((8192, 4096, (4096,), 16, 64), (7000, 4096, (4092,), 16, 64)),
    ((6000, 64, (1024,), 8, 8), (6000, 64, (1020,), 8, 900)),
    ((300, 64, (64, 36), 8, 8), (300, 64, (68,), 8, 8)),
    ((16, 16384, (14336,), 128, 8), (16384, 8, (8,), 8, 1024)),
], ids=str)
def test_layers_share_the_larger_workspace(a, b):
    """A layer whose dy is copied (widths off 8) next to one whose is not, or with
    more tokens or slots."""
    shares(a, b)


def test_every_size_holds_the_largest_exchange_region():
    """Also that of a call whose own regions take next to nothing, and no more
    than that: one slot more costs no exchange counts."""
    small = size(1, 8, (4,), 8, 1)
    assert 0 < data_end(1, 8, (4,), 8, 1) < 16384, small
    for T in (1, 5000):
        grows = size(T, 8, (4,), 8, 1024) - size(T, 8, (4,), 8, 1023)
        assert 0 <= grows <= 256 + 4 * ((T + 1023) // 1024) + 2 * 256 + 2 * 16, grows


def test_segments_of_a_layer_fit_its_workspace():
    """What lora_build_segments writes lies before the layer's other regions."""
    for T, L in ((1, 1), (700, 1024), (8192, 64), (70000, 1024)):
        lay = aa.lora_segment_layout(T, L)
        assert max(v for k, v in lay.items() if not k.startswith("tile_")) < data_end(T, 8, (4,), 8, L)


def test_any_two_layers_share_the_larger_workspace():
    rng = random.Random(7)

    def layer():
        pick = lambda hi: max(1, int(2 ** rng.uniform(0, hi)))
        return (pick(15), 8 * pick(10), tuple(4 * pick(11) for _ in range(rng.randint(1, 8))),
                8 * rng.randint(1, 64), pick(10))

    for _ in range(4000):
        shares(layer(), layer())


def drawn(n, seed):
    rng = random.Random(seed)
    pick = lambda lo, hi: int(2 ** rng.uniform(lo, hi))
    for _ in range(n):
        yield (max(1, pick(0, 13.5)), 8 * pick(0, 10.8),
               tuple(4 * pick(0, 12.8) for _ in range(rng.choice((1, 1, 2, 3, 8)))),
               8 * rng.choice((1, 2, 2, 3, 4, 5, 8, 16, 64)), pick(0, 10))


def test_sums_stay_within_the_workspace():
    """The fp32 sums that any call leaves for a join: within what a workspace
    holds, also at the most rows and columns that a rule takes."""
    edges = [(T, K, N, R, L) for T in (1, 64, 1024, 1025, 8192) for K in (8, 1536, 4096, 16384)
             for N in ((4,), (4096,), (14336, 14336), (32768,), (4096,) * 8) for R in (8, 128, 512) for L in (1, 64, 1024)]
    for c in [*edges, *drawn(20000, 11)]:
        T, K, N, R, L = c
        for _, sums in (layer_rules.forward(*c), *(layer_rules.gradient(*c, weights=w, base=b)
                                                   for w in (True, False) for b in (True, False))):
            assert sums <= min(layer_rules.WS_SUMS, 8 * T * 2 * max(K, sum(N))), c


def test_every_form_is_tested():
    """Each form that the rules choose for a drawn shape is one that the GPU tests
    reach (tests/test_gpu_layer.py, tests/test_gpu_layer_forms.py)."""
    from tests.test_gpu_layer import SHAPES
    from tests.test_gpu_layer_forms import FORMS
    tested = set()
    for s in FORMS + SHAPES:
        T, K, N, R, L = s[:5]
        tested |= {("y", *layer_rules.forward(T, K, N, R, L)[0]), ("dx", *layer_rules.gradient(T, K, N, R, L)[0])}
        if T < 1100:
            tested.add(("dx", *layer_rules.gradient(T, K, N, R, L, weights=False)[0]))
        if s in SHAPES and T in (17, 200, 1000, 2100):
            tested.add(("dx", *layer_rules.gradient(T, K, N, R, L, base=False)[0]))
    missing = {}
    for c in drawn(40000, 12):
        for f in (("y", *layer_rules.forward(*c)[0]), ("dx", *layer_rules.gradient(*c)[0]),
                  ("dx", *layer_rules.gradient(*c, weights=False)[0]), ("dx", *layer_rules.gradient(*c, base=False)[0])):
            if f not in tested:
                missing[f] = c
    assert not missing, missing


@pytest.mark.parametrize("K,N,R,one", [
    (2048, (2048,), 16, True), (4096, (4096,), 16, False), (4096, (4096, 1024, 1024), 16, True),
    (4096, (8192,), 16, True), (4096, (8448,), 16, False), (4096, (14336,), 16, False),
    (2048, (16384,), 16, True), (2048, (12288,), 32, False), (3200, (8192,), 16, True), (3200, (8448,), 16, False)])
def test_one_token_takes_the_form_that_measured_faster(K, N, R, one):
    assert (layer_rules.forward(1, K, N, R, 8)[0][0] == "one") == one


@pytest.mark.parametrize("T,K,N,few", [
    (4, 4096, (4096, 1024, 1024), True), (16, 4096, (4096, 1024, 1024), False), (16, 4096, (4096,), True),
    (2, 8192, (8192,), True), (8, 8192, (8192,), False), (16, 2048, (8192,), True),
    (48, 1032, (2056,), True), (64, 4096, (4096, 1024, 1024), False)])
def test_few_tokens_take_the_form_that_measured_faster(T, K, N, few):
    assert (layer_rules.forward(T, K, N, 16, 1024)[0][0] == "few") == few


@pytest.mark.parametrize("T,K,N,wide", [
    (512, 4096, (4096, 1024, 1024), True), (1024, 4096, (4096, 1024, 1024), False), (640, 8192, (8192,), True),
    (1024, 8192, (8192,), False), (768, 4096, (4096,), True), (512, 14336, (4096,), False)])
def test_dx_alone_takes_the_form_that_measured_faster(T, K, N, wide):
    assert (layer_rules.gradient(T, K, N, 16, 8, weights=False)[0][0] == "wide") == wide
