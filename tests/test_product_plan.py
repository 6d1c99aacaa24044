"""How the linear and grouped products are run: the choice of tile shape,
contraction ranges, slices and shared launches (product_plan and pair_plan in
csrc/products.hip, called as libmoe.so holds them, for an MI355X's 256 compute
units; nothing is launched)."""
import ctypes
import itertools
import math
import random

import pytest

import sparse_moe_layer_fp32_amd as moe
from tests.product_cases import (BIG, DUO, FORWARD, HALF, INPUT, PAIRS, SMALL, THIN8, THIN16, WAYS,
                                 WEIGHT)

CUS = 256


class Plan(ctypes.Structure):
    _fields_ = [("shape", ctypes.c_int), ("splits", ctypes.c_int), ("cus", ctypes.c_int),
                ("slices", ctypes.c_int), ("us", ctypes.c_float)]


@pytest.fixture(scope="module")
def lib():
    lib = moe.load_library()
    plan = lib["_ZN3moe12product_planEiliiii"]
    plan.argtypes = [ctypes.c_int, ctypes.c_int64] + [ctypes.c_int] * 4
    plan.restype = Plan
    pair = lib["_ZN3moe9pair_planEliiiiPNS_11ProductPlanES1_"]
    pair.argtypes = [ctypes.c_int64] + [ctypes.c_int] * 4 + [ctypes.POINTER(Plan)] * 2
    pair.restype = ctypes.c_bool
    return plan, pair


def test_every_gradient_has_an_estimated_time(lib):
    """One launch for both gradients is weighed against the estimates of two:
    none may be free."""
    plan, _ = lib
    for op, P, G, K, F in itertools.product(
            (INPUT, WEIGHT), (1, 5, 16, 17, 40, 64, 200, 1000, 4608, 65536), (1, 2, 8, 64, 288),
            (8, 64, 1280, 4096, 11264), (8, 200, 1024, 11264)):
        p = plan(op, P, G, K, F, CUS)
        assert p.us > 0 and p.splits >= 1, (op, P, G, K, F)


@pytest.mark.parametrize("op", (FORWARD, INPUT))
@pytest.mark.parametrize("P,G,long,short", [
    (17, 2, 11264, 64), (17, 8, 11264, 256), (40, 3, 4096, 64), (64, 16, 4096, 64),
    (150, 10, 8192, 128)])
def test_few_rows_a_group_split_a_long_contraction(lib, op, P, G, long, short):
    """A handful of tiles of many steps each would leave the GPU idle."""
    K, F = (long, short) if op == FORWARD else (short, long)
    assert lib[0](op, P, G, K, F, CUS).splits >= 4


@pytest.mark.parametrize("P,G,K,F", [(65536, 1, 64, 64), (1 << 22, 1, 8, 8), (66_000, 1, 8, 136),
                                     (65536, 1, 1024, 64), (100_000, 4, 64, 128)])
def test_long_narrow_weight_gradients_fill_the_gpu(lib, P, G, K, F):
    """A contraction of many rows and an output of few tiles: more ranges, up
    to a slot of the GPU each, and of at least 16 steps of 64 rows."""
    p = lib[0](WEIGHT, P, G, K, F, CUS)
    assert 8 < p.splits <= 512 and p.splits * 16 * 64 <= P // G + 63
    for op in (FORWARD, INPUT):
        assert lib[0](op, P, G, K, F, CUS).splits <= 8


def ways(lib, op, P, G, K, F):
    p = lib[0](op, P, G, K, F, CUS)
    return p.shape, p.splits, p.slices


def pair_ways(lib, P, G, K, F):
    x, w = Plan(), Plan()
    if not lib[1](P, G, K, F, CUS, x, w):
        return None
    assert x.splits == w.splits == w.slices == 1
    return x.shape, x.slices, w.shape


def test_the_table_of_sizes_takes_every_way(lib):
    """tests/product_cases.py: each size is run as it says, and a sweep of
    sizes finds no other way."""
    for (op, ragged), rows in WAYS.items():
        for shape, splits, slices, P, G, K, F in rows:
            assert (G > 1) == ragged and ways(lib, op, P, G, K, F) == (shape, splits, slices), \
                (op, P, G, K, F)
    for sx, slices, sw, P, G, K, F in PAIRS:
        assert pair_ways(lib, P, G, K, F) == (sx, slices, sw), (P, G, K, F)
    known = {key: {row[:3] for row in rows} for key, rows in WAYS.items()}
    pairs = {(row[4] > 1, row[:3]) for row in PAIRS}
    r = random.Random(1)
    size = lambda a, b: int(math.exp(r.uniform(math.log(a), math.log(b))))  # noqa: E731
    for _ in range(40_000):
        P, G, K, F = size(1, 1 << 18), r.choice((1, size(2, 300))), 8 * size(1, 1408), 8 * size(1, 1408)
        for op in (FORWARD, INPUT, WEIGHT):
            assert ways(lib, op, P, G, K, F) in known[op, G > 1], (op, P, G, K, F)
        pair = pair_ways(lib, P, G, K, F)
        assert pair is None or (G > 1, pair) in pairs, (P, G, K, F)


def sizes_of(name):
    """The sizes of a parametrised test in tests/test_gpu_products.py, as rows
    and groups (with its rows of no group), in and out features."""
    from tests import test_gpu_products as t
    mark, = (m for m in getattr(t, name).pytestmark if m.name == "parametrize" and "K,F" in m.args[0])
    for first, K, F in mark.args[1]:
        yield (first, 1, K, F) if isinstance(first, int) else (sum(first) + 73, len(first), K, F)


def test_sizes_of_the_shape_tests(lib):
    """The sizes that the tests of tile shapes name still take those shapes."""
    got = {name: [ways(lib, op, *s) for s in sizes_of(name)] for name, op in (
        ("test_linear_forward_shapes", FORWARD), ("test_linear_input_gradient_shapes", INPUT),
        ("test_linear_weight_gradient_shapes", WEIGHT), ("test_grouped_forward_shapes", FORWARD),
        ("test_grouped_input_gradient_shapes", INPUT), ("test_grouped_weight_gradient_shapes", WEIGHT))}
    assert got == {
        "test_linear_forward_shapes": [
            (BIG, 1, 2), (BIG, 1, 2), (BIG, 1, 4), (HALF, 1, 1), (HALF, 2, 1), (DUO, 1, 1),
            (DUO, 4, 1), (SMALL, 2, 1), (SMALL, 4, 1), (SMALL, 8, 1)],
        "test_linear_input_gradient_shapes": [
            (BIG, 1, 2), (BIG, 1, 2), (BIG, 1, 4), (HALF, 1, 1), (HALF, 2, 1), (DUO, 1, 1),
            (SMALL, 2, 1), (SMALL, 4, 1), (SMALL, 8, 1)],
        "test_linear_weight_gradient_shapes": [
            (BIG, 1, 1), (BIG, 4, 1), (DUO, 1, 1), (DUO, 4, 1), (DUO, 8, 1), (HALF, 1, 1),
            (HALF, 2, 1), (HALF, 4, 1), (HALF, 8, 1), (SMALL, 2, 1), (SMALL, 4, 1), (SMALL, 8, 1)],
        "test_grouped_forward_shapes": [(BIG, 1, 1), (DUO, 1, 1), (DUO, 1, 1), (SMALL, 4, 1)],
        "test_grouped_input_gradient_shapes": [(BIG, 1, 1), (DUO, 1, 1), (HALF, 1, 1)],
        "test_grouped_weight_gradient_shapes": [
            (DUO, 1, 1), (HALF, 1, 1), (HALF, 2, 1), (SMALL, 8, 1), (SMALL, 2, 1)],
    }
    assert [pair_ways(lib, *s) for s in sizes_of("test_linear_both_gradients_shapes")] == [
        (BIG, 1, BIG), (BIG, 1, HALF), (BIG, 2, HALF), (BIG, 4, BIG), (BIG, 4, HALF),
        (HALF, 1, BIG), (HALF, 1, HALF), (SMALL, 1, SMALL)]
    assert [pair_ways(lib, *s) for s in sizes_of("test_grouped_both_gradients_shapes")] == [
        (BIG, 1, BIG), (BIG, 1, HALF), (HALF, 1, BIG), (HALF, 1, HALF), (SMALL, 1, SMALL)]
    assert ways(lib, FORWARD, 1, 1, 4096, 1280)[0] == THIN8
    assert ways(lib, FORWARD, 2, 1, 72, 4096)[0] == THIN16


def test_long_weight_gradients_run_apart(lib):
    """A weight gradient of few long tiles does not queue behind the input
    gradient's tiles in one launch; even and short ones do share it."""
    for P, K, F in ((27930, 5616, 1000), (11353, 6152, 336), (45079, 1208, 5856), (3800, 728, 608),
                    (4082, 648, 464), (9491, 8304, 440)):
        assert pair_ways(lib, P, 1, K, F) is None, (P, K, F)
    for P, K, F in ((8192, 5120, 7168), (4096, 4096, 11264), (2049, 4096, 1280), (1220, 1928, 1136)):
        assert pair_ways(lib, P, 1, K, F) is not None, (P, K, F)
