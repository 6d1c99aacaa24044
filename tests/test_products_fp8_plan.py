"""How the products of codes are run: the choice of tile shape and contraction
ranges (product_fp8_plan in csrc/products.hip, called as libmoe.so holds it, for
an MI355X's 256 compute units; nothing is launched)."""
import ctypes
import itertools

import pytest

import sparse_moe_layer_fp32_amd as moe
from tests.product_cases import BIG, HALF, SMALL, THIN8, THIN16
from tests.test_product_plan import CUS, Plan


@pytest.fixture(scope="module")
def plan():
    f = moe.load_library()["_ZN3moe16product_fp8_planEliiiib"]
    f.argtypes = [ctypes.c_int64] + [ctypes.c_int] * 4 + [ctypes.c_bool]
    f.restype = Plan
    return lambda P, G, K, F, exact: f(P, G, K // 2, F, CUS, exact)


SIZES = list(itertools.product((1, 3, 16, 17, 64, 65, 300, 1500, 4096, 9000, 65536), (1, 2, 16, 288),
                               (16, 128, 144, 1024, 4096, 11264, 65536),
                               (8, 72, 256, 1280, 4096, 65536)))


def test_every_plan_can_be_run(plan):
    """Thin tiles take up to 64 rows; large ones two steps at least, in one range,
    for bf16 results; ranges are of a step or more; every kind is reached."""
    seen = set()
    for (P, G, K, F), exact in itertools.product(SIZES, (False, True)):
        p = plan(P, G, K, F, exact)
        what = (P, G, K, F, exact, p.shape, p.splits, p.slices)
        steps = -(-K // 128)
        assert p.us > 0 and p.shape in (BIG, HALF, SMALL, THIN8, THIN16), what
        assert 1 <= p.splits <= min(8, steps), what
        if p.shape in (THIN8, THIN16):
            assert P <= 64 and p.splits == 1, what
        if p.shape == BIG:
            assert not exact and steps >= 2 and p.splits == 1 and p.slices in (1, 2, 4), what
            assert G == 1 or p.slices == 1, what
        else:
            assert p.slices == 1, what
        seen.add((p.shape, p.splits > 1, p.slices > 1, exact))
    for exact in (False, True):
        for s, split in itertools.product((HALF, SMALL), (False, True)):
            assert (s, split, False, exact) in seen
        assert {(THIN8, False, False, exact), (THIN16, False, False, exact)} <= seen
    assert {(BIG, False, False, False), (BIG, False, True, False)} <= seen


@pytest.mark.parametrize("P", [64, 512, 2048])
def test_few_rows_of_many_experts_take_small_tiles(plan, P):
    """The stream of the weights bounds them; large tiles would only compute more."""
    assert plan(P, 288, 4096, 1280, False).shape in (HALF, SMALL)


@pytest.mark.parametrize("P,G,K,F", [(8192, 1, 4096, 11264), (65536, 64, 4096, 1280),
                                     (4096, 1, 4096, 4096)])
def test_large_products_take_large_tiles(plan, P, G, K, F):
    assert plan(P, G, K, F, False).shape == BIG
    assert plan(P, G, K, F, True).shape == HALF
