"""How the linear and grouped products are run: the choice of tile shape,
contraction ranges, slices and shared launches (product_plan and pair_plan in
csrc/products.hip, called as libmoe.so holds them, for an MI355X's 256 compute
units; nothing is launched)."""
import ctypes
import itertools

import pytest

import sparse_moe_layer_fp32_amd as moe

CUS = 256
FORWARD, INPUT, WEIGHT = range(3)


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
