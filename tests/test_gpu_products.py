"""Linear and grouped products, SwiGLU and their gradients against plain
64-bit forms, element by element, with bounds by arithmetic
(tests/product_util.py)."""
import itertools

import pytest
import torch

from tests import gpu_util as gu
from tests import product_util as pu
from tests.product_util import Guarded, bf16, d64, f32, half, inp, sum_err, within

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _name_case(request):
    gu.note(f"[gpu-test] {request.node.nodeid}")
    yield


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import sparse_moe_layer_fp32_amd as m
    m.load_library()
    return m


# ------------------------------------------------------------------ linear

LINEAR = [(1, 8, 8), (1, 4096, 1280), (2, 72, 4096), (5, 264, 200), (16, 1280, 72), (17, 64, 136),
          (33, 4096, 64), (64, 520, 264), (65, 128, 712), (130, 1288, 320), (257, 192, 1288),
          (300, 2056, 136), (777, 328, 1032), (1025, 72, 264), (2100, 136, 520)]


def check_linear_forward(moe, T, K, F, act="none", y_dtype="bf16", bias=True, residual=True,
                         keep_z=True, seed=0):
    x, w = bf16(T, K, seed=seed), bf16(F, K, scale=K ** -0.5, seed=seed + 1)
    b = f32(F, seed=seed + 2) if bias else None
    r = bf16(T, F, seed=seed + 3) if residual else None
    cfg = moe.make_linear_config(T, K, F, activation=act, y_dtype=y_dtype)
    ws = moe.alloc_linear_workspace(cfg)
    ws.fill_(0xFF)  # NaN as fp32
    y = Guarded(shape=(T, F), dtype=DT[y_dtype])
    z = Guarded(shape=(T, F), dtype=torch.bfloat16) if keep_z else None
    moe.moe_linear_forward(cfg, inp(x), inp(w), inp(b), inp(r), y.t, z.t if z else None, ws)
    torch.cuda.synchronize()
    xd, wd = d64(x), d64(w)
    zd = xd @ wd.t()
    mag = xd.abs() @ wd.abs().t()
    if bias:
        zd, mag = zd + d64(b), mag + d64(b).abs()
    zerr = sum_err(K, mag)
    if keep_z:
        within(z.check(), zd, (1 + pu.BF16_HALF) * zerr + pu.BF16_HALF * zd.abs(), "z")
    yd = pu.act(zd, act)
    err = pu.MAX_SLOPE[act] * zerr + pu.act_err(zd, act)
    if residual:
        yd = yd + d64(r)
        err = err + 2.0 ** -23 * yd.abs()
    h = half(DT[y_dtype])
    within(y.check(), yd, (1 + h) * err + h * yd.abs(), "y")


@pytest.mark.parametrize("T,K,F", LINEAR)
def test_linear_forward_sizes(moe, T, K, F):
    check_linear_forward(moe, T, K, F)


# Sizes at which an MI355X's launches take each tile shape (256 x 256, 128 x
# 256, 256 x 128, 64 x 64), contraction split (up to 8 ranges) and cut of the
# last round's tiles (halves, quarters).
@pytest.mark.parametrize("T,K,F", [
    (1500, 72, 4096), (5000, 520, 4200), (4100, 520, 4104), (4100, 136, 1032), (1000, 4096, 2056),
    (4100, 72, 1032), (9000, 4096, 72), (2100, 4096, 72), (1500, 2056, 72), (300, 2056, 72)])
def test_linear_forward_shapes(moe, T, K, F):
    check_linear_forward(moe, T, K, F, "silu", keep_z=False, seed=7)


@pytest.mark.parametrize("act,y_dtype", itertools.product(
    ("none", "relu", "gelu", "gelu_tanh", "silu"), ("bf16", "f32")))
@pytest.mark.parametrize("T,K,F", [(3, 512, 264), (150, 136, 200)])
def test_linear_forward_activations(moe, T, K, F, act, y_dtype):
    check_linear_forward(moe, T, K, F, act, y_dtype, residual=y_dtype == "bf16", seed=5)


@pytest.mark.parametrize("bias,residual,keep_z", itertools.product((False, True), repeat=3))
def test_linear_forward_optional_operands(moe, bias, residual, keep_z):
    check_linear_forward(moe, 40, 136, 72, "gelu", "bf16", bias, residual, keep_z, seed=9)
    check_linear_forward(moe, 700, 136, 2056, "silu", "f32", bias, residual, keep_z, seed=9)


def check_linear_backward(moe, T, K, F, act="none", dw_dtype="f32", accumulate=False,
                          want=("dx", "dw", "db"), seed=0):
    dy, x = bf16(T, F, seed=seed), bf16(T, K, seed=seed + 1)
    w, z = bf16(F, K, scale=K ** -0.5, seed=seed + 2), bf16(T, F, scale=2.0, seed=seed + 3)
    dw0, db0 = f32(F, K, seed=seed + 4).to(DT[dw_dtype]), f32(F, seed=seed + 5)
    cfg = moe.make_linear_config(T, K, F, activation=act, dw_dtype=dw_dtype, accumulate=accumulate)
    ws = moe.alloc_linear_workspace(cfg)
    ws.fill_(0xFF)
    fill = accumulate or None
    dz = Guarded(shape=(T, F), dtype=torch.bfloat16) if act != "none" else None
    dx = Guarded(shape=(T, K), dtype=torch.bfloat16) if "dx" in want else None
    dw = Guarded(shape=(F, K), dtype=DT[dw_dtype], fill=fill and dw0) if "dw" in want else None
    db = Guarded(shape=(F,), dtype=torch.float32, fill=fill and db0) if "db" in want else None
    t = lambda g: g.t if g else None  # noqa: E731
    moe.moe_linear_backward(cfg, inp(dy), inp(z) if act != "none" else None,
                            inp(x) if dw else None, inp(w) if dx else None, t(dz), t(dx), t(dw),
                            t(db), ws)
    torch.cuda.synchronize()
    zd = d64(z)
    sl = pu.slope(zd, act)
    dyd = d64(dy)
    dzd, dzerr = dyd * sl, dyd.abs() * pu.slope_err(zd, act) + 2.0 ** -24 * (dyd * sl).abs()
    used = dyd  # what dx and dw are formed from
    if dz:
        got = dz.check()
        within(got, dzd, (1 + pu.BF16_HALF) * dzerr + pu.BF16_HALF * dzd.abs(), "dz")
        used = d64(got)
    if dx:
        want_, mag = used @ d64(w), used.abs() @ d64(w).abs()
        within(dx.check(), want_, 1.01 * sum_err(F, mag) + pu.BF16_HALF * want_.abs(), "dx")
    if dw:
        want_, mag = used.t() @ d64(x), used.abs().t() @ d64(x).abs()
        if accumulate:
            want_, mag = want_ + d64(dw0), mag + d64(dw0).abs()
        within(dw.check(), want_, 1.01 * sum_err(T, mag) + half(DT[dw_dtype]) * want_.abs(), "dw")
    if db:
        want_, mag = dzd.sum(0), dzd.abs().sum(0)
        if accumulate:
            want_, mag = want_ + d64(db0), mag + d64(db0).abs()
        within(db.check(), want_, sum_err(T, mag) + dzerr.sum(0), "db")


@pytest.mark.parametrize("T,K,F", LINEAR)
def test_linear_backward_sizes(moe, T, K, F):
    check_linear_backward(moe, T, K, F)


@pytest.mark.parametrize("T,K,F", [  # as above, for the input gradient
    (1500, 4096, 72), (5000, 4200, 520), (4100, 4104, 520), (4100, 1032, 136), (1000, 2056, 4096),
    (4100, 1032, 72), (2100, 72, 4096), (1500, 72, 2056), (300, 72, 2056)])
def test_linear_input_gradient_shapes(moe, T, K, F):
    check_linear_backward(moe, T, K, F, want=("dx",), seed=7)


@pytest.mark.parametrize("T,K,F", [  # and for the weight gradient
    (300, 2056, 4096), (9000, 520, 4096), (300, 4096, 4096), (4100, 264, 4096), (9000, 264, 2056),
    (300, 1032, 4096), (3000, 1032, 2056), (3000, 1032, 1032), (9000, 520, 1032),
    (3000, 72, 2056), (2100, 72, 1032), (1500, 72, 72)])
def test_linear_weight_gradient_shapes(moe, T, K, F):
    check_linear_backward(moe, T, K, F, want=("dw", "db"), seed=7)


@pytest.mark.parametrize("T,K,F", [  # both in one launch, in each pair of shapes
    (1000, 4104, 1032), (1000, 4104, 264), (4100, 2056, 2056), (700, 2056, 2056),
    (300, 4104, 2056), (500, 4104, 1032), (700, 4104, 264), (300, 264, 264)])
@pytest.mark.parametrize("accumulate,dw_dtype", [(False, "f32"), (True, "bf16")])
def test_linear_both_gradients_shapes(moe, T, K, F, accumulate, dw_dtype):
    check_linear_backward(moe, T, K, F, accumulate=accumulate, dw_dtype=dw_dtype, seed=7)


@pytest.mark.parametrize("act", ("relu", "gelu", "gelu_tanh", "silu"))
@pytest.mark.parametrize("T,K,F,dw_dtype", [(3, 136, 264, "bf16"), (210, 72, 136, "f32")])
def test_linear_backward_activations(moe, T, K, F, dw_dtype, act):
    check_linear_backward(moe, T, K, F, act, dw_dtype, seed=3)


@pytest.mark.parametrize("accumulate,dw_dtype,act", itertools.product(
    (False, True), ("bf16", "f32"), ("none", "silu")))
def test_linear_backward_accumulates(moe, accumulate, dw_dtype, act):
    check_linear_backward(moe, 90, 200, 136, act, dw_dtype, accumulate, seed=4)


@pytest.mark.parametrize("T,F", [  # one strip of rows, several, many blocks, strips of 128 rows
    (1, 520), (17, 8), (64, 520), (65, 520), (1000, 264), (16400, 1032), (66000, 136)])
@pytest.mark.parametrize("accumulate", (False, True))
def test_linear_backward_strips_of_the_activation(moe, T, F, accumulate):
    check_linear_backward(moe, T, 8, F, "silu", "f32", accumulate, want=("dw", "db"), seed=8)


@pytest.mark.parametrize("want", [("dx",), ("dw",), ("db",), ("dx", "db"), ("dw", "db"), ()])
@pytest.mark.parametrize("act", ("none", "gelu"))
@pytest.mark.parametrize("T", (37, 2500))
def test_linear_backward_optional_results(moe, T, act, want):
    check_linear_backward(moe, T, 72, 136, act, want=want, seed=6)


def test_linear_no_tokens(moe):
    for accumulate in (False, True):
        cfg = moe.make_linear_config(0, 64, 72, activation="silu", accumulate=accumulate)
        ws = moe.alloc_linear_workspace(cfg)
        e = lambda n: torch.empty((0, n), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        w = inp(bf16(72, 64))
        moe.moe_linear_forward(cfg, e(64), w, None, None, e(72), None, ws)
        dw, db = torch.ones(72, 64, device="cuda"), torch.ones(72, device="cuda")
        moe.moe_linear_backward(cfg, e(72), e(72), e(64), w, e(72), e(64), dw, db, ws)
        torch.cuda.synchronize()
        assert (dw == float(accumulate)).all() and (db == float(accumulate)).all()


def test_linear_rows_with_nan_and_infinities_stay_apart(moe):
    T, K, F = 70, 136, 72
    x, w = bf16(T, K), bf16(F, K)
    x[3, 7], x[64, 0], x[69, 135] = float("nan"), float("inf"), float("-inf")
    cfg = moe.make_linear_config(T, K, F, y_dtype="f32")
    y = torch.empty(T, F, device="cuda")
    moe.moe_linear_forward(cfg, inp(x), inp(w), None, None, y, None,
                           moe.alloc_linear_workspace(cfg))
    y = y.cpu()
    assert y[3].isnan().all()
    assert not y[64].isfinite().any() and not y[69].isfinite().any()
    rest = [r for r in range(T) if r not in (3, 64, 69)]
    assert y[rest].isfinite().all()


# ------------------------------------------------------------------ grouped

GROUPS = {
    "one": [37],
    "empties": [0, 5, 0, 0, 130, 1, 0],
    "tile_edges": [64, 128, 256, 63, 65, 127, 129, 1],
    "all_in_last": [0, 0, 0, 300],
    "many_small": [(7 * i) % 5 for i in range(200)],
    "long": [700, 3, 1100, 0, 450],
    "none": [0, 0, 0],
}


def group_case(sizes, before, after, K, per=3, seed=0):
    """offsets and gathered rows: `before` rows ahead of the first group and
    `after` behind the last belong to no group."""
    off = torch.tensor([0] + list(itertools.accumulate(sizes)), dtype=torch.int32) + before
    P = before + sum(sizes) + after
    T = max(1, -(-P // per))
    g = torch.Generator().manual_seed(seed + 50)
    ids = torch.randint(0, T * per, (P,), generator=g).to(torch.int32)
    return P, T, off, ids


def spans(off):
    return [(e, int(off[e]), int(off[e + 1])) for e in range(len(off) - 1)]


def source_rows(x, ids, P):
    """The rows that rows 0 .. P - 1 read, in 64 bits: zeros for a source
    outside x."""
    if ids is None:
        return d64(x)
    s = torch.where(ids >= 0, torch.div(ids, 3, rounding_mode="floor"), -1).long().cuda()
    ok = (s >= 0) & (s < x.shape[0])
    return d64(x)[s.clamp(0, x.shape[0] - 1)] * ok.unsqueeze(1)


def check_grouped_forward(moe, sizes, K, F, before=0, after=0, gather=True, bias=True,
                          y_dtype="bf16", bad_ids=(), seed=0):
    P, T, off, ids = group_case(sizes, before, after, K, seed=seed)
    E = len(sizes)
    if not gather:
        T, ids = P, None
    x, w = bf16(T, K, seed=seed), bf16(E, F, K, scale=K ** -0.5, seed=seed + 1)
    b = f32(E, F, seed=seed + 2) if bias else None
    for r, v in bad_ids:
        ids[r] = v
    cfg = moe.make_grouped_config(P, E, K, F, x_rows=T, row_div=3 if gather else 1, y_dtype=y_dtype)
    ws = moe.alloc_grouped_workspace(cfg)
    ws.fill_(0xFF)
    y = Guarded(shape=(P, F), dtype=DT[y_dtype],
                fill=torch.full((P, F), pu.SENTINEL, dtype=DT[y_dtype]))
    moe.moe_grouped_forward(cfg, inp(x), inp(ids), inp(off), inp(w), inp(b), y.t, ws)
    torch.cuda.synchronize()
    got = y.check()
    h = half(DT[y_dtype])
    rows = source_rows(x, ids, P)
    seen = torch.zeros(P, dtype=torch.bool)
    for e, i, j in spans(off):
        seen[i:j] = True
        if j == i:
            continue
        want = rows[i:j] @ d64(w[e]).t()
        mag = rows[i:j].abs() @ d64(w[e]).abs().t()
        if bias:
            want, mag = want + d64(b[e]), mag + d64(b[e]).abs()
        within(got[i:j], want, (1 + h) * sum_err(K, mag) + h * want.abs(), f"y of group {e}")
    assert (got[~seen] == pu.SENTINEL).all(), "a row of no group was written"


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("K,F", [(72, 136), (512, 264)])
def test_grouped_forward(moe, name, K, F):
    check_grouped_forward(moe, GROUPS[name], K, F)


UNEVEN = [1500, 0, 700, 60, 2400, 130, 190, 250, 1, 400, 2000, 369]  # 8000 rows


@pytest.mark.parametrize("sizes,K,F", [
    (UNEVEN, 1032, 2056), ([3000, 900, 2100], 72, 1032), ([1500, 1, 640, 900, 1400, 1300, 259], 72, 1032),
    ([2, 0, 1, 5, 3], 2056, 520)])
def test_grouped_forward_shapes(moe, sizes, K, F):
    """256 x 256 tiles with every size of remainder, the other shapes, and
    few rows."""
    check_grouped_forward(moe, sizes, K, F, before=3, after=70, seed=7)


@pytest.mark.parametrize("sizes,K,F", [
    (UNEVEN, 2056, 1032), ([6000, 1, 5999], 520, 136), ([2500, 900, 2600], 1032, 136)])
def test_grouped_input_gradient_shapes(moe, sizes, K, F):
    check_grouped_backward(moe, sizes, K, F, before=3, after=70, want=("dx",), seed=7)


@pytest.mark.parametrize("sizes,K,F", [
    ([(i * 29) % 61 for i in range(40)], 520, 520), ([100, 0, 300, 1, 640, 209], 1032, 1032),
    ([9000, 3, 2997], 1032, 1032), ([700, 2300, 3000], 72, 136), ([5000, 6000, 1000], 72, 1032)])
@pytest.mark.parametrize("gather", (False, True))
def test_grouped_weight_gradient_shapes(moe, sizes, K, F, gather):
    check_grouped_backward(moe, sizes, K, F, before=3, after=70, gather=gather, want=("dw", "db"),
                           seed=7)


@pytest.mark.parametrize("sizes,K,F", [  # both gradients in one launch
    ([300, 0, 257, 73], 4104, 264), ([400, 1, 90, 0, 64, 65, 130, 190, 0], 2056, 264),
    ([90, 0, 1, 64, 30, 0, 0, 5, 40], 2056, 264), ([90, 0, 1, 64, 30, 0, 0, 5, 40], 2056, 520),
    ([150, 0, 1, 80], 264, 264)])
@pytest.mark.parametrize("gather", (False, True))
def test_grouped_both_gradients_shapes(moe, sizes, K, F, gather):
    check_grouped_backward(moe, sizes, K, F, before=3, after=70, gather=gather, seed=7)


def test_grouped_with_no_rows_of_x(moe):
    """Every source lies outside an x of no rows: the products are zero."""
    P, E, K, F = 40, 3, 72, 136
    off = torch.tensor([0, 10, 10, 40], dtype=torch.int32, device="cuda")
    ids = torch.arange(P, dtype=torch.int32, device="cuda")
    x = torch.empty((0, K), dtype=torch.bfloat16, device="cuda")
    w, dy = bf16(E, F, K).cuda(), bf16(P, F, seed=1).cuda()
    b = f32(E, F, seed=2).cuda()
    cfg = moe.make_grouped_config(P, E, K, F, x_rows=0, y_dtype="f32")
    ws = moe.alloc_grouped_workspace(cfg)
    y, dw = torch.empty(P, F, device="cuda"), torch.ones(E, F, K, device="cuda")
    moe.moe_grouped_forward(cfg, x, ids, off, w, b, y, ws)
    moe.moe_grouped_backward(cfg, dy, x, ids, off, None, None, dw, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(y[:10], b[0].expand(10, F)) and torch.equal(y[10:], b[2].expand(30, F))
    assert (dw == 0).all()


@pytest.mark.parametrize("accumulate", (False, True))
def test_grouped_weight_gradient_larger_than_the_caches(moe, accumulate):
    """Above 256 MB the gradient is stored past the caches."""
    check_grouped_backward(moe, [(i * 29) % 61 for i in range(64)], 1032, 1032,
                           accumulate=accumulate, want=("dw", "db"), seed=8)


@pytest.mark.parametrize("gather,bias,y_dtype", itertools.product((False, True), (False, True),
                                                                  ("bf16", "f32")))
def test_grouped_forward_variants(moe, gather, bias, y_dtype):
    check_grouped_forward(moe, GROUPS["tile_edges"], 136, 72, 5, 9, gather, bias, y_dtype, seed=2)


def test_grouped_forward_most_groups(moe):
    check_grouped_forward(moe, [(i * 37) % 3 for i in range(1024)], 64, 72, before=2, after=3)


def test_grouped_forward_sources_outside_x_read_as_zeros(moe):
    check_grouped_forward(moe, [40, 30], 72, 72,
                          bad_ids=[(0, -1), (41, 2 ** 31 - 1), (69, -2 ** 31), (5, 24 * 3)])


def test_grouped_offsets_are_clamped(moe):
    """Offsets below 0 and beyond P name no rows outside [0, P)."""
    P, K, F = 50, 72, 72
    off = torch.tensor([-9, 20, 2 ** 30], dtype=torch.int32)
    x, w = bf16(P, K), bf16(2, F, K, seed=1)
    cfg = moe.make_grouped_config(P, 2, K, F, y_dtype="f32")
    y = Guarded(shape=(P, F), dtype=torch.float32)
    moe.moe_grouped_forward(cfg, inp(x), None, inp(off), inp(w), None, y.t,
                            moe.alloc_grouped_workspace(cfg))
    got = y.check()
    for e, i, j in ((0, 0, 20), (1, 20, 50)):
        want = x[i:j].double() @ w[e].double().t()
        within(got[i:j], want, sum_err(K, x[i:j].double().abs() @ w[e].double().abs().t()), "y")


def check_grouped_backward(moe, sizes, K, F, before=0, after=0, gather=True, dw_dtype="f32",
                           accumulate=False, want=("dx", "dw", "db"), seed=0):
    P, T, off, ids = group_case(sizes, before, after, K, seed=seed)
    E = len(sizes)
    if not gather:
        T, ids = P, None
    elif P > 3:
        ids[min(P - 1, before + 1)] = -4  # its source reads as zeros
    dy, x = bf16(P, F, seed=seed), bf16(T, K, seed=seed + 1)
    dy[:before], dy[P - after:] = float("nan"), float("nan")  # rows of no group
    w = bf16(E, F, K, scale=K ** -0.5, seed=seed + 2)
    dw0, db0 = f32(E, F, K, seed=seed + 4).to(DT[dw_dtype]), f32(E, F, seed=seed + 5)
    cfg = moe.make_grouped_config(P, E, K, F, x_rows=T, row_div=3 if gather else 1,
                                  dw_dtype=dw_dtype, accumulate=accumulate)
    ws = moe.alloc_grouped_workspace(cfg)
    ws.fill_(0xFF)
    dx = Guarded(shape=(P, K), dtype=torch.bfloat16, fill=torch.full(
        (P, K), pu.SENTINEL, dtype=torch.bfloat16)) if "dx" in want else None
    fill = accumulate or None
    dw = Guarded(shape=(E, F, K), dtype=DT[dw_dtype], fill=fill and dw0) if "dw" in want else None
    db = Guarded(shape=(E, F), dtype=torch.float32, fill=fill and db0) if "db" in want else None
    t = lambda g: g.t if g else None  # noqa: E731
    moe.moe_grouped_backward(cfg, inp(dy), inp(x), inp(ids), inp(off), inp(w), t(dx), t(dw), t(db),
                             ws)
    torch.cuda.synchronize()
    rows = source_rows(x, ids, P)
    gx, gw, gb = (g.check() if g else None for g in (dx, dw, db))
    seen = torch.zeros(P, dtype=torch.bool)
    for e, i, j in spans(off):
        seen[i:j] = True
        d, xe = d64(dy[i:j]), rows[i:j]
        if dx and j > i:
            want_, mag = d @ d64(w[e]), d.abs() @ d64(w[e]).abs()
            within(gx[i:j], want_, 1.01 * sum_err(F, mag) + pu.BF16_HALF * want_.abs(), f"dx {e}")
        if dw:
            want_, mag = d.t() @ xe, d.abs().t() @ xe.abs()
            if accumulate:
                want_, mag = want_ + d64(dw0[e]), mag + d64(dw0[e]).abs()
            within(gw[e], want_, 1.01 * sum_err(j - i, mag) + half(DT[dw_dtype]) * want_.abs(),
                   f"dw {e}")
        if db:
            want_, mag = d.sum(0), d.abs().sum(0)
            if accumulate:
                want_, mag = want_ + d64(db0[e]), mag + d64(db0[e]).abs()
            within(gb[e], want_, sum_err(j - i, mag), f"db {e}")
    if dx:
        assert (gx[~seen] == pu.SENTINEL).all(), "a row of no group was written"


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("K,F", [(72, 136), (264, 320)])
def test_grouped_backward(moe, name, K, F):
    check_grouped_backward(moe, GROUPS[name], K, F)


@pytest.mark.parametrize("gather,dw_dtype,accumulate", itertools.product(
    (False, True), ("bf16", "f32"), (False, True)))
def test_grouped_backward_variants(moe, gather, dw_dtype, accumulate):
    check_grouped_backward(moe, GROUPS["empties"], 136, 72, 5, 9, gather, dw_dtype, accumulate,
                           seed=2)


@pytest.mark.parametrize("want", [("dx",), ("dw",), ("db",), ("dx", "db"), ("dw", "db"), ()])
def test_grouped_backward_optional_results(moe, want):
    check_grouped_backward(moe, GROUPS["tile_edges"], 72, 136, want=want, seed=6)


def test_grouped_beyond_32_bits(moe):
    """Weights, rows and results whose element and byte offsets pass 2^32: the
    first and last groups and rows against the definition."""
    E, K, F, P = 520, 8192, 1032, 540_000
    g = torch.Generator(device="cuda").manual_seed(3)
    normal = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # noqa: E731
    x, w, dy = normal(P, K), normal(E, F, K), normal(P, F)
    assert x.numel() > 2 ** 32 and w.numel() > 2 ** 32
    sizes = [70, 130] + [0] * (E - 4) + [P - 500, 300]
    off = torch.tensor([0] + list(itertools.accumulate(sizes)), dtype=torch.int32, device="cuda")
    cfg = moe.make_grouped_config(P, E, K, F)
    ws = moe.alloc_grouped_workspace(cfg)
    y = torch.empty(P, F, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_forward(cfg, x, None, off, w, None, y, ws)
    dx = torch.empty(P, K, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((E, F, K), 3.0, device="cuda")
    moe.moe_grouped_backward(cfg, dy, x, None, off, w, dx, dw, None, ws)
    torch.cuda.synchronize()
    last = P - 300
    for e, i, j in ((0, 0, 70), (1, 70, 200), (E - 2, last - 90, last), (E - 1, last, P)):
        xe, we, de = x[i:j].double(), w[e].double(), dy[i:j].double()
        want, mag = xe @ we.t(), xe.abs() @ we.abs().t()
        within(y[i:j], want, 1.01 * sum_err(K, mag) + pu.BF16_HALF * want.abs(), f"y of group {e}")
        want, mag = de @ we, de.abs() @ we.abs()
        within(dx[i:j], want, 1.01 * sum_err(F, mag) + pu.BF16_HALF * want.abs(), f"dx {e}")
        if e != E - 2:
            within(dw[e], de.t() @ xe, sum_err(j - i, de.abs().t() @ xe.abs()) + 1e-30, f"dw {e}")
    assert (dw[2:E - 2] == 0).all()


def test_binding_refuses_what_a_kernel_would_misread(moe):
    """Sizes, types, layouts and missing tensors, refused before any launch."""
    z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    cfg = moe.make_linear_config(8, 64, 72)
    ws = moe.alloc_linear_workspace(cfg)
    ok = dict(x=z(8, 64), w=z(72, 64), bias=z(72, d=torch.float32), residual=z(8, 72), y=z(8, 72))
    call = lambda **kw: moe.moe_linear_forward(cfg, *{**ok, **kw}.values(), None, ws)  # noqa: E731
    call()
    for kw, err in ((dict(x=z(7, 64)), ValueError), (dict(w=z(64, 72)[:, :64]), ValueError),
                    (dict(bias=z(72)), TypeError), (dict(y=z(8, 72, d=torch.float32)), TypeError),
                    (dict(x=None), ValueError), (dict(x=z(64, 8).t()), ValueError),
                    (dict(residual=z(8, 72).cpu()), ValueError), (dict(x=[1.0]), TypeError)):
        with pytest.raises(err):
            call(**kw)
    with pytest.raises(ValueError):
        moe.moe_linear_forward(cfg, *ok.values(), None, None)
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.moe_linear_forward(cfg, *ok.values(), None, ws[:-256])
    gc = moe.make_grouped_config(8, 3, 64, 72)
    gws = moe.alloc_grouped_workspace(gc)
    with pytest.raises(ValueError):  # offsets of two groups
        moe.moe_grouped_forward(gc, z(8, 64), None, z(3, d=torch.int32), z(3, 72, 64), None,
                                z(8, 72), gws)
    with pytest.raises(TypeError):  # 64-bit offsets
        moe.moe_grouped_forward(gc, z(8, 64), None, z(4, d=torch.int64), z(3, 72, 64), None,
                                z(8, 72), gws)
    sc = moe.make_swiglu_config(4, 64, ld=128)
    gu_ = z(4, 128)
    moe.moe_swiglu_forward(sc, gu_[:, :64], gu_[:, 64:], z(4, 64))
    with pytest.raises(ValueError):  # another row stride
        moe.moe_swiglu_forward(sc, z(4, 64), gu_[:, 64:], z(4, 64))
    with pytest.raises(ValueError):
        moe.moe_swiglu_forward(sc, gu_[:, ::2], gu_[:, 64:], z(4, 64))


# ------------------------------------------------------------------ SwiGLU

def swiglu_ref(g, u, limit):
    g, u = g.double(), u.double()
    gc, uc = (g.clamp(max=limit), u.clamp(-limit, limit)) if limit > 0 else (g, u)
    s = 1 / (1 + torch.exp(-gc))
    return g, u, gc, uc, s


def check_swiglu(moe, rows, n, limit, fused, keep_h=True, scale=3.0, seed=0):
    gu_ = bf16(rows, 2 * n, scale=scale, seed=seed)
    if limit > 0 and rows * n > 16:  # values at the limit and next to it
        gu_[0, :4] = torch.tensor([limit, -limit, limit * 1.01, limit * 0.99])
        gu_[0, n:n + 4] = torch.tensor([limit, -limit, -limit * 1.01, limit * 1.01])
    dh = bf16(rows, n, seed=seed + 1)
    cfg = moe.make_swiglu_config(rows, n, ld=2 * n if fused else 0, limit=limit)
    g, u = gu_[:, :n], gu_[:, n:]
    if fused:
        dev = inp(gu_)
        dg_, du_ = dev[:, :n], dev[:, n:]
    else:
        dg_, du_ = inp(g.contiguous()), inp(u.contiguous())
    h = Guarded(shape=(rows, n), dtype=torch.bfloat16)
    moe.moe_swiglu_forward(cfg, dg_, du_, h.t)
    out = Guarded(shape=(rows, 2 * n) if fused else (2, rows, n), dtype=torch.bfloat16)
    og, ou = (out.t[:, :n], out.t[:, n:]) if fused else (out.t[0], out.t[1])
    h2 = Guarded(shape=(rows, n), dtype=torch.bfloat16) if keep_h else None
    moe.moe_swiglu_backward(cfg, inp(dh), dg_, du_, og, ou, h2.t if h2 else None)
    torch.cuda.synchronize()
    g, u, gc, uc, s = swiglu_ref(g, u, limit)
    want = gc * s * uc
    hb = 1.01 * 2.0 ** -20 * (gc * uc).abs() + pu.BF16_HALF * want.abs()
    got = h.check()
    within(got, want, hb, "h")
    if h2:
        assert torch.equal(h2.check(), got)
    d = dh.double()
    o = out.check()
    gotg, gotu = (o[:, :n], o[:, n:]) if fused else (o[0], o[1])
    passg = (g <= limit) | (limit <= 0)
    passu = (u.abs() <= limit) | (limit <= 0)
    wg = d * uc * s * (1 + gc * (1 - s)) * passg
    wu = d * gc * s * passu
    within(gotg, wg, 1.01 * 2.0 ** -20 * (d * uc).abs() * (1 + gc.abs()) + pu.BF16_HALF * wg.abs(),
           "dgate")
    within(gotu, wu, 1.01 * 2.0 ** -20 * (d * gc).abs() + pu.BF16_HALF * wu.abs(), "dup")


@pytest.mark.parametrize("rows,n", [(1, 8), (1, 1280), (3, 72), (64, 1280), (257, 264)])
@pytest.mark.parametrize("limit", (0.0, 7.0))
@pytest.mark.parametrize("fused", (False, True))
def test_swiglu(moe, rows, n, limit, fused):
    check_swiglu(moe, rows, n, limit, fused, keep_h=fused)


def test_swiglu_large_values(moe):
    check_swiglu(moe, 9, 64, 0.0, False, scale=1e4, seed=3)
    check_swiglu(moe, 9, 64, 7.0, True, scale=1e4, seed=4)


def test_swiglu_no_rows(moe):
    cfg = moe.make_swiglu_config(0, 64)
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    moe.moe_swiglu_forward(cfg, e, e, e)
    moe.moe_swiglu_backward(cfg, e, e, e, e, e)


# ------------------------------------------------------------------ against differences

@pytest.mark.parametrize("T,K,F", [(5, 72, 64), (130, 264, 136)])
def test_linear_gradients_are_differences_of_the_forward(moe, T, K, F):
    """Without an activation <y, c> is linear in x and w, so it changes by
    exactly <dx, d> and <dw, d> along a direction d (entries 1/4 on values
    that are multiples of 1/4: x + d and w + d are exact in bf16)."""
    g = torch.Generator().manual_seed(1)
    grid = lambda *s: torch.randint(-8, 9, s, generator=g).float().div(4).bfloat16()  # noqa: E731
    x, w, c = grid(T, K), grid(F, K), grid(T, F)
    step = torch.randint(0, 2, (T, K), generator=g).float().div(4).bfloat16()
    wstep = torch.randint(0, 2, (F, K), generator=g).float().div(4).bfloat16()
    cfg = moe.make_linear_config(T, K, F, y_dtype="f32")
    ws = moe.alloc_linear_workspace(cfg)

    def value(x, w):
        y = torch.empty(T, F, device="cuda")
        moe.moe_linear_forward(cfg, x.cuda(), w.cuda(), None, None, y, None, ws)
        return float((y.cpu().double() * c.double()).sum())

    dx = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    dw = torch.empty(F, K, device="cuda")
    moe.moe_linear_backward(cfg, c.cuda(), None, x.cuda(), w.cuda(), None, dx, dw, None, ws)
    # multiples of 1/64 below 2^17: the fp32 sums are exact, and only dx is rounded
    along_x = float((dx.cpu().double() * step.double()).sum())
    bound = pu.BF16_HALF * float((dx.cpu().double().abs() * step.double()).sum()) * 1.01
    assert abs(value(x + step, w) - value(x, w) - along_x) <= bound
    along_w = float((dw.cpu().double() * wstep.double()).sum())
    assert value(x, w + wstep) - value(x, w) == along_w


@pytest.mark.parametrize("act", ("gelu", "gelu_tanh", "silu"))
def test_linear_bias_gradient_is_a_difference(moe, act):
    """dbias against central differences of the forward pass in the bias."""
    T, K, F, h = 24, 64, 16, 2.0 ** -6
    x, w, b, dy = bf16(T, K), bf16(F, K, scale=0.1, seed=1), f32(F, seed=2), bf16(T, F, seed=3)
    cfg = moe.make_linear_config(T, K, F, activation=act, y_dtype="f32")
    ws = moe.alloc_linear_workspace(cfg)
    z = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")

    def value(b, z=None):
        y = torch.empty(T, F, device="cuda")
        moe.moe_linear_forward(cfg, x.cuda(), w.cuda(), b.cuda(), None, y, z, ws)
        return (y.cpu().double() * dy.double()).sum(0)

    value(b, z)
    db = torch.empty(F, device="cuda")
    dz = torch.empty_like(z)
    moe.moe_linear_backward(cfg, dy.cuda(), z, None, None, dz, None, None, db, ws)
    diff = (value(b + h) - value(b - h)) / (2 * h)
    # the slope at the rounded z is off by |act''| <= 1.2 times z's rounding; a
    # central difference by h^2/6 |act'''|, |act'''| <= 2; the forward's own
    # error (2^-20 |z| and sums of 64 terms) is divided by h
    a, zz = dy.double().abs(), z.cpu().double().abs()
    mag = x.double().abs() @ w.double().abs().t() + b.double().abs() + h
    bound = (a * (1.2 * pu.BF16_HALF * zz + h * h / 3 + (2.0 ** -20 * (zz + 1) +
                                                       1.13 * sum_err(K, mag)) / h)).sum(0)
    within(db.cpu(), diff, bound, "dbias")


# ------------------------------------------------------------------ streams, graphs, order

def test_products_in_a_graph_and_on_a_side_stream(moe):
    """Forward and backward of all three operators captured together; every
    replay equals the eager results bit for bit."""
    P, T, E, K, F = 150, 50, 5, 136, 72
    g = torch.Generator().manual_seed(0)
    off = torch.tensor([0, 40, 40, 41, 140, 150], dtype=torch.int32).cuda()
    ids = torch.randint(0, P, (P,), generator=g).to(torch.int32).cuda()
    x, w, dy = bf16(T, K).cuda(), bf16(E, F, K, seed=1).cuda(), bf16(P, F, seed=2).cuda()
    lx, lw = bf16(3, 1024, seed=3).cuda(), bf16(72, 1024, seed=4).cuda()
    gc = moe.make_grouped_config(P, E, K, F, x_rows=T, row_div=3)
    lc = moe.make_linear_config(3, 1024, 72, activation="silu")
    sc = moe.make_swiglu_config(P, F // 2 // 8 * 8, ld=F)
    half_ = F // 2 // 8 * 8
    wg, wl = moe.alloc_grouped_workspace(gc), moe.alloc_linear_workspace(lc)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    o = dict(y=torch.empty(P, F, **bf), dx=torch.empty(P, K, **bf), dw=torch.empty(E, F, K, device="cuda"),
             db=torch.empty(E, F, device="cuda"), ly=torch.empty(3, 72, **bf), lz=torch.empty(3, 72, **bf),
             ldz=torch.empty(3, 72, **bf), ldx=torch.empty(3, 1024, **bf),
             ldw=torch.empty(72, 1024, device="cuda"), ldb=torch.empty(72, device="cuda"),
             h=torch.empty(P, half_, **bf), dgu=torch.zeros(P, F, **bf))

    def step():
        moe.moe_grouped_forward(gc, x, ids, off, w, None, o["y"], wg)
        moe.moe_swiglu_forward(sc, o["y"][:, :half_], o["y"][:, F - half_:], o["h"])
        moe.moe_swiglu_backward(sc, o["h"], o["y"][:, :half_], o["y"][:, F - half_:],
                                o["dgu"][:, :half_], o["dgu"][:, F - half_:])
        moe.moe_grouped_backward(gc, o["dgu"], x, ids, off, w, o["dx"], o["dw"], o["db"], wg)
        moe.moe_linear_forward(lc, lx, lw, None, None, o["ly"], o["lz"], wl)
        moe.moe_linear_backward(lc, o["ly"], o["lz"], lx, lw, o["ldz"], o["ldx"], o["ldw"],
                                o["ldb"], wl)

    step()
    torch.cuda.synchronize()
    ref = {k: v.clone() for k, v in o.items()}
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    assert all(torch.equal(o[k], ref[k]) for k in o), "side stream"
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for rep in range(3):
        for v in o.values():
            v.zero_()
        wg.fill_(0xFF), wl.fill_(0xFF)
        other = torch.randn(256, 256, device="cuda") @ torch.randn(256, 256, device="cuda")
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o[k], ref[k]) for k in o), f"replay {rep}"
        del other


def test_products_are_deterministic(moe):
    T, K, F = 2100, 520, 264
    dy, x, w = bf16(T, F).cuda(), bf16(T, K, seed=1).cuda(), bf16(F, K, seed=2).cuda()
    cfg = moe.make_linear_config(T, K, F)
    ws = moe.alloc_linear_workspace(cfg)
    outs = []
    for _ in range(3):
        dx = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
        dw, db = torch.empty(F, K, device="cuda"), torch.empty(F, device="cuda")
        moe.moe_linear_backward(cfg, dy, None, x, w, None, dx, dw, db, ws)
        outs.append((dx, dw, db))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


# ------------------------------------------------------------------ few groups, long contractions

@pytest.mark.parametrize("sizes,K,F", [
    ([9, 8], 4104, 72), ([0, 5, 0, 16, 1, 9, 0, 0], 2056, 136), ([40, 1, 0, 7], 8200, 64)])
def test_grouped_few_rows_long_contraction(moe, sizes, K, F):
    """Few rows a group and few tiles: the contraction is cut into ranges."""
    for seed in (11, 12):
        check_grouped_forward(moe, sizes, K, F, before=seed % 2, after=2, seed=seed,
                              y_dtype=("bf16", "f32")[seed % 2])
        check_grouped_backward(moe, sizes, F, K, before=seed % 2, after=2, want=("dx",), seed=seed)
        check_grouped_backward(moe, sizes, F, K, seed=seed)


def test_binding_refuses_rows_of_another_length(moe):
    """A transposed weight, and other tensors of the right size in rows of
    another length; batched and flat tensors and rows in parts (heads) are the
    same memory and pass."""
    z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    f = torch.float32
    T, K, F, E = 8, 64, 72, 3
    cfg = moe.make_linear_config(T, K, F, activation="relu")
    ws = moe.alloc_linear_workspace(cfg)
    fwd = dict(x=z(T, K), w=z(F, K), bias=z(F, d=f), residual=z(T, F), y=z(T, F), z=z(T, F))
    bwd = dict(dy=z(T, F), z=z(T, F), x=z(T, K), w=z(F, K), dz=z(T, F), dx=z(T, K),
               dw=z(F, K, d=f), dbias=z(F, d=f))
    for call, ok in ((moe.moe_linear_forward, fwd), (moe.moe_linear_backward, bwd)):
        call(cfg, *ok.values(), ws)
        call(cfg, *[t.view(-1) for t in ok.values()], ws)
        call(cfg, *[t.unflatten(0, (2, -1)) for t in ok.values()], ws)
        call(cfg, *[t.unflatten(-1, (4, -1)) for t in ok.values()], ws)
        for name, t in ok.items():
            if t.dim() == 2:
                with pytest.raises(ValueError, match=f"{name} has shape .*expected rows of"):
                    call(cfg, *{**ok, name: t.view(t.shape[1], t.shape[0])}.values(), ws)
    gc = moe.make_grouped_config(T, E, K, F)
    gws = moe.alloc_grouped_workspace(gc)
    off = z(E + 1, d=torch.int32)
    gf = dict(x=z(T, K), row_ids=None, offsets=off, w=z(E, F, K), bias=z(E, F, d=f), y=z(T, F))
    gb = dict(dy=z(T, F), x=z(T, K), row_ids=None, offsets=off, w=z(E, F, K), dx=z(T, K),
              dw=z(E, F, K, d=f), dbias=z(E, F, d=f))
    for call, ok in ((moe.moe_grouped_forward, gf), (moe.moe_grouped_backward, gb)):
        call(gc, *ok.values(), gws)
        for name, t in ok.items():
            if name not in ("row_ids", "offsets"):
                with pytest.raises(ValueError, match=f"{name} has shape .*expected rows of"):
                    bad = t.transpose(-1, -2).contiguous()
                    call(gc, *{**ok, name: bad}.values(), gws)
    sc = moe.make_swiglu_config(T, K)
    for call, n in ((moe.moe_swiglu_forward, 2), (moe.moe_swiglu_backward, 0)):
        args = [z(T, K) for _ in range(3 if n else 6)]
        call(sc, *args)
        args[n] = z(K, T)
        with pytest.raises(ValueError, match="expected rows of"):
            call(sc, *args)
