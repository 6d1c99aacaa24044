"""Linear and grouped products of block-scaled e4m3 codes against plain 64-bit
forms, element by element, with bounds by arithmetic (tests/fp8_util.py)."""
import itertools

import pytest
import torch

from tests import fp8_util as fu
from tests import gpu_util as gu
from tests import product_util as pu
from tests.product_util import Guarded, bf16, f32, half, inp, within

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


def sum_bound(xc, xs, wc, ws, y_dtype):
    """Bound of the products' sums before any rounding, and the sums in 64 bits."""
    xc, xs, wc, ws = (t.cuda() for t in (xc, xs, wc, ws))
    x, w = fu.values(xc, xs, 1), fu.values(wc, ws, fu.BLOCK)
    err = fu.exact_bound(x.shape[1], x.abs() @ w.abs().t())
    if y_dtype == "bf16":
        err = err + fu.cut_bound(xc, xs, wc, ws)
    return x @ w.t(), err


def check_linear(moe, T, K, F, act="none", y_dtype="bf16", bias=True, residual=True, keep_z=True,
                 seed=0, close=None):
    xc, xs = fu.random_codes(T, K, 1, seed)
    wc, ws = fu.random_codes(F, K, fu.BLOCK, seed + 1, K ** -0.5)
    b = f32(F, seed=seed + 2) if bias else None
    r = bf16(T, F, seed=seed + 3) if residual else None
    cfg = moe.make_linear_config(T, K, F, activation=act, y_dtype=y_dtype)
    work = moe.alloc_linear_fp8_workspace(cfg)
    work.fill_(0xFF)  # NaN as fp32
    y = Guarded(shape=(T, F), dtype=DT[y_dtype])
    z = Guarded(shape=(T, F), dtype=torch.bfloat16) if keep_z else None
    moe.moe_linear_forward_fp8(cfg, fu.codes_in(xc), inp(xs), fu.codes_in(wc), inp(ws), inp(b),
                               inp(r), y.t, z.t if z else None, work)
    torch.cuda.synchronize()
    zd, zerr = sum_bound(xc, xs, wc, ws, y_dtype)
    if bias:
        zd = zd + b.cuda().double()
        zerr = zerr + 2.0 ** -23 * (zd.abs() + b.cuda().double().abs())
    if keep_z:
        within(z.check(), zd, (1 + pu.BF16_HALF) * zerr + pu.BF16_HALF * zd.abs(), "z")
    yd = pu.act(zd, act)
    err = pu.MAX_SLOPE[act] * zerr + pu.act_err(zd, act)
    if residual:
        yd = yd + r.cuda().double()
        err = err + 2.0 ** -23 * yd.abs()
    h = half(DT[y_dtype])
    got = y.check()
    within(got, yd, (1 + h) * err + h * yd.abs(), "y")
    # and in the 2-norm: of normal values, 1/sqrt(3) of half a step of a rounding
    # to bf16 (uniform errors: 2^-8 / sqrt 3 of the values, at most) and 1e-4
    # beside it; fp32 1e-5
    off = ((got.cuda().double() - yd).norm() / yd.norm()).item()
    assert off <= (2.0 ** -8 / 3 ** 0.5 + 1e-4 if y_dtype == "bf16" else 1e-5), off


LINEAR = [(1, 16, 8), (1, 4096, 1280), (2, 80, 4096), (5, 272, 200), (16, 1280, 72), (17, 64, 136),
          (33, 4096, 64), (64, 528, 264), (65, 128, 712), (130, 1296, 320), (257, 192, 1288),
          (300, 2064, 136), (777, 336, 1032), (1025, 80, 264), (2100, 144, 520), (40, 11264, 256)]


@pytest.mark.parametrize("y_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,F", LINEAR)
def test_linear_sizes(moe, T, K, F, y_dtype):
    check_linear(moe, T, K, F, y_dtype=y_dtype)


# Sizes at which an MI355X's launches take each tile shape, contraction split and
# cut of the last round's tiles, for both types of y; and more than 64 blocks a row.
@pytest.mark.parametrize("y_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,F", [
    (1500, 144, 4096), (5000, 528, 4200), (4100, 528, 4104), (4100, 272, 1032), (1000, 4096, 2056),
    (4100, 144, 1032), (9000, 4096, 72), (2100, 8208, 72), (600, 4112, 72), (300, 16400, 264),
    (2048, 9232, 1024), (4224, 8336, 4096), (260, 12304, 2048)])
def test_linear_shapes(moe, T, K, F, y_dtype):
    check_linear(moe, T, K, F, "silu", y_dtype, keep_z=False, seed=7)


@pytest.mark.parametrize("act,y_dtype", itertools.product(pu.MAX_SLOPE, ("bf16", "f32")))
@pytest.mark.parametrize("T,K,F", [(3, 512, 264), (150, 144, 200)])
def test_linear_activations(moe, T, K, F, act, y_dtype):
    check_linear(moe, T, K, F, act, y_dtype, residual=y_dtype == "bf16", seed=5)


@pytest.mark.parametrize("bias,residual,keep_z", itertools.product((False, True), repeat=3))
def test_linear_optional_operands(moe, bias, residual, keep_z):
    check_linear(moe, 40, 144, 72, "gelu", "bf16", bias, residual, keep_z, seed=9)
    check_linear(moe, 700, 144, 2056, "silu", "f32", bias, residual, keep_z, seed=9)


# Whole numbers: codes of small integers and scales of powers of two, so that
# every sum is exact, on the native path too (no product lies 2^-13 below its
# neighbours), and a lost or doubled block, row or scale shows.
@pytest.mark.parametrize("y_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,F", LINEAR + [(300, 16400, 264), (4224, 1040, 4096), (9000, 1296, 72),
                                            (2048, 9232, 1024)])
def test_linear_whole_numbers(moe, T, K, F, y_dtype):
    g = torch.Generator().manual_seed(T + K)
    kb, fb = fu.blocks(K), fu.blocks(F)
    # x: +-1, one in every 16 columns; w: -2 .. 2; scales 1, 2 and 1, 2, 4: a sum's
    # magnitude stays a whole number that bf16 may round, so y is compared with
    # the rounded sum
    x = torch.zeros(T, K)
    at = torch.randint(0, 16, (T, K // 16), generator=g) + 16 * torch.arange(K // 16)
    x.scatter_(1, at, torch.randint(0, 2, (T, K // 16), generator=g).float() * 2 - 1)
    w = torch.randint(-2, 3, (F, K), generator=g).float()
    xs = torch.randint(0, 2, (T, kb), generator=g).float().exp2()
    ws = torch.randint(0, 3, (fb, kb), generator=g).float().exp2()
    xc, wc = (t.to(torch.float8_e4m3fn).view(torch.uint8) for t in (x, w))
    cfg = moe.make_linear_config(T, K, F, y_dtype=y_dtype)
    work = moe.alloc_linear_fp8_workspace(cfg)
    work.fill_(0xFF)
    y = torch.empty(T, F, dtype=DT[y_dtype], device="cuda")
    moe.moe_linear_forward_fp8(cfg, fu.codes_in(xc), xs.cuda(), fu.codes_in(wc), ws.cuda(), None,
                               None, y, None, work)
    want = fu.values(xc.cuda(), xs.cuda(), 1) @ fu.values(wc.cuda(), ws.cuda(), fu.BLOCK).t()
    assert torch.equal(y, want.to(DT[y_dtype]))


# ------------------------------------------------------------------ grouped

def check_grouped(moe, sizes, K, F, x_rows=None, row_div=1, y_dtype="bf16", bias=True, tail=0,
                  before=0, seed=0):
    """Groups of these sizes; `before` and `tail` rows belong to no group."""
    E, P = len(sizes), before + sum(sizes) + tail
    off = before + torch.cat([torch.zeros(1, dtype=torch.long), torch.tensor(sizes).cumsum(0)])
    g = torch.Generator().manual_seed(seed)
    gather = x_rows is not None
    xr = x_rows if gather else P
    xc, xs = fu.random_codes(xr, K, 1, seed)
    wc, ws = zip(*(fu.random_codes(F, K, fu.BLOCK, seed + 2 + e, K ** -0.5) for e in range(E)))
    wc, ws = torch.stack(wc), torch.stack(ws)
    b = f32(E, F, seed=seed + 1) if bias else None
    ids = None
    src = torch.arange(P)
    if gather:
        ids = torch.randint(0, max(1, xr * row_div), (P,), generator=g, dtype=torch.int32)
        if P > 4:  # sources outside x read as zeros
            ids[1], ids[P // 2] = -1, xr * row_div
        src = torch.where((ids >= 0) & (ids < xr * row_div), ids // row_div, -1).long()
    cfg = moe.make_grouped_config(P, E, K, F, x_rows=xr, row_div=row_div, y_dtype=y_dtype)
    work = moe.alloc_grouped_fp8_workspace(cfg)
    work.fill_(0xFF)
    y = Guarded(shape=(P, F), dtype=DT[y_dtype])
    moe.moe_grouped_forward_fp8(cfg, fu.codes_in(xc), inp(xs), inp(ids), inp(off.to(torch.int32)),
                                fu.codes_in(wc), inp(ws), inp(b), y.t, work)
    torch.cuda.synchronize()
    got = y.check()
    h = half(DT[y_dtype])
    for e in range(E):
        i, j = int(off[e]), int(off[e + 1])
        if i == j:
            continue
        have = src[i:j] >= 0
        if xr:
            want, err = sum_bound(xc[src[i:j].clamp(min=0)], xs[src[i:j].clamp(min=0)], wc[e], ws[e],
                                  y_dtype)
            want, err = want * have.cuda()[:, None], err * have.cuda()[:, None]
        else:
            want = torch.zeros(j - i, F, dtype=torch.double, device="cuda")
            err = want
        if bias:
            want = want + b[e].cuda().double()
            err = err + 2.0 ** -23 * (want.abs() + b[e].cuda().double().abs())
        within(got[i:j], want, (1 + h) * err + h * want.abs(), f"group {e}")
    assert (got[:before] == pu.SENTINEL).all() and (got[P - tail:] == pu.SENTINEL).all()


RAGGED = [[3, 0, 1, 9], [16, 17], [0, 0, 5], [64, 1, 63, 0, 65, 128], [200, 0, 31, 500, 7],
          [1] * 40, [300, 260, 190, 130, 70, 10, 600], [1100, 3, 900]]


@pytest.mark.parametrize("y_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sizes", RAGGED, ids=[f"groups{len(s)}rows{sum(s)}" for s in RAGGED])
def test_grouped_ragged(moe, sizes, y_dtype):
    check_grouped(moe, sizes, 272, 200, y_dtype=y_dtype)
    check_grouped(moe, sizes, 1296, 136, x_rows=50, row_div=3, y_dtype=y_dtype, tail=5, before=2)


@pytest.mark.parametrize("y_dtype", ["bf16", "f32"])
def test_grouped_large_tiles(moe, y_dtype):
    """Enough rows for 256-row tiles, with every remainder of a group (64, 128, 192
    and 256 rows), gathered and not."""
    sizes = [2048 + 64, 2048 + 100, 2048 + 190, 2048 + 255, 4096, 0, 1, 777]
    check_grouped(moe, sizes, 400, 1032, y_dtype=y_dtype, bias=False, tail=3)
    check_grouped(moe, sizes, 1040, 520, x_rows=1500, row_div=8, y_dtype=y_dtype)


def test_grouped_empty_x_and_many_groups(moe):
    check_grouped(moe, [4, 0, 9], 128, 72, x_rows=0, row_div=2)
    check_grouped(moe, [700, 300], 128, 72, x_rows=0, row_div=2, y_dtype="f32")
    check_grouped(moe, [1, 0, 2, 0] * 256, 80, 24)
    check_grouped(moe, [0] * 1000 + [3, 40], 80, 24, y_dtype="f32")


def test_grouped_offsets_are_clamped(moe):
    P, E, K, F = 50, 3, 144, 72
    xc, xs = fu.random_codes(P, K)
    parts = [fu.random_codes(F, K, 128, e + 1) for e in range(E)]
    wc, ws = (torch.stack(v).cuda() for v in zip(*parts))
    cfg = moe.make_grouped_config(P, E, K, F)
    work = moe.alloc_grouped_fp8_workspace(cfg)
    ys = [torch.zeros(P, F, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for y, off in zip(ys, ([0, 20, 30, 50], [-7, 20, 30, 2 ** 31 - 1])):
        moe.moe_grouped_forward_fp8(cfg, xc.cuda(), xs.cuda(), None,
                                    torch.tensor(off, dtype=torch.int32).cuda(), wc, ws, None, y, work)
    assert torch.equal(*ys) and ys[0].abs().sum() > 0


def test_weights_beyond_32_bits(moe):
    """The last of 600 groups lies behind 4 GB of codes."""
    E, K, F = 600, 4096, 2048
    off = torch.zeros(E + 1, dtype=torch.int32)
    P = 300
    off[1:], off[E] = 40, P  # rows 0 .. 39 in the first group, the rest in the last
    wc = torch.zeros(E, F, K, dtype=torch.uint8, device="cuda")
    ws = torch.ones(E, F // 128, K // 128, device="cuda")
    parts = {}
    for e in (0, E - 1):
        c, s = fu.random_codes(F, K, 128, e)
        parts[e] = c, s
        wc[e], ws[e] = c.cuda(), s.cuda()
    xc, xs = fu.random_codes(P, K)
    for y_dtype in ("bf16", "f32"):
        cfg = moe.make_grouped_config(P, E, K, F, y_dtype=y_dtype)
        y = torch.empty(P, F, dtype=DT[y_dtype], device="cuda")
        moe.moe_grouped_forward_fp8(cfg, xc.cuda(), xs.cuda(), None, off.cuda(), wc, ws, None, y,
                                    moe.alloc_grouped_fp8_workspace(cfg))
        for e, (i, j) in {0: (0, 40), E - 1: (40, P)}.items():
            want, err = sum_bound(xc[i:j], xs[i:j], *parts[e], y_dtype)
            within(y[i:j], want, 1.01 * err + half(DT[y_dtype]) * want.abs(), f"group {e}")


# ------------------------------------------------------------------ special values, use

@pytest.mark.parametrize("T", [3, 60, 700])
@pytest.mark.parametrize("y_dtype", ["bf16", "f32"])
def test_nan_codes_reach_their_row_and_column_only(moe, T, y_dtype):
    K, F = 400, 264
    xc, xs = fu.random_codes(T, K)
    wc, ws = fu.random_codes(F, K, 128, 1)
    xc[1, 130], wc[200, 7] = 0x7F, 0xFF
    xs[2, 1] = float("nan")
    cfg = moe.make_linear_config(T, K, F, y_dtype=y_dtype)
    y = torch.empty(T, F, dtype=DT[y_dtype], device="cuda")
    moe.moe_linear_forward_fp8(cfg, xc.cuda(), xs.cuda(), wc.cuda(), ws.cuda(), None, None, y, None,
                               moe.alloc_linear_fp8_workspace(cfg))
    want = torch.zeros(T, F, dtype=torch.bool)
    want[1:3], want[:, 200] = True, True
    assert torch.equal(torch.isnan(y.cpu()), want)


def test_input_gradient_through_transposed_codes(moe):
    """dx = dy W in codes is the same product with W's codes transposed: a block of
    128 x 128 keeps its scale."""
    T, K, F = 150, 272, 400
    dyc, dys = fu.random_codes(T, F, 1, 1)
    w = bf16(F, K, seed=2)
    wc = torch.empty(F, K, dtype=torch.uint8, device="cuda")
    ws = torch.empty(fu.blocks(F), fu.blocks(K), device="cuda")
    moe.moe_quantize_weight(w.cuda(), wc, ws)
    cfg = moe.make_linear_config(T, F, K, y_dtype="f32")
    dx = torch.empty(T, K, device="cuda")
    moe.moe_linear_forward_fp8(cfg, dyc.cuda(), dys.cuda(), wc.t().contiguous(), ws.t().contiguous(),
                               None, None, dx, None, moe.alloc_linear_fp8_workspace(cfg))
    dy, wv = fu.values(dyc.cuda(), dys.cuda(), 1), fu.values(wc, ws, 128)
    within(dx, dy @ wv, 1.01 * fu.exact_bound(F, dy.abs() @ wv.abs()), "dx")


@pytest.mark.parametrize("T,K,F", [(1, 4096, 512), (64, 1296, 264), (1000, 4096, 2056),
                                   (4100, 528, 1032)])
def test_graph_replays_streams_and_repeats(moe, T, K, F):
    cfg = moe.make_linear_config(T, K, F, activation="silu")
    xc, xs = (t.cuda() for t in fu.random_codes(T, K))
    wc, ws = (t.cuda() for t in fu.random_codes(F, K, 128, 1))
    work = [moe.alloc_linear_fp8_workspace(cfg) for _ in range(3)]
    ys = [torch.zeros(T, F, dtype=torch.bfloat16, device="cuda") for _ in range(3)]

    def call(i, c=xc):
        moe.moe_linear_forward_fp8(cfg, c, xs, wc, ws, None, None, ys[i], None, work[i])

    call(0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(2)
    torch.cuda.synchronize()
    assert torch.equal(ys[0], ys[2])
    for seed in (0, 5, 6):
        xc.copy_(fu.random_codes(T, K, 1, seed)[0])
        work[1].fill_(0xFF)
        g.replay()
        call(0)
        torch.cuda.synchronize()
        assert torch.equal(ys[0], ys[1])


def test_refused_tensors(moe):
    T, K, F = 8, 144, 72
    cfg = moe.make_linear_config(T, K, F)
    xc, xs = (t.cuda() for t in fu.random_codes(T, K))
    wc, ws = (t.cuda() for t in fu.random_codes(F, K, 128, 1))
    y = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
    work = moe.alloc_linear_fp8_workspace(cfg)
    good = [xc, xs, wc, ws, None, None, y, None, work]
    bad = [(0, xc.cpu(), ValueError), (0, xc.short(), TypeError), (0, xc[:4], ValueError),
           (1, xs[:, :1], ValueError), (1, xs.half(), TypeError), (2, wc.t(), ValueError),
           (3, ws.t().reshape(-1)[:1], ValueError), (4, y[0], TypeError), (6, y.float(), TypeError),
           (8, None, ValueError)]
    for i, t, err in bad:
        args = list(good)
        args[i] = t
        with pytest.raises(err):
            moe.moe_linear_forward_fp8(cfg, *args)
    args = list(good)
    args[8] = torch.empty(4, dtype=torch.uint8, device="cuda")
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.moe_linear_forward_fp8(cfg, *args)
    # (float8_e4m3fn tensors are codes as well)
    args = list(good)
    args[0], args[2] = xc.view(torch.float8_e4m3fn), wc.view(torch.float8_e4m3fn)
    moe.moe_linear_forward_fp8(cfg, *args)
    torch.cuda.synchronize()
