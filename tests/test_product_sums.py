"""Long sums of the gradients, exactly: with entries of 1 and 2 in size every
sum is a whole number below 2^24, so that fp32 in any order gives it exactly,
and a row, a strip of rows or a contraction range that is lost, or taken
twice, shows in every sum that it belongs to (the bounds of rounded sums grow
faster with the rows than one row's share)."""
import itertools

import pytest
import torch

from tests import gpu_util as gu
from tests.product_cases import FORWARD, INPUT, PAIRS, WAYS, WEIGHT

gpu = pytest.mark.gpu


@pytest.fixture
def moe(request):
    gu.note(f"[gpu-test] {request.node.nodeid}")
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import sparse_moe_layer_fp32_amd as m
    m.load_library()
    return m


def whole(*shape, seed):
    """-2, -1, 1 or 2."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(0, 4, shape, generator=g, dtype=torch.int8)
    return (v - 2 + (v >= 2)).to(torch.bfloat16)


def case(T, K, F, relu, seed=0):
    dy, x, z = whole(T, F, seed=seed), whole(T, K, seed=seed + 1), whole(T, F, seed=seed + 2)
    return dy, x, z if relu else None


def sums(dy, x, z):
    """dw and db, exact in 64 bits."""
    dz = dy.double() if z is None else dy.double() * (z > 0)
    return dz.t() @ x.double(), dz.sum(0)


# rows x in features -> out features, relu in front or none: strips of 64 and
# 128 rows of the activation; one to 512 contraction ranges
STRIPS = [(66000, 8, 136), (16400, 8, 1032), (1000, 8, 264), (65, 8, 520), (64, 8, 520)]
RANGES = [(65536, 64, 64), (65537, 8, 8), (300_001, 8, 16), (16384, 256, 64), (40_000, 136, 72),
          (66_000, 1032, 64), (70_000, 1288, 128), (9000, 72, 72), (9000, 264, 2056),
          (9000, 520, 1032), (1500, 72, 72), (600, 8, 8), (5, 8, 8)]


@pytest.mark.parametrize("T,K,F,relu", [(*s, True) for s in STRIPS] +
                         [(*s, False) for s in RANGES if s[0] * s[2] < 3_000_000])
def test_a_lost_row_or_strip_shows(T, K, F, relu):
    """On the CPU, in the oracle: without one row, one strip or one range, or
    with one taken twice, the sums differ."""
    dy, x, z = case(T, K, F, relu)
    dw, db = sums(dy, x, z)
    assert dw.abs().max() < 2 ** 24 and db.abs().max() < 2 ** 24
    for a, b in ((0, 1), (T - 1, T), (T // 2, T // 2 + 1), (T // 3, min(T, T // 3 + 64)),
                 (T - T // 8, T), (0, max(1, T // 512))):
        if a >= b:
            continue
        part = sums(dy[a:b], x[a:b], None if z is None else z[a:b])
        lost_w, lost_b = (part[0] != 0).double().mean(), (part[1] != 0).double().mean()
        assert lost_w > 0.3 and lost_b > 0.3, (a, b)  # of the elements change


def run(moe, dy, x, z, accumulate=False, want=("dw", "db")):
    T, F, K = dy.shape[0], dy.shape[1], x.shape[1]
    cfg = moe.make_linear_config(T, K, F, activation="none" if z is None else "relu",
                                 accumulate=accumulate)
    ws = moe.alloc_linear_workspace(cfg)
    ws.fill_(0xFF)
    dw = torch.full((F, K), 3.0, device="cuda") if "dw" in want else None
    db = torch.full((F,), 5.0, device="cuda") if "db" in want else None
    dz = torch.empty(T, F, dtype=torch.bfloat16, device="cuda") if z is not None else None
    moe.moe_linear_backward(cfg, dy, z, x if dw is not None else None, None, dz, None, dw, db, ws)
    return dw, db


@gpu
@pytest.mark.parametrize("accumulate", (False, True))
@pytest.mark.parametrize("T,K,F", STRIPS)
def test_strips_of_the_activation(moe, T, K, F, accumulate):
    dy, x, z = (t.cuda() for t in case(T, K, F, True))
    want_w, want_b = sums(dy, x, z)
    dw, db = run(moe, dy, x, z, accumulate)
    assert torch.equal(dw.double(), want_w + 3 * accumulate)
    assert torch.equal(db.double(), want_b + 5 * accumulate)


@gpu
@pytest.mark.parametrize("want", [("dw", "db"), ("db",), ("dw",)])
@pytest.mark.parametrize("T,K,F", RANGES)
def test_contraction_ranges(moe, T, K, F, want):
    dy, x, _ = case(T, K, F, False)
    dy, x = dy.cuda(), x.cuda()
    want_w, want_b = sums(dy, x, None)
    for accumulate in (False, True):
        dw, db = run(moe, dy, x, None, accumulate, want)
        assert dw is None or torch.equal(dw.double(), want_w + 3 * accumulate)
        assert db is None or torch.equal(db.double(), want_b + 5 * accumulate)


@gpu
@pytest.mark.parametrize("gather", (False, True))
@pytest.mark.parametrize("sizes,K,F", [
    ([70_000, 3], 64, 64), ([0, 40_000, 0, 21_111], 72, 136), ([9000, 0, 1, 130, 64], 264, 72),
    ([33_000], 8, 8)])
def test_ragged_ranges(moe, sizes, K, F, gather):
    before, after, per = 5, 9, 2
    off = [before + s for s in itertools.accumulate(sizes, initial=0)]
    P = off[-1] + after
    dy, x = whole(P, F, seed=1).cuda(), whole(P, K, seed=2).cuda()
    src, ids = torch.arange(P), None
    if gather:
        ids = torch.randperm(P, generator=torch.Generator().manual_seed(3)).to(torch.int32)
        src = ids.long() // per
    rows = x[src.cuda()].double()
    dy[:before], dy[P - after:] = float("nan"), float("nan")
    cfg = moe.make_grouped_config(P, len(sizes), K, F, x_rows=P, row_div=per if gather else 1)
    ws = moe.alloc_grouped_workspace(cfg)
    ws.fill_(0xFF)
    dw = torch.full((len(sizes), F, K), 3.0, device="cuda")
    db = torch.full((len(sizes), F), 5.0, device="cuda")
    moe.moe_grouped_backward(cfg, dy, x, ids.cuda() if gather else None,
                             torch.tensor(off, dtype=torch.int32, device="cuda"), None, None, dw,
                             db, ws)
    for e, (i, j) in enumerate(zip(off, off[1:])):
        d = dy[i:j].double()
        assert torch.equal(dw[e].double(), d.t() @ rows[i:j]), e
        assert torch.equal(db[e].double(), d.sum(0)), e


def group_offsets(P, G, seed):
    """G uneven groups, some of them empty, with rows of no group before and
    behind them where there are enough."""
    g = torch.Generator().manual_seed(seed)
    cut = torch.randint(P // 16, P - P // 32 + 1, (G + 1,), generator=g).sort().values
    return cut.to(torch.int32)


def on_gpu(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randint(0, 4, shape, generator=g, dtype=torch.int8, device="cuda")
    return (v - 2 + (v >= 2)).to(torch.bfloat16)


def check_exactly(moe, P, G, K, F, want):
    """The products named in `want` for P rows in G groups (1: the linear
    map), against the same in 64 bits, bit for bit."""
    x, w, dy = on_gpu(P, K, seed=1), on_gpu(G, F, K, seed=2), on_gpu(P, F, seed=3)
    off = group_offsets(P, G, seed=P) if G > 1 else torch.tensor([0, P], dtype=torch.int32)
    dev = off.cuda()
    bf = dict(dtype=torch.bfloat16, device="cuda")
    y = torch.full((P, F), 7.5, device="cuda") if FORWARD in want else None
    dx = torch.full((P, K), 7.5, **bf) if INPUT in want else None
    dw = torch.full((G, F, K), 7.5, device="cuda") if WEIGHT in want else None
    db = torch.full((G, F), 7.5, device="cuda") if WEIGHT in want else None
    if G > 1:
        cfg = moe.make_grouped_config(P, G, K, F, y_dtype="f32")
        ws = moe.alloc_grouped_workspace(cfg).fill_(0xFF)
        if y is not None:
            moe.moe_grouped_forward(cfg, x, None, dev, w, None, y, ws)
        if dx is not None or dw is not None:
            moe.moe_grouped_backward(cfg, dy, x, None, dev, w, dx, dw, db, ws)
    else:
        cfg = moe.make_linear_config(P, K, F, y_dtype="f32")
        ws = moe.alloc_linear_workspace(cfg).fill_(0xFF)
        if y is not None:
            moe.moe_linear_forward(cfg, x, w[0], None, None, y, None, ws)
        if dx is not None or dw is not None:
            moe.moe_linear_backward(cfg, dy, None, x, w[0], None, dx, None if dw is None else dw[0],
                                    None if db is None else db[0], ws)
    seen = torch.zeros(P, dtype=torch.bool, device="cuda")
    for e, (i, j) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        seen[i:j] = True
        xe, we, de = x[i:j].double(), w[e].double(), dy[i:j].double()
        if y is not None:
            assert torch.equal(y[i:j].double(), xe @ we.t()), ("y", e)
        if dx is not None:  # rounded once, to nearest even
            assert torch.equal(dx[i:j], (de @ we).float().bfloat16()), ("dx", e)
        if dw is not None:
            assert torch.equal(dw[e].double(), de.t() @ xe), ("dw", e)
            assert torch.equal(db[e].double(), de.sum(0)), ("db", e)
    for t in (y, dx):
        assert t is None or (t[~seen] == 7.5).all(), "a row of no group was written"


@gpu
@pytest.mark.parametrize("ragged", (False, True))
@pytest.mark.parametrize("op", (FORWARD, INPUT, WEIGHT), ids=("forward", "input", "weight"))
def test_every_way_to_run_a_product(moe, op, ragged):
    """Tile shapes, contraction ranges and slices (tests/product_cases.py)."""
    for case_ in WAYS[op, ragged]:
        gu.note(f"  shape, ranges, slices, rows, groups, in, out: {case_}")
        check_exactly(moe, *case_[3:], (op,))


@gpu
def test_every_way_to_run_both_gradients(moe):
    for case_ in PAIRS:
        gu.note(f"  dx shape, slices, dW shape, rows, groups, in, out: {case_}")
        check_exactly(moe, *case_[3:], (INPUT, WEIGHT))


@gpu
@pytest.mark.parametrize("P,G,K,F", [
    (3, 1, 65536, 8), (3, 1, 8, 65536), (300, 1, 65536, 16), (300, 1, 16, 65536), (40, 3, 65536, 8),
    (40, 3, 8, 65536), (5000, 1024, 8, 24), (900, 1024, 136, 8), (1 << 22, 1024, 8, 8)])
def test_ends_of_the_sizes(moe, P, G, K, F):
    """The most features and the most groups."""
    check_exactly(moe, P, G, K, F, (FORWARD, INPUT, WEIGHT))


@gpu
def test_the_most_rows(moe):
    """2^26 rows; sums of entries of either sign stay below 2^24 on the way."""
    T, K, F = 1 << 26, 8, 8
    x, dy, z, w = (on_gpu(n, 8, seed=i) for i, n in enumerate((T, T, T, F)))
    cfg = moe.make_linear_config(T, K, F, activation="relu", accumulate=True)
    ws = moe.alloc_linear_workspace(cfg).fill_(0xFF)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    y, zz = torch.empty(T, F, **bf), torch.empty(T, F, **bf)
    moe.moe_linear_forward(cfg, x, w, None, None, y, zz, ws)
    dz, dx = torch.empty(T, F, **bf), torch.empty(T, K, **bf)
    dw, db = torch.full((F, K), 3.0, device="cuda"), torch.full((F,), 5.0, device="cuda")
    moe.moe_linear_backward(cfg, dy, z, x, w, dz, dx, dw, db, ws)
    sw, sb = torch.full_like(dw, 3.0).double(), torch.full_like(db, 5.0).double()
    for i in range(0, T, 1 << 22):
        part = slice(i, i + (1 << 22))
        xp, zp, dyp = x[part].double(), z[part], dy[part].double()
        assert torch.equal(zz[part].double(), xp @ w.double().t())  # at most 32: exact in bf16
        assert torch.equal(y[part].double(), (xp @ w.double().t()).clamp(min=0))
        d = dyp * (zp > 0)
        assert torch.equal(dz[part].double(), d)
        assert torch.equal(dx[part].double(), d @ w.double())
        sw, sb = sw + d.t() @ xp, sb + d.sum(0)
    assert torch.equal(dw.double(), sw) and torch.equal(db.double(), sb)


@gpu
@pytest.mark.parametrize("T,K,F", [(40_000, 136, 72), (300_001, 8, 16), (600, 72, 72)])
def test_bf16_gradients_of_many_ranges(moe, T, K, F):
    """dw in bf16, added to what is there: rounded once, to nearest even."""
    dy, x = on_gpu(T, F, seed=1), on_gpu(T, K, seed=2)
    cfg = moe.make_linear_config(T, K, F, dw_dtype="bf16", accumulate=True)
    dw = torch.full((F, K), 3.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_linear_backward(cfg, dy, None, x, None, None, None, dw, None,
                            moe.alloc_linear_workspace(cfg).fill_(0xFF))
    want = dy.double().t() @ x.double() + 3
    assert torch.equal(dw, want.float().bfloat16())
