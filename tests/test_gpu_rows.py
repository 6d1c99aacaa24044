"""Rows out to the experts and back, their gradients, and block quantisation,
against plain 64-bit forms element by element, with bounds by arithmetic
(tests/product_util.py, tests/fp8_util.py)."""
import itertools
import math

import pytest
import torch

from tests import fp8_util as fu
from tests import gpu_util as gu
from tests import product_util as pu
from tests.product_util import Guarded, half, sum_err, within

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


def rand(*shape, dtype=torch.bfloat16, scale=1.0, seed=0):
    return (pu.f32(*shape, scale=scale, seed=seed)).to(dtype)


def positions(T, k, rows, seed=0, none=()):
    """pair_pos: different rows for all pairs that have one, in random order;
    values outside [0, rows) of every kind for the others, and for all pairs of
    the tokens in `none`."""
    g = torch.Generator().manual_seed(seed)
    pos = torch.full((T * k,), -1, dtype=torch.int64)
    have = torch.randperm(T * k, generator=g)[:min(rows, T * k)]
    pos[have] = torch.randperm(rows, generator=g)[:len(have)]
    lost = (pos < 0).nonzero().flatten()
    wrong = torch.tensor([-1, rows, -2 ** 31, 2 ** 31 - 1, rows + 7])
    pos[lost] = wrong[torch.arange(len(lost)) % 5]
    pos = pos.view(T, k)
    for t in none:
        pos[t] = -1
    return pos


def valid(pos, rows):
    return (pos >= 0) & (pos < rows)


SIZES = [(1, 1, 8, 1), (1, 8, 4096, 8), (5, 8, 4096, 40), (3, 2, 72, 4), (7, 3, 136, 30),
         (64, 8, 264, 300), (33, 9, 520, 297), (2, 32, 512, 64), (19, 17, 256, 100),
         (130, 4, 1032, 520), (300, 3, 7168, 900), (9, 2, 64, 0), (1000, 2, 128, 1500),
         (17, 1, 65536, 17)]
TYPES = list(itertools.product(("bf16", "f32"), repeat=2))


def check_to_rows(moe, T, k, H, rows, tok="bf16", row="bf16", weights=None, seed=0, none=()):
    """dispatch_forward, or combine_backward's drows."""
    x = rand(T, H, dtype=DT[tok], seed=seed)
    pos = positions(T, k, rows, seed, none)
    cfg = moe.make_dispatch_config(T, rows, k, H, token_dtype=tok, row_dtype=row)
    out = Guarded(shape=(rows, H), dtype=DT[row])
    gpos = Guarded(pos.to(torch.int32)).t
    ok = valid(pos, rows)
    want = torch.full((rows, H), pu.SENTINEL, dtype=torch.double)
    err = torch.zeros(rows, H, dtype=torch.double)
    t = ok.nonzero()[:, 0]
    v = x.double()[t]
    if weights is None:
        moe.moe_dispatch_forward(cfg, Guarded(x).t, gpos, out.t)
    else:
        moe.moe_combine_backward(cfg, Guarded(x).t, None, gpos, Guarded(weights).t, out.t, None)
        v = v * weights.double()[ok].unsqueeze(1)
        err[pos[ok]] = 2.0 ** -24 * v.abs()
    torch.cuda.synchronize()
    want[pos[ok]] = v
    exact = weights is None and (tok == row or row == "f32")
    rounds = torch.zeros_like(want)
    if not exact:
        rounds[pos[ok]] = half(DT[row]) * v.abs()
    within(out.check(), want, 1.01 * err + rounds, "rows")


def check_from_rows(moe, T, k, H, rows, tok="bf16", row="bf16", weights=True, base=True, seed=0,
                    none=()):
    """combine_forward, or (without weights) dispatch_backward."""
    r = rand(rows, H, dtype=DT[row], seed=seed)
    w = rand(T, k, dtype=torch.float32, seed=seed + 1) if weights else None
    b = rand(T, H, dtype=DT[tok], seed=seed + 2) if base else None
    pos = positions(T, k, rows, seed, none)
    cfg = moe.make_dispatch_config(T, rows, k, H, token_dtype=tok, row_dtype=row)
    out = Guarded(shape=(T, H), dtype=DT[tok])
    gpos, gr, gb = Guarded(pos.to(torch.int32)).t, Guarded(r).t, pu.inp(b)
    if weights:
        moe.moe_combine_forward(cfg, gr, gpos, Guarded(w).t, gb, out.t)
    else:
        moe.moe_dispatch_backward(cfg, gr, gpos, gb, out.t)
    torch.cuda.synchronize()
    ok = valid(pos, rows)
    terms = torch.zeros(T, k, H, dtype=torch.double)
    terms[ok] = r.double()[pos[ok]]
    if weights:
        terms = terms * w.double().unsqueeze(2)
    want, mag = terms.sum(1), terms.abs().sum(1)
    if base:
        want, mag = want + b.double(), mag + b.double().abs()
    within(out.check(), want, 1.01 * sum_err(k, mag) + half(DT[tok]) * want.abs(), "tokens")


def check_weight_grad(moe, T, k, H, rows, tok="bf16", row="bf16", with_rows=True, seed=0, none=()):
    dy, r = rand(T, H, dtype=DT[tok], seed=seed), rand(rows, H, dtype=DT[row], seed=seed + 1)
    w = rand(T, k, dtype=torch.float32, seed=seed + 2)
    pos = positions(T, k, rows, seed, none)
    cfg = moe.make_dispatch_config(T, rows, k, H, token_dtype=tok, row_dtype=row)
    dw = Guarded(shape=(T, k), dtype=torch.float32)
    dr = Guarded(shape=(rows, H), dtype=DT[row]) if with_rows else None
    moe.moe_combine_backward(cfg, Guarded(dy).t, Guarded(r).t, Guarded(pos.to(torch.int32)).t,
                             Guarded(w).t, dr.t if dr else None, dw.t)
    torch.cuda.synchronize()
    ok = valid(pos, rows)
    terms = torch.zeros(T, k, H, dtype=torch.double)
    terms[ok] = r.double()[pos[ok]]
    terms = terms * dy.double().unsqueeze(1)
    within(dw.check(), terms.sum(2), sum_err(H, terms.abs().sum(2)), "dweights")
    if dr:
        want = torch.full((rows, H), pu.SENTINEL, dtype=torch.double)
        v = dy.double()[ok.nonzero()[:, 0]] * w.double()[ok].unsqueeze(1)
        want[pos[ok]] = v
        err = torch.zeros_like(want)
        err[pos[ok]] = (1.01 * 2.0 ** -24 + half(DT[row])) * v.abs()
        within(dr.check(), want, err, "drows")


@pytest.mark.parametrize("T,k,H,rows", SIZES)
def test_dispatch_sizes(moe, T, k, H, rows):
    check_to_rows(moe, T, k, H, rows)
    check_from_rows(moe, T, k, H, rows, weights=False, seed=3)


@pytest.mark.parametrize("T,k,H,rows", SIZES)
def test_combine_sizes(moe, T, k, H, rows):
    check_from_rows(moe, T, k, H, rows, seed=5)
    check_weight_grad(moe, T, k, H, rows, seed=7)


@pytest.mark.parametrize("tok,row", TYPES)
@pytest.mark.parametrize("H", [16, 100 * 8, 2048])
def test_types(moe, tok, row, H):
    T, k, rows = 41, 5, 150
    check_to_rows(moe, T, k, H, rows, tok, row, seed=1, none=(0, 40))
    check_to_rows(moe, T, k, H, rows, tok, row, rand(T, k, dtype=torch.float32, seed=9), seed=2)
    for base in (False, True):
        check_from_rows(moe, T, k, H, rows, tok, row, True, base, seed=3, none=(0, 40))
        check_from_rows(moe, T, k, H, rows, tok, row, False, base, seed=4, none=(0, 40))
    check_weight_grad(moe, T, k, H, rows, tok, row, True, seed=5, none=(0, 40))
    check_weight_grad(moe, T, k, H, rows, tok, row, False, seed=6)


def test_ones_for_weights_and_grid_of_many_tokens(moe):
    """combine without weights is dispatch's gradient, and the gradient without
    weights sends dy itself; many narrow tokens."""
    T, k, H, rows = 20011, 3, 24, 50000
    pos = positions(T, k, rows, 1)
    gpos = pos.to(torch.int32).cuda()
    cfg = moe.make_dispatch_config(T, rows, k, H)
    r, dy = rand(rows, H, seed=1).cuda(), rand(T, H, seed=2).cuda()
    y1, y2 = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty_like(dy)
    moe.moe_combine_forward(cfg, r, gpos, None, None, y1)
    moe.moe_dispatch_backward(cfg, r, gpos, None, y2)
    assert torch.equal(y1, y2)
    a, b = torch.zeros(rows, H, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(r)
    moe.moe_combine_backward(cfg, dy, None, gpos, None, a, None)
    moe.moe_dispatch_forward(cfg, dy, gpos, b)
    assert torch.equal(a, b)
    check_from_rows(moe, T, k, H, rows, seed=3)
    check_weight_grad(moe, T, k, H, rows, seed=4)


def test_gradients_against_differences(moe):
    """<dy, y(r + h e) - y(r - h e)> / 2h for directions e of the rows and the
    weights; fp32 throughout, y linear in each, so h has no bias."""
    T, k, H, rows = 13, 4, 136, 40
    pos = positions(T, k, rows, 3)
    gpos = pos.to(torch.int32).cuda()
    cfg = moe.make_dispatch_config(T, rows, k, H, token_dtype="f32", row_dtype="f32")
    f = lambda *s, seed: rand(*s, dtype=torch.float32, seed=seed).cuda()  # noqa: E731
    r, w, dy = f(rows, H, seed=1), f(T, k, seed=2), f(T, H, seed=3)
    er, ew = f(rows, H, seed=4), f(T, k, seed=5)

    def y(r_, w_):
        out = torch.empty(T, H, device="cuda")
        moe.moe_combine_forward(cfg, r_, gpos, w_, None, out)
        return out.double()

    dr, dw = torch.zeros(rows, H, device="cuda"), torch.empty(T, k, device="cuda")
    moe.moe_combine_backward(cfg, dy, r, gpos, w, dr, dw)
    h = 0.5
    for got, plus, minus in (((dr.double() * er.double()).sum(), y(r + h * er, w), y(r - h * er, w)),
                             ((dw.double() * ew.double()).sum(), y(r, w + h * ew), y(r, w - h * ew))):
        want = (dy.double() * (plus - minus)).sum() / (2 * h)
        # fp32 roundings of the moved operands and of y: 8 units of 2^-24 of every
        # term, over h
        scale = (dy.double().abs() * (plus.abs() + minus.abs())).sum() / (2 * h)
        assert abs(got - want) <= (k + H) * 2.0 ** -23 * scale
    # dispatch's gradient is its transpose: <dr, dispatch(x)> = <dx, x>
    x, rows_out = f(T, H, seed=6), torch.zeros(rows, H, device="cuda")
    dx = torch.empty(T, H, device="cuda")
    moe.moe_dispatch_forward(cfg, x, gpos, rows_out)
    moe.moe_dispatch_backward(cfg, r, gpos, None, dx)
    a, b = (r.double() * rows_out.double()).sum(), (dx.double() * x.double()).sum()
    assert abs(a - b) <= k * 2.0 ** -23 * (r.double() * rows_out.double()).abs().sum()


def test_infinities_and_nan_stay_where_they_are(moe):
    """A NaN row reaches only the tokens that name it; rows without a pair are not
    read."""
    T, k, H, rows = 6, 2, 264, 20
    pos = torch.arange(T * k).view(T, k)  # rows 12 .. 19 have no pair
    r = rand(rows, H, seed=1)
    r[12:] = math.nan
    r[3], r[7, 5] = math.nan, math.inf
    cfg = moe.make_dispatch_config(T, rows, k, H)
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(T, k, device="cuda")
    gpos = pos.to(torch.int32).cuda()
    moe.moe_combine_forward(cfg, r.cuda(), gpos, w, None, y)
    bad = ~torch.isfinite(y.cpu().float())
    want = torch.zeros(T, H, dtype=torch.bool)
    want[1], want[3, 5] = True, True
    assert torch.equal(bad, want)
    dw = torch.empty(T, k, device="cuda")
    pos[0, 0] = 12
    gpos[0, 0] = -1  # a pair without a row: weight gradient 0 though all unnamed rows are NaN
    moe.moe_combine_backward(cfg, rand(T, H, seed=2).cuda(), r.cuda(), gpos, w, None, dw)
    assert dw[0, 0] == 0 and torch.isnan(dw[1, 1])
    assert int(torch.isfinite(dw).sum()) == T * k - 2


def test_offsets_beyond_32_bits(moe):
    """Rows at 4 and 8 GB, in both directions and in codes."""
    H, rows = 4096, 2 ** 20 + 5
    T, k = 3, 2
    pos = torch.tensor([[rows - 1, 0], [2 ** 19 + 1, 2 ** 18], [rows - 2, -1]])
    gpos = pos.to(torch.int32).cuda()
    cfg = moe.make_dispatch_config(T, rows, k, H)
    big = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda")
    x = rand(T, H, seed=1).cuda()
    moe.moe_dispatch_forward(cfg, x, gpos, big)
    for t, j in itertools.product(range(T), range(k)):
        if pos[t, j] >= 0:
            assert torch.equal(big[pos[t, j]], x[t])
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    w = torch.tensor([[1.0, 1.0], [0.5, 0.25], [2.0, 1.0]], device="cuda")
    moe.moe_combine_forward(cfg, big, gpos, w, None, y)
    scale = torch.tensor([2.0, 0.75, 2.0], device="cuda").unsqueeze(1)
    assert torch.equal(y, (x.float() * scale).to(torch.bfloat16))
    dw = torch.empty(T, k, device="cuda")
    moe.moe_combine_backward(cfg, x, big, gpos, w, big, dw)
    assert torch.equal(big[rows - 2], x[2] * 2) and dw[2, 1] == 0
    del big
    codes = torch.empty(rows, H, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, H // 128, device="cuda")
    q = moe.make_quantize_config(T, H, rows=rows, top_k=k)
    moe.moe_quantize_rows(q, x, gpos, codes, scales)
    want = fu.encode(x.cpu())
    for t, j in itertools.product(range(T), range(k)):
        if pos[t, j] >= 0:
            check_codes(codes[pos[t, j]][None].cpu(), scales[pos[t, j]][None].cpu(), x[t:t + 1].cpu(), 1)
    assert want[0].shape == (T, H)


# ------------------------------------------------------------------ quantisation

def check_codes(codes, scales, x, rows):
    """Scales to a fp32 rounding; every code the nearest to v 448 / a, with the
    fp32 roundings of 448 / a and of the product (2^-24 each) allowed for."""
    n, k = x.shape
    a = fu.block_max(x.double(), rows).clamp(min=fu.LEAST)
    assert ((scales.double() - a / 448).abs() <= 2.0 ** -24 * a / 448).all()
    v = x.double() * 448 / fu.spread(a, rows, n, k)
    got = fu.decode(codes)
    step = torch.exp2(torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent.double() - 4)
    within(got, v, step / 2 + 2.0 ** -22 * v.abs(), "codes")
    # and where v is clear of a border, exactly torch's conversion
    want = v.float().to(torch.float8_e4m3fn).float().double()
    near = ((v / step - torch.floor(v / step)) - 0.5).abs() < 1e-5
    assert torch.equal(got[~near], want[~near])


COLS = [(1, 16), (1, 4096), (3, 128), (5, 144), (7, 272), (130, 1280), (33, 1296), (9, 528),
        (2, 11264), (65, 2064), (1000, 48), (3, 65536)]


@pytest.mark.parametrize("T,K", COLS)
def test_quantize_rows(moe, T, K):
    x = rand(T, K, seed=T) * torch.exp2(torch.randint(-8, 9, (T, 1)).float()).bfloat16()
    codes = fu.Bytes(shape=(T, K))
    scales = Guarded(shape=(T, fu.blocks(K)), dtype=torch.float32)
    moe.moe_quantize_rows(moe.make_quantize_config(T, K), Guarded(x).t, None, codes.t, scales.t)
    torch.cuda.synchronize()
    check_codes(codes.check(), scales.check(), x, 1)


@pytest.mark.parametrize("T,k,K,rows", [(1, 8, 4096, 8), (5, 3, 144, 11), (40, 32, 1296, 600),
                                        (300, 2, 48, 500), (7, 4, 512, 0), (66, 8, 1280, 528)])
def test_quantize_out_to_rows(moe, T, k, K, rows):
    x = rand(T, K, seed=T)
    pos = positions(T, k, rows, T)
    codes = fu.Bytes(shape=(rows, K))
    scales = Guarded(shape=(rows, fu.blocks(K)), dtype=torch.float32)
    moe.moe_quantize_rows(moe.make_quantize_config(T, K, rows=rows, top_k=k), Guarded(x).t,
                          Guarded(pos.to(torch.int32)).t, codes.t, scales.t)
    torch.cuda.synchronize()
    c, s, ok = codes.check(), scales.check(), valid(pos, rows)
    at = pos[ok]
    check_codes(c[at], s[at], x[ok.nonzero()[:, 0]], 1)
    left = torch.ones(rows, dtype=torch.bool)
    left[at] = False
    assert (c[left] == codes.SENTINEL).all() and (s[left] == pu.SENTINEL).all()


@pytest.mark.parametrize("G,F,K", [(1, 8, 16), (1, 128, 128), (3, 200, 144), (2, 1280, 528),
                                   (5, 136, 1296), (1, 1, 4096), (40, 64, 64)])
def test_quantize_weight(moe, G, F, K):
    w = rand(G, F, K, scale=K ** -0.5, seed=G + F)
    codes = fu.Bytes(shape=(G, F, K))
    scales = Guarded(shape=(G, fu.blocks(F), fu.blocks(K)), dtype=torch.float32)
    moe.moe_quantize_weight(Guarded(w).t, codes.t, scales.t)
    torch.cuda.synchronize()
    c, s = codes.check(), scales.check()
    for g in range(G):
        check_codes(c[g], s[g], w[g], 128)
    if G == 1:  # a matrix by itself
        one = torch.empty(F, K, dtype=torch.float8_e4m3fn, device="cuda")
        moe.moe_quantize_weight(w[0].cuda(), one, scales.t)
        assert torch.equal(one.cpu().view(torch.uint8), c[0])


def test_quantize_extremes(moe):
    """Blocks of zeros, of the smallest and largest numbers, with infinities and
    NaN; each block on its own."""
    K = 128 * 8
    x = torch.zeros(2, K, dtype=torch.bfloat16)
    big = torch.finfo(torch.bfloat16).max
    x[0, 128:256] = big
    x[0, 256:384] = 2.0 ** -133           # the smallest subnormal
    x[0, 300] = 1.0                       # beside an ordinary value
    x[0, 384:512] = -2.0 ** -120          # a block of tiny numbers only
    x[0, 512:640], x[0, 520] = 1.0, math.nan
    x[0, 640:768], x[0, 641] = 2.0, -math.inf
    x[0, 768:896] = -0.0
    x[0, 896:] = 3.0
    x[1] = 1.0
    codes = torch.empty(2, K, dtype=torch.uint8, device="cuda")
    scales = torch.empty(2, 8, device="cuda")
    moe.moe_quantize_rows(moe.make_quantize_config(2, K), x.cuda(), None, codes, scales)
    c, s = fu.decode(codes.cpu()).view(2, 8, 128), scales.cpu().double()
    least = 2.0 ** -90 / 448
    assert (c[0, 0] == 0).all() and abs(s[0, 0] / least - 1) < 2.0 ** -23
    assert (c[0, 1] == 448).all() and abs(s[0, 1] / (big / 448) - 1) < 2.0 ** -23
    assert c[0, 2, 44] == 448 and (c[0, 2] == 0).sum() == 127
    assert (c[0, 3] == 0).all() and abs(s[0, 3] / least - 1) < 2.0 ** -23
    assert torch.isnan(s[0, 4]) and s[0, 5] == math.inf
    for b in (4, 5):  # no value of such a block is finite
        assert not torch.isfinite(c[0, b] * s[0, b]).any()
    assert (c[0, 6] == 0).all() and (c[0, 7] == 448).all()
    assert (c[1] == 448).all() and ((s[1] * 448 - 1).abs() < 2.0 ** -22).all()


# ------------------------------------------------------------------ use

def test_graph_replays_and_streams(moe):
    """All calls captured in one graph and replayed with eager work between, and
    the same on a side stream, bit for bit."""
    T, k, H = 200, 4, 520 + 8
    rows = T * k
    pos = positions(T, k, rows, 1).to(torch.int32).cuda()
    cfg = moe.make_dispatch_config(T, rows, k, H)
    q = moe.make_quantize_config(T, H, rows=rows, top_k=k)
    x, w = rand(T, H, seed=1).cuda(), rand(T, k, dtype=torch.float32, seed=2).cuda()
    bufs = lambda: [torch.zeros(rows, H, dtype=torch.bfloat16, device="cuda"),  # noqa: E731
                    torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"),
                    torch.zeros(rows, H, dtype=torch.bfloat16, device="cuda"),
                    torch.zeros(T, k, device="cuda"),
                    torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"),
                    torch.zeros(rows, H, dtype=torch.uint8, device="cuda"),
                    torch.zeros(rows, fu.blocks(H), device="cuda")]

    def calls(b):
        moe.moe_dispatch_forward(cfg, x, pos, b[0])
        moe.moe_combine_forward(cfg, b[0], pos, w, x, b[1])
        moe.moe_combine_backward(cfg, b[1], b[0], pos, w, b[2], b[3])
        moe.moe_dispatch_backward(cfg, b[2], pos, None, b[4])
        moe.moe_quantize_rows(q, x, pos, b[5], b[6])

    eager, graphed, side = bufs(), bufs(), bufs()
    calls(eager)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls(graphed)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls(side)
    torch.cuda.synchronize()
    for seed in (1, 3, 5):
        x.copy_(rand(T, H, seed=seed))
        calls(eager)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, graphed):
            assert torch.equal(a, b)
        if seed == 1:
            for a, b in zip(eager, side):
                assert torch.equal(a, b)


def test_refused_tensors(moe):
    T, k, H, rows = 8, 2, 64, 16
    cfg = moe.make_dispatch_config(T, rows, k, H)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    r = torch.zeros(rows, H, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    w = torch.ones(T, k, device="cuda")
    for bad, err in ((x.cpu(), ValueError), (x[:4], ValueError), (x.float(), TypeError),
                     (x.t().contiguous().t(), ValueError), (None, ValueError), ([1], TypeError)):
        with pytest.raises(err):
            moe.moe_dispatch_forward(cfg, bad, pos, r)
        with pytest.raises(err):
            moe.moe_combine_forward(cfg, r, pos, w, None, bad)
    for bad, err in ((pos.long(), TypeError), (pos[:, :1], ValueError), (None, ValueError)):
        with pytest.raises(err):
            moe.moe_dispatch_backward(cfg, r, bad, None, x)
        with pytest.raises(err):
            moe.moe_combine_backward(cfg, x, r, bad, w, r, None)
    with pytest.raises(ValueError):
        moe.moe_combine_backward(cfg, x, None, pos, w, None, torch.empty(T, k, device="cuda"))
    q = moe.make_quantize_config(T, H)
    codes = torch.empty(T, H, dtype=torch.uint8, device="cuda")
    scales = torch.empty(T, 1, device="cuda")
    with pytest.raises(ValueError):
        moe.moe_quantize_rows(q, x, None, codes[:4], scales)
    with pytest.raises(TypeError):
        moe.moe_quantize_rows(q, x, None, codes.short(), scales)
    with pytest.raises(ValueError):
        moe.moe_quantize_weight(x, codes, torch.empty(2, 1, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_quantize_weight(x[0], codes, scales)
