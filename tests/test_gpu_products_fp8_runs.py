"""Large products of codes, whose blocks take one tile after the other with their
rings running on (csrc/codes_run.h), at the sizes where that can go wrong: few
steps, more steps than a lane holds scales of, many tiles to a block, tiles cut
along their rows, every remainder of a group, few columns, gathered rows."""
import pytest
import torch

from tests import fp8_util as fu
from tests import gpu_util as gu
from tests import product_util as pu
from tests.product_cases import BIG
from tests.test_gpu_products_fp8 import check_grouped, check_linear
from tests.test_product_plan import CUS
from tests.test_products_fp8_plan import plan  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _name_case(request):
    gu.note(f"[gpu-test] {request.node.nodeid}")
    yield


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import sparse_moe_layer_fp32_amd as m
    m.load_library()
    assert torch.cuda.get_device_properties(0).multi_processor_count == CUS
    return m


def large(plan, P, G, K, F, slices=None):  # noqa: F811
    p = plan(P, G, K, F, False)
    assert p.shape == BIG and (slices is None or p.slices == slices), (p.shape, p.slices)


# two steps (the second of 16 codes, and whole), three, four, and 65 and 97, of
# which a lane holds the columns' scales in two turns
@pytest.mark.parametrize("K", [144, 256, 272, 384, 400, 512, 8208, 12400])
@pytest.mark.parametrize("T,F,slices", [(4100, 4104, 4), (8200, 1032, 1), (2049, 4104, 1)])
def test_steps(moe, plan, T, K, F, slices):  # noqa: F811
    if K > 1024:  # (fewer columns: the reference's work)
        T, F, slices = 8200, 1032, 1
    large(plan, T, 1, K, F, slices)
    check_linear(moe, T, K, F, residual=False, keep_z=False, seed=K)


# up to eight tiles of a block, the last rounds cut in two and in four, and not;
# columns of 8, 64, 72, 136 and 200 in the last tile
@pytest.mark.parametrize("T,F", [(30000, 1032), (40001, 2120), (12300, 4168), (20000, 4232),
                                 (65536, 1480), (4100, 4296), (100000, 264)])
def test_many_tiles(moe, plan, T, F):  # noqa: F811
    large(plan, T, 1, 272, F)
    check_linear(moe, T, 272, F, bias=True, residual=False, keep_z=False, seed=F)


# rows of the last tile: every number of 32-row blocks, whole and cut
@pytest.mark.parametrize("rest", [1, 31, 32, 33, 64, 65, 97, 128, 130, 161, 192, 200, 225, 255])
def test_last_rows(moe, plan, rest):  # noqa: F811
    for T in (2048 + rest, 8192 + rest):
        large(plan, T, 1, 144, 4104)
        check_linear(moe, T, 144, 4104, residual=False, keep_z=False, seed=rest)


@pytest.mark.parametrize("act", list(pu.MAX_SLOPE))
@pytest.mark.parametrize("bias,residual,keep_z", [(True, True, True), (False, True, False),
                                                  (False, False, True)])
def test_ways_out(moe, plan, act, bias, residual, keep_z):  # noqa: F811
    large(plan, 4100, 1, 272, 4104)
    check_linear(moe, 4100, 272, 4104, act, "bf16", bias, residual, keep_z, seed=11)


REMAINDERS = [256 * (i % 3) + r for i, r in enumerate(
    (1, 0, 31, 32, 33, 63, 64, 65, 96, 97, 128, 129, 160, 161, 192, 193, 224, 225, 255, 256))]


@pytest.mark.parametrize("K", [144, 272, 1296])
@pytest.mark.parametrize("F", [776, 1032, 2120])
def test_group_remainders(moe, plan, K, F):  # noqa: F811
    sizes = REMAINDERS + [1500]
    large(plan, sum(sizes) + 9, len(sizes), K, F)
    check_grouped(moe, sizes, K, F, tail=5, before=4, seed=K)
    check_grouped(moe, sizes, K, F, x_rows=700, row_div=3, tail=9, bias=False, seed=F)


@pytest.mark.parametrize("sizes", [[9000], [0, 0, 9000, 0], [1] + [0] * 30 + [9000, 1],
                                   [4500, 4500], [37] * 250])
def test_group_shapes(moe, plan, sizes):  # noqa: F811
    large(plan, sum(sizes), len(sizes), 400, 1032)
    check_grouped(moe, sizes, 400, 1032, x_rows=sum(sizes) // 4, row_div=4)


def whole_numbers(n, k, most, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, (n, k), generator=g).float()


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("K", [256, 8320])
def test_whole_numbers_in_groups(moe, plan, K, gather):  # noqa: F811
    """Sums that are exact in every order: a lost or doubled row, block or scale
    shows."""
    sizes, F = [2048 + 64, 2048 + 100, 0, 2048 + 190, 31, 2048 + 255, 1], 1288
    E, P = len(sizes), sum(sizes)
    large(plan, P, E, K, F)
    xr = 1000 if gather else P
    g = torch.Generator().manual_seed(K)
    x, w = whole_numbers(xr, K, 1, 1), torch.stack([whole_numbers(F, K, 2, 2 + e) for e in range(E)])
    xs = torch.randint(0, 2, (xr, fu.blocks(K)), generator=g).float().exp2()
    ws = torch.randint(0, 3, (E, fu.blocks(F), fu.blocks(K)), generator=g).float().exp2()
    ids = torch.randint(0, xr, (P,), generator=g, dtype=torch.int32) if gather else None
    off = torch.cat([torch.zeros(1, dtype=torch.int32), torch.tensor(sizes).cumsum(0).int()])
    cfg = moe.make_grouped_config(P, E, K, F, x_rows=xr)
    work = moe.alloc_grouped_fp8_workspace(cfg)
    work.fill_(0xFF)
    xc, wc = (t.to(torch.float8_e4m3fn).view(torch.uint8).cuda() for t in (x, w))
    xs, ws = xs.cuda(), ws.cuda()
    y = torch.empty(P, F, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_forward_fp8(cfg, xc, xs, ids.cuda() if gather else None, off.cuda(), wc, ws, None,
                                y, work)
    src = ids.long().cuda() if gather else torch.arange(P, device="cuda")
    for e in range(E):
        i, j = int(off[e]), int(off[e + 1])
        want = fu.values(xc[src[i:j]], xs[src[i:j]], 1) @ fu.values(wc[e], ws[e], fu.BLOCK).t()
        assert torch.equal(y[i:j], want.to(torch.bfloat16)), e


def test_offsets_that_do_not_ascend_write_nothing_outside(moe, plan):  # noqa: F811
    """Not a product that means anything, but one that stays inside its memory:
    more tiles than there is room for are left out."""
    P, E, K, F = 9000, 9, 256, 1032
    large(plan, P, E, K, F)
    xc, xs = fu.random_codes(P, K)
    wc, ws = (torch.stack(v).cuda() for v in zip(*(fu.random_codes(F, K, 128, e) for e in range(E))))
    off = torch.tensor([0, P, 0, P, 0, P, 0, P, 0, P], dtype=torch.int32).cuda()
    cfg = moe.make_grouped_config(P, E, K, F)
    size = moe.moe_grouped_fp8_workspace_size(cfg)
    buf = fu.Bytes(shape=(size,))
    y = pu.Guarded(shape=(P, F), dtype=torch.bfloat16)
    moe.moe_grouped_forward_fp8(cfg, fu.codes_in(xc), pu.inp(xs), None, off, wc, ws, None, y.t, buf.t)
    torch.cuda.synchronize()
    y.check()
    buf.check()


def test_two_calls_at_once_and_in_graphs(moe, plan):  # noqa: F811
    """Two streams with workspaces of their own; two captured calls that share one,
    replayed one after the other."""
    sizes = [3000, 700, 0, 1400]
    E, P, K, F = len(sizes), sum(sizes), 400, 2056
    large(plan, P, E, K, F)
    off = torch.cat([torch.zeros(1, dtype=torch.int32), torch.tensor(sizes).cumsum(0).int()]).cuda()
    cfg = moe.make_grouped_config(P, E, K, F)
    sets = []
    for i in range(2):
        xc, xs = (t.cuda() for t in fu.random_codes(P, K, 1, i))
        wc, ws = (torch.stack(v).cuda()
                  for v in zip(*(fu.random_codes(F, K, 128, 9 * i + e) for e in range(E))))
        sets.append((xc, xs, None, off, wc, ws, None))
    work = [moe.alloc_grouped_fp8_workspace(cfg) for _ in range(2)]
    y = [torch.zeros(P, F, dtype=torch.bfloat16, device="cuda") for _ in range(6)]
    for i in range(2):
        moe.moe_grouped_forward_fp8(cfg, *sets[i], y[i], work[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                moe.moe_grouped_forward_fp8(cfg, *sets[i], y[2 + i], work[i])
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            moe.moe_grouped_forward_fp8(cfg, *sets[i], y[4 + i], work[0])
    for _ in range(3):
        work[0].fill_(0xFF)
        for i, g in enumerate(graphs):
            y[4 + i].zero_()
            g.replay()
        moe.moe_grouped_forward_fp8(cfg, *sets[0], y[2], work[1])
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(y[i], y[2 + i]) and torch.equal(y[i], y[4 + i])


@pytest.mark.parametrize("P,K,F", [(40, 272, 72), (300, 272, 200), (6000, 400, 2056)])
def test_captured_call_follows_its_offsets(moe, P, K, F):
    """A captured product whose groups and sources change between replays."""
    E, xr = 6, 500
    xc, xs = (t.cuda() for t in fu.random_codes(xr, K))
    wc, ws = (torch.stack(v).cuda() for v in zip(*(fu.random_codes(F, K, 128, e + 1) for e in range(E))))
    cfg = moe.make_grouped_config(P, E, K, F, x_rows=xr)
    work = [moe.alloc_grouped_fp8_workspace(cfg) for _ in range(2)]
    ys = [torch.zeros(P, F, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ids = torch.zeros(P, dtype=torch.int32, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    moe.moe_grouped_forward_fp8(cfg, xc, xs, ids, off, wc, ws, None, ys[1], work[1])
    torch.cuda.synchronize()
    assert not ys[1].any()  # no group has rows
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_grouped_forward_fp8(cfg, xc, xs, ids, off, wc, ws, None, ys[0], work[0])
    gen = torch.Generator().manual_seed(P)
    for cuts in ([0, 0, 0, 0, P], [P, P, P, P, P], [P // 3, P // 3, P // 2, P - 1, P - 1], [1, 2, 3, 4, 5]):
        off.copy_(torch.tensor([0] + cuts + [P], dtype=torch.int32))
        ids.copy_(torch.randint(0, xr, (P,), generator=gen, dtype=torch.int32))
        g.replay()
        moe.moe_grouped_forward_fp8(cfg, xc, xs, ids, off, wc, ws, None, ys[1], work[1])
        torch.cuda.synchronize()
        assert torch.equal(*ys) and ys[0].abs().sum(1).min() > 0
        e = next(i for i, c in enumerate(cuts + [P]) if c > 0)
        n = min((cuts + [P])[e], 50)  # the first rows belong to the first group that has any
        want = fu.values(xc[ids[:n].long()], xs[ids[:n].long()], 1) @ fu.values(wc[e], ws[e], fu.BLOCK).t()
        off2 = ((ys[0][:n].double() - want).norm() / want.norm()).item()
        assert off2 <= 2.0 ** -8 / 3 ** 0.5 + 1e-4
