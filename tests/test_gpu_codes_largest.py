"""The largest sizes that the row and code operators take: the most tokens, rows,
features and groups, and outputs beyond 2^32 elements. Whole numbers, compared for
equality where every sum is exact."""
import pytest
import torch

from tests import fp8_util as fu
from tests import gpu_util as gu
from tests import product_util as pu
from tests.product_util import half, within

pytestmark = pytest.mark.gpu
BF = dict(dtype=torch.bfloat16, device="cuda")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _name_case(request):
    gu.note(f"[gpu-test] {request.node.nodeid}")
    yield
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import sparse_moe_layer_fp32_amd as m
    m.load_library()
    return m


def integers(shape, most, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda", dtype=torch.int8)


def as_codes(v):
    """Codes of small whole numbers, by a table."""
    table = torch.arange(-8, 9).float().to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    return table[v.int() + 8]


def powers(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 3, shape, generator=g, device="cuda").float().exp2()


def test_most_tokens_and_rows(moe):
    """2^25 tokens of two pairs each, 2^26 rows, of 8 columns."""
    T, k, H = 2 ** 25, 2, 8
    P = T * k
    cfg = moe.make_dispatch_config(T, P, k, H)
    x = integers((T, H), 8, 1).to(torch.bfloat16)
    pos = (torch.arange(P, device="cuda", dtype=torch.int64) * 5 % P).int().view(T, k)
    rows = torch.empty(P, H, **BF)
    moe.moe_dispatch_forward(cfg, x, pos, rows)
    back = torch.empty(P, H, **BF)
    back[pos[:, 0].long()], back[pos[:, 1].long()] = x, x
    assert torch.equal(rows, back)
    y = torch.empty(T, H, **BF)
    w = torch.full((T, k), 0.5, device="cuda")
    moe.moe_combine_forward(cfg, rows, pos, w, x, y)
    assert torch.equal(y, x + x)
    dw = torch.empty(T, k, device="cuda")
    moe.moe_combine_backward(cfg, x, rows, pos, w, back, dw)
    assert torch.equal(dw, (x.float() ** 2).sum(1, keepdim=True).expand(T, k))
    assert torch.equal(back, rows * 0.5)


def test_most_rows_and_columns_of_codes(moe):
    T, K = 2 ** 25, 16
    x = integers((T, K), 7, 1).to(torch.bfloat16)
    x[:, 3] = 7  # scale 1/64: every whole number is a multiple of a code's step
    codes, scales = torch.empty(T, K, dtype=torch.uint8, device="cuda"), torch.empty(T, 1, device="cuda")
    moe.moe_quantize_rows(moe.make_quantize_config(T, K), x, None, codes, scales)
    assert (scales == scales[0]).all()
    assert torch.equal(fu.decode(codes[-1000:]) * scales[-1000:].double(), x[-1000:].double())
    assert torch.equal(codes, as_codes(x.to(torch.int8)) + ((codes & 0x7F) != 0).byte() * 48)
    T, K = 2 ** 17, 65536
    x = pu.bf16(4, K, seed=3).cuda()
    big = x.repeat(T // 4, 1)
    codes, scales = torch.empty(T, K, dtype=torch.uint8, device="cuda"), torch.empty(T, 512, device="cuda")
    moe.moe_quantize_rows(moe.make_quantize_config(T, K), big, None, codes, scales)
    want, ws = fu.encode(x.cpu())
    near = (codes[:4].cpu() == want).float().mean()
    assert near > 0.999 and within(scales[:4], ws.cuda().double(), 2.0 ** -22 * ws.cuda(), "s") is None
    assert torch.equal(codes[-4:], codes[:4]) and torch.equal(scales[-4:], scales[:4])


def check_whole(moe, T, K, F, y_dtype, groups=None, rows=None):
    """rows: those that are compared (None: all)."""
    x, w = integers((T, K), 1, 1), integers((groups or 1, F, K), 2, 2)
    xs, ws = powers((T, fu.blocks(K)), 3), powers((groups or 1, fu.blocks(F), fu.blocks(K)), 4)
    y = torch.empty(T, F, dtype=DT[y_dtype], device="cuda")
    xc, wc = as_codes(x), as_codes(w)
    if groups is None:
        cfg = moe.make_linear_config(T, K, F, y_dtype=y_dtype)
        moe.moe_linear_forward_fp8(cfg, xc, xs, wc[0], ws[0], None, None, y, None,
                                   moe.alloc_linear_fp8_workspace(cfg))
        off = [0, T]
    else:
        off = [T * g // groups for g in range(groups + 1)]
        cfg = moe.make_grouped_config(T, groups, K, F, y_dtype=y_dtype)
        moe.moe_grouped_forward_fp8(cfg, xc, xs, None, torch.tensor(off, dtype=torch.int32).cuda(), wc,
                                    ws, None, y, moe.alloc_grouped_fp8_workspace(cfg))
    for g in range(len(off) - 1):
        for i, j in rows or [(off[g], off[g + 1])]:
            i, j = max(i, off[g]), min(j, off[g + 1])
            if i < j:
                a = fu.values(xc[i:j], xs[i:j], 1).float()   # whole numbers below 2^24 throughout
                want = a.double() @ fu.values(wc[g], ws[g], fu.BLOCK).t()
                assert torch.equal(y[i:j], want.to(DT[y_dtype])), (g, i)


@pytest.mark.parametrize("y_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,F", [(3, 65536, 8), (300, 65536, 136), (5, 16, 65536), (300, 144, 65536),
                                   (2500, 16384, 2056)])
def test_most_features(moe, T, K, F, y_dtype):
    check_whole(moe, T, K, F, y_dtype)


@pytest.mark.parametrize("y_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("groups", [None, 1024])
def test_most_rows(moe, groups, y_dtype):
    T = 2 ** 26
    ends = [(0, 5000), (2 ** 25 - 3000, 2 ** 25 + 3000), (T - 5000, T)]
    check_whole(moe, T, 16, 8, y_dtype, groups, ends)


@pytest.mark.parametrize("groups", [None, 3, 700])
def test_outputs_beyond_32_bits(moe, groups):
    """Large tiles whose results and codes lie beyond 2^32."""
    T = 2 ** 24 + 77
    ends = [(0, 3000), (2 ** 32 // 264 - 2000, 2 ** 32 // 264 + 2000), (T - 3000, T)]
    check_whole(moe, T, 272, 264, "bf16", groups, ends)


def test_gathered_rows_of_a_large_x(moe):
    """Sources up to the end of the largest x that rows are gathered from."""
    K, F, xr = 4096, 264, (0xF0000000 // 2) // 4096 - 1
    P = 9001
    g = torch.Generator().manual_seed(1)
    ids = torch.randint(0, xr, (P,), generator=g, dtype=torch.int32)
    ids[7], ids[-1], ids[5000] = xr - 1, xr - 1, xr
    xc = torch.zeros(xr, K, dtype=torch.uint8, device="cuda")
    xs = torch.ones(xr, fu.blocks(K), device="cuda")
    live = ids[ids < xr].long().unique().cuda()
    xc[live], xs[live] = as_codes(integers((len(live), K), 1, 2)), powers((len(live), 32), 3)
    w, ws = integers((2, F, K), 1, 4), powers((2, fu.blocks(F), 32), 5)
    wc = as_codes(w)
    off = torch.tensor([0, 4000, P], dtype=torch.int32).cuda()
    for y_dtype in ("bf16", "f32"):
        cfg = moe.make_grouped_config(P, 2, K, F, x_rows=xr, y_dtype=y_dtype)
        y = torch.empty(P, F, dtype=DT[y_dtype], device="cuda")
        moe.moe_grouped_forward_fp8(cfg, xc, xs, ids.cuda(), off, wc, ws, None, y,
                                    moe.alloc_grouped_fp8_workspace(cfg))
        for e, (i, j) in enumerate(((0, 4000), (4000, P))):
            s = ids[i:j].long().cuda()
            have = (s < xr).double()[:, None]
            s = s.clamp(max=xr - 1)
            want = (fu.values(xc[s], xs[s], 1) @ fu.values(wc[e], ws[e], fu.BLOCK).t()) * have
            assert torch.equal(y[i:j], want.to(DT[y_dtype]))
