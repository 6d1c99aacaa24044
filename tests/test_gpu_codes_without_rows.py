"""Rows without a source (row_ids outside x) in grouped products of codes: they
read as zeros, with scales of zero, in every way a product is run."""
import math

import pytest
import torch

from tests import fp8_util as fu
from tests import gpu_util as gu

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


# Few rows a tile (16 x 8 and 16 x 16), 64 x 64 tiles in one range and in several,
# 128 x 256 and 256 x 256 tiles.
@pytest.mark.parametrize("y_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P,K,F", [(5, 400, 264), (40, 400, 1288), (200, 400, 264),
                                   (150, 4096, 264), (9000, 400, 1032)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_zeros_meet_the_weights_scales(moe, P, K, F, y_dtype, bad):
    """0 times a weight block's scale of NaN or infinity is NaN, as 0 times such a
    weight is in bf16; the results of other blocks are the bias."""
    E, X = 2, 30
    xc, xs = (t.cuda() for t in fu.random_codes(X, K))
    wc, ws = (torch.stack(v).cuda() for v in zip(*(fu.random_codes(F, K, 128, e + 1) for e in range(E))))
    ws[1, 1, 2] = bad  # columns 128 .. 255 of the second group
    ids = torch.arange(P, dtype=torch.int32) % X
    ids[1::4] = -1
    ids[3::8] = X
    none = (ids < 0) | (ids >= X)
    half = P // 2
    off = torch.tensor([0, half, P], dtype=torch.int32).cuda()
    bias = torch.arange(E * F, dtype=torch.float32).view(E, F) % 32 + 1
    cfg = moe.make_grouped_config(P, E, K, F, x_rows=X, y_dtype=y_dtype)
    work = moe.alloc_grouped_fp8_workspace(cfg)
    work.fill_(0xFF)  # NaN as fp32
    y = torch.empty(P, F, dtype=DT[y_dtype], device="cuda")
    moe.moe_grouped_forward_fp8(cfg, xc, xs, ids.cuda(), off, wc, ws, bias.cuda(), y, work)
    got = y.float().cpu()
    want = bias[0].expand(P, F).clone()
    want[half:] = bias[1]
    touched = torch.zeros(P, F, dtype=torch.bool)
    touched[half:, 128:256] = True
    missing = none[:, None].expand(P, F)
    assert torch.isnan(got[missing & touched]).all()
    assert torch.equal(got[missing & ~touched], want[missing & ~touched])
    # the other rows: not finite where they meet the block, finite elsewhere
    assert not torch.isfinite(got[~missing & touched]).any()
    assert torch.isfinite(got[~missing & ~touched]).all()


def test_as_in_bf16(moe):
    """The same of the products in bf16."""
    P, K, F = 5, 400, 264
    x = torch.randn(30, K, device="cuda").bfloat16()
    w = torch.randn(1, F, K, device="cuda").bfloat16()
    w[0, 7, 3] = math.inf
    ids = torch.tensor([0, -1, 2, 30, 4], dtype=torch.int32).cuda()
    cfg = moe.make_grouped_config(P, 1, K, F, x_rows=30)
    y = torch.empty(P, F, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_forward(cfg, x, ids, torch.tensor([0, P], dtype=torch.int32).cuda(), w, None, y,
                            moe.alloc_grouped_workspace(cfg))
    bad = ~torch.isfinite(y.cpu().float())
    assert bad[:, 7].all() and bad.sum() == P
    assert torch.isnan(y[[1, 3], 7]).all()
