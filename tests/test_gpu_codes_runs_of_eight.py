"""What bf16 results of codes promise of their sums, run of eight by run of eight:
off by less than 2^-10 of the sum of the runs' largest terms, in which a code below
2^-6 counts as 2^-6, beside the fp32 sums' own errors (tests/fp8_util.py)."""
import pytest
import torch

from tests import fp8_util as fu
from tests import gpu_util as gu
from tests.product_util import BF16_HALF, within

pytestmark = pytest.mark.gpu
# 64 x 64 tiles in one range and in several, 128 x 256 and 256 x 256 tiles
SIZES = [(150, 400, 264), (150, 4096, 264), (1500, 144, 4096), (4100, 528, 1032)]


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


def product(moe, xc, xs, wc, ws):
    (T, K), F = xc.shape, wc.shape[0]
    cfg = moe.make_linear_config(T, K, F)
    y = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
    moe.moe_linear_forward_fp8(cfg, xc, xs, wc, ws, None, None, y, None,
                               moe.alloc_linear_fp8_workspace(cfg))
    return y


def run_bound(xc, xs, wc, ws):
    """2^-10 of the sum of the runs' largest terms, for a few rows of x: [rows][F]."""
    rows, k = xc.shape
    a = fu.decode(xc).abs().clamp(min=2.0 ** -6) * fu.spread(xs, 1, rows, k)
    b = fu.decode(wc).abs().clamp(min=2.0 ** -6) * fu.spread(ws, 128, wc.shape[0], k)
    out = torch.empty(rows, wc.shape[0], dtype=torch.double, device=a.device)
    for i in range(rows):
        out[i] = (a[i] * b).view(-1, k // 8, 8).amax(2).sum(1)
    return 2.0 ** -10 * out


def check(moe, xc, xs, wc, ws, rows):
    xc, xs, wc, ws = (t.cuda() for t in (xc, xs, wc, ws))
    y = product(moe, xc, xs, wc, ws)[rows]
    xc, xs = xc[rows], xs[rows]
    x, w = fu.values(xc, xs, 1), fu.values(wc, ws, 128)
    want = x @ w.t()
    err = run_bound(xc, xs, wc, ws) + fu.exact_bound(x.shape[1], x.abs() @ w.abs().t())
    within(y, want, (1 + BF16_HALF) * err + BF16_HALF * want.abs(), "y")


def scales(rows, k, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.rand(rows, fu.blocks(k), generator=g) + 0.5


@pytest.mark.parametrize("T,K,F", SIZES)
def test_any_codes(moe, T, K, F):
    """Every code but NaN alike, so that runs hold codes of all exponents."""
    g = torch.Generator().manual_seed(T)
    xc, wc = (torch.randint(0, 255, (n, K), generator=g).to(torch.uint8) for n in (T, F))
    for c in (xc, wc):
        c[c == 0x7F] = 0x01
    check(moe, xc, scales(T, K, 1), wc, scales(fu.blocks(F), K, 2),
          torch.tensor([0, 1, 31, 63, T // 2, T - 1], device="cuda"))


@pytest.mark.parametrize("T,K,F", SIZES)
def test_subnormal_code_beside_a_large_one(moe, T, K, F):
    """A run 2^-9 * 448 + 7 * (1.125 * 2^-6) (1.875 * 2^-2), whose largest term is 0.875
    but is summed on the grid of 2^-6 * 2^8, and a run that cancels it exactly."""
    def code(v):
        return torch.tensor(v).to(torch.float8_e4m3fn).view(torch.uint8)
    xc, wc = torch.zeros(T, K, dtype=torch.uint8), torch.zeros(F, K, dtype=torch.uint8)
    xs, ws = torch.ones(T, fu.blocks(K)), torch.ones(fu.blocks(F), fu.blocks(K))
    xc[:, 0], wc[:, 0] = code(2.0 ** -9), code(448.0)
    xc[:, 1:8], wc[:, 1:8] = code(1.125 * 2.0 ** -6), code(1.875 * 2.0 ** -2)
    xc[:, 128], wc[:, 128] = code(1.0), code(-1.0)
    xs[:, 1] = 0.875 + 7 * 1.125 * 1.875 * 2.0 ** -8  # exact: 14 bits
    check(moe, xc, xs, wc, ws, torch.tensor([0, 1, T - 1], device="cuda"))
