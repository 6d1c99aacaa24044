"""The activations of the linear product and SwiGLU by themselves: values and
slopes over their whole range with bounds relative to the result, and the
ends of that range.  With x = 0 the pre-activation is the bias, so a sweep of
z goes straight through the epilogue.

Bounds, from the fp32 forms (2^-24 a rounding, 2^-23 for v_exp_f32 and
v_rcp_f32): the exponent of an exponential is off by its own relative error
times its size, the rest by a few roundings:
  silu       z s(z):      |z| (product, constant: 1.5 2^-24)
  gelu_tanh  z s(2 q(z)): |2 q| (two constants and products, the sum, their
             product, log2 e: 6.5 2^-24)
  gelu       |z| tail(z): z z / 2 (square, product, constant: 2.5 2^-24),
             and the tail's fit, 9.4e-8, with up to ten roundings
"""
import math

import pytest
import torch

from tests import gpu_util as gu
from tests import product_util as pu
from tests.product_util import half, within

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ("relu", "gelu", "gelu_tanh", "silu")
U = 2.0 ** -24


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


def value(z, act):
    """act(z) in 64 bits, without cancellation in the tails."""
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * inner(z)))
    return pu.act(z, act)


def inner(z):
    return math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)


def relative(z, act):
    """Relative error of the sigmoid or tail that the activation is formed from."""
    if act == "relu":
        return torch.zeros_like(z)
    grown = {"gelu": 1.25 * z * z, "gelu_tanh": 6.5 * 2 * inner(z).abs(), "silu": 1.5 * z.abs()}[act]
    return U * (16 + grown)


def through(moe, z, act, y_dtype="f32", T=1):
    """act(z) by the kernel, z from the bias; T rows."""
    F = z.numel()
    cfg = moe.make_linear_config(T, 8, F, activation=act, y_dtype=y_dtype)
    x = torch.zeros(T, 8, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(F, 8, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(T, F, dtype=DT[y_dtype], device="cuda")
    moe.moe_linear_forward(cfg, x, w, z.cuda(), None, y, None, moe.alloc_linear_workspace(cfg))
    y = y.cpu()
    # (bits: a NaN equals itself)
    bits = y.view(torch.int32 if y_dtype == "f32" else torch.int16)
    assert (bits == bits[0]).all(), "rows differ"
    return y[0]


def slopes(moe, z, act):
    """act'(z) in bf16 by the kernel, for dy = 1; z bf16."""
    F = z.numel()
    cfg = moe.make_linear_config(1, 8, F, activation=act)
    dz = torch.empty(1, F, dtype=torch.bfloat16, device="cuda")
    moe.moe_linear_backward(cfg, torch.ones_like(dz), z.view(1, F).cuda(), None, None, dz, None,
                            None, None, moe.alloc_linear_workspace(cfg))
    return dz.cpu()[0]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("y_dtype", ("f32", "bf16"))
@pytest.mark.parametrize("T", (1, 40))  # the kernel for few rows, and the tiles
def test_values_relative_to_themselves(moe, act, y_dtype, T):
    z = torch.linspace(-12, 12, 8192)
    got = through(moe, z, act, y_dtype, T)
    want = value(z.double(), act)
    h = half(DT[y_dtype])
    # (where a sum of exponentials underflows fp32, only to 2^-126 times |z|)
    within(got, want, ((1 + h) * (relative(z.double(), act) + U) + h) * want.abs() + 12 * 2.0 ** -126,
           act)


@pytest.mark.parametrize("act", ACTS)
def test_slopes_relative_to_their_terms(moe, act):
    z = torch.linspace(-12, 12, 4096).bfloat16()
    zd = z.double()
    r = relative(zd, act) + 2 * U
    dq = 1.0
    if act == "gelu":
        a = torch.special.erfc(-zd / math.sqrt(2)) / 2
        b = zd * torch.exp(-zd * zd / 2) / math.sqrt(2 * math.pi)
    elif act == "relu":
        a, b = (zd > 0).double(), torch.zeros_like(zd)
    else:
        q = zd if act == "silu" else 2 * inner(zd)
        if act == "gelu_tanh":
            dq = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * zd * zd)
        a, b = torch.sigmoid(q), zd * dq * torch.sigmoid(q) * torch.sigmoid(-q)
    want = a + b
    # for z > 0 the second term's 1 - s keeps an absolute error: 1 + e rounded,
    # its reciprocal to an ulp, and the difference (gelu's 1 - tail: one of these)
    left = 4 * U * (zd.abs() * dq + 1) * (zd > 0)
    # a sigmoid or gaussian below 2^-126 leaves as 0, and is multiplied by 1 and z dq
    err = r * (a.abs() + b.abs()) + left + 2.0 ** -126 * (1 + zd.abs() * dq)
    within(slopes(moe, z, act), want, (1 + pu.BF16_HALF) * err + pu.BF16_HALF * want.abs(), act)


@pytest.mark.parametrize("T", (1, 40))
def test_ends_of_the_range(moe, T):
    """Huge finite values: the activations are z or 0, the slopes 1 or 0; an
    infinity from a product behaves so in relu and gelu, and a NaN stays."""
    huge = torch.tensor([3e38, 1e30, 1e20, 1e10, 1e5, 400.0, 0.0, -400.0, -1e5, -1e10, -1e20, -1e30,
                         -3e38, -0.0, 64.0, -200.0])
    for act in ACTS:
        assert torch.equal(through(moe, huge, act, T=T), huge.clamp(min=0)), act
        z = huge.bfloat16()
        s = slopes(moe, z, act)
        at0 = z == 0
        assert torch.equal(s[~at0].float(), (z[~at0] > 0).float()), act
        assert (s[at0] == (0.0 if act == "relu" else 0.5)).all(), act
    inf = float("inf")
    ends = torch.tensor([inf, -inf, float("nan"), 1.0] * 2)
    for act in ("relu", "gelu"):
        got = through(moe, ends, act, T=T)
        assert got[0] == inf and got[1] == 0 and got[2].isnan() and got[3].isfinite(), act
    for act in ("gelu_tanh", "silu"):
        got = through(moe, ends, act, T=T)
        assert got[0] == inf and got[2].isnan() and got[3].isfinite(), act


@pytest.mark.parametrize("limit", (0.0, 7.0))
def test_swiglu_ends_of_the_range(moe, limit):
    """Huge gates and ups are clamped to the limit or pass; no gradient beyond
    the limit, whatever dh is; a NaN stays."""
    inf, nan = float("inf"), float("nan")
    g = torch.tensor([[1e30, inf, -1e30, 2.0, 2.0, 2.0, nan, 2.0]]).bfloat16()
    u = torch.tensor([[2.0, 2.0, 2.0, 1e30, inf, -inf, 2.0, nan]]).bfloat16()
    dh = torch.ones(1, 8).bfloat16()
    cfg = moe.make_swiglu_config(1, 8, limit=limit)
    h = torch.empty(1, 8, dtype=torch.bfloat16, device="cuda")
    moe.moe_swiglu_forward(cfg, g.cuda(), u.cuda(), h)
    dg, du, h2 = torch.empty_like(h), torch.empty_like(h), torch.empty_like(h)
    moe.moe_swiglu_backward(cfg, dh.cuda(), g.cuda(), u.cuda(), dg, du, h2)
    h, dg, du, h2 = (t.cpu()[0].double() for t in (h, dg, du, h2))
    s2 = 2 / (1 + math.exp(-2))  # SiLU(2)
    top = limit / (1 + math.exp(-limit)) if limit else inf
    want = [2 * min(float(g[0, 0]), top), 2 * top, 0.0, s2 * min(float(u[0, 3]), limit or inf),
            s2 * (limit or inf), -s2 * (limit or inf)]
    for i, v in enumerate(want):
        assert h[i] == v or abs(h[i] - v) <= 1.01 * pu.BF16_HALF * abs(v), i
    assert h[6].isnan() and h[7].isnan()
    assert torch.equal(h2.nan_to_num(0, 1, -1), h.nan_to_num(0, 1, -1))
    assert h2[6].isnan() and h2[7].isnan()
    if limit:
        assert dg[0] == 0 and dg[1] == 0 and du[3] == 0 and du[4] == 0 and du[5] == 0
    assert dg[2] == 0 and du[2] == 0
