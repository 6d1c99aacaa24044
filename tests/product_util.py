"""Plain 64-bit forms of the linear and grouped products, SwiGLU and their
gradients, error bounds for them by arithmetic, and guarded device buffers.

Bounds.  Operands are bf16, products exact in fp32, sums of L of them in fp32
in some order, with at most one unit of 2^-23 lost per addition:
|error| <= (L + 8) 2^-23 S with S the sum of the terms' magnitudes.  A result
rounded to bf16 is off by up to 2^-8 of its value more (fp32: 2^-24).
Activations: a sigmoid from v_exp_f32 and v_rcp_f32 (1 ulp each, on values up
to 1) is off by less than 2^-21, and so is the normal distribution function by
its published bound of 0.75e-7 and five fp32 roundings; times z, with a factor
of two kept: 2^-20 |z|.
"""
from __future__ import annotations

import math

import torch

BF16_HALF, F32_HALF = 2.0 ** -8, 2.0 ** -24
SENTINEL = 7.5


def half(dtype):
    return BF16_HALF if dtype == torch.bfloat16 else F32_HALF


def sum_err(length, magnitude):
    return (length + 8) * 2.0 ** -23 * magnitude


def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def slope(z, name):
    z = z.clone().requires_grad_()
    with torch.enable_grad():
        g, = torch.autograd.grad(act(z, name).sum(), z)
    return g


def act_err(z, name):
    """|act as computed - act| at the same z."""
    return torch.zeros_like(z) if name in ("none", "relu") else 2.0 ** -20 * z.abs()


def slope_err(z, name):
    """The slopes are s + z s (1 - s) q' forms: s is off by 2^-21, the second
    term's factor s (1 - s) by 2^-20 at most, times |z| q' (q' = 1 for silu;
    for gelu_tanh 2 sqrt(2/pi) (1 + 3 0.044715 z^2)); gelu's second term is a
    product of a gaussian, below 0.4 |z| e^(-z z / 2) < 0.25."""
    if name in ("none", "relu"):
        return torch.zeros_like(z)
    q = 1.6 * (1 + 0.135 * z * z) if name == "gelu_tanh" else 1.0
    return 2.0 ** -20 * (1 + z.abs() * q)


MAX_SLOPE = {"none": 1.0, "relu": 1.0, "gelu": 1.13, "gelu_tanh": 1.13, "silu": 1.1}


def bf16(*shape, scale=1.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


def f32(*shape, scale=1.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g) * scale


def d64(t):
    """On the GPU in 64 bits, where the references are formed."""
    return t.cuda().double()


class Guarded:
    """A device tensor inside a larger buffer whose surroundings are a
    sentinel (outputs: writes outside show) or NaN (inputs: reads outside
    show in the results)."""
    PAD = 4096  # elements on each side

    def __init__(self, host=None, shape=None, dtype=None, fill=None):
        self.inp = host is not None
        if self.inp:
            shape, dtype = host.shape, host.dtype
        n = math.prod(shape)
        bad = (math.nan if self.inp else SENTINEL) if dtype.is_floating_point else -7
        self.buf = torch.full((n + 2 * self.PAD,), bad, dtype=dtype, device="cuda")
        self.t = self.buf[self.PAD:self.PAD + n].view(shape)
        self.n = n
        if self.inp:
            self.t.copy_(host)
        elif fill is not None:
            self.t.copy_(fill)

    def check(self):
        around = torch.cat([self.buf[:self.PAD], self.buf[self.PAD + self.n:]]).cpu()
        want = SENTINEL if around.dtype.is_floating_point else -7
        assert (around == want).all(), "wrote outside the output"
        return self.t.cpu()


def inp(host):
    return None if host is None else Guarded(host).t


def within(got, want, bound, what):
    """got (any dtype) against want in 64 bits, element by element."""
    err = (got.to(want.device).double() - want).abs()
    bad = ~(err <= bound)
    if bad.any():
        i = int(torch.where(bad, err - bound, torch.full_like(err, -1)).flatten().argmax())
        raise AssertionError(
            f"{what}: {int(bad.sum())} of {bad.numel()} off; worst at {i}: got "
            f"{got.flatten()[i].item()}, want {want.flatten()[i].item()}, bound "
            f"{bound.flatten()[i].item() if torch.is_tensor(bound) else bound}")
