"""Block-scaled e4m3 codes in 64 bits for the tests: the encoding by its
definition, decoding, products of codes, and their error bounds by arithmetic.

Bounds of a product of codes.  Products of two codes are exact in fp32 (eight
significand bits).

* fp32 results, and batches of few rows: a block's sum of up to 128 products and
  the sum of blocks, each addition losing at most one unit of 2^-23, the scales'
  product and its multiplication half a unit each:
  (K + 4 blocks + 8) 2^-23 of the sum of magnitudes.
* bf16 results in larger batches: in each run of eight consecutive codes the
  products are cut to a grid of 2^-13 times 2^e, e the largest sum of the two
  codes' exponents; a normal code is at least 2^exponent, a subnormal one has the
  exponent -6.  Seven products are cut by less than a grid step each, the one
  whose exponents are largest by none (its last bit is 2^(e - 6)), so a run is
  off by less than 7 2^-13 M < 2^-10 M with M the largest max(|a|, 2^-6)
  max(|b|, 2^-6) of the run.
"""
from __future__ import annotations

import torch

from tests import product_util as pu

BLOCK, MOST, LEAST = 128, 448.0, 2.0 ** -90


def blocks(n):
    return -(-n // BLOCK)


def decode(codes):
    """Values of uint8 codes in 64 bits."""
    return codes.view(torch.float8_e4m3fn).to(torch.float32).double()


def block_max(x, rows):
    """Largest magnitudes of the blocks rows x 128 of x [n][k]."""
    n, k = x.shape
    pad = torch.zeros(-(-n // rows) * rows, blocks(k) * BLOCK, dtype=x.dtype, device=x.device)
    pad[:n, :k] = x.abs()
    return pad.view(-1, rows, blocks(k), BLOCK).amax((1, 3))


def spread(scales, rows, n, k):
    """Scales of every element."""
    return scales.double().repeat_interleave(rows, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]


def encode(x, rows=1):
    """(codes uint8, scales fp32) of bf16 x [n][k], by torch's own conversion to
    e4m3 (round to nearest even) of fp32 quotients."""
    n, k = x.shape
    a = block_max(x.float(), rows).clamp(min=LEAST)
    inv = spread(MOST / a, rows, n, k).float()
    return (x.float() * inv).to(torch.float8_e4m3fn).view(torch.uint8), a / MOST


def random_codes(n, k, rows=1, seed=0, scale=1.0):
    return encode(pu.bf16(n, k, scale=scale, seed=seed), rows)


def values(codes, scales, rows):
    n, k = codes.shape
    return decode(codes) * spread(scales, rows, n, k)


def cut_bound(xc, xs, wc, ws):
    """The native products' bound (all on one device): [T][F]."""
    t, k = xc.shape
    f = wc.shape[0]
    a = decode(xc).abs().clamp(min=2.0 ** -6)
    b = decode(wc).abs().clamp(min=2.0 ** -6)
    # the largest product of a run is at most the product of its largest factors
    pad = -k % 8
    if pad:
        a, b = (torch.nn.functional.pad(v, (0, pad)) for v in (a, b))
    a, b = a.view(t, -1, 8).amax(2), b.view(f, -1, 8).amax(2)
    runs = a.shape[1]
    sx = xs.double().repeat_interleave(BLOCK // 8, 1)[:, :runs]
    sw = ws.double().repeat_interleave(BLOCK, 0)[:f].repeat_interleave(BLOCK // 8, 1)[:, :runs]
    return 2.0 ** -10 * ((a * sx) @ (b * sw).t())


def exact_bound(k, magnitude):
    return (k + 4 * blocks(k) + 8) * 2.0 ** -23 * magnitude


class Bytes:
    """A uint8 device tensor in a larger buffer: around an input NaN codes, around
    an output a sentinel."""
    PAD, SENTINEL = 4096, 0x55

    def __init__(self, host=None, shape=None):
        self.n = host.numel() if host is not None else torch.Size(shape).numel()
        fill = 0x7F if host is not None else self.SENTINEL
        self.buf = torch.full((self.n + 2 * self.PAD,), fill, dtype=torch.uint8, device="cuda")
        self.t = self.buf[self.PAD:self.PAD + self.n].view(host.shape if host is not None else shape)
        if host is not None:
            self.t.copy_(host)

    def check(self):
        around = torch.cat([self.buf[:self.PAD], self.buf[self.PAD + self.n:]])
        assert (around == self.SENTINEL).all(), "wrote outside the output"
        return self.t.cpu()


def codes_in(host):
    return Bytes(host).t
