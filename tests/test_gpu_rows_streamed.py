"""Rows that go past the last-level cache (more than 256 MB of them named by a call's
pairs), in every pair of types, and weight gradients over several turns of slots:
every element against plain 64-bit forms on the GPU, with the bounds of
tests/product_util.py."""
import itertools
import math

import pytest
import torch

from tests import gpu_util as gu
from tests import product_util as pu
from tests.product_util import half, sum_err, within
from tests.test_gpu_rows import check_weight_grad

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LEFT = 5  # rows that no pair names


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


def rand(*shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


class Case:
    """Operands of a call whose pairs name `named` of R rows, in random order; the
    other rows hold NaN."""

    def __init__(self, moe, tok, row, H, k, named, T, R, seed=1):
        assert named * H * DT[row].itemsize > 2 ** 28 and named <= T * k
        g = torch.Generator().manual_seed(seed)
        pos = torch.tensor([-1, R, -2 ** 31, 2 ** 31 - 1]).repeat(T * k // 4 + 1)[:T * k]
        have = torch.randperm(T * k, generator=g)[:named]
        pos[have] = torch.randperm(R, generator=g)[:named]
        self.moe, self.T, self.R, self.k, self.H = moe, T, R, k, H
        self.pos = pos.view(T, k).cuda()
        self.ok = (self.pos >= 0) & (self.pos < R)
        self.gpos = self.pos.to(torch.int32)
        self.cfg = moe.make_dispatch_config(T, R, k, H, token_dtype=tok, row_dtype=row)
        self.tok, self.row = DT[tok], DT[row]
        self.x = rand(T, H, dtype=self.tok, seed=seed + 1)
        self.base = rand(T, H, dtype=self.tok, seed=seed + 2)
        self.w = rand(T, k, dtype=torch.float32, seed=seed + 3)
        self.r = torch.full((R, H), math.nan, dtype=self.row, device="cuda")
        at = self.pos[self.ok]
        self.r[at] = rand(named, H, dtype=self.row, seed=seed + 4)
        self.left = torch.ones(R, dtype=torch.bool, device="cuda")
        self.left[at] = False

    def slots(self):
        """(slot, tokens with a row there, their rows)."""
        for j in range(self.k):
            t = self.ok[:, j].nonzero().flatten()
            yield j, t, self.pos[t, j]

    def rows(self):
        return torch.full((self.R, self.H), pu.SENTINEL, dtype=self.row, device="cuda")

    def check_rows(self, got, weights, what):
        """r[pos[t][j]] = w x[t], and the other rows as they were."""
        for j, t, at in self.slots():
            v = self.x[t].double()
            if weights:
                v = v * self.w[t, j].double()[:, None]
            exact = not weights and self.row in (self.tok, torch.float32)
            err = 0.0 if exact else (half(self.row) + 1.01 * weights * 2.0 ** -24) * v.abs()
            within(got[at], v, err, f"{what}, slot {j}")

    def check_sums(self, got, weights, base, what):
        want = torch.zeros(self.T, self.H, dtype=torch.double, device="cuda")
        if base:
            want += self.base.double()
        mag = want.abs()
        for j, t, at in self.slots():
            v = self.r[at].double()
            if weights:
                v = v * self.w[t, j].double()[:, None]
            want[t] += v
            mag[t] += v.abs()
        within(got, want, 1.01 * sum_err(self.k, mag) + half(self.tok) * want.abs(), what)

    def check_dots(self, got, r):
        """Pairs without a row: exactly 0."""
        want = torch.zeros(self.T, self.k, dtype=torch.double, device="cuda")
        mag = torch.zeros_like(want)
        for j, t, at in self.slots():
            v = self.x[t].double() * r[at].double()
            want[t, j], mag[t, j] = v.sum(1), v.abs().sum(1)
        within(got, want, sum_err(self.H, mag), "dweights")

    def run(self):
        moe, cfg = self.moe, self.cfg
        out = self.rows()
        moe.moe_dispatch_forward(cfg, self.x, self.gpos, out)
        self.check_rows(out, False, "dispatch")
        assert (out[self.left] == pu.SENTINEL).all()
        y = torch.empty(self.T, self.H, dtype=self.tok, device="cuda")
        moe.moe_combine_forward(cfg, self.r, self.gpos, self.w, self.base, y)
        self.check_sums(y, True, True, "combine")
        moe.moe_dispatch_backward(cfg, self.r, self.gpos, None, y)
        self.check_sums(y, False, False, "dispatch's gradient")
        out.fill_(pu.SENTINEL)
        dw = torch.full((self.T, self.k), pu.SENTINEL, device="cuda")
        moe.moe_combine_backward(cfg, self.x, self.r, self.gpos, self.w, out, dw)
        self.check_rows(out, True, "drows")
        assert (out[self.left] == pu.SENTINEL).all()
        self.check_dots(dw, self.r)
        # over the rows themselves, bit for bit
        kept = self.r.clone()
        dw2 = torch.empty_like(dw)
        moe.moe_combine_backward(cfg, self.x, kept, self.gpos, self.w, kept, dw2)
        assert torch.equal(dw2, dw) and torch.equal(kept[~self.left], out[~self.left])
        assert torch.isnan(kept[self.left]).all()


# Lanes packed, one wave a token (one or two turns of slots), four waves a token.
@pytest.mark.parametrize("H,k", [(264, 3), (520, 2), (520, 11), (4104, 2), (4104, 8), (4104, 11)])
@pytest.mark.parametrize("tok,row", itertools.product(DT, repeat=2))
def test_streamed_rows(moe, tok, row, H, k):
    named = 2 ** 28 // (H * DT[row].itemsize) + 17
    Case(moe, tok, row, H, k, named, T=named * 9 // 8 // k + 3, R=named + LEFT).run()


def test_streamed_rows_beyond_32_bits(moe):
    """Rows anywhere in 8.6 GB."""
    H, named = 4096, 2 ** 15 + 100
    Case(moe, "bf16", "bf16", H, 8, named, T=named // 8 + 40, R=2 ** 20 + 5).run()


@pytest.mark.parametrize("with_rows", [False, True])
@pytest.mark.parametrize("T,k,H,rows", [(37, 9, 1032, 200), (37, 16, 4096, 500), (5, 32, 4104, 160),
                                        (3, 24, 65536, 60)])
def test_four_waves_over_several_turns_of_slots(moe, T, k, H, rows, with_rows):
    check_weight_grad(moe, T, k, H, rows, with_rows=with_rows, seed=k, none=(1,))
    check_weight_grad(moe, T, k, H, rows, "f32", "bf16", with_rows=with_rows, seed=k + 1)


# A few pairs in a buffer with room for more than 256 MB, and the same rows in one
# that fits: the same values, and all other rows left as they were.
def test_few_pairs_in_a_large_buffer(moe):
    T, k, H, R = 64, 8, 4096, 65536
    n = T * k
    g = torch.Generator().manual_seed(3)
    at = torch.randperm(R, generator=g)[:n].view(T, k).to(torch.int32).cuda()
    small = torch.arange(n).view(T, k).to(torch.int32).cuda()
    x, w = rand(T, H, dtype=torch.bfloat16, seed=1), rand(T, k, dtype=torch.float32, seed=2)
    got = []
    for rows, pos in ((R, at), (n, small)):
        cfg = moe.make_dispatch_config(T, rows, k, H)
        q = moe.make_quantize_config(T, H, rows=rows, top_k=k)
        r = torch.full((rows, H), pu.SENTINEL, dtype=torch.bfloat16, device="cuda")
        codes = torch.full((rows, H), 0x55, dtype=torch.uint8, device="cuda")
        scales = torch.full((rows, H // 128), pu.SENTINEL, device="cuda")
        dr, y, dx = torch.full_like(r, pu.SENTINEL), torch.empty_like(x), torch.empty_like(x)
        dw = torch.empty(T, k, device="cuda")
        moe.moe_dispatch_forward(cfg, x, pos, r)
        moe.moe_combine_forward(cfg, r, pos, w, x, y)
        moe.moe_combine_backward(cfg, y, r, pos, w, dr, dw)
        moe.moe_dispatch_backward(cfg, dr, pos, None, dx)
        moe.moe_quantize_rows(q, x, pos, codes, scales)
        i = pos.flatten().long()
        left = torch.ones(rows, dtype=torch.bool, device="cuda")
        left[i] = False
        assert (r[left] == pu.SENTINEL).all() and (dr[left] == pu.SENTINEL).all()
        assert (codes[left] == 0x55).all() and (scales[left] == pu.SENTINEL).all()
        got.append([r[i], dr[i], codes[i], scales[i], y, dx, dw])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert torch.equal(got[0][0], x.repeat_interleave(k, 0))


def test_streamed_codes(moe):
    """More than 256 MB of codes: each row's are those of its token, which stay."""
    T, k, K, R = 8200, 8, 4096, 65541
    named = R - LEFT
    g = torch.Generator().manual_seed(5)
    pos = torch.full((T * k,), -1)
    pos[torch.randperm(T * k, generator=g)[:named]] = torch.randperm(R, generator=g)[:named]
    pos = pos.view(T, k).cuda()
    x = rand(T, K, dtype=torch.bfloat16, seed=6)
    codes = torch.full((R, K), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((R, K // 128), pu.SENTINEL, device="cuda")
    one, one_scales = torch.empty_like(codes[:T]), torch.empty_like(scales[:T])
    moe.moe_quantize_rows(moe.make_quantize_config(T, K, rows=R, top_k=k), x, pos.to(torch.int32),
                          codes, scales)
    moe.moe_quantize_rows(moe.make_quantize_config(T, K), x, None, one, one_scales)
    t, j = (pos >= 0).nonzero(as_tuple=True)
    at = pos[t, j]
    assert torch.equal(codes[at], one[t]) and torch.equal(scales[at], one_scales[t])
    left = torch.ones(R, dtype=torch.bool, device="cuda")
    left[at] = False
    assert int(left.sum()) == LEFT
    assert (codes[left] == 0x55).all() and (scales[left] == pu.SENTINEL).all()
