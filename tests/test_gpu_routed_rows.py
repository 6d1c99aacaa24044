"""Rows out to the experts and back, and products in 8 bits, together as a routed
layer uses them: moe_route and moe_permute give the groups, the rows go out in
memory, in bf16 for training or as codes for serving, through the experts, and
back; also with the experts of one half at a time, as two GPUs would hold them.
Each step is compared with its 64-bit form on the values that it was given."""
import pytest
import torch

import synth
from tests import fp8_util as fu
from tests import gpu_util as gu
from tests import product_util as pu
from tests.product_util import half, sum_err, within

pytestmark = pytest.mark.gpu
BF = dict(dtype=torch.bfloat16, device="cuda")
F32 = dict(dtype=torch.float32, device="cuda")
I32 = dict(dtype=torch.int32, device="cuda")

CASES = {
    "one_token": dict(T=1, H=256, E=16, k=4, I=64, Is=64),
    "few_rows": dict(T=9, H=256, E=16, k=4, I=64, Is=64),
    "ragged": dict(T=300, H=256, E=8, k=2, I=128, Is=128, limit=2.0),
    "many_rows": dict(T=1100, H=512, E=4, k=3, I=192, Is=64),
}


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


class Routed:
    """A workload, its inputs on the GPU, its routing and permutation."""

    def __init__(self, moe, name):
        self.wl = wl = synth.WORKLOADS["tiny"].with_(name=name, **CASES[name])
        self.d = d = gu.upload(synth.make_inputs(wl))
        self.cfg = gu.cfg_of(wl)
        self.T, self.H, self.E, self.k, self.I = wl.T, wl.H, wl.E, wl.k, wl.I
        self.P = wl.T * wl.k
        self.ws = moe.alloc_workspace(self.cfg)
        self.ids, self.gw = torch.empty(self.T, self.k, **I32), torch.empty(self.T, self.k, **F32)
        self.offsets = torch.empty(self.E + 1, **I32)
        self.pairs, pos = torch.empty(self.P, **I32), torch.empty(self.P, **I32)
        moe.moe_route(self.cfg, d.x, d.router_w, d.router_b, self.ids, self.gw, self.ws)
        moe.moe_permute(self.cfg, self.ids, self.offsets, self.pairs, pos, self.ws)
        self.pos = pos.view(self.T, self.k)
        self.x = d.x.view(self.T, self.H)
        self.w = [d.w_gate.view(self.E, self.I, self.H), d.w_up.view(self.E, self.I, self.H),
                  d.w_down.view(self.E, self.H, self.I)]
        self.token = (self.pairs // self.k).long()

    def groups(self):
        off = self.offsets.tolist()
        return [(e, off[e], off[e + 1]) for e in range(self.E) if off[e] < off[e + 1]]


def d64(t):
    return t.double()


@pytest.mark.parametrize("name", list(CASES))
def test_training_step_with_rows_in_memory(moe, name):
    r = Routed(moe, name)
    T, H, E, k, I, P = r.T, r.H, r.E, r.k, r.I, r.P
    rows_cfg = moe.make_dispatch_config(T, P, k, H)
    up_cfg, dn_cfg = moe.make_grouped_config(P, E, H, I), moe.make_grouped_config(P, E, I, H)
    act = moe.make_swiglu_config(P, I, limit=r.wl.limit)
    wu, wd = moe.alloc_grouped_workspace(up_cfg), moe.alloc_grouped_workspace(dn_cfg)
    rows, o, gate, up, h = (torch.empty(P, n, **BF) for n in (H, H, I, I, I))
    base, y = pu.bf16(T, H, seed=3).cuda(), torch.empty(T, H, **BF)

    moe.moe_dispatch_forward(rows_cfg, r.x, r.pos, rows)
    moe.moe_grouped_forward(up_cfg, rows, None, r.offsets, r.w[0], None, gate, wu)
    moe.moe_grouped_forward(up_cfg, rows, None, r.offsets, r.w[1], None, up, wu)
    moe.moe_swiglu_forward(act, gate, up, h)
    moe.moe_grouped_forward(dn_cfg, h, None, r.offsets, r.w[2], None, o, wd)
    moe.moe_combine_forward(rows_cfg, o, r.pos, r.gw, base, y)

    # the rows are the tokens' in the groups' order, and multiply as gathered ones do
    assert torch.equal(rows, r.x[r.token])
    in_place = moe.make_grouped_config(P, E, H, I, x_rows=T, row_div=k)
    gate2 = torch.empty(P, I, **BF)
    moe.moe_grouped_forward(in_place, r.x, r.pairs, r.offsets, r.w[0], None, gate2,
                            moe.alloc_grouped_workspace(in_place))
    for e, i, j in r.groups():
        want, mag = d64(rows[i:j]) @ d64(r.w[0][e]).t(), d64(rows[i:j]).abs() @ d64(r.w[0][e]).abs().t()
        for got in (gate, gate2):
            within(got[i:j], want, 1.01 * sum_err(H, mag) + pu.BF16_HALF * want.abs(), "gate")
    terms = d64(o[r.pos.long()]) * d64(r.gw).unsqueeze(-1)
    want, mag = d64(base) + terms.sum(1), d64(base).abs() + terms.abs().sum(1)
    within(y, want, 1.01 * sum_err(k, mag) + pu.BF16_HALF * want.abs(), "y")

    # backwards
    dy = pu.bf16(T, H, seed=5).cuda()
    do, drows, dr2 = (torch.empty(P, H, **BF) for _ in range(3))
    dh, dgate, dup = (torch.empty(P, I, **BF) for _ in range(3))
    dw, dx = torch.empty(T, k, **F32), torch.empty(T, H, **BF)
    dwd, dwg = torch.empty(E, H, I, **F32), torch.empty(E, I, H, **F32)
    moe.moe_combine_backward(rows_cfg, dy, o, r.pos, r.gw, do, dw)
    moe.moe_grouped_backward(dn_cfg, do, h, None, r.offsets, r.w[2], dh, dwd, None, wd)
    moe.moe_swiglu_backward(act, dh, gate, up, dgate, dup, None)
    moe.moe_grouped_backward(up_cfg, dgate, rows, None, r.offsets, r.w[0], drows, dwg, None, wu)
    moe.moe_grouped_backward(up_cfg, dup, rows, None, r.offsets, r.w[1], dr2, None, None, wu)
    both = torch.empty(T, H, **BF)
    moe.moe_dispatch_backward(rows_cfg, drows, r.pos, dy, both)   # base's gradient is dy itself
    moe.moe_dispatch_backward(rows_cfg, dr2, r.pos, both, dx)

    terms = d64(dy).unsqueeze(1) * d64(o[r.pos.long()])
    within(dw, terms.sum(2), sum_err(H, terms.abs().sum(2)), "dw")
    want = torch.empty(P, H, dtype=torch.double, device="cuda")
    want[r.pos.long().flatten()] = (d64(dy).unsqueeze(1) * d64(r.gw).unsqueeze(2)).view(P, H)
    within(do, want, 1.01 * (2.0 ** -24 + pu.BF16_HALF) * want.abs(), "do")
    for got, given, b in ((both, drows, dy), (dx, dr2, both)):
        terms = d64(given[r.pos.long()])
        want, mag = d64(b) + terms.sum(1), d64(b).abs() + terms.abs().sum(1)
        within(got, want, 1.01 * sum_err(k, mag) + pu.BF16_HALF * want.abs(), "dx")
    for e, i, j in r.groups():
        a, b = d64(dgate[i:j]), d64(rows[i:j])
        within(dwg[e], a.t() @ b, sum_err(j - i, a.abs().t() @ b.abs()) + 1e-30, "dw_gate")
        want, mag = a @ d64(r.w[0][e]), a.abs() @ d64(r.w[0][e]).abs()
        within(drows[i:j], want, 1.01 * sum_err(I, mag) + pu.BF16_HALF * want.abs() + 1e-30, "drows")


class Codes:
    """Experts in codes."""

    def __init__(self, moe, w):
        E, F, K = w.shape
        self.codes = torch.empty(E, F, K, dtype=torch.uint8, device="cuda")
        self.scales = torch.empty(E, fu.blocks(F), fu.blocks(K), **F32)
        moe.moe_quantize_weight(w, self.codes, self.scales)


def check_product(got, xc, xs, w, r, y_dtype):
    for e, i, j in r.groups():
        x, wv = fu.values(xc[i:j], xs[i:j], 1), fu.values(w.codes[e], w.scales[e], fu.BLOCK)
        err = fu.exact_bound(x.shape[1], x.abs() @ wv.abs().t())
        if y_dtype == "bf16":
            err = err + fu.cut_bound(xc[i:j], xs[i:j], w.codes[e], w.scales[e])
        want, hf = x @ wv.t(), half(torch.bfloat16 if y_dtype == "bf16" else torch.float32)
        within(got[i:j], want, (1 + hf) * err + hf * want.abs() + 1e-30, f"expert {e}")


@pytest.mark.parametrize("name", list(CASES))
def test_serving_step_in_codes(moe, name):
    r = Routed(moe, name)
    T, H, E, k, I, P = r.T, r.H, r.E, r.k, r.I, r.P
    wg, wu_, wd = (Codes(moe, w) for w in r.w)
    out_cfg, h_cfg = moe.make_quantize_config(T, H, rows=P, top_k=k), moe.make_quantize_config(P, I)
    up_cfg = moe.make_grouped_config(P, E, H, I)
    dn_cfg = moe.make_grouped_config(P, E, I, H, y_dtype="f32")
    back = moe.make_dispatch_config(T, P, k, H, row_dtype="f32")
    act = moe.make_swiglu_config(P, I, limit=r.wl.limit)
    work = [moe.alloc_grouped_fp8_workspace(c) for c in (up_cfg, dn_cfg)]
    base = pu.bf16(T, H, seed=3).cuda()

    def buffers():
        u8 = dict(dtype=torch.uint8, device="cuda")
        return dict(xc=torch.zeros(P, H, **u8), xs=torch.zeros(P, fu.blocks(H), **F32),
                    gate=torch.zeros(P, I, **BF), up=torch.zeros(P, I, **BF),
                    h=torch.zeros(P, I, **BF), hc=torch.zeros(P, I, **u8),
                    hs=torch.zeros(P, fu.blocks(I), **F32), o=torch.zeros(P, H, **F32),
                    y=torch.zeros(T, H, **BF))

    def step(b):
        moe.moe_quantize_rows(out_cfg, r.x, r.pos, b["xc"], b["xs"])
        moe.moe_grouped_forward_fp8(up_cfg, b["xc"], b["xs"], None, r.offsets, wg.codes, wg.scales,
                                    None, b["gate"], work[0])
        moe.moe_grouped_forward_fp8(up_cfg, b["xc"], b["xs"], None, r.offsets, wu_.codes, wu_.scales,
                                    None, b["up"], work[0])
        moe.moe_swiglu_forward(act, b["gate"], b["up"], b["h"])
        moe.moe_quantize_rows(h_cfg, b["h"], None, b["hc"], b["hs"])
        moe.moe_grouped_forward_fp8(dn_cfg, b["hc"], b["hs"], None, r.offsets, wd.codes, wd.scales,
                                    None, b["o"], work[1])
        moe.moe_combine_forward(back, b["o"], r.pos, r.gw, base, b["y"])

    b = buffers()
    step(b)
    torch.cuda.synchronize()
    check_product(b["gate"], b["xc"], b["xs"], wg, r, "bf16")
    check_product(b["up"], b["xc"], b["xs"], wu_, r, "bf16")
    check_product(b["o"], b["hc"], b["hs"], wd, r, "f32")
    terms = d64(b["o"][r.pos.long()]) * d64(r.gw).unsqueeze(-1)
    want, mag = d64(base) + terms.sum(1), d64(base).abs() + terms.abs().sum(1)
    within(b["y"], want, 1.01 * sum_err(k, mag) + pu.BF16_HALF * want.abs(), "y")

    # codes sent out are the tokens' own, and gathered in place they multiply alike
    tc, ts = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, fu.blocks(H), **F32)
    moe.moe_quantize_rows(moe.make_quantize_config(T, H), r.x, None, tc, ts)
    assert torch.equal(b["xc"], tc[r.token]) and torch.equal(b["xs"], ts[r.token])
    in_place = moe.make_grouped_config(P, E, H, I, x_rows=T, row_div=k)
    gate2 = torch.empty(P, I, **BF)
    moe.moe_grouped_forward_fp8(in_place, tc, ts, r.pairs, r.offsets, wg.codes, wg.scales, None, gate2,
                                moe.alloc_grouped_fp8_workspace(in_place))
    check_product(gate2, b["xc"], b["xs"], wg, r, "bf16")

    # a captured step, and a second one that shares its workspaces, replayed in turn
    # with eager work between them
    graphs, bufs = [], [buffers(), buffers()]
    for c in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(c)
        graphs.append(g)
    first = r.x.clone()
    for n in range(3):
        r.x.copy_(first * (n + 1))
        for w in work:
            w.fill_(0xFF)
        for g in graphs:
            g.replay()
        step(b)
        torch.cuda.synchronize()
        for c in bufs:
            assert all(torch.equal(c[q], b[q]) for q in b), n


@pytest.mark.parametrize("name", ["few_rows", "ragged"])
def test_experts_in_two_halves(moe, name):
    """Each half's pairs have rows in its own buffer, the other's none; the second
    half's sum begins at the first's."""
    r = Routed(moe, name)
    T, H, E, k, P = r.T, r.H, r.E, r.k, r.P
    off = r.offsets.tolist()
    cut = off[E // 2]
    o = pu.f32(P, H, seed=4).cuda()  # what the experts would answer, in the groups' order
    dy = pu.f32(T, H, seed=5).cuda()
    y, dw = None, torch.zeros(T, k, **F32)
    do = torch.full((P, H), float("nan"), **F32)
    for lo, hi in ((0, cut), (cut, P)):
        n = hi - lo
        c = moe.make_dispatch_config(T, n, k, H, token_dtype="f32", row_dtype="f32")
        pos = r.pos - lo   # another half's: below 0 or past the end
        nxt, part, dpart = torch.empty(T, H, **F32), torch.empty(T, k, **F32), torch.empty(n, H, **F32)
        moe.moe_combine_forward(c, o[lo:hi], pos, r.gw, y, nxt)
        moe.moe_combine_backward(c, dy, o[lo:hi], pos, r.gw, dpart, part)
        y = nxt
        dw += part
        do[lo:hi] = dpart
    terms = d64(o[r.pos.long()]) * d64(r.gw).unsqueeze(-1)
    within(y, terms.sum(1), sum_err(k + 1, terms.abs().sum(1)), "y")
    whole = moe.make_dispatch_config(T, P, k, H, token_dtype="f32", row_dtype="f32")
    dw1, do1 = torch.empty(T, k, **F32), torch.empty(P, H, **F32)
    moe.moe_combine_backward(whole, dy, o, r.pos, r.gw, do1, dw1)
    assert torch.equal(dw, dw1) and torch.equal(do, do1)


@pytest.mark.parametrize("T,k,H", [(5, 3, 264), (300, 8, 1024), (40, 2, 4096)])
def test_row_gradients_in_place_of_the_rows(moe, T, k, H):
    """drows may be rows itself: every row is read before it is written."""
    P = T * k
    cfg = moe.make_dispatch_config(T, P, k, H)
    g = torch.Generator().manual_seed(T)
    pos = torch.randperm(P, generator=g).view(T, k).int().cuda()
    dy, o, w = pu.bf16(T, H, seed=1).cuda(), pu.bf16(P, H, seed=2).cuda(), pu.f32(T, k, seed=3).cuda()
    do, dw = torch.empty(P, H, **BF), torch.empty(T, k, **F32)
    moe.moe_combine_backward(cfg, dy, o, pos, w, do, dw)
    dw2 = torch.empty(T, k, **F32)
    moe.moe_combine_backward(cfg, dy, o, pos, w, o, dw2)
    assert torch.equal(o, do) and torch.equal(dw2, dw)


@pytest.mark.parametrize("name", ["few_rows", "ragged", "many_rows"])
def test_gradient_of_the_rows_in_codes(moe, name):
    """The experts' input gradient is the grouped product of dy's codes and of the
    weights' codes transposed, whose blocks of 128 x 128 keep their scales."""
    r = Routed(moe, name)
    H, E, I, P = r.H, r.E, r.I, r.P
    w = Codes(moe, r.w[2])                       # [E][H][I]
    wt = Codes.__new__(Codes)
    wt.codes, wt.scales = w.codes.transpose(1, 2).contiguous(), w.scales.transpose(1, 2).contiguous()
    do = pu.bf16(P, H, seed=3).cuda()
    c, s = torch.empty(P, H, dtype=torch.uint8, device="cuda"), torch.empty(P, fu.blocks(H), **F32)
    moe.moe_quantize_rows(moe.make_quantize_config(P, H), do, None, c, s)
    for y_dtype, t in (("bf16", torch.bfloat16), ("f32", torch.float32)):
        cfg = moe.make_grouped_config(P, E, H, I, y_dtype=y_dtype)
        dh = torch.empty(P, I, dtype=t, device="cuda")
        moe.moe_grouped_forward_fp8(cfg, c, s, None, r.offsets, wt.codes, wt.scales, None, dh,
                                    moe.alloc_grouped_fp8_workspace(cfg))
        check_product(dh, c, s, wt, r, y_dtype)
        # against the gradient of the formula with the weights as coded: W^T dy
        for e, i, j in r.groups():
            want = fu.values(c[i:j], s[i:j], 1) @ fu.values(w.codes[e], w.scales[e], fu.BLOCK)
            off = ((dh[i:j].double() - want).norm() / want.norm()).item()
            assert off <= (2.0 ** -8 / 3 ** 0.5 + 1e-4 if y_dtype == "bf16" else 1e-5), (e, off)
