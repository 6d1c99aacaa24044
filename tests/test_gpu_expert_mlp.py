"""The grouped products and SwiGLU together, as a routed layer in training
uses them: moe_route and moe_permute give the groups, the tokens are gathered
in place, and the forward pass must reproduce moe_forward's own intermediates
and output; the backward pass runs the same calls backwards."""
import pytest
import torch

import synth
from tests import gpu_util as gu
from tests import product_util as pu
from tests.product_util import sum_err, within

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
    return m


CASES = {
    "few_rows": dict(T=9, H=256, E=16, k=4, I=64, Is=64),
    "ragged": dict(T=300, H=256, E=8, k=2, I=128, Is=128, limit=2.0),
    "many_rows": dict(T=1100, H=512, E=4, k=3, I=192, Is=64),
}


@pytest.mark.parametrize("name", list(CASES))
def test_expert_mlp_forward_and_backward(moe, name):
    wl = synth.WORKLOADS["tiny"].with_(name=name, **CASES[name])
    inp = synth.make_inputs(wl)
    d = gu.upload(inp)
    cfg = gu.cfg_of(wl)
    T, H, E, k, I, P = wl.T, wl.H, wl.E, wl.k, wl.I, wl.T * wl.k
    bf = dict(dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    ws = moe.alloc_workspace(cfg)

    # the layer's own forward pass and its intermediates
    ids, gw = torch.empty(T, k, **i32), torch.empty(T, k, dtype=torch.float32, device="cuda")
    y = torch.empty(T, H, **bf)
    moe.moe_forward(cfg, d.x, d.router_w, d.router_b, d.w_gate, d.w_up, d.w_down, d.ws_gate,
                    d.ws_up, d.ws_down, y, ids, gw, ws)
    torch.cuda.synchronize()
    off, nb = moe.moe_workspace_view(cfg, moe.MOE_WS_H)
    h_layer = ws[off:off + nb].view(torch.bfloat16)[:P * I].view(P, I).clone()

    # the same from the parts
    offsets, pairs, pos = torch.empty(E + 1, **i32), torch.empty(P, **i32), torch.empty(P, **i32)
    moe.moe_permute(cfg, ids, offsets, pairs, pos, ws)
    up_cfg = moe.make_grouped_config(P, E, H, I, x_rows=T, row_div=k)
    dn_cfg = moe.make_grouped_config(P, E, I, H, y_dtype="f32")
    act = moe.make_swiglu_config(P, I, ld=2 * I, limit=wl.limit)
    wu, wd = moe.alloc_grouped_workspace(up_cfg), moe.alloc_grouped_workspace(dn_cfg)
    gate, up = torch.empty(P, I, **bf), torch.empty(P, I, **bf)
    gu_ = torch.empty(P, 2 * I, **bf)
    h, o = torch.empty(P, I, **bf), torch.empty(P, H, device="cuda")
    moe.moe_grouped_forward(up_cfg, d.x, pairs, offsets, d.w_gate.view(E, I, H), None, gate, wu)
    moe.moe_grouped_forward(up_cfg, d.x, pairs, offsets, d.w_up.view(E, I, H), None, up, wu)
    gu_[:, :I], gu_[:, I:] = gate, up
    moe.moe_swiglu_forward(act, gu_[:, :I], gu_[:, I:], h)
    moe.moe_grouped_forward(dn_cfg, h, None, offsets, d.w_down.view(E, H, I), None, o, wd)

    # h: the layer rounds once, from unrounded gate and up; here both are
    # rounded on the way: each moves h by its half step, |dh/dg| <= 1.1 |u|
    g_, u_, hl = gate.cpu().double(), up.cpu().double(), h_layer.cpu().double()
    lim = wl.limit if wl.limit > 0 else float("inf")
    gc, uc = g_.clamp(max=lim), u_.clamp(-lim, lim)
    bound = 1.02 * pu.BF16_HALF * (1.1 * gc.abs() * uc.abs() + (gc * uc).abs() + 2 * hl.abs()) + 1e-6
    within(h.cpu(), hl, bound, "h")
    # y: shared + weighted routed rows; against the layer within its own bound
    shared = torch.zeros(T, H, dtype=torch.double)
    if wl.Is:
        xs = inp_f64(d.x)
        wsg, wsu, wsd = (inp_f64(t) for t in (d.ws_gate, d.ws_up, d.ws_down))
        gs, us = xs @ wsg.view(wl.Is, H).t(), xs @ wsu.view(wl.Is, H).t()
        ls = wl.limit_shared if wl.limit_shared > 0 else float("inf")
        shared = pu.act(gs.clamp(max=ls), "silu") * us.clamp(-ls, ls) @ wsd.view(H, wl.Is).t()
    rows = o.cpu().double()[pos.cpu().long()].view(T, k, H)
    y_parts = shared + (gw.cpu().double().unsqueeze(-1) * rows).sum(1)
    m = y.cpu().double().abs().max()
    assert ((y_parts - y.cpu().double()).abs() <= gu.Y_RTOL_M * m + gu.Y_ATOL).all()

    # the backward pass for a random gradient of y
    dy = pu.bf16(T, H, seed=5).cuda()
    w_sorted = gw.view(-1)[pairs.long()]
    do = (dy.float()[(pairs // k).long()] * w_sorted.unsqueeze(1)).to(torch.bfloat16)
    dh, dgu = torch.empty(P, I, **bf), torch.empty(P, 2 * I, **bf)
    h2 = torch.empty(P, I, **bf)
    dxs = [torch.empty(P, H, **bf) for _ in range(2)]
    f32 = dict(dtype=torch.float32, device="cuda")
    dwd, dwg, dwu = (torch.empty(E, H, I, **f32), torch.empty(E, I, H, **f32),
                     torch.empty(E, I, H, **f32))
    moe.moe_grouped_backward(dn_cfg, do, h, None, offsets, d.w_down.view(E, H, I), dh, dwd, None, wd)
    moe.moe_swiglu_backward(act, dh, gu_[:, :I], gu_[:, I:], dgu[:, :I], dgu[:, I:], h2)
    dgate, dup = dgu[:, :I].contiguous(), dgu[:, I:].contiguous()
    moe.moe_grouped_backward(up_cfg, dgate, d.x, pairs, offsets, d.w_gate.view(E, I, H), dxs[0],
                             dwg, None, wu)
    moe.moe_grouped_backward(up_cfg, dup, d.x, pairs, offsets, d.w_up.view(E, I, H), dxs[1], dwu,
                             None, wu)
    torch.cuda.synchronize()
    assert torch.equal(h2, h)

    # every weight's gradient against the definition in 64 bits, from the
    # same rounded rows; and the chain from do to dx in 64 bits throughout,
    # whose intermediate roundings (h, dh, dgate, dup: 2^-8 each) add up to
    # less than 6 2^-8 of the magnitudes that meet in a sum
    off_h, x = offsets.tolist(), inp_f64(d.x)
    tok = (pairs // k).cpu().long()
    wg, wup, wdn = (inp_f64(t) for t in (d.w_gate, d.w_up, d.w_down))
    wg, wup, wdn = wg.view(E, I, H), wup.view(E, I, H), wdn.view(E, H, I)
    for e in range(E):
        i, j = off_h[e], off_h[e + 1]
        for got, a, b in ((dwd[e], do, h), (dwg[e], dgate, None), (dwu[e], dup, None)):
            av = a[i:j].cpu().double()
            bv = h[i:j].cpu().double() if b is not None else x[tok[i:j]]
            within(got.cpu(), av.t() @ bv, sum_err(j - i, av.abs().t() @ bv.abs()) + 1e-30,
                   f"dw of expert {e}")
        if i == j:
            continue
        xe, doe = x[tok[i:j]], do[i:j].cpu().double()
        g, u = (xe @ wg[e].t()).requires_grad_(), (xe @ wup[e].t()).requires_grad_()
        hh = pu.act(g.clamp(max=lim), "silu") * u.clamp(-lim, lim)
        dg, du = torch.autograd.grad((hh * (doe @ wdn[e])).sum(), (g, u))
        want = dg @ wg[e] + du @ wup[e]
        near = (g.detach() - lim).abs() < 0.05  # rounding may cross the clamp there
        near |= (u.detach().abs() - lim).abs() < 0.05
        clean = ~near.any(1)
        dhm = doe.abs() @ wdn[e].abs()
        mg = dhm * u.detach().abs().clamp(max=lim) * 1.1 * 2
        mu = dhm * g.detach().abs().clamp(max=lim) * 1.1 * 2
        bound = 6 * pu.BF16_HALF * (mg @ wg[e].abs() + mu @ wup[e].abs())
        got = (dxs[0][i:j].double() + dxs[1][i:j].double()).cpu()
        within(got[clean], want[clean], bound[clean], f"dx of expert {e}")


def inp_f64(t):
    return t.cpu().double()
