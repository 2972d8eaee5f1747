"""The fp8 products, the combine, the balance loss and their gradients behind
one another on one route build, as a layer's training step uses them: each
step's result against the 64-bit formula of what the step before left, and the
router's gradient as a whole against automatic differentiation in 64 bits.

u = 2^-24. Products: |C - exact| <= (gamma(2K + 4 ceil(K/128)) + 2^-10) sum |a b|, 2^-8 of it more
in bf16. H: SiLU(g) u is off by 1.1 |u| dg + |SiLU(g)| du + 2 dg du + (|g| + 8) 2^-22 |h| for the bounds
dg, du of its products, and 2^-4 of its value or 2^-10 of its scale by its code. Combine:
gamma(K') (|y| + sum |w c|); d_topk_w: gamma(d) sum |dy c|; dC: u, and 2^-8 in bf16. Router: with
R the spread of the logits, (2 (R + 18) + 18 + k) u p (|u| + sum |u| p) for the loss and
(2 (R + 18) + 2 k + 8) u w (|dw| + sum w |dw|) for renormalised weights, and the error of d_topk_w
through the same formulas: w (e + sum w e), or p (e + sum p e)."""
import pytest
import torch

from routed_expert_ffn_top_amd import binding as B
from test_gpu_fp8 import bound, gamma, quantise, rows64, spread, stored, decode, unit64, weights, weights64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


class Chain:
    """Buffers and the calls of a step; everything a graph needs is allocated here."""

    def __init__(self, T, E, k, d, f, renorm, resident, g, dt, S=1, off=None, mask=None):
        self.T, self.E, self.k, self.d, self.f, self.S, self.off, self.mask = T, E, k, d, f, S, off, mask
        P = int((resident >= 0).sum())
        self.P, self.phi = P, resident.tolist()
        self.shape = B.make_shape(T, d, f, E, k, P=P, renorm=renorm)
        self.routes, self.ws = B.alloc_routes(self.shape), B.alloc_workspace(self.shape)
        M = self.M = self.shape.capacity
        u8 = lambda *n: torch.zeros(n, dtype=torch.uint8, device="cuda")
        f32 = lambda *n: torch.zeros(n, device="cuda")
        self.x, self.L, self.dY = f32(T, d), f32(T, E), f32(T, d)
        self.a, self.as_ = u8(T, d), u8(T, B.fp8_scale_bytes(d))
        self.h, self.hs = u8(M, f), u8(M, B.fp8_scale_bytes(f))
        self.c, self.dc = torch.zeros((M, d), dtype=dt, device="cuda"), torch.zeros((M, d), dtype=dt, device="cuda")
        self.y, self.dw, self.dL = f32(T, d), f32(T, k), f32(T, E)
        self.loss, self.d_loss = f32(1), torch.full((1,), 0.01, device="cuda")
        self.counts = torch.zeros((S, E), dtype=torch.int32, device="cuda")
        self.prob, self.slope = f32(S, E), f32(S, E)
        self.bws = B.alloc_balance_workspace(self.shape, S)
        gws = B.moe_gate_up_fp8_workspace_bytes(M, f, d, P)
        self.gws = u8(gws + 256)[:gws] if gws else None
        (self.wg, self.sg), (self.wu, self.su), (self.wd, self.sd) = (weights(g, P, *n, "any") for n in ((f, d), (f, d), (d, f)))
        self.sg, self.su, self.sd = (t * 0.2 for t in (self.sg, self.su, self.sd))

    def go(self):
        r = self.routes
        B.moe_route_build(self.shape, 0, self.T, self.L, self.phi, B.MOE_ROUTE_RESET, r, self.ws)
        B.moe_balance_loss(self.shape, self.L, r["topk_idx"], self.loss, self.counts, self.prob, self.slope, self.bws,
                           seq_offset=self.off, mask=self.mask)
        B.moe_quantize_fp8(self.x, self.a, self.as_)
        B.moe_gate_up_fp8(self.a, self.as_, self.wg, self.sg, self.wu, self.su, self.h, self.hs, slot_offset=r["slot_offset"],
                          row_index=r["rec_token"], ws=self.gws)
        B.moe_matmul_fp8(self.h, self.hs, self.wd, self.sd, self.c, slot_offset=r["slot_offset"])
        self.y.zero_()
        B.moe_combine(self.c, r["route_pos"], r["topk_w"], self.y)
        B.moe_combine_backward(self.c, r["route_pos"], r["topk_w"], self.dY, self.dc, self.dw)
        B.moe_router_backward(self.shape, self.L, r["topk_idx"], self.dL, slope=self.slope, d_loss=self.d_loss, d_topk_w=self.dw,
                              seq_offset=self.off, mask=self.mask)

    def fill(self, g):
        self.x.copy_(torch.randn(self.T, self.d, generator=g))
        self.L.copy_(torch.randn(self.T, self.E, generator=g))
        self.dY.copy_(torch.randn(self.T, self.d, generator=g))

    def results(self):
        return [t.clone() for t in (self.loss, self.counts, self.slope, self.y, self.dc, self.dw, self.dL)]


CASES = [(1, 8, 2, 128, 64), (40, 12, 3, 320, 192), (700, 16, 4, 512, 448), (4000, 8, 2, 832, 256)]


@pytest.mark.parametrize("T,E,k,d,f", CASES)
@pytest.mark.parametrize("renorm,all_resident,dt", [(True, True, torch.float32), (False, True, torch.bfloat16), (True, False, torch.bfloat16)])
def test_training_step(T, E, k, d, f, renorm, all_resident, dt):
    g = torch.Generator().manual_seed(T + E)
    resident = torch.arange(E)
    if not all_resident:   # a third of the experts have no slot: their routes are left out
        resident = torch.where(resident % 3 == 2, -1, (resident % 3 != 2).cumsum(0) - 1)
    S, off, mask = 1, None, None
    if T > 3:
        S, off = 3, torch.tensor([1, T // 3, T // 3, T - 1], dtype=torch.int32).cuda()
        mask = (torch.rand(T, generator=g) < 0.8).to(torch.uint8).cuda()
    c = Chain(T, E, k, d, f, renorm, resident, g, dt, S, off, mask)
    c.fill(g)
    c.go()
    torch.cuda.synchronize()
    r = {n: t.cpu() for n, t in c.routes.items()}
    slots, token, pos, w = r["slot_offset"].long(), r["rec_token"].long(), r["route_pos"].long().view(T, k), r["topk_w"].double()
    n = int(slots[-1])
    assert n == int((resident[r["topk_idx"].long()] >= 0).sum()) and n > 0
    # the products
    codes, byte = stored(c.x, 1)
    assert torch.equal(c.a.cpu(), codes) and torch.equal(c.as_.cpu()[:, : byte.shape[1]], byte)
    a64, fb = rows64(c.a, c.as_), -(-f // 128)
    unit = spread(unit64(c.hs.cpu()[:, :fb]), 1, c.M, f)
    h64, C = decode(c.h) * unit, c.c.cpu().double()
    for s in range(c.P):
        lo, hi = int(slots[s]), int(slots[s + 1])
        if lo == hi:
            continue
        av, G, V, D = a64[token[lo:hi]], weights64(c.wg[s], c.sg[s]), weights64(c.wu[s], c.su[s]), weights64(c.wd[s], c.sd[s])
        gate, up, dg, du = av @ G.t(), av @ V.t(), bound(av, G, d, True), bound(av, V, d, True)
        silu = gate * torch.sigmoid(gate)
        h = silu * up
        err = 1.1 * up.abs() * dg + silu.abs() * du + 2 * dg * du + (gate.abs() + 8) * 2.0 ** -22 * h.abs() + 1e-37
        assert bool(((h64[lo:hi] - h).abs() <= err + torch.maximum(2.0 ** -4 * (h.abs() + err), 2.0 ** -10 * unit[lo:hi])).all())
        out, lim = h64[lo:hi] @ D.t(), bound(h64[lo:hi], D, f, True)
        if dt is torch.bfloat16:
            lim = lim + 2.0 ** -8 * (out.abs() + lim)
        assert bool(((C[lo:hi] - out).abs() <= lim + 1e-37).all())
    # the combine and its gradients
    here = pos >= 0
    rows = torch.where(here[..., None], C[pos.clamp(min=0)], 0.0)
    y, size = (w[..., None] * rows).sum(1), (w[..., None] * rows).abs().sum(1)
    assert bool(((c.y.cpu().double() - y).abs() <= gamma(k + 1) * size).all())
    gy = c.dY.cpu().double()
    dw, dwlim = (gy[:, None] * rows).sum(-1), gamma(d) * (gy[:, None] * rows).abs().sum(-1)
    assert bool(((c.dw.cpu().double() - dw).abs() <= dwlim).all())
    want = w[..., None] * gy[:, None]
    got = c.dc.cpu().double()[pos.clamp(min=0)]
    step = U + (2.0 ** -8 if dt is torch.bfloat16 else 0.0)
    assert bool(((got - want).abs() <= (step * 1.01 * want.abs() + 1e-38))[here].all())
    # the router's gradient as a whole
    L = c.L.cpu().double().requires_grad_()
    ids = r["topk_idx"].long()
    p = torch.softmax(L, -1)
    wt = torch.softmax(L.gather(1, ids), -1) if renorm else p.gather(1, ids)
    seq, live = torch.zeros(T, dtype=torch.int64), torch.ones(T, dtype=torch.bool)
    if off is not None:
        o = off.cpu().long()
        seq = torch.searchsorted(o, torch.arange(T), right=True) - 1
        live = (seq >= 0) & (seq < S) & (mask.cpu() != 0)
    loss, full = 0.0, 0
    for s in range(S):
        t = live & (seq == s)
        m = int(t.sum())
        if m:
            cnt = torch.bincount(ids[t].reshape(-1), minlength=E).double()
            loss, full = loss + E / (k * m) * (cnt * p[t].mean(0)).sum(), full + 1
    loss = loss / max(full, 1)
    R = float(c.L.max() - c.L.min())
    value = float(torch.as_tensor(loss).detach())
    assert abs(float(c.loss) - value) <= (R + 18 + 66 + 3) * U * value
    total = 0.01 * loss + (wt * dw).sum() if full else (wt * dw).sum()
    dL, = torch.autograd.grad(total, L)
    p, wt, slope = p.detach(), wt.detach(), c.slope.cpu().double()
    u = torch.where(live[:, None], 0.01 * slope[seq.clamp(0, S - 1)], 0.0)
    lim = torch.zeros_like(p)
    if renorm:
        v = (2 * (R + 18) + 2 * k + 8) * U * (dw.abs() + dwlim) + dwlim
        lim.scatter_add_(1, ids, wt * (v + (wt * v).sum(-1, keepdim=True)))
    else:
        e = torch.zeros_like(p).scatter_add(1, ids, dwlim)
        lim += p * (e + (p * e).sum(-1, keepdim=True))
        u = u.scatter_add(1, ids, dw)
    lim += (2 * (R + 18) + 18 + k) * U * p * (u.abs() + (u.abs() * p).sum(-1, keepdim=True)) + U * dL.abs() + 1e-37
    err = (c.dL.cpu().double() - dL).abs()
    assert bool((err <= lim).all()), f"{float((err / lim).max()):.3g} of the bound"


def test_training_step_captured_and_on_two_streams():
    """The same bits from a call alone, from two streams at once, and from a graph replayed with eager calls in between."""
    T, E, k, d, f = 700, 16, 4, 512, 448

    def chain():
        return Chain(T, E, k, d, f, False, torch.arange(E), torch.Generator().manual_seed(0), torch.bfloat16)

    one, want = chain(), []
    for i in range(3):
        one.fill(torch.Generator().manual_seed(i))
        one.go()
        want.append(one.results())
    torch.cuda.synchronize()
    two, streams = [one, chain()], [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(4):
        for c, s, j in zip(two, streams, (i % 3, (i + 1) % 3)):
            with torch.cuda.stream(s):
                c.fill(torch.Generator().manual_seed(j))
                c.go()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(two[0].results(), want[0]))
    assert all(torch.equal(a, b) for a, b in zip(two[1].results(), want[1]))
    c, graph = chain(), torch.cuda.CUDAGraph()
    c.fill(torch.Generator().manual_seed(0))
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.go()
    for i in (2, 0, 1, 1):
        c.fill(torch.Generator().manual_seed(i))
        graph.replay()
        torch.cuda.synchronize()
        one.go()
        assert all(torch.equal(a, b) for a, b in zip(c.results(), want[i]))
