"""The combine of record rows with its gradients, the balance loss and the
gradient of the router's logits, against their formulas in 64 bits.

u = 2^-24, gamma(n) = n u / (1 - n u). Combine: one fused multiply-add a route,
|Y - exact| <= gamma(K') (|y| + sum |w c|); a dot product of d terms in whatever
order is within gamma(d) sum |dy c|; w dy is rounded once to fp32, and to bf16
by at most 2^-8 of it.

Probabilities: exp's argument is off by u |v - m|, exp itself by at most 2 u,
the sum of E terms (C = E / 64 a lane, 6 exchanges) by 10 u, the reciprocal and
the product by 2 u each: (R + 18) u of p, R the largest |v - m|. Mean
probabilities add at most 64 + 2 fp32 additions of positive terms, and the
rounding of the result. The gradient p (u - sum u p) is off by the errors of p,
of the sum (10 additions and a product) and of the difference:
(2 (R + 18) + 16) u p (|u| + sum |u| p), u off by 2 u more where the route weights'
gradient is added; the renormalised weights' w (dw - sum w dw) likewise, with
k additions: (2 (R + 18) + 2 k + 8) u w (|dw| + sum w |dw|)."""
import pytest
import torch

from routed_expert_ffn_top_amd import binding as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def gamma(n):
    return n * U / (1 - n * U)


def rows(g, n, d, pad, dt=torch.float32):
    return torch.randn(n, d + pad, generator=g).to(dt).cuda()[:, :d]


def positions(g, n, M, absent):
    """Records of n routes: different ones out of M, some routes left out."""
    pos = torch.full((n,), -1, dtype=torch.int64)
    here = torch.rand(n, generator=g) >= absent
    pos[here] = torch.randperm(M, generator=g)[: int(here.sum())]
    return pos


COMBINE = [(1, 4, 1, 1), (3, 12, 2, 6), (33, 324, 5, 170), (7, 100, 64, 500), (64, 2048, 8, 512), (5, 8200, 9, 45), (257, 64, 3, 771),
           (2, 256, 17, 34)]


@pytest.mark.parametrize("T,d,kp,M", COMBINE)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("absent,pad", [(0.0, 0), (0.3, 4), (1.0, 0)])
def test_combine(T, d, kp, M, dt, absent, pad):
    g = torch.Generator().manual_seed(T + d + kp)
    pos = positions(g, T * kp, M, absent)
    C, w = rows(g, M, d, pad, dt), torch.rand(T, kp, generator=g)
    Y, dY = rows(g, T, d, pad), rows(g, T, d, pad)
    back = torch.full((M, d + pad), 77.0, dtype=dt, device="cuda")
    dC, dw = back[:, :d], torch.full((T, kp), 5.0, device="cuda")
    y0, c, gy = Y.cpu().double(), C.cpu().double(), dY.cpu().double()
    given = pos.clone()
    given[(pos < 0) & (torch.arange(T * kp) % 2 == 0)] = M + 5   # out of range: left out too
    p = given.int().cuda()
    B.moe_combine(C, p, w.cuda(), Y)
    B.moe_combine_backward(C, p, w.cuda(), dY, dC, dw)
    only = torch.full((T, kp), 5.0, device="cuda")
    B.moe_combine_backward(C, p, w.cuda(), dY, None, only)
    torch.cuda.synchronize()
    assert torch.equal(only, dw)
    here = (pos >= 0).reshape(T, kp, 1)
    r = torch.where(here, c[pos.clamp(min=0)].reshape(T, kp, d), 0.0)
    wr = w.double()[..., None] * r
    lim = gamma(kp) * (y0.abs() + wr.abs().sum(1))
    assert bool(((Y.cpu().double() - (y0 + wr.sum(1))).abs() <= lim).all())
    t = gy[:, None, :] * r
    assert bool(((dw.cpu().double() - t.sum(-1)).abs() <= gamma(d) * t.abs().sum(-1)).all())
    want = torch.full((M, d), 77.0, dtype=torch.float64)
    want[pos[pos >= 0]] = (w.double()[..., None] * gy[:, None, :]).reshape(-1, d)[pos >= 0]
    step = 0.0 if dt is torch.float32 else 2.0 ** -8
    got = dC.cpu().double()
    assert bool(((got - want).abs() <= (U + step * (1 + U)) * want.abs()).all())
    assert bool((back[:, d:] == 77.0).all())


def test_combine_rows_nobody_has_do_not_count():
    """Rows of no route may hold anything, NaN among it; a NaN row of a route makes its token NaN alone."""
    C = torch.full((4, 64), float("nan"), device="cuda")
    C[1] = 2.0
    Y, w = torch.ones((2, 64), device="cuda"), torch.ones((2, 2), device="cuda")
    pos = torch.tensor([1, -1, -1, 3], dtype=torch.int32).cuda()
    B.moe_combine(C, pos, w, Y)
    assert bool((Y[0] == 3.0).all()) and bool(Y[1].isnan().all())
    none = torch.full((4,), -1, dtype=torch.int32).cuda()
    Y.fill_(1.0)
    B.moe_combine(C, none, w, Y)
    assert bool((Y == 1.0).all())
    B.moe_combine(C[:0], none, w, Y)      # no record at all
    assert bool((Y == 1.0).all())


def test_combine_gradient_by_differences():
    """d (sum Y G) / dw and / dC by differences in 64 bits: both are linear, so a difference of 1 is exact up to rounding."""
    g = torch.Generator().manual_seed(2)
    T, d, kp, M = 3, 20, 2, 6
    C, w, G = torch.randn(M, d, generator=g), torch.rand(T, kp, generator=g), torch.randn(T, d, generator=g)
    pos = positions(g, T * kp, M, 0.2)

    def f(C, w):
        r = torch.where((pos >= 0)[:, None], C[pos.clamp(min=0)], 0.0).reshape(T, kp, d)
        return ((w[..., None] * r).sum(1) * G.double()).sum()

    dC, dw = torch.zeros((M, d), device="cuda"), torch.empty((T, kp), device="cuda")
    B.moe_combine_backward(C.cuda(), pos.int().cuda(), w.cuda(), G.cuda(), dC, dw)
    C, w = C.double(), w.double()
    for i in range(T * kp):
        e = torch.zeros(T * kp, dtype=torch.float64)
        e[i] = 1.0
        diff = float(f(C, w + e.reshape(T, kp)) - f(C, w))
        assert abs(float(dw.reshape(-1)[i]) - diff) <= 1e-5 * d      # gamma(20) of sums below 20 * 3 * 3
    for i in range(0, M * d, 7):
        e = torch.zeros(M * d, dtype=torch.float64)
        e[i] = 1.0
        assert abs(float(dC.reshape(-1)[i]) - float(f(C + e.reshape(M, d), w) - f(C, w))) <= 1e-6


# ---- balance ----

def probabilities(L):
    L = torch.where(L.isnan(), -float("inf"), L.double())
    m = L.amax(-1, keepdim=True)
    z = torch.exp(L - torch.where(m == -float("inf"), 0.0, m))
    s = z.sum(-1, keepdim=True)
    return torch.where(s > 0, z / s, 0.0), z


def sequences(T, off):
    """Which sequence a token is in, -1 for none."""
    if off is None:
        return torch.zeros(T, dtype=torch.int64)
    s = torch.searchsorted(off, torch.arange(T), right=True) - 1
    return torch.where(s < len(off) - 1, s, -1)


def formula(L, idx, E, k, S, off, mask):
    """loss, counts, P, d loss / d p (less its mean) in 64 bits."""
    p, _ = probabilities(L)
    seq = sequences(len(L), off)
    live = (seq >= 0) & (torch.ones(len(L), dtype=torch.bool) if mask is None else mask != 0)
    counts, P, slope = torch.zeros((S, E), dtype=torch.int64), torch.zeros((S, E), dtype=torch.float64), torch.zeros((S, E), dtype=torch.float64)
    loss, some = 0.0, 0
    for s in range(S):
        m = live & (seq == s)
        n = int(m.sum())
        if n == 0:
            continue
        some += 1
        ids = idx[m][:, :k].reshape(-1)
        counts[s] = torch.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
        P[s] = p[m].mean(0)
        loss = loss + E / (k * n) * (counts[s].double() * P[s]).sum()
        slope[s] = E / (k * n * n) * (counts[s].double() - k * n / E)
    return loss / max(some, 1), counts, P, slope / max(some, 1), seq, live


def run_balance(shape, L, idx, S, off, mask):
    E = shape.E
    new = lambda *n, dt=torch.float32: torch.full(n, 99, dtype=dt, device="cuda")
    o = dict(loss=new(1), counts=new(S, E, dt=torch.int32), prob=new(S, E), slope=new(S, E))
    ws = B.alloc_balance_workspace(shape, S)
    ws.fill_(0xEE)
    B.moe_balance_loss(shape, L, idx, o["loss"], o["counts"], o["prob"], o["slope"], ws, seq_offset=off, mask=mask)
    return o


def choice(L, k, shared, E):
    v = torch.where(L.isnan(), -float("inf"), L)
    i = torch.sort(v, dim=-1, descending=True, stable=True)[1][:, :k]
    return torch.cat([i, torch.arange(E, E + shared).expand(len(L), -1)], 1).int()


def check_balance(T, E, k, shared, S, off, mask, renorm, weights, L=None, idx=None, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(T + E + k + S + seed)
    if L is None:
        L = torch.randn(T, E, generator=g) * scale + torch.randn(E, generator=g)
    if idx is None:
        idx = choice(L, k, shared, E)
    dw = torch.randn(T, k + shared, generator=g) if weights else None
    shape = B.make_shape(T, 64, 64, E, k, shared, renorm=renorm)
    c = lambda t, dt=None: None if t is None else (t if dt is None else t.to(dt)).cuda()
    o = run_balance(shape, c(L), c(idx), S, c(off, torch.int32), c(mask))
    loss, counts, P, slope, seq, live = formula(L, idx.long(), E, k, S, off, mask)
    assert torch.equal(o["counts"].cpu().long(), counts)
    fin = L[L.isfinite()]
    R = float(fin.max() - fin.min()) if fin.numel() else 0.0
    near = (R + 18 + 66 + 2) * U
    assert bool(((o["prob"].cpu().double() - P).abs() <= near * P + 1e-38).all())
    assert abs(float(o["loss"]) - float(loss)) <= near * float(loss) + U * float(loss)
    assert bool(((o["slope"].cpu().double() - slope).abs() <= 1.01 * U * slope.abs() + 1e-38).all())
    # the gradient
    d_loss = torch.tensor([0.37])
    out = torch.full((T, E), 99.0, device="cuda")
    B.moe_router_backward(shape, c(L), c(idx), out, slope=o["slope"], d_loss=c(d_loss), d_topk_w=c(dw),
                          seq_offset=c(off, torch.int32), mask=c(mask))
    p, z = probabilities(L)
    u = torch.where(live[:, None], float(d_loss) * slope[seq.clamp(min=0)], 0.0)
    x, xlim = torch.zeros_like(p), torch.zeros_like(p)
    if weights:
        ids, d = idx[:, :k].long(), dw[:, :k].double()
        ok = (ids >= 0) & (ids < E)
        ids = torch.where(ok, ids, 0)
        if renorm:
            zs = torch.where(ok, z.gather(1, ids), 0.0)
            den = zs.sum(-1, keepdim=True)
            w = torch.where(den > 0, zs / den, 0.0)
            x.scatter_add_(1, ids, w * (d - (w * d).sum(-1, keepdim=True)))
            xlim.scatter_add_(1, ids, (2 * (R + 18) + 2 * k + 8) * U * w * (d.abs() + (w * d.abs()).sum(-1, keepdim=True)))
        else:
            u = u.scatter_add(1, ids, torch.where(ok, d, 0.0))
    want = p * (u - (u * p).sum(-1, keepdim=True)) + x
    lim = (2 * (R + 18) + 16 + k) * U * p * (u.abs() + (u.abs() * p).sum(-1, keepdim=True)) + xlim + U * want.abs() + 1e-37
    err = (out.cpu().double() - want).abs()
    assert bool((err <= lim).all()), f"{float((err / lim).max()):.3g} of the bound"
    return o, out


@pytest.mark.parametrize("T,E,k,shared", [(1, 1, 1, 0), (1, 8, 2, 0), (16, 8, 2, 0), (100, 64, 8, 2), (333, 65, 3, 1), (1000, 128, 6, 0),
                                          (517, 200, 8, 2), (300, 256, 64, 0), (4099, 256, 8, 1), (20000, 6, 2, 0)])
@pytest.mark.parametrize("renorm,weights", [(True, True), (False, True), (True, False)])
@pytest.mark.parametrize("layout", ["all", "sequences", "padded"])
def test_balance(T, E, k, shared, renorm, weights, layout):
    if k > E or k + shared > 64:
        pytest.skip("not a shape")
    g = torch.Generator().manual_seed(T)
    off = mask = None
    S = 1
    if layout == "sequences":   # some empty, tokens before the first and behind the last
        S = min(70, T) + 3
        cut = torch.sort(torch.randint(0, T + 1, (S + 1,), generator=g))[0]
        cut[1] = cut[0]
        off = cut
    elif layout == "padded":
        mask = (torch.rand(T, generator=g) < 0.6).to(torch.uint8)
    check_balance(T, E, k, shared, S, off, mask, renorm, weights)


def test_balance_both_and_many_sequences():
    T, S = 9000, 4096
    g = torch.Generator().manual_seed(0)
    off = torch.sort(torch.randint(0, T, (S + 1,), generator=g))[0]
    mask = (torch.rand(T, generator=g) < 0.3).to(torch.uint8)
    check_balance(T, 24, 3, 0, S, off, mask, True, True)


def test_balance_long():
    """Chunks of 256 tokens."""
    check_balance(70001, 16, 2, 0, 1, None, None, False, True)
    off = torch.tensor([0, 5, 65000, 70001])
    check_balance(70001, 16, 2, 0, 3, off, None, True, True, seed=1)


@pytest.mark.parametrize("renorm", [True, False])
def test_balance_special_logits(renorm):
    """NaN and -infinity, whole rows of them, the lowest number, equal logits, far ones."""
    L = torch.randn(12, 70, generator=torch.Generator().manual_seed(0))
    L[0] = float("nan")
    L[1] = -float("inf")
    L[2, ::2] = float("nan")
    L[3, 5:] = -float("inf")
    L[4] = torch.finfo(torch.float32).min
    L[5] = 1.0
    L[6, :60] = torch.finfo(torch.float32).min
    L[7, 3] = 200.0
    far = L[[0, 1, 2, 3, 5, 7, 8, 9, 10, 11]]
    check_balance(10, 70, 4, 0, 1, None, None, renorm, True, L=far)
    # rows of the lowest number only, whose differences are exact
    low = L[[4, 4, 4]]
    o, out = check_balance(3, 70, 4, 0, 1, None, None, renorm, True, L=low)
    shape = B.make_shape(12, 64, 64, 70, 4, renorm=renorm)
    o = run_balance(shape, L.cuda(), choice(L, 4, 0, 70).cuda(), 1, None, None)
    out = torch.full((12, 70), 9.0, device="cuda")
    B.moe_router_backward(shape, L.cuda(), choice(L, 4, 0, 70).cuda(), out, slope=o["slope"], d_topk_w=torch.ones((12, 4), device="cuda"))
    assert bool(out.isfinite().all()) and bool(o["prob"].isfinite().all())
    assert bool((out[:2] == 0).all())


def test_balance_ids_twice_and_out_of_range():
    g = torch.Generator().manual_seed(6)
    idx = torch.randint(-3, 23, (50, 5), generator=g).int()
    idx[:, 1] = idx[:, 0]
    for renorm in (True, False):
        check_balance(50, 20, 5, 0, 1, None, None, renorm, True, idx=idx)


def test_balance_nothing_counted():
    shape = B.make_shape(6, 64, 64, 8, 2)
    L = torch.randn(6, 8).cuda()
    idx = choice(L.cpu(), 2, 0, 8).cuda()
    zero = torch.zeros(6, dtype=torch.uint8, device="cuda")
    for off, mask, S in ((None, zero, 1), (torch.tensor([3, 3, 3], dtype=torch.int32).cuda(), None, 2)):
        o = run_balance(shape, L, idx, S, off, mask)
        assert all(bool((t == 0).all()) for t in o.values())
        out = torch.full((6, 8), 9.0, device="cuda")
        B.moe_router_backward(shape, L, idx, out, slope=o["slope"], seq_offset=off, mask=mask)
        assert bool((out == 0).all())
    none = B.make_shape(0, 64, 64, 8, 2)
    o = run_balance(none, L[:0], idx[:0], 1, None, None)
    assert all(bool((t == 0).all()) for t in o.values())
    B.moe_router_backward(none, L[:0], idx[:0], L[:0], slope=o["slope"])


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_padding_may_hold_anything(renorm, bad):
    """Tokens that are not counted and whose weights have no gradient: 0, and nothing of theirs anywhere."""
    T, E, k = 40, 100, 3
    g = torch.Generator().manual_seed(11)
    L, dw = torch.randn(T, E, generator=g), torch.randn(T, k, generator=g)
    idx, mask = choice(L, k, 0, E), (torch.arange(T) % 3 != 0).to(torch.uint8)
    dw[mask == 0] = 0.0
    shape = B.make_shape(T, 64, 64, E, k, renorm=renorm)
    got = []
    for logits in (L, torch.where((mask == 0)[:, None] & (torch.arange(E) % 2 == 0), bad, L)):
        o = run_balance(shape, logits.cuda(), idx.cuda(), 1, None, mask.cuda())
        out = torch.full((T, E), 9.0, device="cuda")
        B.moe_router_backward(shape, logits.cuda(), idx.cuda(), out, slope=o["slope"], d_topk_w=dw.cuda(), mask=mask.cuda())
        got.append((o["loss"], o["prob"], out))
    assert all(torch.equal(x, y) for x, y in zip(*got)) and bool((got[1][2][(mask == 0).cuda()] == 0).all())


@pytest.mark.parametrize("E", [126, 128, 252, 256])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_router_rows_of_every_alignment(E, at):
    """Logits and gradients that begin at any multiple of 4 bytes: whether rows are read in pieces or not."""
    T, k = 37, 4
    g = torch.Generator().manual_seed(E)
    L, dw = torch.randn(T, E, generator=g), torch.randn(T, k, generator=g).cuda()
    idx = choice(L, k, 0, E).cuda()
    for renorm in (True, False):
        shape = B.make_shape(T, 64, 64, E, k, renorm=renorm)
        outs = []
        for shift in (0, at):
            place = lambda: torch.empty(T * E + 4, device="cuda")[shift:shift + T * E].view(T, E)
            logits, out = place(), place()
            logits.copy_(L)
            o = run_balance(shape, logits, idx, 1, None, None)
            B.moe_router_backward(shape, logits, idx, out, slope=o["slope"], d_topk_w=dw)
            outs.append((o["loss"], o["slope"], out.cpu().double()))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
        # another distribution of experts over lanes, another order of the same sums: twice their bound at worst
        p = torch.softmax(L.double(), -1)
        u = outs[0][1].cpu().double() + (0 if renorm else torch.zeros_like(p).scatter_add(1, idx.cpu().long(), dw.cpu().double()))
        R = float(L.max() - L.min())
        lim = 2 * (2 * (R + 18) + 16 + k) * U * p * (u.abs() + (u.abs() * p).sum(-1, keepdim=True)) + 2 * U * outs[0][2].abs()
        if renorm:
            c = idx.cpu().long()
            w = torch.softmax(L.double().gather(1, c), -1)
            d = dw.cpu().double().abs()
            lim = lim.scatter_add(1, c, 2 * (2 * (R + 18) + 2 * k + 8) * U * w * (d + (w * d).sum(-1, keepdim=True)))
        assert bool(((outs[0][2] - outs[1][2]).abs() <= lim + 1e-37).all())


def test_balance_uniform_is_one():
    """Uniform routing and probabilities: the loss is 1 and its gradient 0."""
    T, E, k = 64, 8, 2
    idx = torch.stack([torch.arange(T) % E, (torch.arange(T) + 1) % E], 1).int().cuda()
    shape = B.make_shape(T, 64, 64, E, k)
    L = torch.zeros((T, E), device="cuda")
    o = run_balance(shape, L, idx, 1, None, None)
    assert float(o["loss"]) == 1.0 and bool((o["slope"] == 0).all()) and bool((o["counts"] == T * k // E).all())


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_by_differences(renorm):
    """d_logits against central differences of the formula in 64 bits: with steps of e = 2^-9 these are off by e^2 / 6
    of a third derivative, at most 6 max |u| for p (u - sum u p) and as much for the weights, and by 2^-52 / e of the value."""
    T, E, k, S = 5, 9, 3, 2
    g = torch.Generator().manual_seed(8)
    L, off = torch.randn(T, E, generator=g), torch.tensor([0, 2, 5])
    idx = choice(L, k, 0, E)
    dw, d_loss = torch.randn(T, k, generator=g), 0.7
    shape = B.make_shape(T, 64, 64, E, k, renorm=renorm)
    o = run_balance(shape, L.cuda(), idx.cuda(), S, off.int().cuda(), None)
    out = torch.empty((T, E), device="cuda")
    B.moe_router_backward(shape, L.cuda(), idx.cuda(), out, slope=o["slope"], d_loss=torch.tensor([d_loss]).cuda(),
                          d_topk_w=dw.cuda(), seq_offset=off.int().cuda())

    def f(L):
        p, z = probabilities(L)
        w = z.gather(1, idx.long()) if renorm else p.gather(1, idx.long())
        w = w / w.sum(-1, keepdim=True) if renorm else w
        return float(torch.tensor(d_loss)) * formula(L, idx.long(), E, k, S, off, None)[0] + (w * dw.double()).sum()

    e, top = 2.0 ** -9, float(dw.abs().max()) + float(o["slope"].abs().max())
    for t in range(T):
        for j in range(E):
            step = torch.zeros((T, E), dtype=torch.float64)
            step[t, j] = e
            diff = float(f(L.double() + step) - f(L.double() - step)) / (2 * e)
            assert abs(float(out[t, j]) - diff) <= 2 * e * e * top + 1e-5 * top


def test_balance_graph_and_streams():
    """Captured and replayed on new inputs, and on two streams with a workspace each: the bits of a call alone."""
    T, E, k, S = 700, 64, 8, 5
    shape = B.make_shape(T, 64, 64, E, k, renorm=False)
    g = torch.Generator().manual_seed(3)
    off = torch.tensor([0, 100, 100, 333, 600, 690], dtype=torch.int32).cuda()
    Ls = [torch.randn(T, E, generator=g) for _ in range(4)]
    ids = [choice(L, k, 0, E).cuda() for L in Ls]
    dw = torch.randn(T, k, generator=g).cuda()

    class Run:
        def __init__(self):
            new = lambda *n, dt=torch.float32: torch.empty(n, dtype=dt, device="cuda")
            self.L, self.idx, self.out = new(T, E), new(T, k, dt=torch.int32), new(T, E)
            self.o = dict(loss=new(1), counts=new(S, E, dt=torch.int32), prob=new(S, E), slope=new(S, E))
            self.ws = B.alloc_balance_workspace(shape, S)

        def take(self, i):
            self.L.copy_(Ls[i])
            self.idx.copy_(ids[i])

        def go(self):
            o = self.o
            B.moe_balance_loss(shape, self.L, self.idx, o["loss"], o["counts"], o["prob"], o["slope"], self.ws, seq_offset=off)
            B.moe_router_backward(shape, self.L, self.idx, self.out, slope=o["slope"], d_loss=o["loss"], d_topk_w=dw, seq_offset=off)

        def same(self, other):
            return torch.equal(self.out, other.out) and all(torch.equal(self.o[n], other.o[n]) for n in self.o)

    want = []
    for i in range(4):
        r = Run()
        r.take(i)
        r.go()
        want.append(r)
    torch.cuda.synchronize()
    runs, streams = [Run(), Run()], [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(6):
        for r, s, n in zip(runs, streams, (i % 4, (i + 1) % 4)):
            with torch.cuda.stream(s):
                r.take(n)
                r.go()
    torch.cuda.synchronize()
    assert runs[0].same(want[1]) and runs[1].same(want[2])
    r, graph = Run(), torch.cuda.CUDAGraph()
    r.take(0)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        r.go()
    for i in (2, 0, 3, 1):
        r.take(i)
        graph.replay()
        torch.cuda.synchronize()
        assert r.same(want[i])
