"""The expert FFN on MXFP4 activations (MOE_FFN_ACT_MXFP4) against its
definition in 64 bits: X as stored blocks, H = SiLU(g) u quantised from its
fp32 values, both projections on codes.

The bound. g and u are off by at most gamma(2d) of their sums of magnitudes
(see test_gpu_mxfp4.py); |SiLU'| <= 1.1. The exponent g log2(e) is off by
2 u of itself (the constant and the product), so 2 to it by 2 u |g| and its own 2 u,
and the reciprocal and the products add less than 10 u: all within
(16 + 2 |g|) u |h|, so h lies in [h - e, h + e] with
e = 1.1 e_g |u| + |SiLU(g)| e_u + 1.1 e_g e_u + (16 + 2 |g|) u |h|. A block's scale is one
that its largest magnitude can have within its own e, and for a given scale the
stored value never falls as h grows: it lies between the stored values of h - e
and h + e (for most values these are one code). Y is then off by at most
alpha sum |W_d| times that interval's reach, gamma(2f) of its sums of
magnitudes, and gamma(K' + 2) of what is added to the residual."""
import numpy as np
import pytest
import torch

from gpu_util import OracleRun, gpu_inputs, say
from oracle import oracle as oracle_mod
from routed_expert_ffn_top_amd import binding as B
from routed_expert_ffn_top_amd.inputs import MoEConfig, quantize_mxfp4
from routed_expert_ffn_top_amd.layer import MoELayer
from test_gpu_mxfp4 import MAG, U, gamma, quantise, two_to, values

pytestmark = pytest.mark.gpu


def cfg_of(T, d, f, E, k, shared=0):
    return MoEConfig(name=f"mx_layer_{T}_{d}_{f}", index=79, T=T, d=d, f=f, E=E, k=k, n_shared=shared, dtype="bf16_fp4w")


def scale_of(top):
    _, e = torch.frexp(top)
    return torch.where(top > 0, (e - 1 - 2 + 127).clamp(0, 254), 0).int()


def stored_at(h, byte):
    """Values [..][32] as they are stored under the scale byte of their block."""
    unit = two_to(byte - 127)[..., None]
    a = (h.abs() / unit).clamp(max=6.0)
    d = (a[..., None] - MAG).abs()
    near = d == d.amin(-1, keepdim=True)
    code = torch.where(near & (torch.arange(8) % 2 == 0), torch.arange(8) + 100, torch.where(near, torch.arange(8), -1))
    return torch.sign(h) * MAG[code.amax(-1) % 100] * unit


def reference(inp, idx, alpha):
    """(Y, bound) [T][d] in 64 bits, on the CPU."""
    c = inp.cfg
    X = values(*quantise(inp.X))
    orc = oracle_mod.get()
    dec = lambda q, s: torch.from_numpy(orc.mxfp4_decode(q.cpu().numpy(), s.cpu().numpy())).double()
    Wg, Wu, Wd = dec(inp.Wg, inp.Sg), dec(inp.Wu, inp.Su), dec(inp.Wd, inp.Sd)
    Y = inp.A.double().cpu().clone()
    mag, bound = Y.abs(), torch.zeros_like(Y)
    for e in range(Wg.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        x, al = X[t], alpha[t, j][:, None]
        g, u = x @ Wg[e].t(), x @ Wu[e].t()
        eg, eu = (gamma(2 * c.d) * (x.abs() @ w[e].abs().t()) for w in (Wg, Wu))
        silu = g * torch.sigmoid(g)
        h = silu * u
        err = 1.1 * eg * u.abs() + silu.abs() * eu + 1.1 * eg * eu + (16 + 2 * g.abs()) * U * h.abs() + 2.0 ** -120
        b = lambda v: v.reshape(len(t), -1, 32)
        top = scale_of(b(h).abs().amax(-1))
        lo_b = scale_of((b(h).abs() - b(err)).amax(-1).clamp(min=0))
        hi_b = scale_of((b(h).abs() + b(err)).amax(-1))
        H = stored_at(b(h), top)
        reach = torch.zeros_like(H)
        for byte in (lo_b, hi_b):
            for end in (b(h) - b(err), b(h) + b(err)):
                reach = torch.maximum(reach, (stored_at(end, byte) - H).abs())
        H, reach = H.reshape(h.shape), reach.reshape(h.shape)
        wd = Wd[e].abs().t()
        o, m = al * (H @ Wd[e].t()), al * ((H.abs() + reach) @ wd)
        Y.index_put_((t,), o, accumulate=True)
        mag.index_put_((t,), m, accumulate=True)
        bound.index_put_((t,), al * (reach @ wd) + gamma(2 * c.f) * m, accumulate=True)
    return Y, bound + gamma(c.kp + 2) * mag


def run(cfg, logits=None, phi=None):
    inp = gpu_inputs(cfg)
    layer = MoELayer(inp, phi=phi)
    Y = inp.A.clone()
    layer.forward_mxfp4(Y, logits=logits)
    torch.cuda.synchronize()
    return inp, layer, Y


def check(cfg, logits=None, phi=None):
    inp, layer, Y = run(cfg, logits, phi)
    run_ = OracleRun(inp, logits=None if logits is None else logits.cpu().numpy())
    idx, alpha = layer.routes["topk_idx"].cpu(), layer.routes["topk_w"].cpu().double()
    assert np.array_equal(idx.numpy().reshape(run_.idx.shape), run_.idx)
    ref, bound = reference(inp, idx.reshape(cfg.T, -1).long(), alpha.reshape(cfg.T, -1))
    err = (Y.cpu().double() - ref).abs()
    say(f"  max err/bound {float((err / bound).max()):.3g}, rel to the expert sum "
        f"{float(err.norm() / (ref - inp.A.cpu().double()).norm()):.3g}")
    assert bool((err <= bound).all())


@pytest.mark.parametrize("T,d,f,E,k,shared", [(1, 64, 64, 2, 1, 0), (2, 128, 192, 4, 4, 1), (90, 256, 128, 8, 2, 0),
                                              (33, 320, 448, 5, 3, 2), (300, 192, 576, 3, 2, 0), (700, 576, 256, 4, 2, 1),
                                              (130, 1024, 1408, 8, 2, 0)])
def test_layer_on_mxfp4_activations(T, d, f, E, k, shared):
    say(f"MXFP4 activations: T={T} d={d} f={f} E={E} k={k} shared={shared}")
    check(cfg_of(T, d, f, E, k, shared))


def test_skewed_routing_and_another_placement():
    say("MXFP4 activations: one expert takes every token, others none, slots in another order")
    cfg = cfg_of(600, 256, 320, 6, 2)
    logits = torch.full((600, 6), -4.0, device="cuda")
    logits[:, 3] = 2.0
    logits[:599, 1] = 1.0
    logits[599, 5] = 1.0
    check(cfg, logits=logits, phi=[4, 2, 0, 6, 1, 3])


def test_same_bits_in_parts():
    """A capacity of part of the routes, part by part, gives the same bits, whatever the workspace held."""
    say("MXFP4 activations: the token range in parts")
    cfg = cfg_of(300, 256, 192, 6, 2)
    inp, layer, Y = run(cfg)
    part = MoELayer(inp, capacity=202)
    s = part.shape
    L = torch.empty((s.T, s.E), dtype=torch.float32, device="cuda")
    B.moe_router_logits(s, part.X, part.Wr, part.bias, L)
    c, sc = quantise(inp.X)
    xq = torch.cat([c.reshape(-1), sc.reshape(-1)])
    for turn in range(2):
        Z = inp.A.clone()
        for t0 in (0, 101, 202):
            B.moe_route_build(s, t0, min(101, 300 - t0), L, part.phi, B.MOE_ROUTE_RESET, part.routes, part.ws)
            B.moe_expert_ffn(s, xq, None, part.routes, part.arena, part.phi, B.MOE_FFN_EXPERTS | B.MOE_FFN_ACT_MXFP4, part.ws)
        B.moe_expert_ffn(s, None, Z, part.routes, None, None, B.MOE_FFN_FINALIZE, part.ws)
        torch.cuda.synchronize()
        assert torch.equal(Y, Z)
        # the bf16 layer on the same workspace in between
        part.forward(inp.A.clone())


def test_nan_and_infinite_tokens_stay_alone():
    say("MXFP4 activations: a NaN, an infinity and a huge value reach their own tokens only")
    cfg = cfg_of(200, 256, 128, 6, 2)
    logits = torch.randn((200, 6), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    inp = gpu_inputs(cfg)
    a = MoELayer(inp)
    Y = inp.A.clone()
    a.forward_mxfp4(Y, logits=logits)
    inp.X[7, 40], inp.X[99, 3] = float("nan"), float("inf")
    inp.X[150] = 0.0
    Z = inp.A.clone()
    MoELayer(inp).forward_mxfp4(Z, logits=logits)
    torch.cuda.synchronize()
    keep = torch.ones(200, dtype=torch.bool)
    keep[[7, 99, 150]] = False
    assert torch.equal(Y[keep], Z[keep])
    assert bool(torch.isnan(Z[[7, 99]]).all()) and torch.equal(Z[150], inp.A[150])


def test_repeated_and_on_another_stream():
    say("MXFP4 activations: the same bits again and on a side stream")
    cfg = cfg_of(270, 320, 192, 7, 3)
    inp, layer, Y = run(cfg)
    st = torch.cuda.Stream()
    for _ in range(3):
        Z = inp.A.clone()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            layer.forward_mxfp4(Z)
        torch.cuda.current_stream().wait_stream(st)
        torch.cuda.synchronize()
        assert torch.equal(Y, Z)


def test_olmoe_sized_close_to_bf16_activations():
    """Full size: the layer on MXFP4 activations differs from the one on bf16
    activations by the activations' rounding, at most 1/4 of a value (half the
    widest relative step, 4 to 6 and 6 to 8 clipped) in each of X and H."""
    say("MXFP4 activations: OLMoE-sized, against bf16 activations")
    cfg = cfg_of(2048, 2048, 1024, 64, 8)
    inp, layer, Y = run(cfg)
    Z = inp.A.clone()
    layer.forward(Z)
    torch.cuda.synchronize()
    r = float((Y - Z).norm() / (Z - inp.A).norm())
    say(f"  relative difference of the expert sums {r:.3g}")
    assert 0.0 < r < 0.5


def test_refusals():
    cfg = cfg_of(4, 64, 64, 2, 1)
    inp = gpu_inputs(cfg)
    layer = MoELayer(inp)
    xq = torch.zeros(4 * 34, dtype=torch.uint8, device="cuda")
    for other in (B.MOE_FFN_SIMPLE_KERNEL, B.MOE_FFN_FUSED):
        with pytest.raises(B.MoEError) as ei:
            B.moe_expert_ffn(layer.shape, xq, inp.A, layer.routes, layer.arena, layer.phi,
                             B.MOE_FFN_EXPERTS | B.MOE_FFN_ACT_MXFP4 | other, layer.ws)
        assert ei.value.status == B.MOE_ERR_UNSUPPORTED
    for kw in (dict(Y=inp.A[:3]), dict(Y=inp.A, logits=torch.zeros(3, 2, device="cuda")),
               dict(Y=inp.A, logits=torch.zeros(4, 4, device="cuda")[:, :2])):
        with pytest.raises(ValueError):
            layer.forward_mxfp4(**kw)
    bf = gpu_inputs(cfg.with_(dtype="bf16", name="mx_layer_bf16"))
    with pytest.raises(ValueError):
        MoELayer(bf).forward_mxfp4(bf.A)
    with pytest.raises(ValueError):
        MoELayer(inp, capacity=2).forward_mxfp4(inp.A)


def test_far_negative_gates():
    """SiLU(g) u where exp(-g) leaves fp32's range and the product does not: g of
    -86 to -92 with u of 2^116 to 2^126, and -104 with 2^126. g and u are exact
    here, and Y is H as it is stored: each value is (16 + 2 |g|) u off before, far
    from the borders between codes (asserted), so that Y is known to the bit."""
    say("MXFP4 activations: gates far below zero, large up values")
    cfg = cfg_of(3, 64, 64, 1, 1)
    inp = gpu_inputs(cfg)
    near = [-86, -87, -88, -88.5, -89, -89.5, -90, -90.5, -91, -91.5, -92, 1, -2, 0, 3, -40]
    g = torch.tensor(near + near + [-104.0] * 32, dtype=torch.float64)
    silu = g * torch.exp(g) / (1 + torch.exp(g))
    n = torch.where(g == -104, 126, torch.where(silu == 0, 1, (1 - torch.frexp(silu)[1])))
    n[16:32] += 1                                  # other values of a block, up to two powers of two below its top
    n = n.clamp(max=126)
    Wg, Wu, Wd, X = torch.zeros(64, 64), torch.zeros(64, 64), torch.eye(64), torch.zeros(3, 64)
    for j in range(64):                            # 32 ones times codes that add up to g
        rest, c = abs(float(g[j])), 0
        while rest > 0:
            v = max(m for m in (0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0) if m <= rest)
            Wg[j, c], rest, c = (v if g[j] > 0 else -v), rest - v, c + 1
        Wu[j, 32] = 2.0 ** int(n[j] - 63)
    X[:, :32], X[:, 32] = 1.0, 2.0 ** 63
    quant = lambda W: tuple(t.cuda()[None] for t in quantize_mxfp4(W))
    (inp.Wg, inp.Sg), (inp.Wu, inp.Su), (inp.Wd, inp.Sd) = quant(Wg), quant(Wu), quant(Wd)
    inp.X, inp.A = X.to(torch.bfloat16).cuda(), torch.zeros(3, 64, device="cuda")
    h = (silu * two_to(n.int())).reshape(2, 32)
    byte = scale_of(h.abs().amax(-1))
    want = stored_at(h, byte)
    off = (16 + 2 * g.abs().reshape(2, 32)) * U
    for s in (1 - off, 1 + off):
        assert torch.equal(stored_at(h * s, byte), want) and torch.equal(scale_of((h * s).abs().amax(-1)), byte)
    assert int((want[0] != 0).sum()) >= 24 and bool((want[1] != 0).all())
    layer = MoELayer(inp)
    Y = inp.A.clone()
    layer.forward_mxfp4(Y)
    torch.cuda.synchronize()
    t, j = (Y.double().cpu() != want.reshape(64)).nonzero(as_tuple=True)
    assert not len(j), f"g = {sorted(set(g[j].tolist()))}"


# ---- inputs whose g and u are exact: a bound close enough to tell a wrong tile ----

def exact_inputs(cfg, seed=1):
    """Layer inputs whose blocks all have one scale: X's values are E2M1's, each block's
    largest 4 or 6, and the weights' codes any, times 2^-7. Products are at most 144
    units of 2^-9, and d of them less than 2^24 units, so that every partial sum of g
    and u is an fp32 number, whatever the order."""
    assert cfg.d * 36 * 4 < 2 ** 24
    inp = gpu_inputs(cfg)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    mag = MAG.float().cuda()
    pick = torch.randint(8, (cfg.T, cfg.d), generator=gen, device="cuda")
    pick[:, ::32] = 6 + pick[:, ::32] % 2
    sign = torch.randint(2, (cfg.T, cfg.d), generator=gen, device="cuda") * 2 - 1
    inp.X = (mag[pick] * sign).to(torch.bfloat16)
    for q in (inp.Wg, inp.Wu, inp.Wd):
        q.random_(0, 256, generator=gen)
    for s in (inp.Sg, inp.Su, inp.Sd):
        s.fill_(120)
    return inp


def reference_of_exact(inp, idx, alpha):
    """(Y, bound) as in `reference`, where g and u are exact: h is off by SiLU's and
    the product's roundings alone, (16 + 2 |g|) u |h| (and 2^-120, for the range that
    these g do not reach)."""
    c = inp.cfg
    X = values(*quantise(inp.X))
    orc = oracle_mod.get()
    dec = lambda q, s: torch.from_numpy(orc.mxfp4_decode(q.cpu().numpy(), s.cpu().numpy())).double()
    Wg, Wu, Wd = dec(inp.Wg, inp.Sg), dec(inp.Wu, inp.Su), dec(inp.Wd, inp.Sd)
    Y = inp.A.double().cpu().clone()
    mag, bound = Y.abs(), torch.zeros_like(Y)
    for e in range(Wg.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        al = alpha[t, j][:, None]
        g, u = X[t] @ Wg[e].t(), X[t] @ Wu[e].t()
        h = (g * torch.sigmoid(g) * u).reshape(len(t), -1, 32)
        err = (16 + 2 * g.abs().reshape(h.shape)) * U * h.abs() + 2.0 ** -120
        H = stored_at(h, scale_of(h.abs().amax(-1)))
        reach = torch.zeros_like(H)
        for byte in (scale_of((h.abs() - err).amax(-1).clamp(min=0)), scale_of((h.abs() + err).amax(-1))):
            for end in (h - err, h + err):
                reach = torch.maximum(reach, (stored_at(end, byte) - H).abs())
        H, reach = H.reshape(g.shape), reach.reshape(g.shape)
        wd = Wd[e].abs().t()
        o, m = al * (H @ Wd[e].t()), al * ((H.abs() + reach) @ wd)
        Y.index_put_((t,), o, accumulate=True)
        mag.index_put_((t,), m, accumulate=True)
        bound.index_put_((t,), al * (reach @ wd) + gamma(2 * c.f) * m, accumulate=True)
    return Y, bound + gamma(c.kp + 2) * mag


def check_of_exact(inp, Y, routes, at):
    """The tokens `at` within the bound, which has to tell a wrong tile, whose error is
    as large as the expert sums: it is below 1/20 of them. (Of f terms of either sign the
    sum is about sqrt(f) and the magnitudes' sum 0.8 f times a term, so gamma(2f) alone is
    0.8 sqrt(f) 2f u of the sum: 0.6 % for f = 1664, as much again for alpha's spread
    over two routes and for values beside a border between codes.)"""
    T = inp.cfg.T
    idx, alpha = routes["topk_idx"].reshape(T, -1), routes["topk_w"].reshape(T, -1)
    sub = type(inp)(**{**inp.__dict__, "X": inp.X[at].contiguous(), "A": inp.A[at]})
    ref, bound = reference_of_exact(sub, idx[at].cpu().long(), alpha[at].cpu().double())
    err = (Y[at].cpu().double() - ref).abs()
    ffn = (ref - sub.A.cpu().double()).norm()
    say(f"  max err/bound {float((err / bound).max()):.3g}; of the expert sums: error {float(err.norm() / ffn):.3g}, "
        f"bound {float(bound.norm() / ffn):.3g}")
    assert bool((err <= bound).all()) and float(bound.norm()) < 0.05 * float(ffn)


@pytest.mark.parametrize("T,d,f,E,k,shared", [(1, 64, 64, 2, 1, 0), (90, 256, 128, 8, 2, 0), (33, 320, 448, 5, 3, 2),
                                              (700, 576, 256, 4, 2, 1), (130, 1024, 1408, 8, 2, 0)])
def test_exact_projections(T, d, f, E, k, shared):
    say(f"MXFP4 activations, exact g and u: T={T} d={d} f={f} E={E} k={k} shared={shared}")
    cfg = cfg_of(T, d, f, E, k, shared)
    inp = exact_inputs(cfg)
    layer = MoELayer(inp)
    L = torch.empty((T, E), device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(T))
    Y = inp.A.clone()
    layer.forward_mxfp4(Y, logits=L)
    torch.cuda.synchronize()
    check_of_exact(inp, Y, layer.routes, torch.arange(T, device="cuda"))


@pytest.mark.parametrize("d,f", [(3264, 1600), (3200, 1664)])
def test_several_tiles_a_workgroup(d, f):
    """Projections of more than 768 tiles, three or four for each of 256
    workgroups: the same bits as in parts of less than 256 tiles, and within
    the bound for tokens of every part."""
    T, E = 8192, 6
    say(f"MXFP4 activations: several tiles a workgroup, T={T} d={d} f={f}")
    cfg = cfg_of(T, d, f, E, 2)
    inp = exact_inputs(cfg)
    gen = torch.Generator(device="cuda").manual_seed(17)
    L = torch.empty((T, E), device="cuda").normal_(generator=gen)
    L[:, 2] -= 20.0                  # an expert without tokens
    L[:, 4] += 1.5
    layer = MoELayer(inp)
    Y = inp.A.clone()
    layer.forward_mxfp4(Y, logits=L)
    torch.cuda.synchronize()
    count = layer.routes["slot_count"].tolist()
    tiles = lambda counts, N: sum((c + 255) // 256 for c in counts) * ((N + 255) // 256)
    assert tiles(count, 2 * f) > 768 and tiles(count, d) > 768 and 0 in count
    step = 1021
    part = MoELayer(inp, capacity=step * 2)
    s = part.shape
    c, sc = quantise(inp.X)
    xq = torch.cat([c.reshape(-1), sc.reshape(-1)])
    Z = inp.A.clone()
    for t0 in range(0, T, step):
        n = min(step, T - t0)
        B.moe_route_build(s, t0, n, L, part.phi, B.MOE_ROUTE_RESET, part.routes, part.ws)
        torch.cuda.synchronize()
        assert max(tiles(part.routes["slot_count"].tolist(), w) for w in (2 * f, d)) < 256
        B.moe_expert_ffn(s, xq, None, part.routes, part.arena, part.phi, B.MOE_FFN_EXPERTS | B.MOE_FFN_ACT_MXFP4, part.ws)
    B.moe_expert_ffn(s, None, Z, part.routes, None, None, B.MOE_FFN_FINALIZE, part.ws)
    torch.cuda.synchronize()
    assert torch.equal(Y, Z)
    check_of_exact(inp, Y, layer.routes, torch.arange(5, T, 293, device="cuda"))


def test_no_tokens():
    say("MXFP4 activations: a prompt of no tokens, as the bf16 layer takes it")
    inp = gpu_inputs(cfg_of(4, 64, 64, 2, 1))
    c = inp.cfg.with_(T=0)
    layer = MoELayer(type(inp)(**{**inp.__dict__, "cfg": c, "X": inp.X[:0], "A": inp.A[:0]}))
    Y = torch.zeros(0, 64, device="cuda")
    layer.forward(Y)
    layer.forward_mxfp4(Y)
    layer.forward_mxfp4(Y, logits=torch.zeros(0, 2, device="cuda"))
    torch.cuda.synchronize()
