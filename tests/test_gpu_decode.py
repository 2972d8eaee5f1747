"""The layer for a few tokens (moe_layer_decode) against its formulas in 64
bits.

Bound on each output element. All sums are in fp32 with u = 2^-24 a rounding
and gamma_n = n u / (1 - n u) for a sum of n terms in any order; weights and
activations are exact inputs (bf16 products of 8 by 8 bits are exact in fp32,
fp32 ones round once more). With a = |W_g||x|, b = |W_u||x|:
  dg = gamma(d + 4) a, du = gamma(d + 4) b (4: row scale, products, joins)
  dh = 1.1 |u| dg + |silu g| du + 1.1 dg du + 8u (|h| + ...)   (|silu'| < 1.1;
       exp, 1 +, divide and multiply are within 2, 1, 1 and 1 ulp, counted as 8)
  do = |W_d| dh + gamma(3 f + 4) |W_d| (|h| + dh)   (H enters as three terms)
  dy = sum_j alpha (do + 2u (|o| + do)) + gamma(K' + 1) (|A| + sum_j alpha (|o| + do))
Route ids and weights are taken from the call and checked on their own.
"""
import numpy as np
import pytest
import torch

from gpu_util import OracleRun, check_routing_from_gpu_logits, gpu_inputs, say
from routed_expert_ffn_top_amd import binding as B
from routed_expert_ffn_top_amd.inputs import CONFIGS, MoEConfig, make_logits
from routed_expert_ffn_top_amd.layer import MoELayer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = ["bf16", "f32", "bf16_fp8w", "bf16_fp4w"]


def gamma(n):
    return n * U / (1 - n * U)


def plain_weights(inp):
    """Expert weights as fp64 on the GPU, from the stored codes."""
    cfg, o = inp.cfg, OracleRun.__new__(OracleRun)
    if not cfg.quant_weights:
        return tuple(w.double() for w in (inp.Wg, inp.Wu, inp.Wd))
    from oracle import oracle as oracle_mod
    orc = oracle_mod.get()
    out = []
    for q, s in ((inp.Wg, inp.Sg), (inp.Wu, inp.Su), (inp.Wd, inp.Sd)):
        if cfg.fp8_weights:
            w = torch.from_numpy(orc.fp8e4m3_decode(q.cpu().numpy())).cuda().double() * s.double()[..., None]
        else:
            w = torch.from_numpy(orc.mxfp4_decode(q.cpu().numpy(), s.cpu().numpy())).cuda().double()
        out.append(w)
    return tuple(out)


def reference(inp, weights, X, A, idx, w):
    """(y, bound) [T][d] in 64 bits for the given route ids and weights."""
    cfg = inp.cfg
    Wg, Wu, Wd = weights
    x = X.double()
    y, s, err = A.double(), A.double().abs(), torch.zeros_like(A, dtype=torch.float64)
    for e in range(cfg.n_exp):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if not len(t):
            continue
        xe = x[t]
        g, u = xe @ Wg[e].t(), xe @ Wu[e].t()
        dg = gamma(cfg.d + 4) * (xe.abs() @ Wg[e].abs().t())
        du = gamma(cfg.d + 4) * (xe.abs() @ Wu[e].abs().t())
        silu = g * torch.sigmoid(g)
        h = silu * u
        dh = 1.1 * u.abs() * dg + silu.abs() * du + 1.1 * dg * du
        dh = dh + 8 * U * (h.abs() + dh) + 2.0 ** -126
        o = h @ Wd[e].t()
        do = (dh + gamma(3 * cfg.f + 4) * (h.abs() + dh)) @ Wd[e].abs().t()
        al = w[t, j].double()[:, None]
        y[t] += al * o
        s[t] += al * (o.abs() + do)
        err[t] += al * (do + 2 * U * (o.abs() + do))
    return y, err + gamma(cfg.kp + 1) * s + 2.0 ** -140


def check(inp, weights, X, A, Y, routes, name=""):
    torch.cuda.synchronize()
    ref, bound = reference(inp, weights, X, A, routes["topk_idx"].long(), routes["topk_w"])
    err = (Y.double() - ref).abs()
    assert torch.isfinite(Y).all()
    ffn = (ref - A.double()).norm()
    say(f"  {name}: max err/bound {float((err / bound).max()):.3g}, expert sum rel {float(err.norm() / ffn):.3g}")
    assert bool((err <= bound).all())


def tokens(cfg, T, seed=1, pad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.empty((T, cfg.d + pad), device="cuda").normal_(generator=gen).to(cfg.torch_dtype)[:, : cfg.d]
    return X, torch.empty((T, cfg.d), device="cuda").normal_(generator=gen)


SMALL = MoEConfig(name="dec_small", index=71, T=4, d=256, f=192, E=8, k=2)
SHARED = MoEConfig(name="dec_shared", index=72, T=4, d=320, f=128, E=5, k=3, n_shared=2, renorm=False)
ONE = MoEConfig(name="dec_one", index=73, T=4, d=64, f=64, E=1, k=1)
WIDE = MoEConfig(name="dec_wide", index=74, T=4, d=448, f=320, E=96, k=8)
F32ODD = MoEConfig(name="dec_f32odd", index=75, T=4, d=100, f=96, E=6, k=2, dtype="f32")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cfg", [SMALL, SHARED, ONE, WIDE], ids=lambda c: c.name)
def test_decode_token_counts(cfg, dtype):
    cfg = cfg.with_(dtype=dtype)
    inp = gpu_inputs(cfg)
    layer, weights = MoELayer(inp), plain_weights(inp)
    for T in (1, 2, 15, 16, 17, 33, 64):
        say(f"decode {cfg.name} {dtype} T={T}")
        X, A = tokens(cfg, T, seed=T)
        Y = A.clone()
        layer.decode(X, Y)
        check(inp, weights, X, A, Y, layer.decode_routes(T), f"T={T}")
    assert B.moe_device_errors(layer.shape, layer.ws) == 0


def test_decode_f32_odd_widths():
    say("decode, fp32, d = 100 (a last K piece of 4 values), f = 96")
    inp = gpu_inputs(F32ODD)
    layer, weights = MoELayer(inp), plain_weights(inp)
    for T in (1, 20):
        X, A = tokens(F32ODD, T)
        Y = A.clone()
        layer.decode(X, Y)
        check(inp, weights, X, A, Y, layer.decode_routes(T), f"T={T}")


@pytest.mark.parametrize("name,T", [("olmoe_t1024", 1), ("olmoe_t1024_fp4w", 64), ("dsv2lite_t4096_fp8w", 8),
                                    ("mixtral_t256_fp4w", 3)])
def test_decode_model_shapes(name, T):
    say(f"decode {name} T={T}")
    cfg = CONFIGS[name].with_(T=1)
    inp = gpu_inputs(cfg)
    layer, weights = MoELayer(inp), plain_weights(inp)
    X, A = tokens(cfg, T)
    Y = A.clone()
    layer.decode(X, Y)
    check(inp, weights, X, A, Y, layer.decode_routes(T), name)


@pytest.mark.parametrize("dtype", DTYPES)
def test_decode_routes_as_the_prompt_layer(dtype):
    say(f"decode and prompt layer route alike, {dtype}")
    cfg = WIDE.with_(T=40, dtype=dtype)
    inp = gpu_inputs(cfg)
    layer = MoELayer(inp)
    Y = inp.A.clone()
    layer.forward(Y)
    Z = inp.A.clone()
    layer.decode(inp.X, Z)
    torch.cuda.synchronize()
    r = layer.decode_routes(40)
    assert torch.equal(r["topk_idx"], layer.routes["topk_idx"])
    assert torch.equal(r["topk_w"], layer.routes["topk_w"])
    # H is rounded there (bf16: half a step of 2^-8 each value) and not here
    a, b = (Y - inp.A).double(), (Z - inp.A).double()
    assert float((a - b).norm() / b.norm()) < (1e-5 if dtype == "f32" else 2.0 ** -8)


@pytest.mark.parametrize("dtype", DTYPES)
def test_decode_exact_on_integers(dtype):
    """H of up to 22 bits and sums below 2^24: every step is exact in fp32, so
    the outputs are the integers, in whatever order they are summed."""
    say(f"decode on integers, {dtype}")
    cfg = MoEConfig(name="dec_int", index=76, T=17, d=128, f=128, E=2, k=1, dtype=dtype, renorm=True)
    inp = gpu_inputs(cfg)
    gen = torch.Generator(device="cuda").manual_seed(9)
    ints = lambda lo, hi, s: torch.randint(lo, hi + 1, s, generator=gen, device="cuda").float()
    Wg, Wu = ints(1, 6, (2, 128, 128)), ints(-6, 6, (2, 128, 128))
    Wg[Wg == 5] = 4.0
    Wu[Wu.abs() == 5] = 4.0
    # two units an output: |y| <= 2 * 6 * |h|
    Wd = torch.zeros(2, 128, 128, device="cuda")
    for n in range(128):
        Wd[:, n, n], Wd[:, n, (n * 5 + 3) % 128] = 1.0, -1.0
    X = ints(1, 4, (17, 128))
    if cfg.fp4_weights:
        code = {0: 0, 1: 2, 2: 4, 3: 5, 4: 6, 6: 7}
        table = torch.zeros(7, dtype=torch.uint8, device="cuda")
        for v, c in code.items():
            table[v] = c
        enc = lambda W: (table[W.abs().long()] | ((W < 0).to(torch.uint8) << 3))
        pack = lambda W: (enc(W)[..., 0::2] | enc(W)[..., 1::2] << 4).contiguous()
        inp.Wg, inp.Wu, inp.Wd = pack(Wg), pack(Wu), pack(Wd)
        for s in (inp.Sg, inp.Su, inp.Sd):
            s.fill_(127)
    elif cfg.fp8_weights:
        inp.Wg, inp.Wu, inp.Wd = (W.to(torch.float8_e4m3fn).view(torch.uint8) for W in (Wg, Wu, Wd))
        for s in (inp.Sg, inp.Su, inp.Sd):
            s.fill_(1.0)
    else:
        inp.Wg, inp.Wu, inp.Wd = (W.to(cfg.torch_dtype) for W in (Wg, Wu, Wd))
    layer = MoELayer(inp)
    logits = torch.zeros(17, 2, device="cuda")
    logits[::2, 1] = 1.0
    Y = torch.zeros(17, 128, device="cuda")
    layer.decode(X.to(cfg.torch_dtype), Y, logits=logits)
    torch.cuda.synchronize()
    e = (torch.arange(17, device="cuda") % 2 == 0).long()
    x = X.double()
    g = torch.einsum("td,tfd->tf", x, Wg[e].double())
    h = g * torch.einsum("td,tfd->tf", x, Wu[e].double())
    assert float(g.min()) > 40 and 2 ** 18 < float(h.abs().max()) < 2 ** 22    # SiLU(g) = g in fp32, more than 16 bits
    ref = torch.einsum("tf,tnf->tn", h, Wd[e].double())
    assert float(ref.abs().max()) < 2 ** 24
    assert torch.equal(Y.double(), ref)


def test_decode_strides_and_untouched_columns():
    say("decode with padded rows of X and Y")
    inp = gpu_inputs(SMALL)
    layer, weights = MoELayer(inp), plain_weights(inp)
    for T in (1, 5):
        X, A = tokens(SMALL, T, pad=40)
        buf = torch.full((T + 1, SMALL.d + 12), 7.5, device="cuda")
        Y = buf[:T, : SMALL.d]
        Y.copy_(A)
        layer.decode(X, Y)
        check(inp, weights, X, A, Y, layer.decode_routes(T), f"T={T}")
        assert bool((buf[:, SMALL.d:] == 7.5).all()) and bool((buf[T] == 7.5).all())
        Y2 = A.clone()
        layer.decode(X.contiguous(), Y2)
        assert torch.equal(Y2, Y)


@pytest.mark.parametrize("dtype", ["bf16", "bf16_fp4w"])
def test_decode_same_bits_for_any_placement(dtype):
    say(f"decode: same bits for any phi and P, {dtype}")
    cfg = WIDE.with_(dtype=dtype)
    inp = gpu_inputs(cfg)
    X, A = tokens(cfg, 9)
    ys = []
    gen = torch.Generator().manual_seed(3)
    for phi in (None, torch.randperm(96, generator=gen).tolist(), (torch.randperm(200, generator=gen)[:96]).tolist()):
        layer = MoELayer(inp, phi=phi)
        Y = A.clone()
        layer.decode(X, Y)
        torch.cuda.synchronize()
        ys.append(Y)
        layer.close()
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


def test_decode_bad_tokens_stay_alone():
    say("decode: a NaN or infinite token leaves the others alone")
    inp = gpu_inputs(SMALL)
    layer = MoELayer(inp)
    X, A = tokens(SMALL, 20)
    L = make_logits(20, SMALL.E, 5, device="cuda")
    Y = A.clone()
    layer.decode(X, Y, logits=L)
    X2, L2 = X.clone(), L.clone()
    X2[3, 7], X2[11] = float("nan"), float("inf")
    L2[17] = float("nan")
    Z = A.clone()
    layer.decode(X2, Z, logits=L2)
    torch.cuda.synchronize()
    keep = torch.ones(20, dtype=torch.bool)
    keep[[3, 11, 17]] = False
    assert torch.equal(Y[keep], Z[keep])
    assert bool(torch.isnan(Z[3]).any()) and not bool(torch.isfinite(Z[11]).all())
    # a row of NaN logits takes ids in order with weight 0
    r = layer.decode_routes(20)
    assert r["topk_idx"][17].tolist() == [0, 1] and r["topk_w"][17].tolist() == [0.0, 0.0]
    assert torch.equal(Z[17], A[17])


def test_decode_infinite_hidden_unit():
    say("decode: an overflowing hidden unit is an infinity, not a NaN")
    cfg = ONE.with_(dtype="bf16")
    inp = gpu_inputs(cfg)
    inp.Wg.fill_(0), inp.Wu.fill_(0), inp.Wd.fill_(0)
    inp.Wg[0, 0, 0] = inp.Wu[0, 0, 0] = 2.0 ** 100
    inp.Wd[0, 5, 0] = 1.0
    layer = MoELayer(inp)
    X = torch.zeros(1, 64, dtype=torch.bfloat16, device="cuda")
    X[0, 0] = 1.0
    Y = torch.zeros(1, 64, device="cuda")
    layer.decode(X, Y, logits=torch.zeros(1, 1, device="cuda"))
    torch.cuda.synchronize()
    assert float(Y[0, 5]) == float("inf")


def test_decode_after_prompt_and_between():
    """As a server runs it: a prompt through the prompt layer, then tokens one
    batch after another of changing size, all on one stream, unsynchronised."""
    say("decode: prompt, then batches of changing size")
    cfg = SHARED.with_(T=150)
    inp = gpu_inputs(cfg)
    layer, weights = MoELayer(inp), plain_weights(inp)
    alone = MoELayer(inp)
    Yp = inp.A.clone()
    layer.forward(Yp)
    runs = []
    for i, T in enumerate((1, 7, 64, 1, 33, 7)):
        X, A = tokens(cfg, T, seed=40 + i)
        Y = A.clone()
        layer.decode(X, Y)
        runs.append((X, A, Y))
    layer.forward(Yp)
    torch.cuda.synchronize()
    for X, A, Y in runs:
        Z = A.clone()
        alone.decode(X, Z)
        torch.cuda.synchronize()
        assert torch.equal(Y, Z)
    check(inp, weights, *runs[-1], layer.decode_routes(7), "last")
    Ya = inp.A.clone()
    alone.forward(Ya)
    alone.forward(Ya)
    torch.cuda.synchronize()
    assert torch.equal(Ya, Yp)


def test_decode_two_streams():
    say("decode: two layers on two streams at once")
    inps = [gpu_inputs(SMALL), gpu_inputs(WIDE)]
    layers = [MoELayer(i) for i in inps]
    ins = [tokens(i.cfg, 8, seed=3 + k) for k, i in enumerate(inps)]
    want = []
    for l, (X, A) in zip(layers, ins):
        Y = A.clone()
        l.decode(X, Y)
        torch.cuda.synchronize()
        want.append(Y)
    streams = [torch.cuda.Stream() for _ in layers]
    outs = [[] for _ in layers]
    for rep in range(20):
        for k, (l, (X, A)) in enumerate(zip(layers, ins)):
            with torch.cuda.stream(streams[k]):
                Y = A.clone()
                l.decode(X, Y)
                outs[k].append(Y)
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(y, want[k]) for y in outs[k])


def test_decode_one_arena_on_two_streams():
    say("decode: one arena, two workspaces, two streams")
    inp = gpu_inputs(SMALL)
    layer = MoELayer(inp)
    X, A = tokens(SMALL, 8)
    Y = A.clone()
    layer.decode(X, Y)
    torch.cuda.synchronize()
    shape = B.make_shape(8, SMALL.d, SMALL.f, SMALL.E, SMALL.k, dtype=SMALL.dtype)
    bufs = [(B.alloc_routes(shape), B.alloc_decode_workspace(shape), torch.cuda.Stream()) for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for rep in range(40):
        for routes, ws, st in bufs:
            with torch.cuda.stream(st):
                Z = A.clone()
                B.moe_layer_decode(shape, X, layer.Wr, None, None, Z, layer.arena, routes, ws)
                outs.append(Z)
    torch.cuda.synchronize()
    assert all(torch.equal(Z, Y) for Z in outs)


def test_decode_captured_and_replayed():
    say("decode: captured into a graph, replayed between eager calls, and the arena loaded again")
    inp = gpu_inputs(SMALL)
    layer = MoELayer(inp)
    X, A = tokens(SMALL, 6)
    Xs, Ys = X.clone(), A.clone()
    eager = MoELayer(inp)
    g = torch.cuda.CUDAGraph()
    layer.decode(Xs, Ys)       # buffers exist before the capture
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        layer.decode(Xs, Ys)
    for i in range(6):
        X, A = tokens(SMALL, 6, seed=60 + i)
        Xs.copy_(X)
        Ys.copy_(A)
        g.replay()
        Z = A.clone()
        eager.decode(X, Z)
        if i == 2:
            W = A.clone()
            layer2 = MoELayer(inp)
            layer2.decode(X, W)
        torch.cuda.synchronize()
        assert torch.equal(Ys, Z), f"replay {i}"
    # eager calls on the captured layer still run, and so does a load after the replays
    for _ in range(40):
        Z = A.clone()
        layer.decode(X, Z)
    torch.cuda.synchronize()
    assert torch.equal(Z, Ys)
    Wg, Wu, Wd = inp.Wg, inp.Wu, inp.Wd
    B.arena_release_slot(layer.arena, 0)
    B.moe_pack_gate_up(layer.shape, Wg[0], Wu[0], layer.arena.plane_gu[0], 1, 0, 0)
    B.moe_pack_down(layer.shape, Wd[0], layer.arena.plane_d[0], 1, 0, 0)
    B.arena_publish_slot(layer.arena, 0, 0)
    Z = A.clone()
    layer.decode(X, Z)
    torch.cuda.synchronize()
    assert torch.equal(Z, Ys)


def test_decode_on_an_absent_expert_is_refused():
    inp = gpu_inputs(SMALL)
    layer = MoELayer(inp)
    B.arena_release_slot(layer.arena, 3)
    X, A = tokens(SMALL, 2)
    with pytest.raises(B.MoEError) as e:
        layer.decode(X, A.clone())
    assert e.value.status == B.MOE_ERR_SLOT_STATE


def test_decode_no_tokens():
    inp = gpu_inputs(SMALL)
    layer = MoELayer(inp)
    X, A = tokens(SMALL, 0)
    layer.decode(X, A)
    torch.cuda.synchronize()


# ---- routing: skewed, within the gate/up launch, at the limits ----

def skewed(T, E, k, seed=1):
    """Logits that send every token to experts 3, 4, .. (k of them), in an order of its own."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    L = torch.empty((T, E), device="cuda").uniform_(-1, 0, generator=gen)
    L[:, 3:3 + k] += 5.0
    return L


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [7, 16, 23, 64])
def test_decode_skewed_routing(T, dtype):
    """Far more routes on an expert than the mean: several entries of the lists
    for one slot, the last of them short."""
    say(f"decode, every token on the same experts, T={T} {dtype}")
    cfg = MoEConfig(name="dec_skew", index=79, T=4, d=192, f=128, E=96, k=2, n_shared=1, dtype=dtype)
    inp = gpu_inputs(cfg)
    layer, weights = MoELayer(inp), plain_weights(inp)
    X, A = tokens(cfg, T)
    Y = A.clone()
    layer.decode(X, Y, logits=skewed(T, 96, 2))
    r = layer.decode_routes(T)
    check(inp, weights, X, A, Y, r, f"T={T}")
    assert set(r["topk_idx"][:, :2].unique().tolist()) == {3, 4} and r["topk_idx"][:, 2].eq(96).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cfg", [SMALL, SHARED, F32ODD.with_(d=128)], ids=lambda c: c.name)
def test_decode_given_logits(cfg, dtype):
    """Few tokens, experts and given logits: routed within the gate/up launch."""
    say(f"decode with given logits, {cfg.name} {dtype}")
    cfg = cfg.with_(dtype=dtype, f=128)
    inp = gpu_inputs(cfg)
    layer, weights = MoELayer(inp), plain_weights(inp)
    for T in (1, 3, 8, 16):
        X, A = tokens(cfg, T)
        L = make_logits(T, cfg.E, T, device="cuda")
        if T > 1:
            L[1, 2] = float("nan")
            L[0, 1] = L[0, 0] = 2.0      # a tie
        Y = A.clone()
        layer.decode(X, Y, logits=L)
        r = layer.decode_routes(T)
        check(inp, weights, X, A, Y, r, f"T={T}")
        prompt = MoELayer(type(inp)(**{**inp.__dict__, "cfg": cfg.with_(T=T), "X": X, "A": A}))
        prompt.forward(A.clone(), logits=L)
        torch.cuda.synchronize()
        assert torch.equal(r["topk_idx"], prompt.routes["topk_idx"]) and torch.equal(r["topk_w"], prompt.routes["topk_w"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cfg", [SMALL, ONE, WIDE, F32ODD.with_(d=128), MoEConfig(name="dec_d1088", index=80, T=4, d=1088, f=64, E=8, k=2)],
                         ids=lambda c: c.name)
def test_decode_routes_few_tokens_as_the_prompt_layer(cfg, dtype):
    say(f"decode routes few tokens as the prompt layer does, {cfg.name} {dtype}")
    for T in (1, 2, 4, 5, 9):
        c = cfg.with_(T=T, dtype=dtype, f=64)
        inp = gpu_inputs(c)
        layer = MoELayer(inp)
        layer.forward(inp.A.clone())
        layer.decode(inp.X, inp.A.clone())
        torch.cuda.synchronize()
        r = layer.decode_routes(T)
        assert torch.equal(r["topk_idx"], layer.routes["topk_idx"]) and torch.equal(r["topk_w"], layer.routes["topk_w"])


@pytest.mark.parametrize("dtype", ["bf16", "bf16_fp4w"])
def test_decode_largest_expert_table_and_route_count(dtype):
    say(f"decode: 256 + 2 experts in 512 slots; 1024 routes, {dtype}")
    from routed_expert_ffn_top_amd.inputs import random_phi
    cfg = MoEConfig(name="dec_e256", index=81, T=4, d=128, f=64, E=256, k=6, n_shared=2, dtype=dtype, renorm=False)
    inp = gpu_inputs(cfg)
    layer, weights = MoELayer(inp, phi=random_phi(258, 512, 4).tolist(), P=512), plain_weights(inp)
    for T in (1, 64):
        X, A = tokens(cfg, T)
        Y = A.clone()
        layer.decode(X, Y)
        check(inp, weights, X, A, Y, layer.decode_routes(T), f"T={T}")
    layer.close()
    cfg = MoEConfig(name="dec_r1024", index=82, T=4, d=64, f=64, E=40, k=40, n_shared=24, dtype=dtype)
    inp = gpu_inputs(cfg)
    layer, weights = MoELayer(inp), plain_weights(inp)
    for T in (1, 16):
        X, A = tokens(cfg, T)
        Y = A.clone()
        layer.decode(X, Y)
        check(inp, weights, X, A, Y, layer.decode_routes(T), f"T={T}, 64 routes a token")


def test_decode_arena_past_4_gib():
    say("decode: a gate/up plane of 5.4 GB, slots past 2^32 bytes")
    cfg = MoEConfig(name="dec_big", index=83, T=4, d=4096, f=4096, E=80, k=4)
    inp = gpu_inputs(cfg)
    layer = MoELayer(inp)
    X, A = tokens(cfg, 3)
    L = torch.full((3, 80), -1.0, device="cuda")
    L[:, 76:] = torch.arange(4, device="cuda") * 0.3
    Y = A.clone()
    layer.decode(X, Y, logits=L)
    torch.cuda.synchronize()
    weights = [torch.zeros(80, 1, 1)] * 3
    small = [w[76:].double() for w in (inp.Wg, inp.Wu, inp.Wd)]
    sub = type(inp)(**{**inp.__dict__, "cfg": cfg.with_(E=4)})
    r = layer.decode_routes(3)
    assert int(r["topk_idx"].min()) >= 76
    ref, bound = reference(sub, small, X, A, r["topk_idx"].long() - 76, r["topk_w"])
    assert bool(((Y.double() - ref).abs() <= bound).all())


def test_decode_workspace_serves_several_shapes_and_layers():
    say("decode: one workspace for two layers and three token counts, call after call")
    cfgs = [SMALL, WIDE]
    layers = [MoELayer(gpu_inputs(c)) for c in cfgs]
    shapes = [(l, c, T, B.make_shape(T, c.d, c.f, c.E, c.k, dtype=c.dtype)) for l, c in zip(layers, cfgs) for T in (64, 1, 9)]
    ws = max((B.alloc_decode_workspace(s) for *_, s in shapes), key=lambda w: w.numel())
    for rep in range(3):
        got = []
        for l, c, T, s in shapes:
            X, A = tokens(c, T, seed=90 + rep)
            Y = A.clone()
            B.moe_layer_decode(s, X, l.Wr, None, None, Y, l.arena, B.alloc_routes(s), ws)
            got.append((l, X, A, Y))
        torch.cuda.synchronize()
        for l, X, A, Y in got:
            Z = A.clone()
            l.decode(X, Z)
            torch.cuda.synchronize()
            assert torch.equal(Y, Z)


def test_decode_first_call_not_captured_and_strided_logits_refused():
    """The workspace's clearing, recorded and not run, would leave the next eager
    call with counters of anything."""
    say("decode: a first call within a capture, logits that would be copied")
    cfg = SMALL
    inp = gpu_inputs(cfg)
    layer = MoELayer(inp)
    X, Y = inp.X[:2].contiguous(), inp.A[:2].contiguous()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        X.mul_(1.0)
        with pytest.raises(RuntimeError):
            layer.decode(X, Y)
    with pytest.raises(ValueError):
        layer.decode(X, Y, logits=torch.zeros(2, 2 * cfg.E, device="cuda")[:, : cfg.E])
    Z = Y.clone()
    layer.decode(X, Y)                   # makes the workspace; a stream of its own may come next
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    layer.decode(X, Z, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(Y, Z)


@pytest.mark.parametrize("dtype", DTYPES)
def test_decode_skewed_routing_within_gate_up(dtype):
    """Every workgroup of gate/up sorts the routes for itself: their entries have
    to agree where a slot has several and its routes are those of several waves."""
    say(f"decode, every token on the same experts, routed within gate/up, {dtype}")
    cfg = MoEConfig(name="dec_skew_self", index=82, T=4, d=128, f=1024, E=64, k=8, dtype=dtype)
    inp = gpu_inputs(cfg)
    layer, weights = MoELayer(inp), plain_weights(inp)
    X, A = tokens(cfg, 16)
    L = skewed(16, 64, 8)
    first = A.clone()
    layer.decode(X, first, logits=L)
    check(inp, weights, X, A, first, layer.decode_routes(16), "first")
    for _ in range(200):
        Y = A.clone()
        layer.decode(X, Y, logits=L)
        assert torch.equal(Y, first)


@pytest.mark.parametrize("T", [19, 64])
@pytest.mark.parametrize("dtype,d,f", [("bf16", 2048, 5632), ("f32", 2048, 2816), ("bf16_fp8w", 2048, 11264), ("bf16_fp4w", 4096, 10304)])
def test_decode_large_experts_many_routes(dtype, d, f, T):
    """Experts of more than 64 MB with many routes each: entries of 32 routes, one or two of them a slot."""
    say(f"decode, experts of {d} x {f} {dtype}, T={T}")
    cfg = MoEConfig(name="dec_large", index=83, T=4, d=d, f=f, E=2, k=1, dtype=dtype)
    inp = gpu_inputs(cfg)
    layer, weights = MoELayer(inp), plain_weights(inp)
    X, A = tokens(cfg, T)
    L = torch.zeros(T, 2, device="cuda")
    L[: T - 3, 1] = 1.0
    Y = A.clone()
    layer.decode(X, Y, logits=L)
    check(inp, weights, X, A, Y, layer.decode_routes(T), f"T={T}")


@pytest.mark.parametrize("dtype", DTYPES)
def test_decode_far_negative_gates(dtype):
    """SiLU(g) u where exp(-g) leaves fp32's range and the product does not. g, u
    and W_d H are exact (one term each, or 32 whose sums are), so Y is H, off by
    the roundings of SiLU(g) u alone: exp of g / 2 within 1 ulp (2u) in each of two
    factors and three products (u each), or exp, 1 +, a division and a product:
    8u in either form, and one more for alpha = 1 times it."""
    say(f"decode: gates far below zero, large up values, {dtype}")
    cfg = MoEConfig(name="dec_far", index=86, T=4, d=64, f=64, E=1, k=1, dtype=dtype)
    inp = gpu_inputs(cfg)
    g = torch.tensor([-80, -86, -87, -87.5, -88, -88.5, -89, -89.5, -90, -91, -92, -96, -100, -104, -120, -150] * 4,
                     dtype=torch.float64)
    silu = g * torch.exp(g) / (1 + torch.exp(g))
    n = (-torch.frexp(silu)[1]).clamp(max=126)     # u = 2^n: H near 1, or as near as fp32 allows
    Wg, Wu, Wd, X = torch.zeros(64, 64), torch.zeros(64, 64), torch.eye(64), torch.zeros(3, 64)
    for j in range(64):
        rest, c = abs(float(g[j])), 0
        while rest > 0:
            v = max(m for m in (0.5, 1.0, 2.0, 4.0, 6.0) if m <= rest)
            Wg[j, c], rest, c = -v, rest - v, c + 1
        Wu[j, 32] = 2.0 ** int(n[j] - 63)
    X[:, :32], X[:, 32] = 1.0, 2.0 ** 63
    if cfg.fp8_weights:
        q8 = lambda W: W.to(torch.float8_e4m3fn).view(torch.uint8).cuda()[None]
        one = torch.ones(1, 64, device="cuda")
        inp.Wg, inp.Sg, inp.Wd, inp.Sd = q8(Wg), one, q8(Wd), one.clone()
        inp.Wu, inp.Su = q8((Wu > 0).float()), Wu.sum(-1).cuda()[None]
    elif cfg.fp4_weights:
        from routed_expert_ffn_top_amd.inputs import quantize_mxfp4
        (inp.Wg, inp.Sg), (inp.Wu, inp.Su), (inp.Wd, inp.Sd) = (tuple(t.cuda()[None] for t in quantize_mxfp4(W))
                                                                for W in (Wg, Wu, Wd))
    else:
        inp.Wg, inp.Wu, inp.Wd = (W.to(cfg.torch_dtype).cuda()[None] for W in (Wg, Wu, Wd))
    layer = MoELayer(inp)
    for logits in (torch.zeros(3, 1, device="cuda"), None):
        Y = torch.zeros(3, 64, device="cuda")
        layer.decode(X.to(cfg.torch_dtype).cuda(), Y, logits=logits)
        torch.cuda.synchronize()
        want = (silu * torch.pow(2.0, n.double())).expand(3, 64)
        off = (Y.cpu().double() - want).abs() / want.abs()
        say(f"  largest error {float(off.max() / U):.3g} u")
        assert bool((off <= 9 * U).all()), f"g = {sorted(set(g.expand(3, 64)[off > 9 * U].tolist()))}"


def integer_layer(cfg, at):
    """A layer whose every step is exact in fp32, for tokens that are zero but at
    the hidden indices `at`: g in [64, 1536], so SiLU(g) = g, |h| < 2^21, and two
    units an output. Returns (layer, Wg, Wu [E][f][len(at)], Wd [E][d][f])."""
    inp = gpu_inputs(cfg)
    gen = torch.Generator(device="cuda").manual_seed(9)
    E, d, f = cfg.E, cfg.d, cfg.f
    W = torch.zeros(2, E, f, d, device="cuda")
    some = torch.randint(1, 7, (2, E, f, len(at)), generator=gen, device="cuda").float()
    some[some == 5] = 4.0
    some[1] *= torch.where(torch.rand(some[1].shape, generator=gen, device="cuda") < 0.5, -1.0, 1.0)
    W[..., at] = some
    Wd = torch.zeros(E, d, f, device="cuda")
    n = torch.arange(d, device="cuda")
    for e in range(E):
        Wd[e, n, n % f], Wd[e, n, (n * 5 + 3 + e) % f] = 1.0, -1.0
    if cfg.fp4_weights:
        table = torch.zeros(7, dtype=torch.uint8, device="cuda")
        for v, c in {1: 2, 2: 4, 3: 5, 4: 6, 6: 7}.items():
            table[v] = c
        enc = lambda w: (table[w.abs().long()] | ((w < 0).to(torch.uint8) << 3))
        pack = lambda w: (enc(w)[..., 0::2] | enc(w)[..., 1::2] << 4).contiguous()
        inp.Wg, inp.Wu, inp.Wd = pack(W[0]), pack(W[1]), pack(Wd)
        for s in (inp.Sg, inp.Su, inp.Sd):
            s.fill_(127)
    elif cfg.fp8_weights:
        inp.Wg, inp.Wu, inp.Wd = (w.to(torch.float8_e4m3fn).view(torch.uint8) for w in (W[0], W[1], Wd))
        for s in (inp.Sg, inp.Su, inp.Sd):
            s.fill_(1.0)
    else:
        inp.Wg, inp.Wu, inp.Wd = (w.to(cfg.torch_dtype) for w in (W[0], W[1], Wd))
    return MoELayer(inp), some[0].double(), some[1].double(), Wd


@pytest.mark.parametrize("d,f,dtype", [(131072, 64, "bf16"), (131072, 64, "f32"), (131072, 64, "bf16_fp8w"),
                                       (131072, 64, "bf16_fp4w"), (65600, 64, "bf16"), (49152, 256, "bf16"),
                                       (49156, 224, "f32")])
def test_decode_widest_layers(d, f, dtype):
    """More chunks of output columns than workgroups, to the last counter: a
    workgroup of down takes several chunks, and is the only arrival at each.
    Up to 16 routes an entry and, for experts of 64 MB and more, 32."""
    say(f"decode, d={d} f={f} {dtype}")
    cfg = MoEConfig(name="dec_widest", index=87, T=4, d=d, f=f, E=2, k=1, dtype=dtype)
    at = sorted({0, 31, 32, 127, 128, d // 2, d - 129, d - 64, d - 1} | set(range(7, d, d // 55)))[:64]
    layer, Wg, Wu, Wd = integer_layer(cfg, at)
    gen = torch.Generator(device="cuda").manual_seed(3)
    for T in (1, 5, 45):
        X = torch.zeros(T, d, device="cuda")
        x = torch.randint(1, 5, (T, len(at)), generator=gen, device="cuda").float()
        X[:, at] = x
        X = X.to(cfg.torch_dtype)
        L = torch.zeros(T, 2, device="cuda")
        L[1::2, 1] = 1.0
        for logits in (L, None):
            Y = torch.zeros(T, d, device="cuda")
            layer.decode(X, Y, logits=logits)
            torch.cuda.synchronize()
            r = layer.decode_routes(T)
            e = r["topk_idx"][:, 0].long()
            if logits is not None:
                assert torch.equal(e, L.argmax(-1))
            g = (Wg[e] * x.double()[:, None]).sum(-1)
            h = g * (Wu[e] * x.double()[:, None]).sum(-1)
            assert float(g.min()) > 40 and float(h.abs().max()) < 2 ** 22
            # column n holds W_d's two entries: +1 at n % f, -1 beside it (or 0, where both fall on one unit)
            n = torch.arange(d, device="cuda")
            for t in range(T):
                w = Wd[e[t]]
                ref = h[t, (n * 5 + 3 + e[t]) % f] * w[n, (n * 5 + 3 + e[t]) % f].double()
                two = (n % f) != (n * 5 + 3 + e[t]) % f
                ref = ref + torch.where(two, h[t, n % f] * w[n, n % f].double(), 0.0)
                assert torch.equal(Y[t].double(), ref), f"T={T} token {t}"
            for _ in range(2):      # the counters are clear again
                Z = torch.zeros(T, d, device="cuda")
                layer.decode(X, Z, logits=logits)
                torch.cuda.synchronize()
                assert torch.equal(Z, Y)


def test_decode_captured_while_a_slot_loads():
    """Refused, and nothing is left of it: neither in the capture nor as an error
    that the next launch would report."""
    say("decode: a capture while a slot is being loaded")
    inp = gpu_inputs(SMALL)
    layer = MoELayer(inp)
    X, A = tokens(SMALL, 3)
    want = A.clone()
    layer.decode(X, want)
    torch.cuda.synchronize()
    st, cap = torch.cuda.Stream(), torch.cuda.Stream()
    B.arena_release_slot(layer.arena, 0)
    with torch.cuda.stream(st):
        torch.cuda._sleep(400_000_000)
        B.moe_pack_gate_up(layer.shape, inp.Wg[0], inp.Wu[0], layer.arena.plane_gu[0], 1, 0, 0)
        B.moe_pack_down(layer.shape, inp.Wd[0], layer.arena.plane_d[0], 1, 0, 0)
        B.arena_publish_slot(layer.arena, 0, 0)
    n = torch.zeros(1, device="cuda")
    Y = A.clone()
    g = torch.cuda.CUDAGraph()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap):
        g.capture_begin(capture_error_mode="thread_local")
        n.add_(1)
        with pytest.raises(B.MoEError) as e:
            layer.decode(X, Y)
        n.add_(1)
        g.capture_end()
    assert e.value.status == B.MOE_ERR_SLOT_STATE
    layer.decode(X, Y)               # eager: waits for the load on its stream
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, want) and float(n) == 2.0
    with torch.cuda.graph(g2 := torch.cuda.CUDAGraph()):     # loaded now
        layer.decode(X, Y)
    Y.copy_(A)
    g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, want)


@pytest.mark.parametrize("d,f", [(4, 32), (12, 64), (20, 32)])
def test_decode_narrowest_layers(d, f):
    say(f"decode, fp32, d={d} f={f}")
    cfg = MoEConfig(name="dec_narrow", index=88, T=4, d=d, f=f, E=5, k=2, n_shared=1, dtype="f32")
    inp = gpu_inputs(cfg)
    layer, weights = MoELayer(inp), plain_weights(inp)
    for T in (1, 6, 64):
        X, A = tokens(cfg, T)
        buf = torch.full((T, d + 4), 7.5, device="cuda")
        Y = buf[:, :d]
        Y.copy_(A)
        layer.decode(X, Y)
        check(inp, weights, X, A, Y, layer.decode_routes(T), f"T={T}")
        assert bool((buf[:, d:] == 7.5).all())
