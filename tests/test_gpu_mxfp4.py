"""MXFP4 quantisation, reading back and products against their definitions in
64 bits. Quantisation and reading back are exact, bit for bit.

Product: a product of two stored values has at most 4 significant bits and is
exact in fp32; K of them are added. An fp32 addition that rounds is off by at
most u = 2^-24 of the sum, one that cuts by at most 2u, so whatever the order
|C - exact| <= gamma(2K) sum_k |a b|, gamma(n) = n u / (1 - n u); bf16 results
add half a step: 8 significant bits make a step 2^(e-7) for a value in [2^e,
2^(e+1)), so half of one is at most 2^-8 of the value."""
import numpy as np
import pytest
import torch

from gpu_util import gpu_inputs, say
from oracle import oracle as oracle_mod
from routed_expert_ffn_top_amd import binding as B
from routed_expert_ffn_top_amd.inputs import MoEConfig, quantize_mxfp4
from routed_expert_ffn_top_amd.layer import MoELayer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
MAG = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def gamma(n):
    return n * U / (1 - n * U)


def two_to(n):
    """2^n in 64 bits, by its exponent (pow() need not be exact)."""
    return torch.from_numpy(np.ldexp(1.0, n.cpu().numpy()))


def stored(x):
    """(codes [rows][K], scale bytes) from the definition, on the CPU in 64 bits: the
    nearest magnitude by distance, ties to the even code."""
    b = x.detach().cpu().double().reshape(x.shape[0], -1, 32)
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad[..., None], 0.0, b)
    top = b.abs().amax(-1)
    _, e = torch.frexp(top)                     # top in [2^(e-1), 2^e)
    byte = torch.where(top > 0, (e - 1 - 2 + 127).clamp(0, 254), 0)
    v = b.abs() / two_to(byte.int() - 127)[..., None]
    d = (v.clamp(max=6.0)[..., None] - MAG).abs()
    near = d == d.amin(-1, keepdim=True)        # one code, or two neighbours
    code = torch.where(near & (torch.arange(8) % 2 == 0), torch.arange(8) + 100, torch.where(near, torch.arange(8), -1))
    code = code.amax(-1) % 100
    code = code + 8 * ((b < 0) & (code > 0))
    code = torch.where(bad[..., None], 0, code)
    return code.reshape(x.shape).to(torch.uint8), torch.where(bad, 255, byte).to(torch.uint8)


def quantise(x):
    rows, K = x.shape
    codes = torch.full((rows, K // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, K // 32), 0xEE, dtype=torch.uint8, device="cuda")
    B.moe_quantize_mxfp4(x, codes, scales)
    torch.cuda.synchronize()
    return codes, scales


def unpack(codes):
    c = codes.cpu()
    return torch.stack([c & 15, c >> 4], -1).reshape(c.shape[0], -1)


def check_quantise(x):
    codes, scales = quantise(x)
    want, byte = stored(x)
    assert torch.equal(scales.cpu(), byte), "scales"
    assert torch.equal(unpack(codes), want), "codes"
    return codes, scales


def values(codes, scales):
    """Stored values in 64 bits (the oracle's decoder is fp32: exact where it does not overflow)."""
    c = unpack(codes).long()
    s = scales.cpu().double().repeat_interleave(32, -1)
    v = torch.where(c >= 8, -1.0, 1.0).double() * MAG[c & 7] * two_to(s.int() - 127)
    return torch.where(s == 255, float("nan"), v)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,K,pad", [(1, 32, 0), (1, 2048, 0), (3, 96, 8), (65, 1408, 0), (257, 160, 64), (1030, 64, 0)])
def test_quantise_normal(rows, K, pad, dtype):
    say(f"quantise {rows} x {K}, rows {K + pad} apart, {dtype}")
    gen = torch.Generator(device="cuda").manual_seed(rows + K)
    x = torch.empty((rows, K + pad), device="cuda").normal_(generator=gen).to(dtype)[:, :K]
    codes, scales = check_quantise(x)
    want, byte = quantize_mxfp4(x.float())
    assert torch.equal(codes, want) and torch.equal(scales, byte)      # the benchmark inputs' own quantiser


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantise_borders(dtype):
    """Every border between codes, its neighbours on both sides, both signs, at
    scales from the smallest to the largest."""
    say(f"quantise: borders, {dtype}")
    edge = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9375, 0.0, 0.5, 1.0, 1.5, 2.0, 3.0]
    eps = torch.finfo(dtype).eps
    rows = []
    for e in (-126, -125, -124, -100, -3, 0, 1, 60, 124):
        for base in (4.0, 7.5):
            for sign in (1.0, -1.0):
                for off in (0.0, eps, -eps):
                    v = torch.tensor([x * (1 + off) for x in edge] + [-x for x in edge[:15]] + [base], dtype=torch.float64)
                    if e == 124:
                        v = v.clamp(-7.9, 7.9)
                    rows.append((sign * v * 2.0 ** e).float())
    check_quantise(torch.stack(rows).to(dtype).cuda())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantise_extremes(dtype):
    say(f"quantise: zeros, subnormals, the largest, infinities, NaN, {dtype}")
    x = torch.zeros(12, 64, dtype=dtype)
    fin = torch.finfo(dtype)
    x[1, 3] = -0.0
    x[2, :32] = torch.linspace(-1, 1, 32).to(dtype) * fin.tiny * 0.5      # subnormals
    x[2, 40] = fin.smallest_normal
    x[3, 5], x[3, 6] = fin.max, -fin.max
    x[4, 7] = float("inf")
    x[5, 33] = float("-inf")
    x[6, 2], x[6, 3] = float("nan"), 1.0
    x[7, :32], x[7, 9] = 1.0, float("nan")
    x[8, :32] = 2.0 ** -126
    x[9, 0], x[9, 1] = 2.0 ** -133, 2.0 ** -126      # a subnormal beside a normal
    x[10, 0], x[10, 1] = 2.0 ** 127, -(2.0 ** 126)
    x[11] = -(2.0 ** -124)
    codes, scales = check_quantise(x.cuda())
    assert scales[4, 0] == 255 and scales[4, 1] == 0 and scales[6, 0] == 255 and int(codes[6, 0]) == 0


def test_quantise_fp32_subnormal_blocks():
    say("quantise: blocks of fp32 subnormals")
    gen = torch.Generator().manual_seed(1)
    bits = torch.randint(0, 1 << 23, (40, 64), generator=gen, dtype=torch.int32)
    bits[:20] = bits[:20] >> torch.randint(0, 23, (20, 1), generator=gen, dtype=torch.int32)
    bits |= torch.randint(0, 2, bits.shape, generator=gen, dtype=torch.int32) << 31
    check_quantise(bits.view(torch.float32).cuda())


def test_quantise_long_rows_of_weights():
    say("quantise: 2.2e9 values, offsets past 2^31 elements")
    rows, K = 2050, 1 << 20
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(4)
    at = [0, 1, 1023, 2047, 2048, 2049]
    for r in at:
        x[r].normal_(generator=gen)
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, K // 32), dtype=torch.uint8, device="cuda")
    B.moe_quantize_mxfp4(x, codes, scales)
    want, byte = quantize_mxfp4(x[at].float())
    assert torch.equal(codes[at], want) and torch.equal(scales[at], byte)
    assert int(codes[2:1000].max()) == 0 and int(scales[2:1000].max()) == 0
    y = torch.empty_like(x)
    B.moe_dequantize_mxfp4(codes, scales, y)
    torch.cuda.synchronize()
    assert torch.equal(y[2049].double().cpu(), values(codes[2049:], scales[2049:])[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_dequantise_every_code_and_scale(dtype):
    say(f"read back: 16 codes x 256 scales, {dtype}")
    codes = torch.arange(16, dtype=torch.uint8).repeat(2)
    codes = (codes[0::2] | codes[1::2] << 4).repeat(256, 1).cuda()
    scales = torch.arange(256, dtype=torch.uint8).reshape(256, 1).cuda()
    buf = torch.full((256, 40), 3.5, dtype=dtype, device="cuda")
    B.moe_dequantize_mxfp4(codes, scales, buf[:, :32])
    torch.cuda.synchronize()
    want = values(codes, scales).to(dtype)       # 64 bits to the type: overflow gives infinities
    got = buf[:, :32].cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(nan=1.0), want.nan_to_num(nan=1.0))
    assert bool((buf[:, 32:] == 3.5).all())
    orc = oracle_mod.get()
    ref = torch.from_numpy(orc.mxfp4_decode(codes.cpu().numpy()[1:254], scales.cpu().numpy()[1:254]))
    if dtype == torch.float32:
        assert torch.equal(got[1:254], ref)


def pack(w):
    """fp32 weights [P][N][K] to packed slices on the GPU; also the stored values in 64 bits."""
    P, N, K = w.shape
    shape = B.make_shape(1, N, K, 1, 1, dtype="bf16_fp4w")
    packed = torch.empty((P, B.fp4_slice_bytes(N, K)), dtype=torch.uint8, device="cuda")
    vals = []
    for p in range(P):
        sl = B.mxfp4_slice(w[p])
        B.moe_pack_down(shape, sl, packed[p], 1, 0, 0)
        vals.append(values(sl[: N * K // 2].reshape(N, -1), sl[N * K // 2:].reshape(N, -1)))
    return packed, torch.stack(vals).cuda()


def product(A, W, off, rec):
    """(exact, sum of magnitudes) in 64 bits; A [rows][K], W [P][N][K] values."""
    out = torch.zeros(len(rec), W.shape[1], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    for p in range(W.shape[0]):
        r = slice(off[p], off[p + 1])
        out[r] = A[rec[r]] @ W[p].t()
        mag[r] = A[rec[r]].abs() @ W[p].abs().t()
    return out, mag


def run_matmul(M, N, K, P, sizes, gather, dtype, seed=0, tail=0, scale_spread=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + M + N + K)
    w = torch.empty((P, N, K), device="cuda").normal_(generator=gen)
    rows = max(1, M // 3) if gather else M
    x = torch.empty((rows, K), device="cuda").normal_(generator=gen)
    if scale_spread:
        e = torch.randint(-scale_spread, scale_spread + 1, (rows, K // 32, 1), generator=gen, device="cuda").float()
        x = (x.reshape(rows, -1, 32) * torch.pow(2.0, e)).reshape(rows, K)
        e = torch.randint(-scale_spread, scale_spread + 1, (P, N, K // 32, 1), generator=gen, device="cuda").float()
        w = (w.reshape(P, N, -1, 32) * torch.pow(2.0, e)).reshape(P, N, K)
    packed, W = pack(w)
    codes, scales = quantise(x)
    A = values(codes, scales).cuda()
    off = [0] + list(np.cumsum(sizes))
    used = off[-1]
    assert used + tail == M
    rec = torch.randint(rows, (M,), generator=gen, device="cuda", dtype=torch.int32) if gather else None
    C = torch.full((M, N + 16), -77.0, dtype=dtype, device="cuda")
    B.moe_matmul_mxfp4(codes, scales, packed, C[:, :N], slot_offset=torch.tensor(off, dtype=torch.int32, device="cuda"),
                       row_index=rec)
    torch.cuda.synchronize()
    r = rec.long() if gather else torch.arange(M, device="cuda")
    ref, mag = product(A, W, off, r)
    err = (C[:used, :N].double() - ref[:used]).abs()
    bound = gamma(2 * K) * mag[:used] + 2.0 ** -126
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (ref[:used].abs() + bound)
    assert torch.isfinite(C[:used, :N]).all()
    if used:
        say(f"  max err/bound {float((err / bound).max()):.3g}, rel {float(err.norm() / ref[:used].norm()):.3g}")
    assert bool((err <= bound).all())
    assert bool((C[used:] == -77.0).all()) and bool((C[:, N:] == -77.0).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (1, 2048, 1024), (2, 320, 448), (31, 64, 128), (33, 128, 192), (64, 64, 64),
                                   (65, 576, 320), (255, 256, 256), (256, 512, 128), (257, 320, 1408), (700, 1088, 576)])
def test_matmul_one_slice(M, N, K, dtype):
    say(f"matmul {M} x {N} x {K} {dtype}")
    run_matmul(M, N, K, 1, [M], False, dtype)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("sizes,tail", [([0, 5, 0, 64, 1, 300, 0], 0), ([1] * 66, 0), ([0, 0, 0], 7), ([257, 0, 255, 513], 31),
                                        ([0] * 100 + [3] + [0] * 50 + [129], 2)])
def test_matmul_groups(sizes, tail, gather):
    say(f"matmul groups {sizes[:8]}.. of {len(sizes)}, {tail} rows behind, gather {gather}")
    run_matmul(sum(sizes) + tail, 192, 320, len(sizes), sizes, gather, torch.float32, tail=tail)


def test_matmul_spread_scales():
    say("matmul: scales spread over 2^-20 .. 2^20")
    run_matmul(130, 320, 448, 3, [30, 0, 100], True, torch.float32, scale_spread=20)
    run_matmul(300, 256, 512, 1, [300], False, torch.float32, scale_spread=20)


@pytest.mark.parametrize("M", [3, 300])
def test_matmul_exact_where_a_scale_is_wrong_elsewhere(M):
    """One code 1.0 and one scale byte a row and weight, all others 0 or
    another power of two: each result is one product, 2^(i + j)."""
    say(f"matmul: every scale in its place, M={M}")
    N, K = 320, 448
    gen = torch.Generator(device="cuda").manual_seed(2)
    codes = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
    wc = torch.zeros(N, K, dtype=torch.uint8, device="cuda")
    k = torch.randint(K, (M,), generator=gen, device="cuda")
    codes[torch.arange(M), k] = 2
    wc[:, :] = 2
    As = torch.randint(100, 140, (M, K // 32), generator=gen, device="cuda", dtype=torch.int32).to(torch.uint8)
    Ws = torch.randint(100, 140, (N, K // 32), generator=gen, device="cuda", dtype=torch.int32).to(torch.uint8)
    two = lambda c: (c[:, 0::2] | c[:, 1::2] << 4).contiguous()
    shape = B.make_shape(1, N, K, 1, 1, dtype="bf16_fp4w")
    packed = torch.empty(B.fp4_slice_bytes(N, K), dtype=torch.uint8, device="cuda")
    B.moe_pack_down(shape, torch.cat([two(wc).reshape(-1), Ws.reshape(-1)]), packed, 1, 0, 0)
    C = torch.empty(M, N, device="cuda")
    B.moe_matmul_mxfp4(two(codes), As, packed, C)
    torch.cuda.synchronize()
    b = k // 32
    n = (As[torch.arange(M), b].int()[:, None] + Ws[:, b].int().t() - 254).cpu().numpy()
    bad = np.argwhere(C.cpu().numpy() != np.ldexp(1.0, n))       # a power of two by its exponent: no pow()
    assert not len(bad), f"{len(bad)} differ, first {bad[:4].tolist()}: {C.cpu().numpy()[tuple(bad[0])]!r}, 2^{n[tuple(bad[0])]}"


def test_matmul_nan_and_infinite_blocks():
    say("matmul: a NaN block reaches its own row only; out-of-range rows are brought into range")
    M, N, K = 70, 128, 128
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty((M, K), device="cuda").normal_(generator=gen)
    w = torch.empty((1, N, K), device="cuda").normal_(generator=gen)
    packed, _ = pack(w)
    c, s = quantise(x)
    C = torch.empty(M, N, device="cuda")
    B.moe_matmul_mxfp4(c, s, packed[0], C)
    x[5, 40], x[69, 3] = float("nan"), float("inf")
    c2, s2 = quantise(x)
    D = torch.empty(M, N, device="cuda")
    B.moe_matmul_mxfp4(c2, s2, packed[0], D)
    w[0, 17, 100] = float("nan")
    packed2, _ = pack(w)
    E = torch.empty(M, N, device="cuda")
    B.moe_matmul_mxfp4(c, s, packed2[0], E)
    torch.cuda.synchronize()
    keep = torch.ones(M, dtype=torch.bool)
    keep[[5, 69]] = False
    assert torch.equal(C[keep], D[keep]) and bool(torch.isnan(D[~keep]).all())
    cols = torch.ones(N, dtype=torch.bool)
    cols[17] = False
    assert torch.equal(C[:, cols], E[:, cols]) and bool(torch.isnan(E[:, 17]).all())
    rec = torch.tensor([-5, M + 9, 3], dtype=torch.int32, device="cuda")
    F = torch.empty(3, N, device="cuda")
    B.moe_matmul_mxfp4(c, s, packed[0], F, row_index=rec)
    G = torch.zeros(3, N, device="cuda")
    B.moe_matmul_mxfp4(c, s, packed, G, slot_offset=torch.tensor([-4, 900], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(F, C[[0, M - 1, 3]]) and torch.equal(G, C[:3])


def test_matmul_same_bits_alone_and_in_groups():
    """A record's result hangs neither on its group's size nor on its place."""
    say("matmul: same bits alone and in groups")
    gen = torch.Generator(device="cuda").manual_seed(8)
    x = torch.empty((600, 512), device="cuda").normal_(generator=gen)
    w = torch.empty((2, 256, 512), device="cuda").normal_(generator=gen)
    packed, _ = pack(w)
    c, s = quantise(x)
    C = torch.empty(600, 256, device="cuda")
    B.moe_matmul_mxfp4(c, s, packed, C, slot_offset=torch.tensor([0, 590, 600], dtype=torch.int32, device="cuda"))
    D = torch.empty(600, 256, device="cuda")
    for lo, hi, p in ((0, 1, 0), (1, 40, 0), (40, 590, 0), (590, 600, 1)):
        B.moe_matmul_mxfp4(c[lo:hi], s[lo:hi], packed[p], D[lo:hi])
    torch.cuda.synchronize()
    assert torch.equal(C, D)


def test_matmul_of_a_layer_route_map():
    """Quantised activations through the gate/up slices of an arena, grouped by
    a route build, as the expert projections take them."""
    say("matmul over a route map and an arena's plane")
    cfg = MoEConfig(name="mx_route", index=77, T=90, d=256, f=128, E=8, k=2, dtype="bf16_fp4w")
    inp = gpu_inputs(cfg)
    layer = MoELayer(inp)
    layer.forward(inp.A.clone())
    codes, scales = quantise(inp.X)
    n = cfg.T * cfg.kp
    C = torch.empty(n, 2 * cfg.f, device="cuda")
    r = layer.routes
    B.moe_matmul_mxfp4(codes, scales, layer.arena.plane_gu, C, slot_offset=r["slot_offset"], row_index=r["rec_token"])
    torch.cuda.synchronize()
    A = values(codes, scales).cuda()
    orc = oracle_mod.get()
    dec = lambda q, s: torch.from_numpy(orc.mxfp4_decode(q.cpu().numpy(), s.cpu().numpy())).cuda().double()
    Wg, Wu = dec(inp.Wg, inp.Sg), dec(inp.Wu, inp.Su)
    # packed rows alternate 32 gate, 32 up
    W = torch.stack([Wg.reshape(8, 4, 32, 256), Wu.reshape(8, 4, 32, 256)], 2).reshape(8, 256, 256)
    ref, mag = product(A, W, r["slot_offset"].tolist(), r["rec_token"][:n].long())
    assert bool(((C.double() - ref).abs() <= gamma(512) * mag).all())


def test_arena_from_unquantised_weights():
    """Weights quantised by the library on the way into an arena give the layer
    that the stored codes give, for prompts and for tokens."""
    say("an MXFP4 arena loaded from fp32 and bf16 weights")
    cfg = MoEConfig(name="mx_load", index=78, T=70, d=320, f=192, E=6, k=2, n_shared=1, dtype="bf16_fp4w")
    inp = gpu_inputs(cfg)
    gen = torch.Generator(device="cuda").manual_seed(12)
    ws = [torch.empty(s, device="cuda").normal_(0, 0.02, generator=gen) for s in
          ((7, 192, 320), (7, 192, 320), (7, 320, 192))]
    for dt in (torch.float32, torch.bfloat16):
        src = [w.to(dt) for w in ws]
        (inp.Wg, inp.Sg), (inp.Wu, inp.Su), (inp.Wd, inp.Sd) = (quantize_mxfp4(w.float()) for w in src)
        a, b = MoELayer(inp), MoELayer(inp)
        b.arena.plane_gu.fill_(0xFF)
        b.arena.plane_d.fill_(0xFF)
        for s in range(7):
            B.arena_release_slot(b.arena, s)
        b.arena.load_resident(*src, phi=list(range(7)))
        assert torch.equal(a.arena.plane_gu, b.arena.plane_gu) and torch.equal(a.arena.plane_d, b.arena.plane_d)
        Y, Z = inp.A.clone(), inp.A.clone()
        a.forward(Y)
        b.forward(Z)
        y, z = inp.A[:5].clone(), inp.A[:5].clone()
        a.decode(inp.X[:5], y)
        b.decode(inp.X[:5], z)
        torch.cuda.synchronize()
        assert torch.equal(Y, Z) and torch.equal(y, z)


def test_mxfp4_captured_and_on_another_stream():
    say("quantise, product and read back: captured, replayed, on a side stream")
    gen = torch.Generator(device="cuda").manual_seed(21)
    packed, _ = pack(torch.empty((1, 128, 256), device="cuda").normal_(generator=gen))
    x = torch.empty((37, 256), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    c, s = torch.empty(37, 128, dtype=torch.uint8, device="cuda"), torch.empty(37, 8, dtype=torch.uint8, device="cuda")
    C, V = torch.empty(37, 128, device="cuda"), torch.empty(37, 256, device="cuda")

    def step():
        B.moe_quantize_mxfp4(x, c, s)
        B.moe_matmul_mxfp4(c, s, packed[0], C)
        B.moe_dequantize_mxfp4(c, s, V)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        x.normal_(generator=gen)
        C.fill_(0)
        g.replay()
        got = (C.clone(), V.clone())
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            step()
        torch.cuda.current_stream().wait_stream(st)
        torch.cuda.synchronize()
        assert torch.equal(got[0], C) and torch.equal(got[1], V)


# ---- sizes that the ring kernel takes (whole tiles of 256 x 256, stages of 128 k) ----

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(769, 2176, 128), (1100, 1408, 576), (2049, 832, 64), (1025, 1600, 640), (513, 4160, 1408),
                                   (1024, 2048, 512)])
def test_matmul_large_one_slice(M, N, K, dtype):
    say(f"matmul, large, {M} x {N} x {K} {dtype}")
    run_matmul(M, N, K, 1, [M], False, dtype)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("sizes,tail,N,K", [([257, 0, 255, 513, 1, 600], 31, 1088, 320), ([0] * 100 + [3000] + [0] * 50 + [129], 2, 256, 256),
                                            ([40] * 66, 0, 512, 384), ([128, 129, 0, 256, 700], 5, 1152, 1024)])
def test_matmul_large_groups(sizes, tail, N, K, gather):
    say(f"matmul, large groups of {len(sizes)}, N={N} K={K}, {tail} rows behind, gather {gather}")
    run_matmul(sum(sizes) + tail, N, K, len(sizes), sizes, gather, torch.float32, tail=tail, scale_spread=6)


@pytest.mark.parametrize("off", [0, 2, 4, 6])
def test_matmul_large_unaligned_scales(off):
    """Scale bytes that start at any even address, at the end of their allocation."""
    say(f"matmul, large, scales {off} bytes from a 16-byte address")
    M, N, K = 900, 2048, 256
    gen = torch.Generator(device="cuda").manual_seed(off)
    x = torch.empty((M, K), device="cuda").normal_(generator=gen)
    packed, W = pack(torch.empty((1, N, K), device="cuda").normal_(generator=gen))
    c, s = quantise(x)
    buf = torch.full((off + s.numel(),), 255, dtype=torch.uint8, device="cuda")
    t = buf[off:].view(s.shape)
    t.copy_(s)
    C = torch.empty(M, N, device="cuda")
    B.moe_matmul_mxfp4(c, t, packed[0], C)
    torch.cuda.synchronize()
    ref, mag = product(values(c, s).cuda(), W, [0, M], torch.arange(M, device="cuda"))
    assert bool(((C.double() - ref).abs() <= gamma(2 * K) * mag).all())


def test_matmul_large_same_bits_as_small():
    say("matmul: a record's bits are the same in large and in small calls")
    gen = torch.Generator(device="cuda").manual_seed(18)
    for K in (448, 512):
        x = torch.empty((1300, K), device="cuda").normal_(generator=gen)
        w = torch.empty((2, 1600, K), device="cuda").normal_(generator=gen)
        packed, _ = pack(w)
        c, s = quantise(x)
        C = torch.empty(1300, 1600, device="cuda")
        B.moe_matmul_mxfp4(c, s, packed, C, slot_offset=torch.tensor([0, 1290, 1300], dtype=torch.int32, device="cuda"))
        D = torch.empty(1300, 1600, device="cuda")
        for lo, hi, p in ((0, 1, 0), (1, 40, 0), (40, 160, 0), (1250, 1290, 0), (1290, 1300, 1)):
            B.moe_matmul_mxfp4(c[lo:hi].clone(), s[lo:hi].clone(), packed[p], D[lo:hi])
        torch.cuda.synchronize()
        assert torch.equal(C[:160], D[:160]) and torch.equal(C[1250:], D[1250:])


def test_matmul_large_nan_blocks_and_ranges():
    say("matmul, large: NaN blocks stay in their rows and columns; rows and offsets out of range")
    M, N, K = 800, 2048, 256
    gen = torch.Generator(device="cuda").manual_seed(31)
    x = torch.empty((M, K), device="cuda").normal_(generator=gen)
    w = torch.empty((1, N, K), device="cuda").normal_(generator=gen)
    packed, _ = pack(w)
    c, s = quantise(x)
    C = torch.empty(M, N, device="cuda")
    B.moe_matmul_mxfp4(c, s, packed[0], C)
    c2, s2, bad = c.clone(), s.clone(), [5, 255, 256, 799]
    for i, r in enumerate(bad):
        s2[r, i * 2] = 255
    w2 = packed.clone()
    B.moe_pack_down(B.make_shape(1, N, K, 1, 1, dtype="bf16_fp4w"), with_nan(w[0], 1500, 130), w2[0], 1, 0, 0)
    D, E = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    B.moe_matmul_mxfp4(c2, s2, packed[0], D)
    B.moe_matmul_mxfp4(c, s, w2[0], E)
    rec = torch.arange(M, dtype=torch.int32, device="cuda")
    rec[3], rec[700] = -9, M + 70
    F = torch.zeros(M + 40, N, device="cuda")
    far = torch.tensor([-7, M + 1000], dtype=torch.int32, device="cuda")
    B.moe_matmul_mxfp4(c, s, packed, F[:M], slot_offset=far, row_index=rec)
    torch.cuda.synchronize()
    keep = torch.ones(M, dtype=torch.bool)
    keep[bad] = False
    assert torch.equal(C[keep], D[keep]) and bool(torch.isnan(D[~keep]).all())
    cols = torch.arange(N) != 1500
    assert torch.equal(C[:, cols], E[:, cols]) and bool(torch.isnan(E[:, 1500]).all())
    want = C.clone()
    want[3], want[700] = C[0], C[M - 1]
    assert torch.equal(F[:M], want) and bool((F[M:] == 0).all())


def with_nan(w, n, k):
    w = w.clone()
    w[n, k] = float("nan")
    return B.mxfp4_slice(w)


# ---- ring workgroups with several tiles each ----

def ring_tiles(sizes, N):
    """Tiles of 256 x 256; 256 workgroups take them, so more than 768 are four for some and three for all others."""
    return sum((n + 255) // 256 for n in sizes) * ((N + 255) // 256)


def ring_pieces(sizes, tail, N):
    """What the choice between the two kernels looks at: 32 x 64 pieces at the mean rows a slot."""
    M = sum(sizes) + tail
    slots = min(len(sizes), M)
    return slots * ((M // slots + 31) // 32) * (N // 64)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [64, 128, 192, 448, 512, 640])
def test_matmul_several_tiles_a_workgroup(K, dtype, gather):
    """A tile requested while the one before it is stored: its rows, scales and
    shifts stand beside the old ones. Partial and empty slots, columns past N."""
    sizes, tail, N = [0, 5000, 0, 257, 1, 9000, 256, 0, 3000, 255, 4000, 7], 77, 2112
    say(f"matmul, {ring_tiles(sizes, N)} tiles, K={K}, {dtype}, gather {gather}")
    assert ring_tiles(sizes, N) > 768 and ring_pieces(sizes, tail, N) >= 768
    run_matmul(sum(sizes) + tail, N, K, len(sizes), sizes, gather, dtype, tail=tail, scale_spread=5)


@pytest.mark.parametrize("K,off", [(64, 2), (128, 2), (320, 6)])
def test_matmul_several_tiles_unaligned_scales(K, off):
    say(f"matmul, several tiles a workgroup, scales {off} bytes from a 16-byte address, K={K}")
    M, N = 24001, 2240
    assert ring_tiles([M], N) > 768
    gen = torch.Generator(device="cuda").manual_seed(off + K)
    x = torch.empty((8000, K), device="cuda").normal_(generator=gen)
    packed, W = pack(torch.empty((1, N, K), device="cuda").normal_(generator=gen))
    c, s = quantise(x)
    buf = torch.full((off + s.numel(),), 255, dtype=torch.uint8, device="cuda")
    t = buf[off:].view(s.shape)
    t.copy_(s)
    rec = torch.randint(8000, (M,), generator=gen, device="cuda", dtype=torch.int32)
    C = torch.empty(M, N, device="cuda")
    B.moe_matmul_mxfp4(c, t, packed[0], C, row_index=rec)
    torch.cuda.synchronize()
    ref, mag = product(values(c, s).cuda(), W, [0, M], rec.long())
    assert bool(((C.double() - ref).abs() <= gamma(2 * K) * mag).all())


@pytest.mark.parametrize("gather", [False, True])
def test_matmul_large_groups_uneven(gather):
    say(f"matmul, large, uneven groups with an empty one, gather {gather}")
    sizes, tail, N, K = [128, 129, 0, 256, 700], 5, 1280, 1024
    assert ring_pieces(sizes, tail, N) >= 768
    run_matmul(sum(sizes) + tail, N, K, len(sizes), sizes, gather, torch.float32, tail=tail, scale_spread=6)
