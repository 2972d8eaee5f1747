"""Operators around a layer whose experts are stored in 8-bit floating point with a scale for each block of 128, and
around the training of its router, as cases that can be timed and compared:

  quant    values to e4m3 codes with one scale for each block (128 of a row, or 128 x 128 of a matrix) and back
  matmul   rows quantised as they come, times such weight slices, one slice for each group of rows
  experts  the same with SwiGLU and the second product behind it: a whole expert FFN in record order
  combine  the records' rows summed into their tokens with the route weights, and the gradients of both
  balance  the load-balancing loss of a routing with the counts behind it, and the gradient of the router's logits

`run` computes them in elementary torch operations, or, with `own`, with the library's entry points.
"""
import math

import torch

own = False

STD_W = 0.02


def listed():
    return [
        # one token's activations on their way into an 8-bit product
        dict(name="quant_row_bf16", kind="quant", src="bf16", rows=1, K=2048, pad=0, block=1),
        # the gate weights of a layer when a model is loaded
        dict(name="quant_weights_f32", kind="quant", src="f32", rows=65536, K=2048, pad=0, block=128),
        # the down projections of one answering token: 8 of 64 experts, a record each
        dict(name="matmul_olmoe_one_token", kind="matmul", M=8, N=2048, K=1024, P=64, gather=False, out="bf16", pow2=True),
        # 32 sequences answering, two of eight large experts each: nothing but reading the weights
        dict(name="matmul_mixtral_t32", kind="matmul", M=64, N=4096, K=14336, P=8, gather=False, out="f32", pow2=False),
        # the down projection of a prompt of 4096 tokens, the shared experts among the slots, a checkpoint's own scales
        dict(name="matmul_dsv2lite_down", kind="matmul", M=32768, N=2048, K=1408, P=66, gather=False, out="bf16", pow2=False),
        # a short prompt: groups of uneven size, some empty, widths that end inside a block
        dict(name="matmul_ragged", kind="matmul", M=777, N=320, K=448, P=7, gather=True, out="f32", pow2=False),
        # an expert FFN for one answering token
        dict(name="experts_olmoe_one_token", kind="experts", T=1, k=8, d=2048, f=1024, P=64, pow2=True),
        # an expert FFN over a prompt of 4096 tokens, 8 of 64 experts each
        dict(name="experts_olmoe_t4096", kind="experts", T=4096, k=8, d=2048, f=1024, P=64, pow2=False),
        # a short prompt at odd sizes, a tenth of the routes left out: their experts are not resident
        dict(name="combine_ragged_f32", kind="combine", T=33, k=5, d=324, rows="f32", absent=0.1, pad=4),
        # the end of a prompt's layer in training the router: every route of 4096 tokens
        dict(name="combine_olmoe_t4096", kind="combine", T=4096, k=8, d=2048, rows="bf16", absent=0.0, pad=0),
        # the smallest layer that the library is run on, a batch of 16 tokens
        dict(name="balance_tiny", kind="balance", T=16, E=8, k=2, shared=0, S=1, masked=0.0, renorm=True, weights=True),
        # a long batch of 16 sequences, padded, on the widest router
        dict(name="balance_t65536_e256", kind="balance", T=65536, E=256, k=8, shared=1, S=16, masked=0.2, renorm=False,
             weights=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 1e-9)))))


def draw(rng):
    kind = rng.choice(["quant", "matmul", "matmul", "experts", "combine", "balance"])
    if kind == "quant":
        while True:
            c = dict(kind=kind, src=rng.choice(["bf16", "f32"]), rows=_log(rng, 1, 65536), K=64 * _log(rng, 1, 224),
                     pad=rng.choice([0, 0, 8, 64]), block=rng.choice([1, 128]))
            if c["rows"] * c["K"] <= 1 << 27:
                return c
    if kind == "matmul":
        while True:
            c = dict(kind=kind, M=_log(rng, 1, 32768), N=64 * _log(rng, 1, 64), K=64 * _log(rng, 1, 224),
                     P=_log(rng, 1, 66), gather=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]),
                     pow2=rng.random() < 0.4)
            if c["M"] * c["N"] * c["K"] <= 1 << 36 and c["P"] * c["N"] * c["K"] <= 1 << 28 and c["M"] * c["N"] <= 1 << 26:
                return c
    if kind == "experts":
        while True:
            c = dict(kind=kind, T=_log(rng, 1, 4096), d=64 * _log(rng, 2, 64), f=64 * _log(rng, 1, 64),
                     P=_log(rng, 1, 66), pow2=rng.random() < 0.4)
            c["k"] = rng.randint(1, min(8, c["P"]))
            if c["T"] * c["k"] * c["d"] * c["f"] <= 1 << 36 and c["P"] * c["d"] * c["f"] <= 1 << 27:
                return c
    if kind == "combine":
        return dict(kind=kind, T=_log(rng, 1, 4096), k=rng.randint(1, 8), d=4 * _log(rng, 1, 512),
                    rows=rng.choice(["bf16", "f32"]), absent=rng.choice([0.0, 0.1, 0.5]), pad=rng.choice([0, 0, 4, 64]))
    E = _log(rng, 2, 256)
    T = _log(rng, 1, 65536)
    return dict(kind=kind, T=T, E=E, k=rng.randint(1, min(8, E)), shared=rng.choice([0, 0, 1, 2]),
                S=_log(rng, 1, min(64, T)), masked=rng.choice([0.0, 0.0, 0.2, 0.9]), renorm=rng.random() < 0.5,
                weights=rng.random() < 0.6)


# ---- inputs ----

def _normal(gen, shape, std=1.0, dtype=torch.float32):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen).to(dtype)


def _rows(gen, shape, pad, dtype, std=1.0):
    """A matrix whose rows lie `pad` elements further apart than they are long."""
    return _normal(gen, (shape[0], shape[1] + pad), std, dtype)[:, : shape[1]]


def _cut(x, rows, cols):
    """x [..., R, C] padded with zeros to whole blocks, as [..., R / rows, rows, C / cols, cols]."""
    R, C = x.shape[-2:]
    x = torch.nn.functional.pad(x, (0, -C % cols, 0, -R % rows))
    return x.reshape(*x.shape[:-2], x.shape[-2] // rows, rows, x.shape[-1] // cols, cols)


def _whole(b, R, C):
    """_cut undone."""
    return b.reshape(*b.shape[:-4], b.shape[-4] * b.shape[-3], b.shape[-2] * b.shape[-1])[..., :R, :C]


def _quantise(x, rows):
    """e4m3 codes (as fp32 values) and exponent bytes of fp32 x [..., R, C] in blocks of rows x 128: the byte is the
    least in 1 .. 247 with max |x| <= 448 * 2^(byte - 127); a block with an infinity or a NaN has 255 and codes 0."""
    b = _cut(x, rows, 128)
    top = b.abs().amax((-3, -1))
    bad = ~torch.isfinite(top)
    m, e = torch.frexp(torch.where(bad, 0.0, top))   # top = m 2^e, m in [1/2, 1): 448 = (7/8) 2^9
    byte = (e - 9 + (m > 0.875) + 127).clamp(1, 247)
    byte = torch.where(bad, 255, torch.where(top == 0, 1, byte))
    v = torch.where(bad[..., None, :, None], 0.0, b * _pow2(254 - byte)[..., None, :, None])
    return _whole(v.to(torch.float8_e4m3fn).float(), *x.shape[-2:]), byte


def _pow2(field):
    """2^(field - 127) in fp32 for exponent fields 1 .. 254, which pow() and ldexp() need not give exactly."""
    return (field.to(torch.int32) << 23).view(torch.float32)


def _unit(byte):
    return torch.where(byte == 255, math.nan, _pow2(byte))


def _spread(s, rows, R, C):
    """A scale for each block of rows x 128 as one for each element of [R, C]."""
    return s.repeat_interleave(rows, -2)[..., :R, :].repeat_interleave(128, -1)[..., :C]


def _weights(gen, shape, pow2):
    """Codes (uint8) and fp32 scales of a stack of weight matrices: with powers of two as scales, or max / 448."""
    codes, scales = [], []
    for _ in range(shape[0]):   # one at a time: they are made in fp32
        w = _normal(gen, shape[1:], STD_W)
        if pow2:
            v, byte = _quantise(w, 128)
            s = _unit(byte)
        else:
            s = _cut(w, 128, 128).abs().amax((-3, -1)) / 448.0
            v = w / _spread(s, 128, *shape[1:])
        codes.append(v.to(torch.float8_e4m3fn).view(torch.uint8))
        scales.append(s)
    return torch.stack(codes), torch.stack(scales)


def _sizes(P, M, seed):
    """How many rows each group has: uneven, and now and then none."""
    cpu = torch.Generator().manual_seed(seed)
    p = torch.rand(P, generator=cpu) + 0.5
    if P > 4:
        p[torch.randint(P, (1,), generator=cpu)] = 0.0
    return torch.bincount(torch.multinomial(p, M, replacement=True, generator=cpu), minlength=P)


def _offset(n):
    return torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)]).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    return {"quant": _prepare_quant, "matmul": _prepare_matmul, "experts": _prepare_experts,
            "combine": _prepare_combine, "balance": _prepare_balance}[c["kind"]](c, seed, gen)


def _row_blocks(rows, K):
    """Memory for the codes and scales of quantised rows."""
    from routed_expert_ffn_top_amd import binding as B
    return (torch.empty((rows, K), dtype=torch.uint8, device="cuda"),
            torch.empty((rows, B.fp8_scale_bytes(K)), dtype=torch.uint8, device="cuda"))


def _prepare_quant(c, seed, gen):
    x = _rows(gen, (c["rows"], c["K"]), c["pad"], torch.float32 if c["src"] == "f32" else torch.bfloat16, STD_W)
    s = dict(case=c, x=x)
    if own:
        codes, scales = _row_blocks(c["rows"], c["K"])
        if c["block"] == 128:
            scales = torch.empty((-(-c["rows"] // 128), -(-c["K"] // 128)), device="cuda")
        s.update(codes=codes, scales=scales, out=torch.empty((c["rows"], c["K"]), dtype=torch.bfloat16, device="cuda"))
    return s


def _prepare_matmul(c, seed, gen):
    n = _sizes(c["P"], c["M"], seed)
    rows = max(1, c["M"] // 8) if c["gather"] else c["M"]
    x = _normal(gen, (rows, c["K"]), 1.0, torch.bfloat16)
    take = torch.randint(rows, (c["M"],), generator=gen, device="cuda", dtype=torch.int32) if c["gather"] else None
    w, ws = _weights(gen, (c["P"], c["N"], c["K"]), c["pow2"])
    s = dict(case=c, x=x, offset=_offset(n).cuda(), take=take, most=int(n.max()), w=w, ws=ws)
    if own:
        s["a"], s["as"] = _row_blocks(rows, c["K"])
        s["out"] = torch.empty((c["M"], c["N"]), dtype=torch.float32 if c["out"] == "f32" else torch.bfloat16, device="cuda")
    return s


def _prepare_experts(c, seed, gen):
    # every token goes to k different experts; records in the order of the experts, then of the routes
    cpu = torch.Generator().manual_seed(seed)
    p = torch.rand(c["P"], generator=cpu) + 0.5
    to = torch.multinomial(p.expand(c["T"], -1), c["k"], generator=cpu).reshape(-1)
    n = torch.bincount(to, minlength=c["P"])
    take = torch.sort(to, stable=True)[1] // c["k"]
    x = _normal(gen, (c["T"], c["d"]), 1.0, torch.bfloat16)
    s = dict(case=c, x=x, offset=_offset(n).cuda(), take=take.to(torch.int32).cuda(), most=int(n.max()))
    for name, N, K in (("wg", c["f"], c["d"]), ("wu", c["f"], c["d"]), ("wd", c["d"], c["f"])):
        s[name], s[name + "s"] = _weights(gen, (c["P"], N, K), c["pow2"])
    if own:
        M = c["T"] * c["k"]
        s["a"], s["as"] = _row_blocks(c["T"], c["d"])
        s["h"], s["hs"] = _row_blocks(M, c["f"])
        s["out"] = torch.empty((M, c["d"]), dtype=torch.bfloat16, device="cuda")
    return s


def _prepare_combine(c, seed, gen):
    n, dt = c["T"] * c["k"], torch.float32 if c["rows"] == "f32" else torch.bfloat16
    out = torch.rand(n, generator=gen, device="cuda") < c["absent"]
    # the routes that are there, in the order of the records
    order = torch.argsort(torch.rand(n, generator=gen, device="cuda") + out)
    pos = torch.empty(n, dtype=torch.int64, device="cuda")
    pos[order] = torch.arange(n, device="cuda")
    pos = torch.where(out, -1, pos).to(torch.int32)
    w = torch.rand((c["T"], c["k"]), generator=gen, device="cuda")
    s = dict(case=c, C=_rows(gen, (n, c["d"]), c["pad"], dt, 0.1), pos=pos, w=w / w.sum(-1, keepdim=True),
             y=_rows(gen, (c["T"], c["d"]), c["pad"], torch.float32), dy=_rows(gen, (c["T"], c["d"]), c["pad"], torch.float32))
    # records that no route points at keep what their gradient's memory held: zeros here
    s["dC"] = torch.zeros((n, c["d"]), dtype=dt, device="cuda")
    if own:
        s["dw"] = torch.empty_like(s["w"])
    return s


def _prepare_balance(c, seed, gen):
    cpu = torch.Generator().manual_seed(seed)
    cuts = torch.randperm(c["T"] - 1, generator=cpu)[: c["S"] - 1].sort()[0] + 1 if c["T"] > 1 else torch.empty(0, dtype=torch.int64)
    ends = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([c["T"]])]).to(torch.int32)
    logits = _normal(gen, (c["T"], c["E"])) + _normal(gen, (c["E"],), 0.5)
    idx = torch.topk(logits, c["k"], -1)[1]
    more = torch.arange(c["E"], c["E"] + c["shared"], device="cuda").expand(c["T"], -1)
    s = dict(case=c, logits=logits, idx=torch.cat([idx, more], -1).to(torch.int32), ends=ends.cuda(),
             mask=(torch.rand(c["T"], generator=gen, device="cuda") >= c["masked"]).to(torch.uint8) if c["masked"] else None,
             dw=_normal(gen, (c["T"], c["k"] + c["shared"])) / c["T"] if c["weights"] else None,
             d_loss=torch.full((1,), 0.01, device="cuda"))
    if own:
        from routed_expert_ffn_top_amd import binding as B
        shape = B.make_shape(c["T"], 64, 64, c["E"], c["k"], c["shared"], renorm=c["renorm"])
        new = lambda *n, dt=torch.float32: torch.empty(n, dtype=dt, device="cuda")
        s.update(shape=shape, ws=B.alloc_balance_workspace(shape, c["S"]), loss=new(1), prob=new(c["S"], c["E"]),
                 counts=new(c["S"], c["E"], dt=torch.int32), slope=new(c["S"], c["E"]), dlogits=new(c["T"], c["E"]))
    return s


# ---- one pass ----

def run(s):
    return {"quant": _quant, "matmul": _matmul, "experts": _experts, "combine": _combine,
            "balance": _balance}[s["case"]["kind"]](s)


def _quant(s):
    c = s["case"]
    if own:
        from routed_expert_ffn_top_amd import binding as B
        B.moe_quantize_fp8(s["x"], s["codes"], s["scales"], block_rows=c["block"])
        B.moe_dequantize_fp8(s["codes"], s["scales"], s["out"], block_rows=c["block"])
        return {"values": s["out"]}
    v, byte = _quantise(s["x"].float(), c["block"])
    return {"values": (v * _spread(_unit(byte), c["block"], c["rows"], c["K"])).to(torch.bfloat16)}


def _values(x):
    """What quantised rows stand for."""
    v, byte = _quantise(x, 1)
    return v * _spread(_unit(byte), 1, *x.shape[-2:])


def _decoded(w, ws):
    return w.view(torch.float8_e4m3fn).float() * _spread(ws, 128, *w.shape[-2:])


def _grouped(a, off, most, M, w, ws):
    """a [M][K] times the slice of its group, [M][N] in fp32."""
    r = torch.arange(M, device=a.device)
    g = torch.searchsorted(off, r, right=True) - 1
    if M <= w.shape[0]:   # a slice a row
        return torch.bmm(_decoded(w[g], ws[g]), a[:, :, None])[:, :, 0]
    # the groups' rows side by side, each padded to the largest group's length
    at = (off[:-1, None] + torch.arange(most, device=a.device)).clamp(max=M - 1)
    return torch.bmm(a[at], _decoded(w, ws).transpose(1, 2).contiguous())[g, r - off[g]]


def _matmul(s):
    c = s["case"]
    if own:
        from routed_expert_ffn_top_amd import binding as B
        B.moe_quantize_fp8(s["x"], s["a"], s["as"])
        B.moe_matmul_fp8(s["a"], s["as"], s["w"], s["ws"], s["out"], slot_offset=s["offset"], row_index=s["take"])
        return {"out": s["out"]}
    a = _values(s["x"].float())
    if s["take"] is not None:
        a = a[s["take"].long()]
    o = _grouped(a, s["offset"].long(), s["most"], c["M"], s["w"], s["ws"])
    return {"out": o.to(torch.float32 if c["out"] == "f32" else torch.bfloat16)}


def _experts(s):
    c = s["case"]
    M = c["T"] * c["k"]
    if own:
        from routed_expert_ffn_top_amd import binding as B
        B.moe_quantize_fp8(s["x"], s["a"], s["as"])
        B.moe_gate_up_fp8(s["a"], s["as"], s["wg"], s["wgs"], s["wu"], s["wus"], s["h"], s["hs"], slot_offset=s["offset"],
                          row_index=s["take"])
        B.moe_matmul_fp8(s["h"], s["hs"], s["wd"], s["wds"], s["out"], slot_offset=s["offset"])
        return {"out": s["out"]}
    a, off = _values(s["x"].float())[s["take"].long()], s["offset"].long()
    g, u = (_grouped(a, off, s["most"], M, s[n], s[n + "s"]) for n in ("wg", "wu"))
    h = _values(g / (1 + torch.exp(-g)) * u)
    return {"out": _grouped(h, off, s["most"], M, s["wd"], s["wds"]).to(torch.bfloat16)}


def _combine(s):
    c = s["case"]
    if own:
        from routed_expert_ffn_top_amd import binding as B
        B.moe_combine(s["C"], s["pos"], s["w"], s["y"])
        B.moe_combine_backward(s["C"], s["pos"], s["w"], s["dy"], s["dC"], s["dw"])
        return {"y": s["y"], "dC": s["dC"], "dw": s["dw"]}
    pos = s["pos"].long().reshape(c["T"], c["k"])
    here = pos >= 0
    rows = s["C"][pos.clamp(min=0)].float() * here[..., None]
    s["y"] += (rows * s["w"][..., None]).sum(1)
    # the records of the routes that are left out are nobody's: one row more takes what they would write
    n, g = c["T"] * c["k"], (s["w"][..., None] * s["dy"][:, None, :]).reshape(-1, c["d"]).to(s["dC"].dtype)
    dC = torch.cat([s["dC"], s["dC"][:1]]).index_copy(0, torch.where(here, pos, n).reshape(-1), g)[:n]
    return {"y": s["y"], "dC": dC, "dw": (rows * s["dy"][:, None, :]).sum(-1)}


def _balance(s):
    c = s["case"]
    if own:
        from routed_expert_ffn_top_amd import binding as B
        B.moe_balance_loss(s["shape"], s["logits"], s["idx"], s["loss"], s["counts"], s["prob"], s["slope"], s["ws"],
                           seq_offset=s["ends"], mask=s["mask"])
        B.moe_router_backward(s["shape"], s["logits"], s["idx"], s["dlogits"], slope=s["slope"], d_loss=s["d_loss"],
                              d_topk_w=s["dw"], seq_offset=s["ends"], mask=s["mask"])
        return {"loss": s["loss"], "counts": s["counts"], "prob": s["prob"], "dlogits": s["dlogits"]}
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    idx = s["idx"][:, :k].long()
    z = torch.exp(s["logits"] - s["logits"].amax(-1, keepdim=True))
    p = z / z.sum(-1, keepdim=True)
    seq = torch.searchsorted(s["ends"].long(), torch.arange(T, device=p.device), right=True) - 1
    live = torch.ones(T, device=p.device, dtype=torch.float64) if s["mask"] is None else s["mask"].double()
    of = (seq == torch.arange(S, device=p.device)[:, None]).double() * live   # which tokens a sequence counts
    n, chosen = of.sum(-1), torch.zeros((T, E), device=p.device, dtype=torch.float64).scatter(1, idx, 1.0)
    counts, prob = of @ chosen, of @ p.double()
    some = n.clamp(min=1)[:, None]
    prob, full = prob / some, (n > 0).double().sum()
    loss = (E / k * counts * prob / some).sum() / full.clamp(min=1)
    # a softmax's backward drops what all experts have alike
    slope = E / k * (counts - counts.mean(-1, keepdim=True)) / some ** 2 / full.clamp(min=1)
    u = (slope * s["d_loss"])[seq].float() * live.float()[:, None]
    if s["dw"] is None:
        return {"loss": loss.float()[None], "counts": counts.int(), "prob": prob.float(),
                "dlogits": p * (u - (u * p).sum(-1, keepdim=True))}
    dw = s["dw"][:, :k]
    if c["renorm"]:
        sel = z.gather(1, idx)
        sel = sel / sel.sum(-1, keepdim=True)
        extra = torch.zeros_like(p).scatter(1, idx, sel * (dw - (sel * dw).sum(-1, keepdim=True)))
    else:
        u, extra = u.scatter_add(1, idx, dw), 0.0
    return {"loss": loss.float()[None], "counts": counts.int(), "prob": prob.float(),
            "dlogits": p * (u - (u * p).sum(-1, keepdim=True)) + extra}


# ---- what a pass cannot do without ----

def work(case):
    c = case
    if c["kind"] == "quant":
        n = c["rows"] * c["K"]   # the source, the codes written and read, the values read back
        nb = n // 128 if c["block"] == 1 else n // 4096
        return {"bytes": n * (4 if c["src"] == "f32" else 2) + 2 * n + 2 * nb + 2 * n, "flops": 0}
    if c["kind"] == "matmul":
        rows = max(1, c["M"] // 8) if c["gather"] else c["M"]
        w = min(c["P"], c["M"]) * c["N"] * c["K"]   # groups that can have rows
        return {"bytes": rows * c["K"] * 2 + w + w // 4096 + c["M"] * c["N"] * (4 if c["out"] == "f32" else 2),
                "flops": 2 * c["M"] * c["N"] * c["K"]}
    if c["kind"] == "experts":
        M = c["T"] * c["k"]
        w = min(c["P"], M) * 3 * c["d"] * c["f"]
        return {"bytes": c["T"] * c["d"] * 2 + w + w // 4096 + M * c["d"] * 2 + 4 * M, "flops": 6 * M * c["d"] * c["f"]}
    if c["kind"] == "combine":
        n, b = c["T"] * c["k"] * (1 - c["absent"]), 4 if c["rows"] == "f32" else 2
        return {"bytes": int(n * c["d"] * 2 * b + c["T"] * c["d"] * 12 + c["T"] * c["k"] * 12),
                "flops": int(5 * n * c["d"])}
    per = c["E"] * 8 + (c["k"] + c["shared"]) * (8 if c["weights"] else 4) + (1 if c["masked"] else 0)
    return {"bytes": c["T"] * per + c["S"] * c["E"] * 12, "flops": 20 * c["T"] * c["E"]}


# ---- the definition, in 64 bits ----

def _two(e):
    """2^e in 64 bits for whole numbers e."""
    return (e.to(torch.int64) + 1023 << 52).view(torch.float64)


def _blocks64(x, rows):
    """Values that fp8 blocks of rows x 128 of x [R][C] stand for, from the definition, in 64 bits."""
    x = x.double()
    R, C = x.shape
    top = torch.zeros((-(-R // rows), -(-C // 128)), dtype=torch.float64, device=x.device)
    for j in range(top.shape[1]):
        m = x[:, 128 * j: 128 * j + 128].abs().amax(-1)
        m = torch.nn.functional.pad(m, (0, -R % rows)).reshape(-1, rows)
        top[:, j] = m.amax(-1)
    e = torch.ceil(torch.log2(top / 448.0))
    e = torch.where(top > 0, e, -126.0).clamp(-126, 120)
    e = torch.where(448.0 * _two(e - 1) >= top, e - 1, torch.where(448.0 * _two(e) < top, e + 1, e))
    unit = _two(e.clamp(-126, 120))
    out = torch.empty_like(x)
    for j in range(top.shape[1]):
        cols = slice(128 * j, 128 * j + 128)
        u = unit[:, j].repeat_interleave(rows)[:R, None]
        v = x[:, cols] / u
        # e4m3's distance of neighbours: 2^-3 of the power of two below, not under 2^-9; round() ties to even
        step = _two(torch.frexp(v)[1] - 4).clamp(min=2.0 ** -9)
        out[:, cols] = torch.round(v / step) * step * u
    return out


def _decoded64(w, ws):
    """A slice [N][K] in 64 bits, from the codes' bit fields."""
    n = w.int()
    exp, man = (n >> 3) & 15, (n & 7).double()
    mag = torch.where(exp == 0, man * 2.0 ** -9, (1 + man / 8) * _two(exp - 7))
    v = torch.where(n >= 128, -mag, mag)
    for i in range(ws.shape[0]):
        for j in range(ws.shape[1]):
            v[128 * i: 128 * i + 128, 128 * j: 128 * j + 128] *= ws[i, j].double()
    return v


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["kind"] == "quant":
        return {"values": _blocks64(s["x"], c["block"])}
    if c["kind"] == "combine":
        return _exact_combine(c, s)
    if c["kind"] == "balance":
        return _exact_balance(c, s)
    a, off = _blocks64(s["x"], 1), s["offset"].tolist()
    M = c["M"] if c["kind"] == "matmul" else c["T"] * c["k"]
    out = torch.empty((M, c["N"] if c["kind"] == "matmul" else c["d"]), dtype=torch.float64, device="cuda")
    for g in range(c["P"]):
        r = slice(off[g], off[g + 1])
        if off[g] == off[g + 1]:
            continue
        rows = a[r] if s["take"] is None else a[s["take"][r].long()]
        if c["kind"] == "matmul":
            out[r] = rows @ _decoded64(s["w"][g], s["ws"][g]).t()
            continue
        gate, up = (rows @ _decoded64(s[n][g], s[n + "s"][g]).t() for n in ("wg", "wu"))
        out[r] = _blocks64(gate * torch.sigmoid(gate) * up, 1) @ _decoded64(s["wd"][g], s["wds"][g]).t()
    return {"out": out}


def _exact_combine(c, s):
    y, dy = s["y"].double(), s["dy"].double()
    dC, dw = s["dC"].double(), torch.zeros((c["T"], c["k"]), dtype=torch.float64, device="cuda")
    pos = s["pos"].long().reshape(c["T"], c["k"])
    for j in range(c["k"]):
        t = torch.nonzero(pos[:, j] >= 0)[:, 0]
        rows, w = s["C"][pos[t, j]].double(), s["w"][t, j].double()[:, None]
        y[t] += w * rows
        dC[pos[t, j]] = w * dy[t]
        dw[t, j] = (rows * dy[t]).sum(-1)
    return {"y": y, "dC": dC, "dw": dw}


def _exact_balance(c, s):
    E, k = c["E"], c["k"]
    p = torch.softmax(s["logits"].double(), -1)
    ends, idx = s["ends"].tolist(), s["idx"][:, :k].long()
    live = torch.ones(c["T"], dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"] != 0
    counts = torch.zeros((c["S"], E), dtype=torch.int64, device="cuda")
    prob, u = torch.zeros((c["S"], E), dtype=torch.float64, device="cuda"), torch.zeros_like(p)
    loss, full = 0.0, 0
    for q in range(c["S"]):
        r = slice(ends[q], ends[q + 1])
        n = int(live[r].sum())
        if n == 0:
            continue
        full += 1
        counts[q] = torch.bincount(idx[r][live[r]].reshape(-1), minlength=E)
        prob[q] = p[r][live[r]].mean(0)
        loss = loss + E / (k * n) * (counts[q] * prob[q]).sum()
        u[r] = live[r, None] * (E / (k * n * n) * counts[q].double())
    u = u * s["d_loss"].double() / max(full, 1)
    extra = torch.zeros_like(p)
    if s["dw"] is not None:
        dw = s["dw"][:, :k].double()
        if c["renorm"]:
            w = torch.softmax(s["logits"].double().gather(1, idx), -1)
            extra = extra.scatter(1, idx, w * (dw - (w * dw).sum(-1, keepdim=True)))
        else:
            u = u.scatter_add(1, idx, dw)
    loss = torch.as_tensor(loss, dtype=torch.float64, device="cuda").reshape(1) / max(full, 1)
    return {"loss": loss, "counts": counts, "prob": prob, "dlogits": p * (u - (p * u).sum(-1, keepdim=True)) + extra}
