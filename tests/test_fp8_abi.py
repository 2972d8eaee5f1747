"""The checks of their arguments of the fp8 operators, the combine, the balance
loss and the router's gradient, on the CPU: every call below ends in its
checks, before any GPU work."""
import ctypes

import pytest
import torch

from routed_expert_ffn_top_amd import binding as B

INV, UN, WS = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE
L = B.load()


def test_scale_bytes():
    assert [B.fp8_scale_bytes(K) for K in (64, 128, 2048, 2112, 4096, 14336)] == [16, 16, 16, 32, 32, 112]


@pytest.mark.parametrize("call", [L.moe_quantize_fp8, L.moe_dequantize_fp8], ids=["quantize", "dequantize"])
def test_values_and_blocks(call):
    def status(v=0x1000, dt=B.MOE_DT_BF16, rows=4, K=64, ld=64, br=1, codes=0x2000, scales=0x3000):
        if call is L.moe_quantize_fp8:
            return call(v, dt, rows, K, ld, br, codes, scales, None)
        return call(codes, scales, rows, K, br, v, dt, ld, None)
    assert status(rows=0, v=None, codes=None, scales=None) == B.MOE_OK     # nothing to do
    for kw in (dict(dt=B.MOE_DT_BF16_FP8W), dict(rows=-1), dict(K=0), dict(K=-64), dict(ld=63), dict(br=0), dict(br=64), dict(v=None),
               dict(codes=None), dict(scales=None), dict(v=0x1008), dict(codes=0x2008), dict(ld=68), dict(dt=B.MOE_DT_F32, ld=66),
               dict(br=128, scales=0x3002)):
        assert status(**kw) == INV, kw
    for kw in (dict(K=96, ld=96), dict(rows=1 << 28), dict(rows=1 << 60)):
        assert status(**kw) == UN, kw


PRODUCT = dict(M=4, N=64, K=64, A=0x1000, As=0x2000, rows=4, ri=None, off=None, P=1, W=0x4000, Ws=0x5000, stride=0, sstride=0,
               C=0x8000, dt=B.MOE_DT_F32, ldc=64)
BAD = (dict(M=-1), dict(N=0), dict(K=0), dict(rows=-1), dict(P=0), dict(P=513, off=0x10, stride=4096, sstride=1), dict(P=2, stride=4096),
       dict(rows=3), dict(rows=0, ri=0x10), dict(A=None), dict(As=None), dict(W=None), dict(Ws=None), dict(C=None), dict(A=0x1008),
       dict(As=0x2008), dict(W=0x4008), dict(Ws=0x5002), dict(C=0x8008), dict(P=2, off=0x10, stride=4095, sstride=1),
       dict(P=2, off=0x10, stride=4104, sstride=1), dict(P=2, off=0x10, stride=4096, sstride=0))
UNSUPPORTED = (dict(N=96, ldc=96), dict(K=96), dict(K=(1 << 20) + 64), dict(M=1 << 30, rows=1 << 30, N=1 << 15, ldc=1 << 15),
               dict(rows=(1 << 30) + 1))


def test_matmul_refusals():
    def status(**kw):
        a = dict(PRODUCT, **kw)
        return L.moe_matmul_fp8(a["M"], a["N"], a["K"], a["A"], a["As"], a["rows"], a["ri"], a["off"], a["P"], a["W"], a["Ws"],
                                a["stride"], a["sstride"], a["C"], a["dt"], a["ldc"], None)
    assert status(M=0, A=None, As=None, W=None, Ws=None, C=None, rows=0) == B.MOE_OK
    for kw in BAD + (dict(dt=B.MOE_DT_BF16_FP8W), dict(ldc=63), dict(ldc=66), dict(dt=B.MOE_DT_BF16, ldc=68)):
        assert status(**kw) == INV, kw
    for kw in UNSUPPORTED + (dict(ldc=1 << 21),):
        assert status(**kw) == UN, kw


@pytest.mark.parametrize("which", ["Wg", "Wu"])
def test_gate_up_refusals(which):
    def status(Hs=0x9000, ws=0xa0000, n=1 << 40, **kw):
        a = dict(PRODUCT, **kw)
        good = (PRODUCT["W"], PRODUCT["Ws"])
        g, u = ((a["W"], a["Ws"]), good) if which == "Wg" else (good, (a["W"], a["Ws"]))
        return L.moe_gate_up_fp8(a["M"], a["N"], a["K"], a["A"], a["As"], a["rows"], a["ri"], a["off"], a["P"], *g, *u, a["stride"],
                                 a["sstride"], a["C"], Hs, ws, n, None)
    assert status(M=0, A=None, As=None, W=None, Ws=None, C=None, rows=0) == B.MOE_OK
    for kw in BAD + (dict(Hs=None),):
        assert status(**kw) == INV, kw
    for kw in UNSUPPORTED:
        assert status(**kw) == UN, kw
    need = B.moe_gate_up_fp8_workspace_bytes(4, 64, 64, 1)
    assert need == 4 * 4 * 64 and B.moe_gate_up_fp8_workspace_bytes(0, 64, 64, 1) == 0
    assert B.moe_gate_up_fp8_workspace_bytes(32768, 1024, 2048, 64) == 0      # many records a slot
    for kw in (dict(ws=None), dict(ws=0xa0010), dict(n=need - 1)):
        assert status(**kw) == WS, kw


def test_combine_refusals():
    base = dict(T=2, d=8, kp=2, M=4, C=0x1000, dt=B.MOE_DT_BF16, ldc=8, pos=0x2000, w=0x3000, Y=0x4000, ldy=8)

    def status(back=False, dC=0x5000, lddc=8, dw=0x6000, **kw):
        a = dict(base, **kw)
        args = [a[k] for k in ("T", "d", "kp", "M", "C", "dt", "ldc", "pos", "w", "Y", "ldy")]
        return L.moe_combine_backward(*args, dC, lddc, dw, None) if back else L.moe_combine(*args, None)
    for back in (False, True):
        assert status(back, T=0, C=None, pos=None, w=None, Y=None, dC=None, dw=None) == B.MOE_OK
        for kw in (dict(T=-1), dict(d=0), dict(M=-1), dict(kp=0), dict(kp=65), dict(dt=B.MOE_DT_BF16_FP8W), dict(ldc=4), dict(ldy=4),
                   dict(ldc=10), dict(ldy=10), dict(C=None), dict(pos=None), dict(w=None), dict(Y=None), dict(C=0x1004), dict(Y=0x4008),
                   dict(dt=B.MOE_DT_F32, C=0x1008)):
            assert status(back, **kw) == INV, kw
        for kw in (dict(d=6), dict(d=(1 << 20) + 4, ldc=1 << 21, ldy=1 << 21), dict(T=1 << 24), dict(T=1 << 23, d=1028, ldc=1028, ldy=1028)):
            assert status(back, **kw) == UN, kw
    for kw in (dict(dw=None), dict(lddc=4), dict(lddc=10), dict(dC=0x5004), dict(dt=B.MOE_DT_F32, dC=0x5008)):
        assert status(True, **kw) == INV, kw


def test_balance_refusals():
    s = B.make_shape(100, 64, 64, 8, 2, 1)
    n = B.moe_balance_workspace_bytes(s, 3)
    assert n > B.moe_balance_workspace_bytes(s, 1) > 0
    assert B.moe_balance_workspace_bytes(s, 0) == 0 and B.moe_balance_workspace_bytes(s, 4097) == 0
    assert B.moe_balance_workspace_bytes(B.make_shape(100, 64, 64, 0, 1), 1) == 0
    base = dict(shape=s, L=0x1000, idx=0x2000, off=0x3000, S=3, mask=None, loss=0x4000, counts=0x5000, prob=0x6000, slope=0x7000,
                ws=0x10000, n=n)

    def status(**kw):
        a = dict(base, **kw)
        return L.moe_balance_loss(ctypes.byref(a["shape"]), a["L"], a["idx"], a["off"], a["S"], a["mask"], a["loss"], a["counts"],
                                  a["prob"], a["slope"], a["ws"], a["n"], None)
    for kw in (dict(S=0), dict(S=4097), dict(off=None), dict(L=None), dict(idx=None), dict(loss=None), dict(counts=None),
               dict(prob=None), dict(slope=None), dict(shape=B.make_shape(100, 64, 64, 300, 2))):
        assert status(**kw) == INV, kw
    for kw in (dict(ws=None), dict(ws=0x10010), dict(n=n - 1)):
        assert status(**kw) == WS, kw

    def back(shape=s, L_=0x1000, idx=0x2000, slope=0x3000, off=0x4000, S=3, dw=0x5000, out=0x6000):
        return L.moe_router_backward(ctypes.byref(shape), L_, idx, slope, None, off, S, None, dw, out, None)
    for kw in (dict(S=0), dict(off=None), dict(L_=None), dict(idx=None), dict(out=None), dict(slope=None, dw=None),
               dict(shape=B.make_shape(100, 64, 64, 4, 5))):
        assert back(**kw) == INV, kw
    none = B.make_shape(0, 64, 64, 8, 2)
    assert back(shape=none, L_=None, idx=None, out=None) == B.MOE_OK


def test_router_backward_refuses_more_tokens_than_a_launch_has_waves():
    shape = B.make_shape(1 << 26, 64, 64, 1, 1)
    assert L.moe_router_backward(ctypes.byref(shape), 0x1000, 0x2000, 0x3000, None, None, 1, None, None, 0x4000, None) == UN


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def test_binding_refuses_other_blocks():
    x = torch.zeros(4, 64)
    ok = dict(values=x, codes=u8(4, 64), scales=u8(4, 16))
    for kw in (dict(values=x.half()), dict(codes=u8(4, 63)), dict(codes=u8(64, 4).t()), dict(scales=u8(4, 1)), dict(scales=u8(4, 32)[:, :16]),
               dict(values=torch.zeros(64, 4).t()), dict(values=torch.zeros(2, 2, 128)[..., :64]), dict(block_rows=128),
               dict(block_rows=128, scales=torch.zeros(2, 1)), dict(scales=torch.zeros(4, 16))):
        for call in (B.moe_quantize_fp8, B.moe_dequantize_fp8):
            with pytest.raises(ValueError):
                call(**dict(ok, **kw))


def test_binding_refuses_other_products():
    f = torch.zeros
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    ok = dict(A_codes=u8(4, 64), A_scales=u8(4, 16), B_codes=u8(2, 64, 64), B_scales=f(2, 1, 1), C=f(4, 64), slot_offset=i32(3))
    for kw in (dict(A_scales=u8(4, 1)), dict(A_codes=f(4, 64)), dict(B_codes=u8(2, 64, 128)), dict(B_codes=u8(2, 64, 128)[..., :64]),
               dict(B_scales=f(1, 1, 1)), dict(B_scales=f(2, 1, 2)), dict(B_scales=f(2, 1)), dict(B_scales=f(2, 1, 1).double()),
               dict(B_codes=u8(2, 64, 64).float()), dict(C=f(4, 128)), dict(C=f(64, 4).t()), dict(C=f(4, 64).half()),
               dict(slot_offset=i32(2)), dict(row_index=i32(3)), dict(row_index=i32(4).long()), dict(B_codes=u8(64), B_scales=f(1))):
        with pytest.raises(ValueError):
            B.moe_matmul_fp8(**dict(ok, **kw))
    w = dict(Wg_codes=u8(2, 64, 64), Wg_scales=f(2, 1, 1), Wu_codes=u8(2, 64, 64), Wu_scales=f(2, 1, 1))
    ok = dict(A_codes=u8(4, 64), A_scales=u8(4, 16), H_codes=u8(4, 64), H_scales=u8(4, 16), slot_offset=i32(3), **w)
    for kw in (dict(H_codes=u8(4, 128), H_scales=u8(4, 16)), dict(H_scales=u8(4, 1)), dict(Wu_codes=u8(2, 128, 64)),
               dict(Wu_codes=u8(2, 128, 64)[:, :64]), dict(Wu_codes=u8(64, 64), Wu_scales=f(1, 1)), dict(slot_offset=i32(2))):
        with pytest.raises(ValueError):
            B.moe_gate_up_fp8(**dict(ok, **kw))


def test_binding_refuses_other_rows_and_routings():
    f, i32 = torch.zeros, lambda *n: torch.zeros(n, dtype=torch.int32)
    ok = dict(C=f(4, 8), route_pos=i32(4), topk_w=f(2, 2))
    for kw in (dict(C=f(4, 12)), dict(C=f(4, 8).half()), dict(C=f(8, 4).t()), dict(C=f(8).expand(4, 8)), dict(route_pos=i32(3)),
               dict(route_pos=i32(4).long()), dict(topk_w=f(3, 2)), dict(topk_w=f(2, 2).double()), dict(topk_w=f(2, 4)[:, ::2])):
        with pytest.raises(ValueError):
            B.moe_combine(Y=f(2, 8), **dict(ok, **kw))
        with pytest.raises(ValueError):
            B.moe_combine_backward(dY=f(2, 8), dC=None, d_topk_w=f(2, 2), **dict(ok, **kw))
    for kw in (dict(dC=f(3, 8)), dict(dC=f(4, 8).bfloat16()), dict(dC=f(8, 4).t()), dict(d_topk_w=f(4)), dict(d_topk_w=f(2, 4)[:, ::2])):
        with pytest.raises(ValueError):
            B.moe_combine_backward(dY=f(2, 8), **dict(ok, dC=None, d_topk_w=f(2, 2)) | kw)
    s = B.make_shape(6, 64, 64, 8, 2)
    ok = dict(logits=f(6, 8), topk_idx=i32(6, 2), loss=f(1), counts=i32(2, 8), prob=f(2, 8), slope=f(2, 8), ws=u8(4096), seq_offset=i32(3))
    for kw in (dict(logits=f(6, 9)), dict(logits=f(8, 6).t()), dict(topk_idx=i32(6, 3)), dict(topk_idx=i32(6, 2).long()), dict(loss=f(2)),
               dict(counts=i32(1, 8)), dict(prob=f(8, 2)), dict(slope=f(2, 8).double()), dict(seq_offset=i32(3).long()),
               dict(mask=f(6)), dict(mask=u8(5))):
        with pytest.raises(ValueError):
            B.moe_balance_loss(s, **dict(ok, **kw))
    ok = dict(logits=f(6, 8), topk_idx=i32(6, 2), d_logits=f(6, 8), slope=f(1, 8))
    for kw in (dict(d_logits=f(6, 9)), dict(slope=f(2, 8)), dict(d_loss=f(2)), dict(d_topk_w=f(6, 3)), dict(topk_idx=i32(6, 1))):
        with pytest.raises(ValueError):
            B.moe_router_backward(s, **dict(ok, **kw))
    # host tensors
    with pytest.raises(ValueError):
        B.moe_router_backward(s, **ok)


def test_products_refuse_more_records_than_tiles_are_counted_of():
    """A slot's records are rounded up to whole tiles of 256 in 32 bits."""
    for M in (2 ** 31 - 1, 2 ** 31 - 255):
        p = (M, 64, 64, 0x1000, 0x2000, 1, 0x10, None, 1)
        assert L.moe_matmul_fp8(*p, 0x4000, 0x5000, 0, 0, 0x8000, B.MOE_DT_BF16, 64, None) == UN
        assert L.moe_gate_up_fp8(*p, 0x4000, 0x5000, 0x6000, 0x7000, 0, 0, 0x8000, 0x9000, 0xa0000, 1 << 40, None) == UN
        assert B.moe_gate_up_fp8_workspace_bytes(M, 64, 64) == 0


def test_quantise_refuses_more_blocks_than_a_launch_has_threads():
    """256 threads a block of 128 x 128, fewer than 2^32 a launch."""
    K = 2 ** 31 - 64
    for rows in (1, 4):
        assert L.moe_quantize_fp8(0x1000, B.MOE_DT_BF16, rows, K, K, 128, 0x2000, 0x3000, None) == UN
