"""The MXFP4 operators' checks of their arguments, on the CPU: every call
below ends in its checks, before any GPU work."""
import contextlib

import pytest
import torch

from routed_expert_ffn_top_amd import binding as B
from test_abi import _FakeWs, _fake_routes

INV, UN = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED
L = B.load()


@pytest.mark.parametrize("call", [L.moe_quantize_mxfp4, L.moe_dequantize_mxfp4], ids=["quantize", "dequantize"])
def test_values_and_blocks(call):
    def status(v=0x1000, dt=B.MOE_DT_BF16, rows=4, K=64, ld=64, codes=0x2000, scales=0x3000):
        if call is L.moe_quantize_mxfp4:
            return call(v, dt, rows, K, ld, codes, scales, None)
        return call(codes, scales, rows, K, v, dt, ld, None)
    assert status(rows=0, v=None, codes=None, scales=None) == B.MOE_OK     # nothing to do
    assert status(dt=B.MOE_DT_BF16_FP4W) == INV
    assert status(rows=-1) == INV
    assert status(K=0) == INV and status(K=-32) == INV
    assert status(ld=63) == INV
    assert status(K=48) == UN
    assert status(rows=1 << 30, K=32, ld=32) == UN                         # 2^35 values
    for k in ("v", "codes", "scales"):
        assert status(**{k: None}) == INV
    assert status(v=0x1008) == INV and status(codes=0x2008) == INV
    assert status(ld=68) == INV                                            # rows 136 bytes apart
    assert status(dt=B.MOE_DT_F32, ld=66) == INV


def test_matmul_refusals():
    base = dict(M=4, N=64, K=64, A=0x1000, As=0x2000, rows=4, ri=None, off=None, P=1, W=0x4000, stride=0, C=0x8000,
                dt=B.MOE_DT_F32, ldc=64)

    def status(**kw):
        a = dict(base, **kw)
        return L.moe_matmul_mxfp4(a["M"], a["N"], a["K"], a["A"], a["As"], a["rows"], a["ri"], a["off"], a["P"], a["W"],
                                  a["stride"], a["C"], a["dt"], a["ldc"], None)
    assert status(M=0, A=None, As=None, W=None, C=None, rows=0) == B.MOE_OK
    for kw in (dict(M=-1), dict(N=0), dict(K=0), dict(rows=-1), dict(P=0), dict(P=513, off=0x10), dict(dt=B.MOE_DT_BF16_FP4W),
               dict(ldc=63), dict(P=2, stride=4096), dict(rows=3), dict(rows=0, ri=0x10), dict(A=None), dict(As=None),
               dict(W=None), dict(C=None), dict(A=0x1008), dict(As=0x2001), dict(W=0x4008), dict(C=0x8004),
               dict(ldc=66), dict(dt=B.MOE_DT_BF16, ldc=68), dict(P=2, off=0x10, stride=2175), dict(P=2, off=0x10, stride=2184)):
        assert status(**kw) == INV, kw
    for kw in (dict(N=96), dict(K=96), dict(M=1 << 30, rows=1 << 30), dict(ldc=1 << 21)):
        assert status(**kw) == UN, kw


def test_binding_refuses_other_layouts():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        B.moe_quantize_mxfp4(x.half(), u8(4, 32), u8(4, 2))
    with pytest.raises(ValueError):
        B.moe_quantize_mxfp4(x, u8(4, 31), u8(4, 2))
    with pytest.raises(ValueError):
        B.moe_quantize_mxfp4(x, u8(4, 32), u8(4, 4)[:, :2])
    with pytest.raises(ValueError):
        B.moe_quantize_mxfp4(torch.zeros(64, 4).t(), u8(4, 32), u8(4, 2))
    with pytest.raises(ValueError):
        B.moe_quantize_mxfp4(torch.zeros(2, 2, 128)[..., :64], u8(4, 32), u8(4, 2))
    ok = dict(A_codes=u8(4, 32), A_scales=u8(4, 2), B=u8(B.fp4_slice_bytes(64, 64)), C=torch.zeros(4, 64))
    for kw in (dict(A_scales=u8(4, 3)), dict(B=u8(B.fp4_slice_bytes(64, 64) - 1)), dict(C=torch.zeros(64, 4).t()),
               dict(C=torch.zeros(4, 64).half()), dict(row_index=torch.zeros(4, dtype=torch.int64)),
               dict(row_index=torch.zeros(3, dtype=torch.int32)), dict(slot_offset=torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            B.moe_matmul_mxfp4(**dict(ok, **kw))


@pytest.mark.parametrize("dtype,flags", [("bf16", 0), ("f32", 0), ("bf16_fp8w", 0), ("bf16_fp4w", B.MOE_FFN_SIMPLE_KERNEL),
                                         ("bf16_fp4w", B.MOE_FFN_FUSED)])
def test_mxfp4_activations_refused(dtype, flags):
    """Before the arena's state is looked at (nothing is loaded here)."""
    s = B.make_shape(4, 128, 64, 8, 2, dtype=dtype)
    h = B.moe_arena_create(s, 0x100000, 0x200000, 4 * s.f * s.d, 2 * s.f * s.d, s.P)
    arena = type("Arena", (), {"handle": h})()
    with pytest.raises(B.MoEError) as e:
        B.moe_expert_ffn(s, 0x1000, 0x3000, _fake_routes(s), arena, list(range(8)),
                         B.MOE_FFN_EXPERTS | B.MOE_FFN_ACT_MXFP4 | flags, _FakeWs(B.moe_workspace_bytes(s)), 0)
    assert e.value.status == UN
    B.moe_arena_destroy(h)


class _On:
    """A tensor or stream of some device, as far as the check looks."""

    def __init__(self, device):
        self.device_index = device

    def get_device(self):
        return self.device_index


def test_other_devices_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(B, "_raw_stream", lambda device: 100 + device)
    assert B._stream_of(_On(1), None) == 101
    assert B._stream_of(0x1000, 7) == 7
    with pytest.raises(ValueError):
        B._stream_of(_On(0), None)
    with pytest.raises(ValueError):
        B._stream_of(torch.zeros(4), None)      # host memory
    with pytest.raises(ValueError):
        B._stream_of(_On(1), _On(0))


def test_weights_of_another_shape_refused():
    """Weights that are quantised on their way into an arena: a smaller slice would be
    read past its end by the packing."""
    arena = B.Arena.__new__(B.Arena)
    arena.shape, arena.handle = B.make_shape(4, 128, 64, 2, 1, dtype="bf16_fp4w"), None
    ok = dict(Wg=(2, 64, 128), Wu=(2, 64, 128), Wd=(2, 128, 64))
    for kw in (dict(Wg=(2, 64, 64)), dict(Wu=(2, 32, 128)), dict(Wd=(2, 64, 128)), dict(Wd=(2, 128, 32)),
               dict(Wg=(64, 128))):
        w = {k: torch.zeros(v) for k, v in dict(ok, **kw).items()}
        with pytest.raises(ValueError, match="load_resident: need"):
            arena.load_resident(w["Wg"], w["Wu"], w["Wd"], phi=[0, 1])


def test_handles_of_streams_without_an_address(monkeypatch):
    """0 and 1 name the default stream; the per-thread one (2) torch cannot name, and
    as an address it would be another stream."""
    class Stream:
        device = "cuda:0"

        def __init__(self, handle=0):
            self.handle = handle

        def wait_stream(self, other):
            used.append(self.handle)

    used = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(5))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    for handle in (0, 1, 0x7f0000000100):
        with B.on_stream(handle):
            pass
    assert used == [0, 0, 0x7f0000000100]
    with pytest.raises(ValueError):
        with B.on_stream(2):
            pass
