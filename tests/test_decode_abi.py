"""moe_layer_decode's checks of its arguments, on the CPU: every call below
ends in its checks, before any GPU work."""
import pytest
import torch

from routed_expert_ffn_top_amd import binding as B
from test_abi import _FakeWs, _fake_routes


def _shape(**kw):
    base = dict(T=4, d=128, f=64, E=8, k=2, dtype="bf16")
    base.update(kw)
    return B.make_shape(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(T=65), B.MOE_ERR_UNSUPPORTED),
    (dict(T=64, E=64, k=17), B.MOE_ERR_UNSUPPORTED),       # 1088 routes
    (dict(T=64, E=64, k=15, n_shared=2), B.MOE_ERR_UNSUPPORTED),
    (dict(T=-1), B.MOE_ERR_INVALID_ARG),
    (dict(d=96), B.MOE_ERR_UNSUPPORTED),
    (dict(d=131136), B.MOE_ERR_UNSUPPORTED),
    (dict(d=65536, f=8192), B.MOE_ERR_UNSUPPORTED),        # a gate/up slice of 2 GiB
])
def test_decode_shapes_refused(kw, status):
    assert B.moe_decode_workspace_bytes(_shape(**kw)) == 0
    assert B.moe_last_error()[0] == status


def test_decode_workspace_sizes():
    a, b = (B.moe_decode_workspace_bytes(_shape(T=t)) for t in (1, 64))
    assert 0 < a < b and a % 256 == 0
    # H as three bf16 terms and one fp32 row of d per route
    assert b >= 64 * 2 * (64 * 6 + 128 * 4) + 64 * 8 * 4
    assert B.moe_decode_workspace_bytes(_shape(T=64, E=64, k=16)) > 0      # 1024 routes
    assert B.moe_decode_workspace_bytes(_shape(T=0)) > 0


class _Arena:
    def __init__(self, handle):
        self.handle = handle


@pytest.fixture
def arena():
    s = _shape()
    # planes are never touched: the calls below fail first
    h = B.moe_arena_create(s, 0x100000, 0x200000, 2 * s.f * s.d, s.f * s.d, s.P)
    yield _Arena(h)
    B.moe_arena_destroy(h)


def _call(arena, s=None, X=0x1000, Wr=0x2000, logits=None, Y=0x3000, routes=None, ws=None):
    s = s or _shape()
    ws = ws or _FakeWs(B.moe_decode_workspace_bytes(s))
    r = _fake_routes(s) if routes is None else routes
    with pytest.raises(B.MoEError) as e:
        B.moe_layer_decode(s, X, Wr, None, logits, Y, arena, r, ws, 0)
    return e.value


def test_decode_refusals(arena):
    inv, un, wk = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE
    n = B.moe_decode_workspace_bytes(_shape())
    assert _call(arena, X=None).status == inv
    assert _call(arena, Y=None).status == inv
    assert _call(_Arena(None)).status == inv
    assert _call(arena, Wr=None, logits=None).status == inv
    assert _call(arena, X=0x1008).status == inv
    assert _call(arena, Y=0x3004).status == inv
    assert _call(arena, Wr=0x2004).status == inv
    assert _call(arena, routes=dict(topk_idx=0x1000)).status == inv
    assert _call(arena, ws=_FakeWs(n - 1)).status == wk
    assert _call(arena, ws=_FakeWs(n, 0x7f0000000080)).status == wk
    assert _call(arena, s=_shape(T=65), ws=_FakeWs(1 << 30)).status == un
    for other in (dict(d=192), dict(f=128), dict(E=9, P=8), dict(n_shared=1, P=8), dict(P=9), dict(dtype="f32")):
        assert _call(arena, s=_shape(**other)).status == inv, other
    f32 = _shape(dtype="f32", ldx=130)
    assert _call(arena, s=f32).status == un


def test_decode_needs_contiguous_rows():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        B.check_rows(x, torch.float32, 8, "X")          # not on the GPU
    assert B.row_stride(torch.zeros(4, 24)[:, :8]) == 24
    assert B.row_stride(torch.zeros(1, 8)) == 8


class _On:
    """A tensor of some device and address, as far as the binding looks."""

    def __init__(self, device, addr=0x1000, n=1 << 30):
        self.device, self.addr, self.n = device, addr, n

    def get_device(self):
        return self.device

    def data_ptr(self):
        return self.addr

    def numel(self):
        return self.n

    def element_size(self):
        return 1


def test_decode_operands_on_one_device(monkeypatch):
    """Every operand, not X alone: a kernel of one GPU would follow the pointer
    into another's memory, or the host's."""
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, a)) or B.MOE_OK

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(B, "_raw_stream", lambda device: 100 + device)
    monkeypatch.setattr(B, "load", lambda: Lib())
    s = _shape()
    arena = _Arena(0x5000)
    arena.plane_gu = arena.plane_d = _On(1)
    base = dict(X=_On(1), W_r=_On(1), bias=_On(1), logits=_On(1), Y=_On(1), ws=_On(1), idx=_On(1), w=_On(1), arena=arena)

    def call(**kw):
        a = dict(base, **kw)
        B.moe_layer_decode(s, a["X"], a["W_r"], a["bias"], a["logits"], a["Y"], a["arena"],
                           dict(topk_idx=a["idx"], topk_w=a["w"]), a["ws"])
    call()
    call(bias=None, logits=None)
    assert [c[0] for c in calls] == ["moe_layer_decode"] * 2 and calls[0][1][-1] == 101
    other = _Arena(0x5000)
    other.plane_gu = other.plane_d = _On(0)
    for dev in (0, -1):
        for name in ("X", "W_r", "bias", "logits", "Y", "ws", "idx", "w"):
            with pytest.raises(ValueError):
                call(**{name: _On(dev)})
        with pytest.raises(ValueError):
            B.moe_decode_workspace_init(s, _On(dev))
    with pytest.raises(ValueError):
        call(arena=other)
    B.moe_decode_workspace_init(s, _On(1))
    with pytest.raises(ValueError):       # all of them on a GPU that is not the current one
        call(**{k: _On(0) for k in base if k != "arena"}, arena=other)
    assert len(calls) == 3


def test_layer_operands_on_the_layers_device(monkeypatch):
    """forward_mxfp4 looks before its first launch, which is the router's."""
    from routed_expert_ffn_top_amd.inputs import MoEConfig
    from routed_expert_ffn_top_amd.layer import MoELayer
    layer = MoELayer.__new__(MoELayer)
    layer.cfg = MoEConfig(name="on_device", index=85, T=4, d=128, f=64, E=8, k=2, dtype="bf16_fp4w")
    layer.shape, layer.paged, layer.X = _shape(dtype="bf16_fp4w"), False, _On(1)
    launched = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(B, "_raw_stream", lambda device: 100 + device)
    monkeypatch.setattr(B, "check_rows", lambda *a: None)
    for f in ("moe_router_logits", "moe_quantize_mxfp4"):
        monkeypatch.setattr(B, f, lambda *a: launched.append(a))
    layer._xq, layer._logits = torch.zeros(1), None
    with pytest.raises(ValueError):
        layer.forward_mxfp4(torch.zeros(4, 128))       # in host memory
    layer.X = _On(0)
    with pytest.raises(ValueError):
        layer.forward_mxfp4(torch.zeros(4, 128))
    assert not launched
