"""Loading an arena on a stream of its own: the temporaries of the load (blocks
quantised on the way, codes joined with their scales) must hold what was put into
them until the packing has read them, whatever the current stream does meanwhile."""
import pytest
import torch

from gpu_util import gpu_inputs, say
from routed_expert_ffn_top_amd import binding as B
from routed_expert_ffn_top_amd.inputs import MoEConfig
from routed_expert_ffn_top_amd.layer import MoELayer

pytestmark = pytest.mark.gpu

PAUSE = 20_000_000   # cycles that a stream is kept busy for: some ms


def cfg_of(dtype):
    return MoEConfig(name=f"load_{dtype}", index=84, T=2, d=320, f=192, E=6, k=2, dtype=dtype)


def sources(kind):
    """dtype of the arena, and (Wg, Wu, Wd, scales) to load."""
    if kind in ("fp32", "bf16"):
        gen = torch.Generator(device="cuda").manual_seed(6)
        ws = [torch.empty(s, device="cuda").normal_(0, 0.02, generator=gen) for s in
              ((6, 192, 320), (6, 192, 320), (6, 320, 192))]
        return "bf16_fp4w", [w.to(torch.float32 if kind == "fp32" else torch.bfloat16) for w in ws], None
    inp = gpu_inputs(cfg_of(kind))
    return kind, [inp.Wg, inp.Wu, inp.Wd], [inp.Sg, inp.Su, inp.Sd]


def fresh_arena(dtype):
    c = cfg_of(dtype)
    a = B.Arena(B.make_shape(c.T, c.d, c.f, c.E, c.k, dtype=dtype))
    a.plane_gu.view(torch.uint8).fill_(0xEE)
    a.plane_d.view(torch.uint8).fill_(0xEE)
    return a


@pytest.mark.parametrize("handle", ["stream", "int", "default"])
@pytest.mark.parametrize("kind", ["fp32", "bf16", "bf16_fp4w", "bf16_fp8w"])
def test_load_on_another_stream(kind, handle):
    say(f"load of {kind} on a side stream ({handle}) while the current one allocates and writes")
    dtype, ws, scales = sources(kind)
    phi = [3, 0, 5, 1, 4, 2]
    want, got = fresh_arena(dtype), fresh_arena(dtype)
    want.load_resident(*ws, phi=phi, scales=scales)
    torch.cuda.synchronize()

    cur, st = torch.cuda.Stream(), torch.cuda.default_stream() if handle == "default" else torch.cuda.Stream()
    give = {"stream": st, "int": st.cuda_stream, "default": 0}[handle]
    with torch.cuda.stream(cur):
        sizes = [320 * 192 * 17 // 32, 320 * 192 + 4 * 192, 320 * 192 + 4 * 320]
        junk = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in sizes * 4]
        del junk                                  # blocks of the temporaries' sizes, in use by what is queued here
        torch.cuda._sleep(PAUSE)
        src = [w.clone() for w in ws]             # made behind the pause
        sc = None if scales is None else [s.clone() for s in scales]
    with torch.cuda.stream(st):
        torch.cuda._sleep(PAUSE)
    with torch.cuda.stream(cur):
        got.load_resident(*src, phi=phi, stream=give, scales=sc)
        # what the load has dropped may come back here: written at once
        junk = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in sizes * 24]
    torch.cuda.synchronize()
    assert torch.equal(got.plane_gu, want.plane_gu) and torch.equal(got.plane_d, want.plane_d)
    del junk


def test_slice_on_another_stream():
    say("a slice quantised on a side stream, packed there, dropped at once")
    _, (Wg, _, Wd), _ = sources("fp32")
    c = cfg_of("bf16_fp4w")
    shape = B.make_shape(c.T, c.d, c.f, c.E, c.k, dtype=c.dtype)
    want = torch.empty(B.fp4_slice_bytes(c.d, c.f), dtype=torch.uint8, device="cuda")
    B.moe_pack_down(shape, B.mxfp4_slice(Wd[0]), want, 1, 0, 0)
    got = torch.zeros_like(want)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        torch.cuda._sleep(PAUSE)
    W = Wd[0] * 1.0
    B.moe_pack_down(shape, B.mxfp4_slice(W, st), got, 1, 0, 0, st)
    junk = [torch.full((c.d * c.f * 17 // 32,), 0x55, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    del junk


@pytest.mark.parametrize("dtype", ["bf16", "bf16_fp8w", "bf16_fp4w"])
def test_paged_layer_set_up_on_another_stream(dtype):
    """The host planes of a paged layer hold each expert's slices as they are
    after its packing, also where that is queued on a busy stream."""
    say(f"paged layer set up on a busy side stream, {dtype}")
    inp = gpu_inputs(cfg_of(dtype).with_(P=4, G=2))
    want = MoELayer(inp, paged=True)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        torch.cuda._sleep(PAUSE)
    got = MoELayer(inp, paged=True, stream=st)
    for a, b in ((want.host_gu_plane, got.host_gu_plane), (want.host_d_plane, got.host_d_plane)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
