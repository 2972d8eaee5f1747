"""The balance loss and the router's gradient at the edges of what they take: offsets past the tokens, workspaces that
hold an earlier call's sums."""
import pytest
import torch

from routed_expert_ffn_top_amd import binding as B
from test_gpu_train import check_balance, choice

pytestmark = pytest.mark.gpu


def balance(shape, L, idx, off, ws):
    S, E = len(off) - 1, shape.E
    new = lambda *n, dt=torch.float32: torch.full(n, 99, dtype=dt, device="cuda")
    o = [new(1), new(S, E, dt=torch.int32), new(S, E), new(S, E)]
    B.moe_balance_loss(shape, L, idx, *o, ws, seq_offset=torch.tensor(off, dtype=torch.int32).cuda())
    return o


@pytest.mark.parametrize("T", [100, 112, 20000])
def test_offsets_past_the_tokens(T):
    """They count as the number of tokens, whatever the workspace held: the bits of a call with that number in their place."""
    E, k, S = 12, 2, 6
    g = torch.Generator().manual_seed(T)
    L = torch.randn(T, E, generator=g)
    idx, L, shape = choice(L, k, 0, E).cuda(), L.cuda(), B.make_shape(T, 64, 64, E, k)
    ws, clean = B.alloc_balance_workspace(shape, S), B.alloc_balance_workspace(shape, S)
    full = [T * i // S for i in range(S + 1)]
    for far in ([0, T // 2, T + 20, T + 30, T + 40, 2 * T, 3 * T], [0, T // 3, T // 2, T - 1, T, T + 1, T + 2], [T + 1] * 7):
        balance(shape, L, idx, full, ws)   # every entry filled
        clean.fill_(0xEE)
        got, want = balance(shape, L, idx, far, ws), balance(shape, L, idx, [min(o, T) for o in far], clean)
        assert all(torch.equal(x, y) for x, y in zip(got, want)), far


def test_slope_with_ids_out_of_range():
    """slope = E / (k n^2 S+) (c - k n / E) whether or not every route counts, one rounding to fp32 off; and its
    gradient is that of the loss, from which a constant over the experts drops out."""
    T, E, k = 60, 10, 3
    g = torch.Generator().manual_seed(2)
    L, idx = torch.randn(T, E, generator=g), torch.randint(-4, E + 4, (T, k), generator=g).int()
    shape = B.make_shape(T, 64, 64, E, k)
    loss, counts, prob, slope = balance(shape, L.cuda(), idx.cuda(), [0, T], B.alloc_balance_workspace(shape, 1))
    c = torch.bincount(idx[(idx >= 0) & (idx < E)].long(), minlength=E).double()
    assert torch.equal(counts.cpu()[0].double(), c) and float(c.sum()) < k * T
    want = E / (k * T * T) * (c - k * T / E)
    assert bool(((slope.cpu()[0].double() - want).abs() <= 1.01 * 2.0 ** -24 * want.abs()).all())
    assert abs(float((slope.cpu()[0].double() + 1 / T).mean()) - E / (k * T * T) * float(c.mean())) <= 2.0 ** -23 / T
    # the gradient of the loss as it is defined: p (u - sum u p) with u = E / (k n^2) c
    out = torch.empty((T, E), device="cuda")
    B.moe_router_backward(shape, L.cuda(), idx.cuda(), out, slope=slope)
    p, u = torch.softmax(L.double(), -1), E / (k * T * T) * c
    R = float(L.max() - L.min())
    shifted = (slope.cpu()[0].double().abs()).expand(T, E)
    lim = (2 * (R + 18) + 16) * 2.0 ** -24 * p * (shifted + (shifted * p).sum(-1, keepdim=True))
    grad = p * (u - (u * p).sum(-1, keepdim=True))
    # 2^-50: this formula's own differences, of numbers below 1, in 64 bits
    assert bool(((out.cpu().double() - grad).abs() <= lim + 2.0 ** -24 * grad.abs() + 2.0 ** -50).all())


@pytest.mark.parametrize("T", [16385, 40001, 131073, 262145, 300001])
def test_chunks_of_every_length(T):
    """Chunks of 64 tokens and, past 65536, of more in steps of 4 up to 256."""
    off = torch.tensor([0, 7, T // 3, T // 3 + 1, T])
    check_balance(T, 5, 2, 0, 4, off, (torch.rand(T, generator=torch.Generator().manual_seed(T)) < 0.7).to(torch.uint8), True, True)
