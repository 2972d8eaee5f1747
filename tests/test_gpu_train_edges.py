"""The balance loss and the router's gradient at the edges of what they take: offsets past the tokens, workspaces that
hold an earlier call's sums."""
import pytest
import torch

from routed_expert_ffn_top_amd import binding as B
from test_gpu_train import choice

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
