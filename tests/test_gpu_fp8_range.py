"""Products on fp8 blocks of 128 at the ends of the scales' range: large rows against small weights and the other
way round, weight scales up to the largest fp32 number, scales of 0, every scale byte of a row. Each for few
records a slot, many with bf16 C and many with fp32 C, which are multiplied in three ways.

u = 2^-24. |C - exact| <= gamma(2K + 4 ceil(K/128)) sum |a b| as at ordinary scales, 2^-10 of it more where the fp8
matrix instructions cut (bf16 C), half a step of bf16; K 2^-149 where products leave the normal numbers, 2^-134
for bf16 C that does. fp32 C of many records takes rows as bf16: a value below 2^-126 is off by at most 2^-133, its product by that
times the weight."""
import pytest
import torch

from routed_expert_ffn_top_amd import binding as B
from test_gpu_fp8 import bound, quantise, rows64, weights, weights64

pytestmark = pytest.mark.gpu

N = 1600   # with 4000 records the persistent kernel, with 5 the other one


def check(C, av, wv, K):
    want = av @ wv.t()
    lim = bound(av, wv, K, C.dtype is torch.bfloat16) + K * 2.0 ** -149 + 2.0 ** -133 * wv.abs().sum(1)
    if C.dtype is torch.bfloat16:
        lim = lim + 2.0 ** -8 * (want.abs() + lim) + 2.0 ** -134
    err = (C.cpu().double() - want).abs()
    assert bool((err <= lim).all()), f"{float((err / lim).nan_to_num(float('inf')).max()):.3g} of the bound"


def product(a, as_, w, ws, out):
    C = torch.full((a.shape[0], N), 3.0, device="cuda", dtype=out)
    B.moe_matmul_fp8(a, as_, w, ws, C)
    torch.cuda.synchronize()
    return C


ENDS = [((-60, 0), (1.9 * 2.0 ** 125, 2.0 ** 60)), ((118, 0), (1.3 * 2.0 ** -60, 2.0 ** 56)), ((118, 0), (0.0, 1.0)),
        ((118, 118), (0.0, 2.0 ** -70)), ((-118, 0), (1.7 * 2.0 ** 100, 2.0 ** -18)), ((-118, -118), (2.0 ** 118, 1.5 * 2.0 ** 110)),
        ((0, 0), (1.5 * 2.0 ** -126, 2.0 ** -120)), ((110, 110), (2.0 ** -126, 1.1 * 2.0 ** -110)),
        ((-60, -60), (-1.5 * 2.0 ** 127, 2.0 ** 127)), ((-60, 10), (1.99 * 2.0 ** 119, 2.0 ** -100)), ((0, -70), (1.0, 2.0 ** 127))]


@pytest.mark.parametrize("M,out", [(5, torch.float32), (5, torch.bfloat16), (4000, torch.bfloat16), (4000, torch.float32)])
@pytest.mark.parametrize("rows,scales", ENDS)
def test_scales_at_either_end(M, out, rows, scales):
    """Row values near 2^rows[b] and the weight scale scales[b] in block b of k."""
    g = torch.Generator().manual_seed(3)
    K = 256
    x = torch.randn(M, K, generator=g)
    for b in range(2):
        x[:, 128 * b:128 * b + 128] *= 2.0 ** rows[b]
    a, as_ = quantise(x.cuda())
    w, _ = weights(g, 1, N, K, "any")
    ws = torch.tensor(scales, dtype=torch.float64).float().repeat(-(-N // 128), 1).cuda()
    C = product(a, as_, w[0], ws, out)
    check(C, rows64(a, as_), weights64(w[0], ws), K)


@pytest.mark.parametrize("M,out,bytes_", [(16, torch.float32, (0, 254)), (16, torch.bfloat16, (0, 254)), (4000, torch.bfloat16, (0, 254)),
                                          (4000, torch.float32, (1, 247))])
def test_every_row_byte(M, out, bytes_):
    """Rows of each scale byte, against weights that bring the result back among the numbers."""
    g = torch.Generator().manual_seed(5)
    K, lo, hi = 192, *bytes_
    w, ws = weights(g, 1, N, K, "any")
    for part in (range(lo, 128), range(128, hi + 1)):
        s = ws[0] * 2.0 ** (60 if part[0] < 128 else -60)
        for first in range(0, len(part), M):
            b = torch.tensor([part[min(first + i, len(part) - 1)] for i in range(M)])
            a, _ = weights(g, 1, M, K, "any")
            as_ = torch.full((M, B.fp8_scale_bytes(K)), 0xEE, dtype=torch.uint8)
            as_[:, 0], as_[:, 1] = b, b.flip(0)
            C = product(a[0], as_.cuda(), w[0], s, out)
            check(C, rows64(a[0], as_), weights64(w[0], s), K)
