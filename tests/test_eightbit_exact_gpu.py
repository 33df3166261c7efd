"""Sums of the 8-bit product that are whole numbers, so that every bit is known.

Codes are -2 to 2 and scales 1 or 2, drawn for each row and group: a term is a
whole number of at most 16 in magnitude, and 147,456 of them stay below 2^22.
Every partial sum, in any order and wherever a sum is cut, is then exact in
fp32 (and in the plain product on the CPU), and a term that is lost, counted
twice or multiplied by another group's scale shows."""
import pytest
import torch

from protein_folding_attention_gb300 import evoattn

pytestmark = pytest.mark.gpu
DEV = "cuda"


def whole(R, K, seed, blocks=False):
    """An operand on the device (NaN codes beside its rows), and its values."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-2, 3, (R, K), generator=g).float()
    rows, groups = -(-R // 128) if blocks else R, -(-K // 128)
    k = torch.randint(0, 2, (rows, groups), generator=g)
    scale = torch.exp2(k.float()).repeat_interleave(128, 1)[:, :K]
    values = q * (scale.repeat_interleave(128, 0)[:R] if blocks else scale)
    full = torch.full((R, -(-K // 16) * 16), 0x7F, dtype=torch.uint8, device=DEV)
    full[:, :K] = q.to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)
    scales = (k + 127).to(torch.uint8).to(DEV).view(torch.float8_e8m0fnu)
    return full.view(torch.float8_e4m3fn)[:, :K], scales, values


def check(M, N, K, blocks, dtype=torch.float32):
    a, sa, va = whole(M, K, 1)
    b, sb, vb = whole(N, K, 2, blocks)
    want = va @ vb.t()
    assert want.abs().max() < 2 ** 22
    for _ in range(3):
        got = evoattn.matmul8(a, sa, b, sb, dtype)
        assert evoattn.device_status() == evoattn.OK
        assert torch.equal(got.cpu(), want.to(dtype))


@pytest.mark.parametrize("M, N, K", [
    (1, 700, 2048), (3, 20000, 4100), (30, 10000, 2500), (60, 10000, 2500),      # b on the lanes, sums whole
    (1, 4096, 8000), (5, 40, 20001), (17, 300, 9000), (40, 129, 20000), (64, 64, 20000), (100, 130, 20001),  # in pieces
    (300, 516, 128), (700, 257, 1024), (20000, 128, 3300), (2000, 1000, 260)])   # a on the lanes
@pytest.mark.parametrize("blocks", [False, True])
def test_scales_of_many_groups(M, N, K, blocks):
    """Scales that change from group to group, many groups to a sum and many sums
    to a CTA: the columns of tensor memory that hold them are used again and again."""
    check(M, N, K, blocks)


@pytest.mark.parametrize("M, N, K", [
    (1300, 4096, 4096), (5000, 400, 3001), (4097, 1500, 1100), (2500, 1999, 1290),           # 192 columns at a time
    (2000, 2000, 9000), (1000, 4000, 4000), (20000, 240, 1281), (4096, 4096, 1200),          # 240
    (3840, 192, 1153)])                                                                      # 128 are as good
@pytest.mark.parametrize("blocks", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_wide_tiles(M, N, K, blocks, dtype):
    check(M, N, K, blocks, dtype)


LONG = [(64, 64, 20000), (3, 200, 20001), (100, 130, 20001), (512, 128, 147456),   # in pieces
        (40, 10000, 3001), (2000, 128, 3001), (2000, 2000, 3001)]                  # b, a on the lanes; wide tiles


@pytest.mark.parametrize("M, N, K", LONG)
def test_no_term_of_a_long_sum_is_lost(M, N, K):
    check(M, N, K, False)


@pytest.mark.parametrize("M, N, K", LONG)
def test_single_terms_of_a_long_sum(M, N, K):
    """One term alone: the first and the last, both sides of the last border
    between groups, and of every third of the others."""
    a, sa, va = whole(M, K, 3)
    b, sb, vb = whole(N, K, 4)
    last = (K - 1) // 128 * 128
    borders = sorted({0, K - 1, last - 1, last, *range(128, last, 384), *range(127, last, 384)})
    for k in borders[:20] + borders[20::40] + borders[-3:]:
        one = torch.zeros((M, -(-K // 16) * 16), dtype=torch.uint8, device=DEV)
        one[:, k] = a.view(torch.uint8)[:, k]
        got = evoattn.matmul8(one.view(torch.float8_e4m3fn)[:, :K], sa, b, sb, torch.float32)
        assert torch.equal(got.cpu(), va[:, k:k + 1] * vb[:, k]), k
    assert evoattn.device_status() == evoattn.OK
