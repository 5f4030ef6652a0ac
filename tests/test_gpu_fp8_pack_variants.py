"""The pack's row kernels that take several blocks per warp, which only many rows reach: every alignment of the rows,
K tails inside a warp's blocks, infinities and NaN in one of them, and rows by index.

Codes and scales are compared bit for bit with a vectorised form of the definition, itself checked against the oracle."""
import numpy as np
import pytest
import torch

import oracle.lowp as ref
import xnor_popcount_gemm_bnn_b200 as bnn
from gpu_util import assert_no_device_error, dev

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
BLOCK = 128


def packed_rows(x):
    """The definition for blocks of 1 x 128, on whole arrays: (codes with NaN as 0x7F, scales)."""
    x = x.float()
    rows, K = x.shape
    kb = -(-K // BLOCK)
    full = torch.zeros(rows, kb * BLOCK, device=x.device)
    full[:, :K] = x
    t = full.view(rows, kb, BLOCK)
    fin = t.isfinite()
    amax = torch.where(fin, t.abs(), torch.zeros_like(t)).amax(dim=2, keepdim=True)
    s = (amax.double() / 448.0).float().clamp_min(2.0 ** -126)
    least = amax.double() < 448.0 * 2.0 ** -126
    q = t.double() * torch.where(least, 2.0 ** 126, 448.0) / torch.where(least, torch.ones_like(amax.double()), amax.double())
    c = torch.where(fin, q, torch.zeros_like(q)).float().to(torch.float8_e4m3fn).view(torch.uint8)
    c = torch.where(fin, c, torch.full_like(c, 0x7F))
    return c.view(rows, kb * BLOCK)[:, :K], s[:, :, 0].t().contiguous()


def rows_with_specials(rows, K, dtype, seed):
    """Uneven rows; an infinity, a NaN, a block of NaN, a block of zeros and a tiny block, each in one block of a row."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    x = torch.randn(rows, K, generator=g, device=dev()) * torch.exp(torch.randn(rows, 1, generator=g, device=dev()))
    x = x.to(DT[dtype])
    c = min(K - 1, 5 * BLOCK + 17)
    x[3, c], x[10, K - 1], x[17, 0] = float("inf"), float("-inf"), float("nan")
    x[24, K // BLOCK * BLOCK - BLOCK:K // BLOCK * BLOCK] = float("nan")
    x[31, BLOCK:2 * BLOCK] = -0.0
    x[38, :BLOCK] = 1e-39
    x[rows - 1, c] = float("inf")
    return x


def same_codes(got, want):
    return torch.equal(torch.where((got & 0x7F) == 0x7F, torch.full_like(got, 0x7F), got), want)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_definition_on_whole_arrays_matches_the_oracle(dtype):
    x = rows_with_specials(40, 700, dtype, 1)
    c, s = packed_rows(x)
    wc, ws = ref.fp8_pack(x.float().cpu().numpy(), 1)
    assert np.array_equal(c.cpu().numpy(), wc) and np.array_equal(s.cpu().numpy(), ws)


# The row's alignment in bytes follows from the stride and the offset, in elements: 32, 16, 8, 4 and 2.
@pytest.mark.parametrize("dtype,ld,offset,K", [
    ("bf16", 4112, 0, 4090), ("bf16", 4104, 0, 4096), ("bf16", 4100, 0, 2049), ("bf16", 4098, 2, 1000),
    ("bf16", 1001, 1, 1000), ("bf16", 2051, 0, 2049), ("bf16", 1040, 0, 1024),
    ("fp32", 4096, 0, 4090), ("fp32", 2052, 0, 2049), ("fp32", 1002, 0, 1000), ("fp32", 4091, 3, 4090)])
@pytest.mark.parametrize("gather", [False, True])
def test_rows_of_many_blocks_per_warp(dtype, ld, offset, K, gather):
    rows = 2500
    x_rows = 700 if gather else rows
    flat = torch.full((x_rows * ld + offset,), float("nan"), dtype=DT[dtype], device=dev())
    x = flat.as_strided((x_rows, K), (ld, 1), offset)
    x.copy_(rows_with_specials(x_rows, K, dtype, ld + K))
    width = bnn.bnn_fp8_ld_bytes(K)
    codes = torch.full((rows, width + 16), 0x5A, dtype=torch.uint8, device=dev())
    scales = torch.full((-(-K // BLOCK), rows + 2), -7.0, device=dev())
    index, keep = None, torch.ones(rows, dtype=torch.bool, device=dev())
    if gather:
        g = torch.Generator(device=dev()).manual_seed(K)
        index = torch.randint(0, x_rows, (rows,), generator=g, device=dev(), dtype=torch.int32)
        index[::97], index[5], index[2499] = -1, x_rows, 2 ** 31 - 1
        keep = (index >= 0) & (index < x_rows)
    bnn.bnn_fp8_pack(x, codes, scales, row_index=index, K=K)
    wc, ws = packed_rows(x if index is None else x[index.clamp(0, x_rows - 1).long()])
    assert same_codes(codes[keep][:, :K], wc[keep])
    assert (codes[keep][:, K:width] == 0).all() and (codes[:, width:] == 0x5A).all()
    assert torch.equal(scales[:, :rows][:, keep], ws[:, keep]) and (scales[:, rows:] == -7.0).all()
    assert (codes[~keep] == 0x5A).all() and (scales[:, :rows][:, ~keep] == -7.0).all()
    assert_no_device_error()


def near_middles():
    """(x, amax), 24-bit integers, whose quotient x * 448 / amax is the middle of two fp32 numbers or very near it, and
    next to the middle of two codes: T * 2^b - or + half a unit, T odd with five bits."""
    found = []
    for T in range(17, 32, 2):
        for b in range(3, 7):
            step = 2 ** (20 - b)
            for m in range(2 ** 23 // step, 2 ** 24 // step):
                for j in (-2, -1, 0, 1, 2):
                    for sign in (-1, 1):
                        amax = m * step + j
                        n = T * amax * 2 ** b + sign * m
                        if n % 448 == 0 and 2 ** 23 <= amax < 2 ** 24 and 2 ** 23 <= n // 448 < 2 ** 24:
                            found.append((n // 448, amax))
    return found


@pytest.mark.parametrize("shift", [0, -60, 80])
@pytest.mark.parametrize("block_rows", [1, BLOCK])
def test_fp32_quotients_next_to_a_middle(block_rows, shift):
    """fp32 quotients that 2^-21 of a unit may send to either neighbour: the code is one of those next to the real
    quotient, and no farther from it than the nearest by more than the quotient's own rounding, 2^-24 (1 + 2^-20) of it
    on both sides of the middle."""
    from fractions import Fraction as F
    pairs = [p for p in near_middles() if p[0] <= p[1]] + [(10335963, 12582912), (10335963 // 2 * 2, 12582912)]
    assert len(pairs) > 10
    rows = len(pairs) * block_rows                            # a pair in a block of its own
    x = torch.zeros(rows, 40)
    for i, (v, amax) in enumerate(pairs):
        x[i * block_rows, :3] = torch.tensor([float(amax), float(v), -float(v)]) * 2.0 ** shift
    codes, scales = bnn.empty_fp8(rows, 40, dev()), bnn.empty_fp8_scales(rows, 40, block_rows, dev())
    bnn.bnn_fp8_pack(x.to(dev()), codes, scales, block_rows=block_rows)
    got = codes.double().cpu()[::block_rows, :3].tolist()
    positive = [F(v) for v in ref.VALUES[:127].tolist()]
    for (v, amax), (top, up, down) in zip(pairs, got):
        q = F(v * 448, amax)
        best = min(abs(q - c) for c in positive)
        assert top == 448.0 and down == -up
        assert abs(q - F(up)) <= best + 2 * q * F(1 + 2 ** -20) / 2 ** 24, (v, amax, up)
