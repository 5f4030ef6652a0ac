"""The variants of the 8-bit products that only larger calls reach: every ring depth and split of K, groups with more
rows than the few-rows kernel takes at a time, and CTA pairs with several tiles.

The shapes are those that the launchers' rules send to each variant on 148 SMs.  Every element is compared, within the
bound of test_gpu_fp8.py, with float64 products of the codes' values on the GPU, and two runs bit for bit."""
import numpy as np
import pytest
import torch

import oracle.lowp as ref
import xnor_popcount_gemm_bnn_b200 as bnn
from gpu_util import assert_no_device_error, dev

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
BLOCK = 128


def codes_of(shape, K, seed):
    """Codes over the whole range but NaN, garbage in the padding past K."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    c = torch.randint(0, 256, (*shape, bnn.bnn_fp8_ld_bytes(K)), generator=g, dtype=torch.uint8, device=dev())
    c[..., :K][(c[..., :K] & 0x7F) == 0x7F] = 0
    return c


def scales_of(shape, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    return torch.exp(torch.randn(shape, generator=g, device=dev())) * 0.01


def values(codes, scales, K, block_rows):
    """float64 values of codes [rows, ld] with block-major scales [blocks of K, row blocks]."""
    table = torch.from_numpy(ref.VALUES).to(dev())
    rows = codes.shape[0]
    i, b = torch.arange(rows, device=dev()) // block_rows, torch.arange(K, device=dev()) // BLOCK
    return table[codes[:, :K].long()] * scales.double()[b[None, :], i[:, None]]


def check(out, a, w, K):
    """|C - C64| <= (128 * 2^-23 + (2 * blocks + 2) * 2^-24) * sum |a w| and half a step of the output type."""
    c64, mag = a @ w.t(), a.abs() @ w.abs().t()
    half = torch.finfo(out.dtype).eps / 2
    blocks = -(-K // BLOCK)
    tol = (128 * 2.0 ** -23 + (2 * blocks + 2) * 2.0 ** -24) * mag * (1 + half) + half * c64.abs()
    bad = ~((out.double() - c64).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3].tolist())


# rows per MMA and split of K of the few-rows kernel; the shallow ring first (with 3 and 2 parts)
FEW = [(1, 11008, 4096), (16, 12800, 4096), (9, 300, 896), (5, 300, 640), (10, 300, 900), (20, 12800, 4096),
       (30, 260, 900), (60, 12600, 4000), (40, 300, 760), (70, 200, 900), (100, 6200, 4000), (128, 4600, 4000),
       (128, 9400, 4096)]
# CTA pairs: 256 columns with more than 74 tiles, an odd number of K blocks and a second band of row tiles; 128 columns
MANY = [(2300, 4000, 610), (2560, 4096, 256), (2500, 2000, 290)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("M,N,K", FEW + MANY)
def test_dense(M, N, K, dtype):
    A, W = codes_of((M,), K, M + K), codes_of((N,), K, N + K + 1)
    kb = -(-K // BLOCK)
    sa, sw = scales_of((kb, M), 5), scales_of((kb, -(-N // BLOCK)), 6)
    out, again = (torch.full((M, N), float("nan"), dtype=DT[dtype], device=dev()) for _ in range(2))
    bnn.bnn_fp8_gemm(A, sa, W, sw, K, out)
    bnn.bnn_fp8_gemm(A, sa, W, sw, K, again)
    check(out, values(A, sa, K, 1), values(W, sw, K, BLOCK), K)
    assert torch.equal(out, again)
    assert_no_device_error()


def uneven(E, R, most, seed):
    """Row counts of E groups, R in all: one of `most` rows, every third group empty, the others uneven."""
    g = np.random.default_rng(seed)
    p = g.random(E) * (np.arange(E) % 3 != 1)
    p[E // 2] = 0
    c = np.floor(p / p.sum() * (R - most)).astype(np.int64)
    c[E // 2] = most
    c[0 if E // 2 else -1] += R - c.sum()
    return c


GROUPED = [  # R, rows of the largest group, N, K, E
    (200, 70, 260, 300, 40),        # 16 rows at a time, K not split, up to 5 turns of a group
    (200, 200, 260, 300, 40),       # all rows one group's
    (200, 70, 260, 2000, 40),       # the shallow ring, 2 parts: the ring is reused after the parts' sums
    (120, 50, 260, 2000, 20),       # 4 parts
    (240, 90, 260, 300, 20),        # 32 rows at a time
    (260, 101, 130, 1300, 20),      # 6 parts
    (900, 300, 300, 700, 20),       # 64 rows at a time
    (1300, 333, 140, 900, 30),      # 4 parts
    (2100, 600, 520, 300, 40),      # pairs of 128 columns, more groups than the tile walk looks at together
    (2000, 700, 2048, 200, 16),     # pairs of 256 columns
    (9000, 2500, 1000, 610, 36),    # pairs with several tiles, an odd number of K blocks, two bands in a group
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("R,most,N,K,E", GROUPED)
def test_grouped(R, most, N, K, E, dtype):
    first, tail = 3, 5
    counts = uneven(E, R - first - tail, most, E + R) if most < R else np.eye(E, dtype=np.int64)[E // 2] * (R - first - tail)
    off = np.concatenate([[0], np.cumsum(counts)]) + first
    assert off[-1] == R - tail and (counts >= 0).all() and (counts == 0).any()
    A, W = codes_of((R,), K, 1), codes_of((E, N), K, 2)
    kb = -(-K // BLOCK)
    sa, sw = scales_of((kb, R), 3), scales_of((E, kb, -(-N // BLOCK)), 4)
    offsets = torch.tensor(off, dtype=torch.int32, device=dev())
    out, again = (torch.full((R, N), 99.0, dtype=DT[dtype], device=dev()) for _ in range(2))
    bnn.bnn_fp8_gemm_grouped(A, sa, offsets, W, sw, K, out)
    bnn.bnn_fp8_gemm_grouped(A, sa, offsets, W, sw, K, again)
    for e in np.nonzero(counts)[0]:
        r = slice(int(off[e]), int(off[e + 1]))
        check(out[r], values(A[r], sa[:, r], K, 1), values(W[e], sw[e], K, BLOCK), K)
    assert (out[:first] == 99.0).all() and (out[R - tail:] == 99.0).all()
    assert torch.equal(out, again)
    assert_no_device_error()


def test_no_experts():
    """A product with an empty set of experts leaves its outputs as they were."""
    A, sa, out = codes_of((4,), 64, 1), scales_of((1, 4), 2), torch.full((4, 8), 99.0, device=dev())
    bnn.bnn_fp8_gemm_grouped(A, sa, torch.zeros(1, dtype=torch.int32, device=dev()), A.new_empty(0, 8, 64),
                             sa.new_empty(0, 1, 1), 64, out)
    assert (out == 99.0).all()
    assert_no_device_error()


@pytest.mark.parametrize("M", [5, 70, 150])
@pytest.mark.parametrize("low", [-126, -140, -148])
def test_small_scale_products(M, low):
    """Products of scales down to 2^low.  From 2^-126 on the usual bound holds; below it a product is rounded to a
    multiple of 2^-149, off by 2^-150 at most, times the block's sum; and each block's addition to a sum that may be
    subnormal is off by 2^-150."""
    N, K = 140, 500
    kb = -(-K // BLOCK)
    A, W = codes_of((M,), K, 1), codes_of((N,), K, 2)
    sa = (1.0 + scales_of((kb, M), 3).clamp(0, 0.9)) * 2.0 ** (low // 2)
    sw = (1.0 + scales_of((kb, 2), 4).clamp(0, 0.9)) * 2.0 ** (low - low // 2)
    out = torch.empty(M, N, device=dev())
    bnn.bnn_fp8_gemm(A, sa, W, sw, K, out)
    a, w = values(A, sa, K, 1), values(W, sw, K, BLOCK)
    one = torch.ones(kb, M, device=dev()), torch.ones(kb, 2, device=dev())
    inner = values(A, one[0], K, 1).abs() @ values(W, one[1], K, BLOCK).abs().t()
    c64, mag = a @ w.t(), a.abs() @ w.abs().t()
    tol = (128 * 2.0 ** -23 + (2 * kb + 2) * 2.0 ** -24) * mag + 2.0 ** -150 * (kb + (inner if low < -126 else 0.0))
    assert ((out.double() - c64).abs() <= tol).all()
    assert (out != 0).any()
    assert_no_device_error()


@pytest.mark.parametrize("M", [5, 70, 150])
def test_large_scale_products(M):
    """Products of scales up to the largest fp32 number, beside one past it: that row's outputs in those columns are not
    finite, all others are right."""
    N, K = 140, 500
    kb = -(-K // BLOCK)
    A, W = codes_of((M,), K, 1), codes_of((N,), K, 2)
    A = torch.where((A & 0x7F) > 0x30, A & 0x87, A)          # |values| of at most 2^-1, so that the sums stay finite
    W = torch.where((W & 0x7F) > 0x30, W & 0x87, W)
    sa = torch.full((kb, M), 2.0 ** 60, device=dev())
    sw = torch.full((kb, 2), 2.0 ** 50, device=dev())
    sw[1, 1] = 2.0 ** 67
    sa[1, 3] = 1.5 * 2.0 ** 60
    sa[1, 2] = 2.0 ** 61
    out = torch.empty(M, N, device=dev())
    bnn.bnn_fp8_gemm(A, sa, W, sw, K, out)
    ok = torch.ones(M, N, dtype=torch.bool, device=dev())
    ok[2, BLOCK:] = False
    assert not out[~ok].isfinite().any()
    a, w = values(A, sa, K, 1), values(W, sw, K, BLOCK)
    c64, mag = a @ w.t(), a.abs() @ w.abs().t()
    ok &= mag < 2.0 ** 127
    assert ok.sum() >= M * BLOCK
    tol = (128 * 2.0 ** -23 + (2 * kb + 2) * 2.0 ** -24) * mag
    assert ((out.double() - c64).abs() <= tol)[ok].all()
    assert_no_device_error()


@pytest.mark.parametrize("rows", [2, 60])
def test_experts_past_32_bits(rows):
    """Experts' weights and scales more than 2^32 bytes from the first's."""
    E, N, K = 70, 130, 200
    far = 1 << 26                                             # 70 experts apart by 2^26 bytes, of either
    W = torch.empty(E * far, dtype=torch.uint8, device=dev()).as_strided((E, N, 208), (far, 208, 1))
    sw = torch.empty(E * far // 4, device=dev()).as_strided((E, 2, 2), (far // 4, 2, 1))
    W.copy_(codes_of((E, N), K, 1))
    sw.copy_(scales_of((E, 2, 2), 2))
    A, sa = codes_of((E * rows,), K, 3), scales_of((2, E * rows), 4)
    out = torch.empty(E * rows, N, device=dev())
    bnn.bnn_fp8_gemm_grouped(A, sa, torch.arange(0, E * rows + 1, rows, dtype=torch.int32, device=dev()), W, sw, K, out)
    for e in range(E):
        r = slice(e * rows, (e + 1) * rows)
        check(out[r], values(A[r], sa[:, r], K, 1), values(W[e], sw[e], K, BLOCK), K)
    assert_no_device_error()
