"""8-bit block-scaled operands through the C ABI against the oracle.

Packed codes and scales are compared bit for bit (every step of their definition is one IEEE operation).  Products:
every product of two codes is exact in fp32 (4-bit significands), so a block's sum of 128 has at most 128 additions,
each off by at most 2^-23 of a partial sum (truncation), and the sum over blocks adds a product of two scales and one
fused multiply-add per block (2^-24 each):
    |C - C64| <= (128 * 2^-23 + (2 * blocks + 2) * 2^-24) * sum |a w| + (half a step of the output type) * |C64|."""
import numpy as np
import pytest
import torch

import oracle.lowp as ref
import xnor_popcount_gemm_bnn_b200 as bnn
from gpu_util import assert_no_device_error, dev

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def u8(t):
    return t.view(torch.uint8).cpu().numpy()


def make(rows, K, seed, dtype="fp32"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))
    return x.to(DT[dtype])


def packed(x, block_rows, ld=None, lds=None):
    """Packed on the GPU, with guard bytes where ld and lds are larger."""
    rows, K = x.shape
    ld = ld or bnn.bnn_fp8_ld_bytes(K)
    nr = -(-rows // block_rows)
    codes = torch.full((rows, ld), 0x5A, dtype=torch.uint8, device=dev())
    scales = torch.full(((K + 127) // 128, lds or nr), -7.0, device=dev())
    bnn.bnn_fp8_pack(x.to(dev()), codes, scales, block_rows=block_rows)
    return codes, scales


def same_codes(got, want):
    """Equal codes; NaN codes may differ in their sign."""
    nan = (want & 0x7F) == 0x7F
    assert np.array_equal(np.where(nan, 0x7F, want), np.where((got & 0x7F) == 0x7F, 0x7F, got))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 16), (5, 129), (128, 128), (130, 1000), (257, 517), (1, 4096), (40, 4090)])
def test_pack(rows, K, block_rows, dtype):
    x = make(rows, K, rows + K, dtype)
    codes, scales = packed(x, block_rows, ld=bnn.bnn_fp8_ld_bytes(K) + 16, lds=-(-rows // block_rows) + 3)
    c, s = ref.fp8_pack(x.float().numpy(), block_rows)
    got = u8(codes)
    assert np.array_equal(got[:, :K], c)
    assert not got[:, K:bnn.bnn_fp8_ld_bytes(K)].any()              # padding
    assert (got[:, bnn.bnn_fp8_ld_bytes(K):] == 0x5A).all()         # past the packed row: as it was
    assert np.array_equal(scales.cpu().numpy()[:, :s.shape[1]], s)
    assert (scales.cpu().numpy()[:, s.shape[1]:] == -7.0).all()
    assert_no_device_error()


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_pack_special_values(dtype, block_rows):
    x = make(6, 300, 9, dtype)
    x[0] = 0.0
    x[1, 128:256] = -0.0
    x[2, 5], x[2, 130] = float("inf"), float("-inf")
    x[3, :] = float("nan")
    x[4, :128] = 1e-42 if dtype == "fp32" else 1e-39                # below the smallest scale
    x[5, 0], x[5, 1] = 3.3e38, -3.3e38
    codes, scales = packed(x, block_rows)
    c, s = ref.fp8_pack(x.float().numpy(), block_rows)
    same_codes(u8(codes)[:, :300], c)
    assert np.array_equal(scales.cpu().numpy(), s)


@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (2, 2), (4, 4), (3, 1)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_pack_strides_and_alignment(dtype, offset, pad, block_rows):
    """Rows of any element alignment and stride."""
    rows, K = 33, 260
    buf = make(rows, K + pad + offset, 21, dtype).to(dev())
    flat = torch.full((rows * (K + pad) + offset,), float("nan"), dtype=DT[dtype], device=dev())
    x = flat[offset:].as_strided((rows, K), (K + pad, 1), offset)
    x.copy_(buf[:, :K])
    codes = bnn.empty_fp8(rows, K, dev())
    scales = bnn.empty_fp8_scales(rows, K, block_rows, dev())
    bnn.bnn_fp8_pack(x, codes, scales, block_rows=block_rows)
    c, s = ref.fp8_pack(x.float().cpu().numpy(), block_rows)
    assert np.array_equal(u8(codes)[:, :K], c)
    assert np.array_equal(scales.cpu().numpy(), s)


def test_pack_gather():
    """Rows by index: repeated, in any order; an index outside x leaves the packed row as it was."""
    x = make(10, 200, 33, "bf16")
    index = torch.tensor([9, 0, 0, -1, 4, 10, 2**31 - 1, 7], dtype=torch.int32)
    codes = torch.full((8, 208), 0x11, dtype=torch.uint8, device=dev())
    scales = torch.full((2, 8), -1.0, device=dev())
    bnn.bnn_fp8_pack(x.to(dev()), codes, scales, row_index=index.to(dev()))
    c, s = ref.fp8_pack(x.float().numpy(), 1)
    for r, i in enumerate(index.tolist()):
        if 0 <= i < 10:
            assert np.array_equal(u8(codes)[r, :200], c[i])
            assert np.array_equal(scales.cpu().numpy()[:, r], s[:, i])
        else:
            assert (u8(codes)[r] == 0x11).all() and (scales[:, r] == -1.0).all()


def random_codes(rows, K, seed, ld=None):
    """Codes over the whole range (no NaN), garbage in the padding."""
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, 256, (rows, ld or bnn.bnn_fp8_ld_bytes(K)), generator=g, dtype=torch.uint8)
    c[:, :K] = torch.where((c[:, :K] & 0x7F) == 0x7F, torch.zeros_like(c[:, :K]), c[:, :K])
    return c


def random_scales(K, n, seed, lds=None):
    g = torch.Generator().manual_seed(seed)
    s = torch.full(((K + 127) // 128, lds or n), float("nan"))
    s[:, :n] = torch.exp(torch.randn((K + 127) // 128, n, generator=g)) * 0.01
    return s


def check(out, c64, mag, K, dtype):
    blocks = -(-K // 128)
    half = torch.finfo(DT[dtype]).eps / 2
    tol = (128 * 2.0 ** -23 + (2 * blocks + 2) * 2.0 ** -24) * mag * (1 + half) + half * np.abs(c64)
    y = out.float().cpu().numpy().astype(np.float64)
    bad = ~(np.abs(y - c64) <= tol)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:3], y[bad][:3], c64[bad][:3])


SHAPES = [(1, 1, 1), (1, 128, 128), (2, 130, 129), (7, 100, 16), (16, 129, 300), (17, 513, 1000), (33, 256, 4096),
          (64, 300, 700), (65, 127, 640), (128, 640, 257), (129, 128, 128), (200, 1000, 513), (256, 257, 128),
          (300, 96, 2000), (515, 385, 260), (1, 2000, 11008), (3, 4096, 130)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(M, N, K, dtype):
    A, W = random_codes(M, K, M + K), random_codes(N, K, N + K + 1)
    sa, sw = random_scales(K, M, 5), random_scales(K, -(-N // 128), 6)
    out = torch.full((M, N), float("nan"), dtype=DT[dtype], device=dev())
    bnn.bnn_fp8_gemm(A.to(dev()), sa.to(dev()), W.to(dev()), sw.to(dev()), K, out)
    c64, mag = ref.fp8_gemm(A.numpy(), sa.numpy(), W.numpy(), sw.numpy(), K)
    check(out, c64, mag, K, dtype)
    assert_no_device_error()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("M", [5, 70, 150])
def test_gemm_strides(M, dtype):
    """Row strides larger than the rows everywhere, an output of odd alignment, its padding as it was."""
    N, K = 150, 333
    A, W = random_codes(M, K, 1, ld=368), random_codes(N, K, 2, ld=352)
    sa, sw = random_scales(K, M, 3, lds=M + 5), random_scales(K, 2, 4, lds=7)
    buf = torch.full((M * (N + 9) + 1,), -3.0, dtype=DT[dtype], device=dev())
    out = buf[1:].as_strided((M, N), (N + 9, 1), 1)
    bnn.bnn_fp8_gemm(A.to(dev()), sa.to(dev()), W.to(dev()), sw.to(dev()), K, out)
    c64, mag = ref.fp8_gemm(A.numpy(), sa.numpy(), W.numpy(), sw.numpy(), K)
    check(out, c64, mag, K, dtype)
    rest = buf[1:].view(M, N + 9)[:, N:]
    assert (rest == -3.0).all() and buf[0] == -3.0


@pytest.mark.parametrize("M", [9, 140])
def test_gemm_nan_codes_stay_in_their_row_and_column(M):
    N, K = 140, 256
    A, W = random_codes(M, K, 7), random_codes(N, K, 8)
    A[3, 200], W[130, 5] = 0x7F, 0xFF
    sa, sw = random_scales(K, M, 9), random_scales(K, 2, 10)
    out = torch.zeros(M, N, device=dev())
    bnn.bnn_fp8_gemm(A.to(dev()), sa.to(dev()), W.to(dev()), sw.to(dev()), K, out)
    nan = torch.isnan(out).cpu()
    want = torch.zeros(M, N, dtype=torch.bool)
    want[3], want[:, 130] = True, True
    assert torch.equal(nan, want)


def test_gemm_exact_integers():
    """Codes of small whole numbers and unit scales: every sum is exact, so the product is."""
    M, N, K = 150, 140, 1000
    g = torch.Generator().manual_seed(2)
    a, w = (torch.randint(-8, 9, s, generator=g).float() for s in ((M, 1008), (N, 1008)))
    one = torch.ones(8, max(M, 2))
    for m in (M, 20, 1):
        out = torch.empty(m, N, device=dev())
        bnn.bnn_fp8_gemm(a[:m].to(torch.float8_e4m3fn).to(dev()), one[:, :m].contiguous().to(dev()),
                         w.to(torch.float8_e4m3fn).to(dev()), one[:, :2].contiguous().to(dev()), K, out)
        assert torch.equal(out.cpu().double(), a[:m, :K].double() @ w[:, :K].double().t())


def grouped(counts, N, K, dtype, first=0, tail=0, seed=0, interleave=False):
    E = len(counts)
    off = np.concatenate([[0], np.cumsum(counts)]) + first
    R = int(off[-1]) + tail
    A = random_codes(max(R, 1), K, seed + 1)[:R]
    sa = random_scales(K, max(R, 1), seed + 2)[:, :R]
    W = torch.stack([random_codes(N, K, seed + 10 + e) for e in range(E)])
    sw = torch.stack([random_scales(K, -(-N // 128), seed + 50 + e) for e in range(E)])
    swd = sw.to(dev())
    if interleave:                                     # [blocks of K, E, row blocks] in memory
        swd = swd.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.full((R, N), 99.0, dtype=DT[dtype], device=dev())
    bnn.bnn_fp8_gemm_grouped(A.to(dev()), sa.contiguous().to(dev()), torch.from_numpy(off.astype(np.int32)).to(dev()),
                             W.to(dev()), swd, K, out)
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if counts[e]:
            c64, mag = ref.fp8_gemm(A[r].numpy(), sa[:, r].numpy(), W[e].numpy(), sw[e].numpy(), K)
            check(out[r], c64, mag, K, dtype)
    assert (out[:first] == 99.0).all() and (out[R - tail:] == 99.0).all()
    assert_no_device_error()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 128, 128), ([0, 0, 3, 0], 130, 200), ([1, 2, 3, 4, 5, 6, 7, 8], 257, 300), ([40, 0, 17, 1], 128, 1000),
    ([130, 1, 0, 300], 200, 513), ([257, 255, 256], 300, 128), ([0, 0], 64, 64), ([600], 129, 640),
    ([5] * 70, 96, 150), ([700, 3, 2, 1, 0, 0, 0, 50], 384, 384)])
def test_grouped(counts, N, K, dtype):
    grouped(counts, N, K, dtype, seed=sum(counts))


@pytest.mark.parametrize("counts", [[3, 4], [200, 90]])
def test_grouped_rows_outside_every_group_stay(counts):
    grouped(counts, 140, 260, "bf16", first=5, tail=9)


@pytest.mark.parametrize("counts", [[3, 4, 0], [200, 90, 8]])
def test_grouped_interleaved_scales(counts):
    grouped(counts, 300, 700, "fp32", interleave=True)


@pytest.mark.parametrize("rows", [20, 500])
def test_grouped_bad_offsets_are_clamped(rows):
    """Offsets outside [0, R] or decreasing never reach outside the arrays."""
    N, K = 100, 130
    A, sa = random_codes(rows, K, 1), random_scales(K, rows, 2)
    W, sw = random_codes(3 * N, K, 3).view(3, N, -1), torch.stack([random_scales(K, 1, 4)] * 3)
    buf = torch.full((rows + 64, N), 5.0, device=dev())
    out = buf[32:32 + rows]
    for off in ([-40, rows // 2, rows + 9, 2 ** 31 - 1], [-2 ** 31, -1, 3, 2], [rows, 4, 0, -7]):
        bnn.bnn_fp8_gemm_grouped(A.to(dev()), sa.to(dev()), torch.tensor(off, dtype=torch.int32, device=dev()),
                                 W.to(dev()), sw.to(dev()), K, out)
        torch.cuda.synchronize()
        assert (buf[:32] == 5.0).all() and (buf[32 + rows:] == 5.0).all()
    assert_no_device_error()


@pytest.mark.parametrize("M", [4, 300])
def test_gemm_on_a_side_stream_and_captured(M):
    """Calls on another stream, two at once, and a captured call replayed on new values."""
    N, K = 300, 400
    A, W = random_codes(M, K, 1).to(dev()), random_codes(N, K, 2).to(dev())
    sa, sw = random_scales(K, M, 3).to(dev()), random_scales(K, 3, 4).to(dev())
    want = torch.empty(M, N, device=dev())
    bnn.bnn_fp8_gemm(A, sa, W, sw, K, want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty(M, N, device=dev()) for _ in range(8)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i, o in enumerate(outs):
        bnn.bnn_fp8_gemm(A, sa, W, sw, K, o, stream=streams[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    out = torch.empty(M, N, device=dev())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bnn.bnn_fp8_gemm(A, sa, W, sw, K, out)
    A2 = random_codes(M, K, 11).to(dev())
    A.copy_(A2)
    graph.replay()
    bnn.bnn_fp8_gemm(A2, sa, W, sw, K, want)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert_no_device_error()


def test_binding_refuses_wrong_tensors():
    d = dev()
    A, W = random_codes(4, 64, 1).to(d), random_codes(8, 64, 2).to(d)
    sa, sw = random_scales(64, 4, 3).to(d), random_scales(64, 1, 4).to(d)
    out = torch.empty(4, 8, device=d)
    for bad in ((A.float(), sa, W, sw, 64, out), (A, sa.double(), W, sw, 64, out), (A, sa, W, sw, 65, out),
                (A, sa, W, sw, 64, out[:3]), (A.cpu(), sa, W, sw, 64, out), (A, sa[:, :3], W, sw, 64, out),
                (A, sa, W, sw, 64, torch.empty(8, 4, device=d).t())):
        with pytest.raises((ValueError, TypeError, bnn.BnnError)):
            bnn.bnn_fp8_gemm(*bad)
    with pytest.raises(TypeError):
        bnn.bnn_fp8_gemm(A, sa, W, sw, 64, out.half())


@pytest.mark.parametrize("dtype,ld,offset,K", [
    ("bf16", 264, 0, 261), ("bf16", 268, 4, 263), ("bf16", 262, 2, 259), ("bf16", 261, 1, 130), ("bf16", 272, 8, 129),
    ("fp32", 264, 0, 261), ("fp32", 266, 2, 259), ("fp32", 261, 1, 261), ("fp32", 268, 4, 255), ("fp32", 136, 8, 3)])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows", [7, 400])
def test_pack_rows_that_end_inside_a_vector(rows, dtype, ld, offset, K, block_rows):
    """Every alignment of the rows with a K that ends inside a load; what follows a row (NaN) is not read into it."""
    flat = torch.full((rows * ld + offset,), float("nan"), dtype=DT[dtype], device=dev())
    x = flat.as_strided((rows, K), (ld, 1), offset)
    x.copy_(make(rows, K, ld + K, dtype).to(dev()))
    codes = torch.full((rows, bnn.bnn_fp8_ld_bytes(K) + 16), 0x5A, dtype=torch.uint8, device=dev())
    scales = bnn.empty_fp8_scales(rows, K, block_rows, dev())
    bnn.bnn_fp8_pack(x, codes, scales, block_rows=block_rows)
    c, s = ref.fp8_pack(x.float().cpu().numpy(), block_rows)
    assert np.array_equal(u8(codes)[:, :K], c)
    assert not u8(codes)[:, K:bnn.bnn_fp8_ld_bytes(K)].any()
    assert (u8(codes)[:, bnn.bnn_fp8_ld_bytes(K):] == 0x5A).all()
    assert np.array_equal(scales.cpu().numpy(), s)


def test_single_row_and_column_views():
    """M = 1 and N = 1 as torch hands them over: scales of one column and outputs whose strides say nothing."""
    K = 300
    A, W = random_codes(1, K, 1), random_codes(1, K, 2)
    sa, sw = random_scales(K, 1, 3), random_scales(K, 1, 4)
    out = torch.empty(1, 1, device=dev())
    bnn.bnn_fp8_gemm(A.to(dev()), sa.t().contiguous().t().to(dev()), W.to(dev()), sw.t().contiguous().t().to(dev()), K,
                     out)
    c64, mag = ref.fp8_gemm(A.numpy(), sa.numpy(), W.numpy(), sw.numpy(), K)
    check(out, c64, mag, K, "fp32")


def test_offsets_past_32_bits():
    """Rows far apart: element offsets beyond 2^32 in the input of a pack, in codes and in the output of a product."""
    rows, K, N = 300, 200, 130
    far = 1 << 24                                          # 300 rows apart by 2^24 elements
    big = torch.empty(rows * far, dtype=torch.bfloat16, device=dev())
    x = big.as_strided((rows, K), (far, 1))
    x.copy_(make(rows, K, 5, "bf16").to(dev()))
    codes, scales = bnn.empty_fp8(rows, K, dev()), bnn.empty_fp8_scales(rows, K, 1, dev())
    bnn.bnn_fp8_pack(x, codes, scales)
    c, s = ref.fp8_pack(x.float().cpu().numpy(), 1)
    assert np.array_equal(u8(codes)[:, :K], c)
    W, sw = random_codes(N, K, 2), random_scales(K, 2, 4)
    for m in (300, 100):
        spread = big.view(torch.uint8).as_strided((m, 208), (far, 1), 1 << 20)
        spread.copy_(codes.view(torch.uint8)[:m])
        out = big.as_strided((m, N), (far, 1), 1 << 22)
        bnn.bnn_fp8_gemm(spread, scales[:, :m].contiguous(), W.to(dev()), sw.to(dev()), K, out)
        c64, mag = ref.fp8_gemm(c[:m], s[:, :m], W.numpy(), sw.numpy(), K)
        check(out, c64, mag, K, "bf16")
    assert_no_device_error()


def test_calls_back_to_back_see_one_another():
    """Each launch may set up beside the one before it: a chain in which every call reads what the last one wrote."""
    M, K = 40, 512
    x = make(M, K, 3, "bf16").to(dev())
    W = torch.stack([bnn.empty_fp8(K, K, dev()) for _ in range(2)])
    sw = torch.stack([bnn.empty_fp8_scales(K, K, 128, dev()) for _ in range(2)])
    for i in range(2):
        bnn.bnn_fp8_pack((make(K, K, 20 + i) * 0.02).to(dev()), W[i], sw[i], block_rows=128)

    def chain(wait):
        y = x.clone()
        codes, scales = bnn.empty_fp8(M, K, dev()), bnn.empty_fp8_scales(M, K, 1, dev())
        for i in range(24):
            bnn.bnn_fp8_pack(y, codes, scales)
            if wait:
                torch.cuda.synchronize()
            bnn.bnn_fp8_gemm(codes, scales, W[i % 2], sw[i % 2], K, y)
            if wait:
                torch.cuda.synchronize()
        return y

    want = chain(True)
    for _ in range(5):
        assert torch.equal(chain(False).view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("counts", [[3, 2, 4], [40, 30, 35], [300, 10, 200]])
def test_two_streams_of_different_kernels(counts):
    """Grouped and dense products of several widths at once on two streams give what they give alone."""
    N, K = 260, 900
    R = sum(counts)
    A, sa = random_codes(R, K, 1).to(dev()), random_scales(K, R, 2).to(dev())
    W = torch.stack([random_codes(N, K, 10 + e) for e in range(3)]).to(dev())
    sw = torch.stack([random_scales(K, 3, 50 + e) for e in range(3)]).to(dev())
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=dev())
    sizes = [m for m in (1, 20, 60, 100, 200) if m <= R]
    sas = [sa[:, :m].contiguous() for m in sizes]

    def all_of(stream, outs):
        bnn.bnn_fp8_gemm_grouped(A, sa, off, W, sw, K, outs[0], stream=stream)
        for m, s, o in zip(sizes, sas, outs[1:]):
            bnn.bnn_fp8_gemm(A[:m], s, W[0], sw[0], K, o, stream=stream)

    new = lambda: [torch.empty(R, N, device=dev())] + [torch.empty(m, N, device=dev()) for m in sizes]
    want = new()
    all_of(None, want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [new() for _ in range(6)]
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        all_of(streams[i % 2], o)
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
    assert_no_device_error()
