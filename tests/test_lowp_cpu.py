"""Without a GPU: the oracle of the 8-bit products and the routing against torch's own conversions and sorts, and the
refusals of the C entries (host checks, before any CUDA call)."""
import ctypes
import re

import numpy as np
import pytest
import torch

import oracle.lowp as ref
import xnor_popcount_gemm_bnn_b200 as bnn

L = bnn.lib
FAKE = ctypes.c_void_p(0x10000)
FAKE4 = ctypes.c_void_p(0x10004)     # not 16-byte aligned
FAKE2 = ctypes.c_void_p(0x10002)     # not 4-byte aligned
NULL = None
OK, INV, ALN, UNS = bnn.BNN_OK, bnn.BNN_ERR_INVALID_ARG, bnn.BNN_ERR_ALIGNMENT, bnn.BNN_ERR_UNSUPPORTED


def test_oracle_code_values_match_torch():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref.VALUES, equal_nan=True)


def test_oracle_rounding_matches_torch():
    g = torch.Generator().manual_seed(3)
    q = torch.cat([torch.randn(4000, generator=g) * s for s in (1e-3, 0.1, 1.0, 30.0, 150.0)])
    pos = torch.tensor(ref.VALUES[:127])
    ties = ((pos[1:] + pos[:-1]) / 2).float()            # exactly between two codes
    q = torch.cat([q, ties, -ties, pos.float(), torch.tensor([0.0, -0.0])]).clamp(-448, 448)
    want = q.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_nearest(q.numpy()), want)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_oracle_route_matches_sort(score):
    g = torch.Generator().manual_seed(5)
    l = torch.randn(40, 24, generator=g).to(torch.bfloat16)      # bf16: equal logits occur
    idx, w = ref.route(l.float().numpy(), 5, score)
    s = torch.softmax(l.double(), 1) if score == "softmax" else torch.sigmoid(l.double())
    order = torch.sort(l.double(), dim=1, descending=True, stable=True).indices[:, :5]
    assert np.array_equal(idx, order.int().numpy())
    picked = s.gather(1, order)
    np.testing.assert_allclose(w, (picked / picked.sum(1, keepdim=True)).numpy(), rtol=1e-12)


def test_fp8_row_bytes():
    for K, want in ((1, 16), (16, 16), (17, 32), (4096, 4096), (4090, 4096)):
        assert bnn.bnn_fp8_ld_bytes(K) == want
    assert bnn.bnn_fp8_ld_bytes(0) == -1


def test_route_constants_match_header():
    import os
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "bnn.h")).read()
    for name in ("BNN_ROUTE_SOFTMAX", "BNN_ROUTE_SIGMOID"):
        assert int(re.search(rf"\b{name}\s*=\s*(\d+)", text).group(1)) == getattr(bnn, name)


def test_fp8_pack_refusals():
    def call(x=FAKE, dt=0, x_rows=8, K=200, ld_x=200, index=NULL, rows=8, block=1, codes=FAKE, ldc=208, scales=FAKE,
             lds=8):
        return L.bnn_fp8_pack(x, dt, x_rows, K, ld_x, index, rows, block, codes, ldc, scales, lds, NULL)
    assert call(x=NULL) == INV
    assert call(codes=NULL) == INV
    assert call(scales=NULL) == INV
    assert call(dt=2) == INV
    assert call(K=0) == INV
    assert call(ld_x=199) == INV
    assert call(rows=9, lds=9) == INV                       # more rows than x has, and no index
    assert call(rows=-1) == INV
    assert call(x_rows=-1) == INV
    assert call(block=64) == INV
    assert call(ldc=192) == INV                             # K rounded up to 16 is 208
    assert call(lds=7) == INV
    assert call(K=2 ** 31, ld_x=2 ** 31, ldc=2 ** 31) == INV
    assert call(ldc=216) == ALN
    assert call(codes=FAKE4) == ALN
    assert call(scales=FAKE2) == ALN
    assert call(x=FAKE2) == ALN
    assert call(index=FAKE2) == ALN
    assert call(index=FAKE, block=128) == UNS
    assert call(rows=0, lds=0) == OK
    assert call(x=NULL, x_rows=0, rows=0, codes=NULL, scales=NULL, lds=0) == OK


def test_fp8_gemm_refusals():
    def call(A=FAKE, lda=208, sa=FAKE, ldsa=8, W=FAKE, ldw=208, sw=FAKE, ldsw=2, M=8, N=200, K=200, out=FAKE, dt=1,
             ldo=200):
        return L.bnn_fp8_gemm(A, lda, sa, ldsa, W, ldw, sw, ldsw, M, N, K, out, dt, ldo, NULL)
    for name in ("A", "sa", "W", "sw", "out"):
        assert call(**{name: NULL}) == INV, name
    assert call(lda=192) == INV
    assert call(ldw=192) == INV
    assert call(ldsa=7) == INV
    assert call(ldsw=1) == INV
    assert call(ldo=199) == INV
    assert call(K=0) == INV
    assert call(M=-1) == INV
    assert call(N=-1) == INV
    assert call(dt=3) == INV
    assert call(M=2 ** 31, ldsa=2 ** 31) == INV
    assert call(lda=216) == ALN
    assert call(ldw=216) == ALN
    assert call(A=FAKE4) == ALN
    assert call(W=FAKE4) == ALN
    assert call(sa=FAKE2) == ALN
    assert call(sw=FAKE2) == ALN
    assert call(out=ctypes.c_void_p(0x10001)) == ALN
    assert call(out=FAKE2, dt=0) == ALN
    assert call(M=0, A=NULL, sa=NULL, out=NULL) == OK
    assert call(N=0, W=NULL) == OK


def test_fp8_gemm_grouped_refusals():
    def call(A=FAKE, lda=208, sa=FAKE, ldsa=8, R=8, off=FAKE, E=3, W=FAKE, ldw=208, ws=200 * 208, sw=FAKE, ldsw=2,
             sws=4, N=200, K=200, out=FAKE, dt=1, ldo=200):
        return L.bnn_fp8_gemm_grouped(A, lda, sa, ldsa, R, off, E, W, ldw, ws, sw, ldsw, sws, N, K, out, dt, ldo, NULL)
    assert call(off=NULL) == INV
    assert call(E=-1) == INV
    assert call(ws=200 * 208 - 16) == INV
    assert call(sws=-1) == INV
    assert call(ldsa=7) == INV
    assert call(A=NULL) == INV
    assert call(ws=200 * 208 + 8) == ALN
    assert call(off=FAKE2) == ALN
    assert call(E=1025) == UNS
    assert call(E=0) == OK
    assert call(R=0, A=NULL, sa=NULL, out=NULL, ldsa=0) == OK
    assert call(N=0) == OK


def params(**kw):
    p = dict(score=0, k=2, n_groups=1, kept_groups=1, group_top=2, renormalize=1, scale=1.0, bias=None)
    p.update(kw)
    return ctypes.byref(bnn.bnn_route_params(*p.values()))


def test_route_refusals():
    def call(l=FAKE, dt=0, T=4, E=16, ld=16, p=None, idx=FAKE, w=FAKE, off=NULL, tok=NULL, slot=NULL):
        return L.bnn_route(l, dt, T, E, ld, params() if p is None else p, idx, w, off, tok, slot, NULL)
    assert L.bnn_route(FAKE, 0, 4, 16, 16, None, FAKE, FAKE, NULL, NULL, NULL, NULL) == INV
    assert call(l=NULL) == INV
    assert call(idx=NULL) == INV
    assert call(w=NULL) == INV
    assert call(dt=5) == INV
    assert call(off=FAKE) == INV                            # a plan needs all three
    assert call(tok=FAKE, slot=FAKE) == INV
    assert call(T=-1) == INV
    assert call(E=0) == INV
    assert call(ld=15) == INV
    assert call(p=params(k=0)) == INV
    assert call(p=params(k=17), E=16) == INV                # more than there are
    assert call(p=params(k=17), E=32, ld=32) == UNS
    assert call(E=513, ld=513) == UNS
    assert call(p=params(score=2)) == INV
    assert call(p=params(n_groups=0)) == INV
    assert call(p=params(n_groups=3)) == INV                # 16 experts
    assert call(p=params(n_groups=4, kept_groups=5)) == INV
    assert call(p=params(n_groups=4, kept_groups=0)) == INV
    assert call(p=params(group_top=3)) == INV
    assert call(p=params(renormalize=2)) == INV
    assert call(p=params(scale=float("inf"))) == INV
    assert call(p=params(scale=float("nan"))) == INV
    assert call(T=2 ** 30) == INV                           # T * k
    assert call(l=FAKE2) == ALN
    assert call(idx=FAKE2) == ALN
    assert call(w=FAKE2) == ALN
    assert call(p=params(bias=0x10002)) == ALN
    assert call(off=FAKE2, tok=FAKE, slot=FAKE) == ALN
    assert call(T=0) == OK
    assert call(T=0, l=NULL, idx=NULL, w=NULL) == OK


def test_route_combine_refusals():
    def call(Y=FAKE, dt=1, R=8, N=40, ldy=40, slot=FAKE, w=FAKE, T=4, k=2, out=FAKE, odt=1, ldo=40):
        return L.bnn_route_combine(Y, dt, R, N, ldy, slot, w, T, k, out, odt, ldo, NULL)
    for name in ("Y", "slot", "w", "out"):
        assert call(**{name: NULL}) == INV, name
    assert call(dt=4) == INV
    assert call(odt=4) == INV
    assert call(k=0) == INV
    assert call(ldy=39) == INV
    assert call(ldo=39) == INV
    assert call(T=-1) == INV
    assert call(R=-1) == INV
    assert call(k=65) == UNS
    assert call(Y=ctypes.c_void_p(0x10001)) == ALN
    assert call(out=FAKE2, odt=0) == ALN
    assert call(slot=FAKE2) == ALN
    assert call(w=FAKE2) == ALN
    assert call(T=0, slot=NULL, w=NULL, out=NULL) == OK
    assert call(N=0, Y=NULL) == OK


def test_fp8_gemm_grouped_without_experts():
    """E = 0 is allowed and launches nothing: the empty arrays W, w_scales and offsets may be NULL, also through the
    binding's torch tensors of no elements, whose address is 0."""
    def call(W=NULL, sw=NULL, off=NULL, E=0, N=200, ldsa=8):
        return L.bnn_fp8_gemm_grouped(FAKE, 208, FAKE, ldsa, 8, off, E, W, 208, 200 * 208, sw, 2, 4, N, 200, FAKE, 1,
                                      200, NULL)
    assert call() == OK
    assert call(W=FAKE) == OK
    assert call(off=FAKE2) == ALN                           # what is given is still checked
    assert call(ldsa=7) == INV
    assert call(E=1) == INV
    assert call(E=1, W=FAKE, off=FAKE) == INV
    assert call(E=1, W=FAKE, sw=FAKE) == INV
    assert torch.empty(0, 200, 208).data_ptr() == 0
