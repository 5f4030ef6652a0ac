"""The weights of bnn_route against the oracle's fp64 ones: rounded once, and their range."""
import numpy as np
import pytest
import torch

import oracle.lowp as ref
import xnor_popcount_gemm_bnn_b200 as bnn
from gpu_util import assert_no_device_error, dev

pytestmark = pytest.mark.gpu
SCORE = {"softmax": bnn.BNN_ROUTE_SOFTMAX, "sigmoid": bnn.BNN_ROUTE_SIGMOID}


def draw(T, E, seed, std):
    return torch.randn(T, E, generator=torch.Generator().manual_seed(seed)) * std


def weights(logits, k, score, bias=None, **kw):
    """(idx, weights) of the kernel and of the oracle, weights in float64."""
    T = logits.shape[0]
    idx, w = torch.empty(T, k, dtype=torch.int32, device=dev()), torch.empty(T, k, device=dev())
    bnn.bnn_route(logits.to(dev()), idx, w, score=SCORE[score], bias=None if bias is None else bias.to(dev()), **kw)
    want_i, want_w = ref.route(logits.float().numpy(), k, score, None if bias is None else bias.numpy(), **kw)
    assert_no_device_error()
    return idx.cpu().numpy(), w.cpu().numpy().astype(np.float64), want_i, want_w


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("scale", [1e39, -1e40, 1e45, 3e38, 1e-40, 2.0 ** -149])
def test_scale_beyond_fp32(score, renormalize, scale):
    """The scale is a double: a weight is infinite (or 0) only where the product itself leaves fp32.  An fp32
    evaluation's bound as in test_gpu_route.py, 2 (2^-21 + (range + E) 2^-24), and one step of the smallest numbers."""
    E = 48
    logits = draw(64, E, 3, 6.0)                           # chosen scores from 1 down to about 1e-7
    gi, gw, wi, ww = weights(logits, 8, score, renormalize=renormalize, scale=scale)
    assert np.array_equal(gi, wi)
    rel = 2 * (2.0 ** -21 + (float(logits.max() - logits.min()) + E) * 2.0 ** -24)
    top = float(np.finfo(np.float32).max)
    sure = np.abs(np.abs(ww) - top) > 2 * rel * top        # not so near the largest number that either may come
    over = sure & (np.abs(ww) > top)
    fine = sure & (np.abs(ww) < top)
    assert sure.any() and np.array_equal(gw[over], np.sign(ww[over]) * np.inf)
    assert (np.abs(gw - ww)[fine] <= rel * np.abs(ww[fine]) + 2.0 ** -149).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("T,E,k,std,groups,with_bias", [
    (1, 8, 2, 1.5, 1, False), (16, 64, 4, 1.5, 1, True), (40, 64, 6, 8.0, 1, False), (300, 128, 8, 1.5, 8, False),
    (200, 256, 8, 4.0, 1, True), (100, 257, 7, 8.0, 1, False), (100, 512, 16, 3.0, 16, True),
    (60, 60, 6, 30.0, 6, False), (60, 40, 40 // 4, 0.01, 1, False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_weights_are_rounded_once(T, E, k, std, groups, with_bias, score, renormalize, dtype):
    """fp64 scores rounded to fp32 at the end: half a step, 2^-24 of the weight (and 2^-150 where it is subnormal),
    whichever way the choice was settled; 1e-12 covers the fp64 sums of up to 512 terms on both sides."""
    logits = draw(T, E, T + E, std).to(dtype)
    bias = draw(1, E, 9, 0.1)[0] if with_bias else None
    gi, gw, wi, ww = weights(logits, k, score, bias, renormalize=renormalize, scale=1.7, n_groups=groups,
                             kept_groups=max(1, groups // 2))
    assert np.array_equal(gi, wi)
    assert (np.abs(gw - ww) <= (2.0 ** -24 + 1e-12) * np.abs(ww) + 2.0 ** -150).all()
