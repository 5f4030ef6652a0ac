"""The weights of bnn_route against the oracle's fp64 ones: their range."""
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
