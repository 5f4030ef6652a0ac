"""Routing to experts through the C ABI against the oracle: choices, plan and offsets equal, weights within the
bound of an fp32 evaluation, and the layer of experts as a whole.

Weights: an fp32 softmax (or sigmoid) has a relative error of at most 2^-22 for the exponential, |argument| 2^-24 for
its argument's rounding, E 2^-24 for the sum and 2^-23 for two divisions; renormalising doubles it:
    |w - w64| <= 2 (2^-21 + (range + E) 2^-24) |w64|, and 2^-126 where the score underflows."""
import numpy as np
import pytest
import torch

import oracle.lowp as ref
import xnor_popcount_gemm_bnn_b200 as bnn
from gpu_util import assert_no_device_error, dev

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
SCORE = {"softmax": bnn.BNN_ROUTE_SOFTMAX, "sigmoid": bnn.BNN_ROUTE_SIGMOID}


def run(logits, k, score="softmax", plan=True, ld=None, stream=None, **kw):
    T, E = logits.shape
    d = dev()
    l = logits.to(d)
    if ld is not None:
        wide = torch.full((T, ld), float("inf"), dtype=l.dtype, device=d)
        wide[:, :E] = l
        l = wide[:, :E]
    idx = torch.full((T, k), -9, dtype=torch.int32, device=d)
    w = torch.full((T, k), float("nan"), device=d)
    more = {}
    if plan:
        more = dict(offsets=torch.full((E + 1,), -9, dtype=torch.int32, device=d),
                    row_token=torch.full((T * k,), -9, dtype=torch.int32, device=d),
                    slot_row=torch.full((T, k), -9, dtype=torch.int32, device=d))
    bias = kw.pop("bias", None)
    bnn.bnn_route(l, idx, w, score=SCORE[score], bias=None if bias is None else bias.to(d), stream=stream, **kw, **more)
    return idx, w, more


def check(logits, k, score="softmax", **kw):
    T, E = logits.shape
    idx, w, more = run(logits, k, score, **kw)
    kw.pop("ld", None)
    kw.pop("plan", None)
    bias = kw.pop("bias", None)
    l = logits.float().numpy()
    want_i, want_w = ref.route(l, k, score, None if bias is None else bias.numpy(), **kw)
    got_i, got_w = idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    assert np.array_equal(got_i, want_i), np.argwhere(got_i != want_i)[:5]
    fin = l[np.isfinite(l)]
    rng = min(200.0, float(fin.max() - fin.min()) if fin.size else 0.0)
    tol = 2 * (2.0 ** -21 + (rng + E) * 2.0 ** -24) * np.abs(want_w) + 2.0 ** -126 * max(1.0, abs(kw.get("scale", 1.0)))
    assert (np.abs(got_w - want_w) <= tol).all()
    if more:
        off, tok, slot = ref.route_plan(want_i, E)
        assert np.array_equal(more["offsets"].cpu().numpy(), off)
        assert np.array_equal(more["row_token"].cpu().numpy(), tok)
        assert np.array_equal(more["slot_row"].cpu().numpy(), slot)
    assert_no_device_error()


def draw(T, E, seed, dtype="fp32", std=1.5):
    return (torch.randn(T, E, generator=torch.Generator().manual_seed(seed)) * std).to(DT[dtype])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 4), (2, 3, 3), (7, 33, 2), (31, 64, 8), (33, 100, 5), (100, 128, 16),
                                   (65, 256, 8), (300, 257, 7), (40, 512, 16), (1000, 16, 2)])
def test_route(T, E, k, dtype, score):
    check(draw(T, E, T + E, dtype), k, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,G,kept,top", [(5, 16, 4, 4, 2, 2), (60, 256, 8, 8, 4, 2), (60, 256, 8, 8, 3, 1),
                                              (33, 60, 6, 6, 2, 2), (20, 512, 16, 32, 1, 2), (9, 96, 3, 32, 5, 1),
                                              (11, 8, 2, 8, 2, 2), (50, 64, 8, 2, 1, 2), (50, 64, 8, 2, 2, 2)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_groups_and_bias(T, E, k, G, kept, top, score, with_bias):
    bias = draw(1, E, 77, std=0.1)[0] if with_bias else None
    check(draw(T, E, G + E), k, score, bias=bias, n_groups=G, kept_groups=kept, group_top=top)


@pytest.mark.parametrize("renormalize,scale", [(False, 1.0), (True, 2.5), (False, -0.5), (True, 0.0)])
def test_route_weights(renormalize, scale):
    for score in ("softmax", "sigmoid"):
        check(draw(50, 40, 3), 6, score, renormalize=renormalize, scale=scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_ties_go_to_the_lowest_index(score, with_bias):
    """Equal logits everywhere, and pairs of equal experts far apart."""
    bias = torch.zeros(96) if with_bias else None
    check(torch.zeros(4, 96), 7, score, bias=bias)
    l = draw(64, 96, 8)
    l[:, 50:] = l[:, :46]
    check(l, 9, score, bias=bias)
    check(l, 9, score, bias=bias, n_groups=3, kept_groups=2)
    check(draw(200, 96, 9, "bf16", std=0.05), 8, score, bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_near_ties_with_a_bias(score):
    """Choice values closer than fp32 tells apart: the order is that of the 64-bit values."""
    g = torch.Generator().manual_seed(4)
    l = 1.0 + torch.randint(0, 64, (300, 128), generator=g).float() * 2.0 ** -23
    check(l, 8, score, bias=torch.randint(0, 3, (128,), generator=g).float() * 2.0 ** -30)
    check(l, 8, score, bias=torch.full((128,), 2.0 ** -28), n_groups=4, kept_groups=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masks_and_extremes(score):
    """-inf and NaN mask experts, rows left with none or too few, the type's lowest value, +inf."""
    l = draw(12, 40, 5)
    l[0] = float("-inf")
    l[1] = float("nan")
    l[2, 3:] = float("-inf")
    l[3, :] = torch.finfo(torch.float32).min
    l[4, 7] = float("inf")
    l[5, 7], l[5, 9] = float("inf"), float("inf")
    l[6, :20] = float("nan")
    l[7] = -200.0
    l[8] = -1000.0
    l[9] = 90.0
    l[10, ::2] = -1e30
    check(l, 6, score)
    check(l, 6, score, n_groups=4, kept_groups=2)
    bias = draw(1, 40, 6, std=0.1)[0]
    bias[2], bias[11] = float("-inf"), float("nan")
    check(l, 6, score, bias=bias)
    check(l, 6, score, bias=bias, n_groups=8, kept_groups=2)


def test_route_strided_rows_and_no_plan():
    check(draw(20, 50, 2, "bf16"), 4, ld=53)
    check(draw(20, 50, 2), 4, "sigmoid", ld=64, plan=False)


def test_route_no_tokens():
    idx, w, more = run(torch.empty(0, 20), 3)
    assert (more["offsets"] == 0).all()


@pytest.mark.parametrize("T,E,k", [(4096, 8, 2), (9000, 256, 8), (3001, 512, 7)])
def test_route_plan_of_many_tokens(T, E, k):
    """The plan of long prompts against a stable sort."""
    idx, w, more = run(draw(T, E, 1), k)
    flat = idx.long().flatten()
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(more["row_token"].long(), order // k)
    assert torch.equal(more["slot_row"].long().flatten()[order], torch.arange(T * k, device=idx.device))
    assert torch.equal(more["offsets"].long(),
                       torch.searchsorted(flat[order], torch.arange(E + 1, device=idx.device)))
    assert_no_device_error()


@pytest.mark.parametrize("dt,odt", [("bf16", "bf16"), ("fp32", "fp32"), ("bf16", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (3, 2, 7), (5, 8, 130), (40, 4, 1000), (2, 64, 33), (9, 3, 4096)])
def test_combine(T, k, N, dt, odt):
    """Rows missing from the sum (-1 and past the end), repeated rows, strides.  fp32 sums of k terms:
    k 2^-24 sum |terms|, plus half a step of the output type."""
    g = torch.Generator().manual_seed(T * k + N)
    R = T * k + 2
    Y = torch.randn(R, N + 3, generator=g).to(DT[dt]).to(dev())[:, :N]
    slot = torch.randint(-1, R + 2, (T, k), generator=g, dtype=torch.int32)
    w = torch.randn(T, k, generator=g)
    buf = torch.full((T, N + 5), 3.0, dtype=DT[odt], device=dev())
    bnn.bnn_route_combine(Y, slot.to(dev()), w.to(dev()), buf[:, :N])
    want, mag = ref.route_combine(Y.float().cpu().numpy(), slot.numpy(), w.numpy())
    half = torch.finfo(DT[odt]).eps / 2
    tol = k * 2.0 ** -24 * mag * (1 + half) + half * np.abs(want)
    assert (np.abs(buf[:, :N].float().cpu().numpy() - want) <= tol).all()
    assert (buf[:, N:] == 3.0).all()


@pytest.mark.parametrize("T,E,k,D,F", [(1, 8, 2, 256, 384), (37, 8, 3, 200, 130), (300, 4, 2, 384, 260)])
def test_layer_of_experts(T, E, k, D, F):
    """Route, gather and pack, the experts' product, combine: as they are used together, against the oracle's chain
    (the oracle packs the same real rows, so codes agree and only the product's and the sum's rounding differ)."""
    d = dev()
    x = draw(T, D, 1, "bf16", 1.0)
    router = draw(E, D, 2, std=0.1)
    w = draw(E * F, D, 3, std=0.05)
    logits = (x.float() @ router.t())
    logits[T // 2, :] = float("-inf")                      # a padded token: no expert
    idx, wt, plan = run(logits, k, "softmax")
    codes, scales = bnn.empty_fp8(T * k, D, d), bnn.empty_fp8_scales(T * k, D, 1, d)
    codes.view(torch.uint8).zero_()
    scales.fill_(1.0)
    bnn.bnn_fp8_pack(x.to(d), codes, scales, row_index=plan["row_token"])
    W = torch.stack([bnn.empty_fp8(F, D, d) for _ in range(E)])
    sw = torch.stack([bnn.empty_fp8_scales(F, D, 128, d) for _ in range(E)])
    for e in range(E):
        bnn.bnn_fp8_pack(w[e * F:(e + 1) * F].to(d), W[e], sw[e], block_rows=128)
    Y = torch.full((T * k, F), float("nan"), dtype=torch.bfloat16, device=d)
    bnn.bnn_fp8_gemm_grouped(codes, scales, plan["offsets"], W, sw, D, Y)
    out = torch.empty(T, F, dtype=torch.bfloat16, device=d)
    bnn.bnn_route_combine(Y, plan["slot_row"], wt, out)

    ri, rw = ref.route(logits.numpy(), k, "softmax")
    xc, xs = ref.fp8_pack(x.float().numpy(), 1)
    want, mag = np.zeros((T, F)), np.zeros((T, F))
    for e in range(E):
        wc, ws = ref.fp8_pack(w[e * F:(e + 1) * F].numpy(), 128)
        y, m = ref.fp8_gemm(xc, xs, wc, ws, D)
        for t in range(T):
            for j in range(k):
                if ri[t, j] == e:
                    want[t] += rw[t, j] * y[t]
                    mag[t] += rw[t, j] * m[t]
    # the product (derived in the fp8 tests), its rounding to bf16, the weights (2^-20 covers E <= 8 and the logits'
    # range here), the fp32 sum, the rounding to bf16
    blocks = -(-D // 128)
    tol = (128 * 2.0 ** -23 + (2 * blocks + 2) * 2.0 ** -24 + 2.0 ** -8 + 2.0 ** -17 + k * 2.0 ** -24) * 1.01 * mag
    assert (np.abs(out.float().cpu().numpy() - want) <= tol + 2.0 ** -8 * np.abs(want)).all()
    assert (out[T // 2] == 0).all()
    assert_no_device_error()


def test_layer_of_experts_captured():
    """The four calls captured in one graph and replayed on other tokens give what eager calls give."""
    d = dev()
    T, E, k, D, F = 19, 8, 2, 256, 256
    W = torch.stack([bnn.empty_fp8(F, D, d) for _ in range(E)])
    sw = torch.stack([bnn.empty_fp8_scales(F, D, 128, d) for _ in range(E)])
    for e in range(E):
        bnn.bnn_fp8_pack(draw(F, D, 100 + e, std=0.05).to(d), W[e], sw[e], block_rows=128)

    def buffers():
        return dict(x=torch.empty(T, D, dtype=torch.bfloat16, device=d), l=torch.empty(T, E, device=d),
                    idx=torch.empty(T, k, dtype=torch.int32, device=d), w=torch.empty(T, k, device=d),
                    off=torch.empty(E + 1, dtype=torch.int32, device=d),
                    tok=torch.empty(T * k, dtype=torch.int32, device=d),
                    slot=torch.empty(T, k, dtype=torch.int32, device=d), codes=bnn.empty_fp8(T * k, D, d),
                    scales=bnn.empty_fp8_scales(T * k, D, 1, d),
                    Y=torch.empty(T * k, F, dtype=torch.bfloat16, device=d),
                    out=torch.empty(T, F, dtype=torch.bfloat16, device=d))

    def layer(b):
        bnn.bnn_route(b["l"], b["idx"], b["w"], offsets=b["off"], row_token=b["tok"], slot_row=b["slot"])
        bnn.bnn_fp8_pack(b["x"], b["codes"], b["scales"], row_index=b["tok"])
        bnn.bnn_fp8_gemm_grouped(b["codes"], b["scales"], b["off"], W, sw, D, b["Y"])
        bnn.bnn_route_combine(b["Y"], b["slot"], b["w"], b["out"])

    one, two = buffers(), buffers()
    def fill(b, seed):
        b["x"].copy_(draw(T, D, seed, "bf16", 1.0))
        b["l"].copy_(draw(T, E, seed + 1))
    fill(one, 1)
    layer(one)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(one)
    for seed in (5, 9, 13):
        fill(one, seed)
        fill(two, seed)
        graph.replay()
        layer(two)
        torch.cuda.synchronize()
        for name in ("idx", "w", "off", "tok", "slot", "out"):
            assert torch.equal(one[name], two[name]), name
    assert_no_device_error()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("scale", [1e-6, 1e-3, 30.0])
@pytest.mark.parametrize("groups", [1, 8])
def test_route_crowded_and_spread_logits(score, scale, groups):
    """Logits so near that many tokens are decided beyond fp32, and so far apart that scores saturate."""
    l = draw(200, 128, 3) * scale
    bias = draw(1, 128, 4, std=1e-7)[0]
    check(l, 8, score, n_groups=groups, kept_groups=max(1, groups // 2))
    check(l, 8, score, bias=bias, n_groups=groups, kept_groups=max(1, groups // 2))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("E,G", [(128, 8), (64, 16), (40, 4), (256, 8)])
def test_route_groups_near_the_border(score, top, E, G):
    """Groups whose two best experts are clear of the rest, and whose scores are a few steps of fp32 apart."""
    T, per = 120, E // G
    l = (draw(T, E, 11) * 0.2 - 3.0).reshape(T, G, per)
    step = torch.randint(-3, 4, (T, G, 2), generator=torch.Generator().manual_seed(5)) * 2.0 ** -22
    at = torch.argsort(torch.rand(T, G, per, generator=torch.Generator().manual_seed(6)), dim=2)[:, :, :2]
    l.scatter_(2, at, torch.tensor([2.0, 1.0]) + step)
    l[::7, 0] = float("-inf")
    l = l.reshape(T, E)
    check(l, 4, score, n_groups=G, kept_groups=G // 2, group_top=top)
    if score == "sigmoid":
        check(l, 4, score, bias=draw(1, E, 12, std=1e-7)[0], n_groups=G, kept_groups=G // 2, group_top=top)


def test_route_is_the_same_on_every_run_and_stream():
    l = draw(3000, 64, 6)
    first = run(l, 6)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, s, s, None):
        again = run(l, 6, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        assert all(torch.equal(first[2][n], again[2][n]) for n in first[2])


def test_combine_of_no_rows_and_bad_values():
    """R = 0 gives zeros; a slot left out counts for nothing even where its weight is NaN."""
    d = dev()
    out = torch.full((3, 40), 7.0, device=d)
    slot = torch.full((3, 2), -1, dtype=torch.int32, device=d)
    w = torch.full((3, 2), float("nan"), device=d)
    bnn.bnn_route_combine(torch.empty(0, 40, device=d), slot, w, out)
    assert (out == 0).all()
    Y = torch.full((4, 40), float("inf"), device=d)
    Y[2] = 1.5
    slot = torch.tensor([[2, 4], [-1, 2], [2, 2]], dtype=torch.int32, device=d)
    w = torch.tensor([[2.0, float("nan")], [float("inf"), 1.0], [1.0, -1.0]], device=d)
    bnn.bnn_route_combine(Y, slot, w, out)
    assert torch.equal(out[:, 0].cpu(), torch.tensor([3.0, 1.5, 0.0]))


def test_combine_offsets_past_32_bits():
    d = dev()
    far = 1 << 24
    big = torch.zeros(300 * far, dtype=torch.bfloat16, device=d)
    Y = big.as_strided((300, 24), (far, 1))
    Y.copy_(draw(300, 24, 2, "bf16").to(d))
    slot = torch.tensor([[299, 0], [150, 298]], dtype=torch.int32, device=d)
    w = torch.tensor([[0.5, 0.25], [1.0, -2.0]], device=d)
    out = torch.empty(2, 24, device=d)
    bnn.bnn_route_combine(Y, slot, w, out)
    want, mag = ref.route_combine(Y.float().cpu().numpy(), slot.cpu().numpy(), w.cpu().numpy())
    assert (np.abs(out.cpu().numpy() - want) <= 2 * 2.0 ** -24 * mag + 2.0 ** -24 * np.abs(want)).all()
