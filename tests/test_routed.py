"""The operators whose weight depends on the row (awq_route_experts,
awq_w4a16_experts_up / _down, awq_lora_add) against float64, and what they
refuse."""
import ctypes
import math
import types

import numpy as np
import pytest
import torch

import oracle as O
from tests.gpu_util import f32, gpu

awq = pytest.importorskip("weight_only_int4_stats_amd")
E = awq._abi

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture
def on_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    awq.lib()


# ---- tolerances ----------------------------------------------------------------
# One output rounding is at most eps / 2 of the value (half the smallest
# subnormal near 0).  A matrix-core sum of n products that are exact in fp32 is
# off by at most n units of 2^-23 of the sum of their sizes (each addition is
# within one unit of the running size, whatever its rounding).


def rounding(ref, dtype):
    i = torch.finfo(dtype)
    return np.abs(ref) * (i.eps / 2) + (i.tiny * i.eps / 2 if dtype != torch.bfloat16 else i.tiny)


def check(got, ref, slack, dtype, what=""):
    """|got - ref| <= slack (what the computation may be off) + the rounding of
    a value that far from ref."""
    got = f32(got).astype(np.float64)
    bound = slack + rounding(np.abs(ref) + slack, dtype)
    off = np.abs(got - ref)
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(np.max(off / np.maximum(bound, 1e-300))),
                           np.argwhere(bad)[:5].tolist())


def product_slack(size, K, g):
    """z = sum over groups of step (sum q x - z sum x): each group's sums have g
    terms plus its start, the groups are added in fp32; five roundings per
    group beside (the sum of x, its product with z, the step's and the row
    scale's products, the addition)."""
    return size * (g + K // g + 13) * 2.0 ** -23


# ---- routing ---------------------------------------------------------------------


def route_case(T, n, dtype, seed, spread=1.5, levels=0):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, spread, (T, n))
    if levels:                                       # few different values: ties everywhere
        x = np.round(x * levels) / levels
    return torch.from_numpy(x).to(dtype)


ROUTES = [
    # T, E, top_k, n_group, topk_group, group_top, sigmoid, bias, renormalize, scale, dtype, tie levels
    (1, 1, 1, 1, 1, 1, False, False, True, 1.0, "f32", 0),
    (1, 64, 8, 1, 1, 1, False, False, True, 1.0, "bf16", 0),
    (5, 3, 2, 1, 1, 1, True, True, False, 1.5, "f16", 0),
    (257, 60, 4, 1, 1, 1, False, True, False, 1.0, "f32", 0),
    (33, 64, 64, 1, 1, 1, True, False, True, 1.0, "bf16", 2),
    (70, 65, 7, 1, 1, 1, False, False, True, 1.0, "f16", 1),
    (130, 128, 6, 4, 2, 1, False, False, False, 16.0, "bf16", 4),
    (130, 256, 8, 8, 4, 2, True, True, True, 2.5, "bf16", 0),
    (67, 256, 8, 8, 4, 2, True, False, True, 2.5, "f32", 2),
    (19, 96, 5, 32, 3, 2, False, True, True, 1.0, "f32", 0),     # groups of 3
    (23, 160, 16, 8, 3, 2, False, True, True, 1.0, "f16", 3),    # groups of 20 over lanes of 4
    (9, 64, 3, 64, 9, 2, True, True, False, 1.0, "f32", 0),      # groups of 1
    (11, 512, 33, 2, 1, 2, False, False, True, 1.0, "bf16", 0),
    (7, 1000, 50, 1, 1, 1, True, True, True, 1.0, "f32", 0),
    (6, 1024, 64, 64, 8, 2, False, True, True, 1.0, "bf16", 0),
]


def compare_route(got, ref, what):
    ids, weights = got[0].cpu().numpy(), got[1].cpu().numpy().astype(np.float64)
    assert np.array_equal(ids, ref[0]), (what, np.argwhere(ids != ref[0])[:5].tolist())
    # formed in double, rounded once to float
    assert np.all(np.abs(weights - ref[1]) <= np.abs(ref[1]) * (2.0 ** -24 + 1e-12) + 2.0 ** -150), what


@pytest.mark.gpu
@pytest.mark.parametrize("case", ROUTES, ids=lambda c: "x".join(str(v) for v in c[:6]))
def test_route(on_gpu, case):
    T, n, k, ng, tg, gt, sig, with_bias, renorm, scale, dt, levels = case
    x = route_case(T, n, DTYPES[dt], n + T, levels=levels)
    bias = np.random.default_rng(n).normal(0, 0.05, n).astype(np.float32) if with_bias else None
    got = awq.awq_route_experts(gpu(x), k, bias=None if bias is None else gpu(torch.from_numpy(bias)),
                                score="sigmoid" if sig else "softmax", n_group=ng, topk_group=tg, group_top=gt,
                                renormalize=renorm, scale=scale)
    ref = O.route_experts(f32(x), k, bias, sig, ng, tg, gt, renorm, scale)
    compare_route(got, ref, case)


@pytest.mark.gpu
@pytest.mark.parametrize("sig", [False, True])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("groups", [(1, 1), (4, 2), (4, 4)])
def test_route_masked_and_extreme_logits(on_gpu, sig, dt, groups):
    """Rows of -inf, of NaN, with fewer usable experts than top_k, masked by the
    type's lowest value, with +inf, and far apart."""
    dtype = DTYPES[dt]
    x = route_case(12, 48, dtype, 5)
    low = torch.finfo(dtype).min
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 3:] = -math.inf
    x[3] = low
    x[4, :45] = low
    x[5, 7] = math.inf
    x[6, 11], x[6, 29] = math.inf, math.inf
    x[7] = 60 * torch.arange(48).to(dtype)
    x[8, ::2] = math.nan
    x[9, 12:] = -math.inf                            # with groups: only the first has anyone
    bias = torch.linspace(-0.1, 0.1, 48)
    for b in (None, bias):
        got = awq.awq_route_experts(gpu(x), 6, bias=None if b is None else gpu(b), score="sigmoid" if sig else "softmax",
                                    n_group=groups[0], topk_group=groups[1], group_top=2)
        ref = O.route_experts(f32(x), 6, None if b is None else b.numpy(), sig, groups[0], groups[1], 2)
        compare_route(got, ref, (sig, dt, groups, b is not None))


@pytest.mark.gpu
def test_route_close_choices(on_gpu):
    """Choices one double step apart in the scores but equal as floats keep
    their order, and exact ties go to the lowest index."""
    x = torch.zeros(64, 128)
    for t in range(64):
        x[t, 100 - t] = 2.0 ** -22                   # score differs by about 2e-9
        x[t, 20] = 2.0 ** -22 if t % 2 else 0.0
    got = awq.awq_route_experts(gpu(x), 4)
    compare_route(got, O.route_experts(x.numpy(), 4), "close")


@pytest.mark.gpu
@pytest.mark.parametrize("sig", [False, True])
@pytest.mark.parametrize("n", [24, 256, 600])
def test_route_close_choices_under_a_bias(on_gpu, sig, n):
    """Biases that bring choices within a few double steps of each other, and
    groups whose values meet."""
    rng = np.random.default_rng(n)
    x = np.round(rng.normal(0, 1, (80, n)) * 4) / 4
    x[:, n // 2:] = x[:, :n // 2]                    # the second half of the groups repeats the first
    ref = O.route_experts(x, n, None, sig, renormalize=False)
    score = np.zeros((80, n))
    np.put_along_axis(score, ref[0], ref[1], axis=1)
    # pulls the experts of row 0 to one choice, up to the bias's own rounding
    bias = (0.5 - score[0]).astype(np.float32)
    xt = torch.from_numpy(x).float()
    for ng, tg, gt in ((1, 1, 1), (4, 2, 2), (n // 3, n // 6, 1) if n // 3 <= 64 else (8, 3, 1)):
        got = awq.awq_route_experts(gpu(xt), 5, bias=gpu(torch.from_numpy(bias)), score="sigmoid" if sig else "softmax",
                                    n_group=ng, topk_group=tg, group_top=gt)
        compare_route(got, O.route_experts(x, 5, bias, sig, ng, tg, gt), (sig, n, ng))
        got = awq.awq_route_experts(gpu(xt), 5, score="sigmoid" if sig else "softmax", n_group=ng, topk_group=tg,
                                    group_top=gt)
        compare_route(got, O.route_experts(x, 5, None, sig, ng, tg, gt), (sig, n, ng, "no bias"))


@pytest.mark.gpu
@pytest.mark.parametrize("sig", [False, True])
@pytest.mark.parametrize("size", [10.0, 1e3, 1e4, 1e6])
@pytest.mark.parametrize("n,groups", [(4, (2, 1)), (64, (8, 3)), (96, (32, 9)), (256, (8, 4)), (1000, (4, 1))])
def test_route_groups_whose_two_choices_cancel(on_gpu, sig, size, n, groups):
    """A group's two choices of opposite sign leave a worth far below either, so
    that what float loses of each choice decides."""
    n_group, topk_group = groups
    x = route_case(3000 if n <= 256 else 200, n, torch.float32, n, spread=0.5)
    bias = np.full(n, -2 * size, np.float32)
    bias[::n // n_group], bias[1::n // n_group] = size, -size   # the two largest of a group, the others far below
    got = awq.awq_route_experts(gpu(x), 1, bias=gpu(torch.from_numpy(bias)), score="sigmoid" if sig else "softmax",
                                n_group=n_group, topk_group=topk_group, group_top=2)
    compare_route(got, O.route_experts(f32(x), 1, bias, sig, n_group, topk_group, 2), (sig, size, n))


@pytest.mark.gpu
def test_route_group_lost_by_float(on_gpu):
    """Worths 1.00088 and 1.00054, in float 1.0 and 1.000977."""
    x = torch.tensor([[0.0017578, 0.0017578, 0.0021484, 0.0]])
    bias = np.array([1e4, -1e4, 1e4, -1e4], np.float32)
    got = awq.awq_route_experts(gpu(x), 1, bias=gpu(torch.from_numpy(bias)), score="sigmoid", n_group=2, topk_group=1,
                                group_top=2)
    ref = O.route_experts(f32(x), 1, bias, True, 2, 1, 2)
    assert ref[0][0, 0] == 0
    compare_route(got, ref, "cancelling")


@pytest.mark.gpu
@pytest.mark.parametrize("groups", [(1, 1), (4, 2), (4, 1)])
@pytest.mark.parametrize("top_k", [1, 5, 12])
def test_route_sigmoid_near_saturation(on_gpu, groups, top_k):
    """Logits of 20 to 40 whose sigmoids meet in double though the logits differ:
    the lowest index wins wherever they are equal."""
    rng = np.random.default_rng(top_k)
    T, n = 400, 64
    start = rng.uniform(20, 40, (T, 1))
    x = start + np.cumsum(10.0 ** rng.uniform(-4, -2.5, (T, n)), axis=1)   # the larger logit at the higher index
    x[::4] = x[::4, ::-1]
    x[1::4, 32:] -= 60                               # half of the experts far down
    xt = torch.from_numpy(x).float()
    ref = O.route_experts(f32(xt), top_k, None, True, *groups, 1)
    got = awq.awq_route_experts(gpu(xt), top_k, score="sigmoid", n_group=groups[0], topk_group=groups[1])
    compare_route(got, ref, groups)


@pytest.mark.gpu
@pytest.mark.parametrize("sig", [False, True])
@pytest.mark.parametrize("groups", [(1, 1, 1), (4, 2, 1), (4, 2, 2), (12, 5, 2)])
def test_route_bias_switches_experts_off(on_gpu, sig, groups):
    """A bias of -inf: never chosen, in a group worth less for it, whole groups off."""
    n_group, topk_group, group_top = groups
    x = route_case(40, 48, torch.float32, 8)
    bias = np.random.default_rng(3).normal(0, 0.05, 48).astype(np.float32)
    bias[::3] = -np.inf
    bias[13:36] = -np.inf
    for b in (bias, np.full(48, -np.inf, np.float32)):
        got = awq.awq_route_experts(gpu(x), 8, bias=gpu(torch.from_numpy(b)), score="sigmoid" if sig else "softmax",
                                    n_group=n_group, topk_group=topk_group, group_top=group_top)
        ref = O.route_experts(f32(x), 8, b, sig, n_group, topk_group, group_top)
        assert not np.isin(ref[0], np.nonzero(~np.isfinite(b))[0]).any()
        compare_route(got, ref, groups)


@pytest.mark.gpu
def test_route_strided_rows_and_given_outputs(on_gpu):
    big = route_case(40, 100, torch.bfloat16, 9)
    x = gpu(big)[:, 10:74]
    ids = torch.full((42, 5), 77, dtype=torch.int32, device="cuda")
    w = torch.full((42, 5), 7.0, device="cuda")
    awq.awq_route_experts(x, 5, ids=ids[1:41], weights=w[1:41])
    compare_route((ids[1:41], w[1:41]), O.route_experts(f32(big)[:, 10:74], 5), "strided")
    assert (ids[0] == 77).all() and (ids[41] == 77).all() and (w[0] == 7).all() and (w[41] == 7).all()
    i0, w0 = awq.awq_route_experts(x[:0], 5)
    assert i0.shape == (0, 5) and w0.shape == (0, 5)


# ---- the routed products -------------------------------------------------------------


def stack(n_exp, N, K, g, seed):
    rng = np.random.default_rng(seed)
    words = rng.integers(-2 ** 31, 2 ** 31, (n_exp, N, K // 8), dtype=np.int64).astype(np.int32)
    step = rng.uniform(2e-4, 4e-3, (n_exp, N, K // g)).astype(np.float16)
    zero = rng.integers(0, 16, (n_exp, N, K // g)).astype(np.uint8)
    return words, step, zero


def acts(rows, K, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 1, (rows, K)) * np.where(rng.random(K) < 0.02, 20.0, 1.0)
    return torch.from_numpy(x).to(dtype)


def packed(w):
    return tuple(gpu(torch.from_numpy(t)) for t in w)


def choices(T, n_exp, k, seed, kind):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(n_exp)[:k] for _ in range(T)]).astype(np.int32)
    if kind == "one":                                # every slot one expert
        ids[:] = n_exp - 1
    if kind == "holes":
        ids[rng.random(ids.shape) < 0.3] = -1
        ids[T // 2] = [-1, n_exp, 2 ** 31 - 1, -2 ** 31][T % 4]
    if kind == "none":
        ids[:] = -7
    if kind == "twice":                              # a token's choices all one expert
        ids[:] = ids[:, :1]
    return ids


def check_up(x, ids, w, g, act, out, y, what):
    k = ids.shape[1]
    K = x.shape[1]
    z, size = O.expert_rows(np.repeat(f32(x), k, axis=0), ids.reshape(-1), *w)
    slack = product_slack(size, K, g)
    if act == "swiglu":
        n = z.shape[1] // 2
        ref = O.swiglu(z)
        gate, up = np.abs(z[:, :n]), np.abs(z[:, n:])
        dg, du = slack[:, :n], slack[:, n:]
        # |silu'| <= 1.1, silu <= |gate|; exp, the sum, the division and the product: under 8 roundings
        slack = 1.1 * dg * (up + du) + gate * du + 8 * 2.0 ** -24 * np.abs(ref)
        z = ref
    check(y, z, slack, out, what)


def check_down(x, ids, weights, w, g, out, y, what):
    T, k = ids.shape
    K = x.shape[1]
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < w[0].shape[0])
    xx = np.where(ok[:, None], f32(x), 0.0)
    z, size = O.expert_rows(xx, flat, *w)
    wt = np.where(ok, weights.reshape(-1).astype(np.float64), 0.0)[:, None]
    ref = (z * wt).reshape(T, k, -1).sum(1)
    # each term's own error, and k additions (and products) of the terms' sizes
    slack = (product_slack(size, K, g) * np.abs(wt)).reshape(T, k, -1).sum(1)
    terms = np.abs(z * wt).reshape(T, k, -1).sum(1)
    slack += (k + 1) * 2.0 ** -23 * terms
    if out == torch.bfloat16:                        # terms kept in fp16 (one rounding of 2^-11 each)
        slack += 2.0 ** -11 * (terms + slack)
    check(y, ref, slack, out, what)


PRODUCTS = [
    # T, experts, top_k, K, N, group, x type, y type, choices
    (1, 1, 1, 64, 2, 64, "f16", "f32", ""),
    (1, 8, 2, 128, 16, 128, "bf16", "bf16", ""),
    (1, 64, 8, 512, 130, 128, "f16", "f16", ""),
    (2, 5, 3, 192, 66, 64, "bf16", "f32", "holes"),
    (2, 40, 9, 2176, 70, 64, "bf16", "f32", "holes"),
    (1, 20, 1, 4160, 34, 64, "f16", "f32", ""),
    (4, 30, 3, 1792, 50, 256, "bf16", "f16", "holes"),
    (3, 64, 8, 1920, 47 * 2, 128, "f16", "f32", "holes"),
    (1, 12, 5, 3968, 18, 128, "bf16", "f32", "none"),
    (3, 4, 4, 256, 200, 256, "f16", "f32", "holes"),
    (7, 3, 2, 384, 62, 128, "bf16", "f16", "holes"),
    (40, 2, 1, 1152, 34, 128, "bf16", "f32", "one"),
    (17, 16, 1, 2176, 18, 64, "f16", "f32", "one"),
    (33, 7, 3, 2304, 66, 256, "bf16", "bf16", "holes"),
    (50, 6, 2, 4224, 32, 128, "f16", "f32", ""),
    (3, 2, 2, 320, 64, 64, "f16", "bf16", "none"),
    (150, 4, 2, 320, 258, 64, "bf16", "f32", "holes"),
    (300, 8, 2, 256, 130, 128, "f16", "f16", "holes"),
    (700, 3, 2, 512, 390, 256, "bf16", "f32", ""),
    (260, 2, 2, 128, 514, 128, "f16", "f32", "one"),
    (1030, 16, 8, 192, 70, 64, "bf16", "bf16", "holes"),
    (40, 9, 2, 2176, 34, 128, "bf16", "f32", "holes"),
    (2, 32, 4, 512, 50, 128, "f16", "f32", "twice"),
    (9, 20, 4, 512, 50, 128, "f16", "f32", "twice"),
    (200, 5, 4, 256, 130, 128, "bf16", "f32", "twice"),
    (5, 40, 40, 576, 70, 64, "bf16", "f32", ""),
    (3001, 5, 3, 128, 66, 128, "f16", "f32", "holes"),
    (4099, 3, 2, 64, 18, 64, "bf16", "f32", "one"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("case", PRODUCTS, ids=lambda c: "x".join(str(v) for v in c))
def test_experts_up(on_gpu, case, act):
    T, n_exp, k, K, N, g, xdt, ydt, kind = case
    w = stack(n_exp, N, K, g, T + K)
    x = acts(T, K, DTYPES[xdt], N)
    ids = choices(T, n_exp, k, T * N, kind)
    y = awq.awq_w4a16_experts_up(gpu(x), gpu(torch.from_numpy(ids)), *packed(w), act=act, out_dtype=DTYPES[ydt],
                                 group_size=g)
    check_up(x, ids, w, g, act, DTYPES[ydt], y, case)


@pytest.mark.gpu
@pytest.mark.parametrize("case", PRODUCTS, ids=lambda c: "x".join(str(v) for v in c))
def test_experts_down(on_gpu, case):
    T, n_exp, k, K, N, g, xdt, ydt, kind = case
    N += N // 2 % 2                                  # odd numbers of outputs among them
    w = stack(n_exp, N, K, g, T + K)
    x = acts(T * k, K, DTYPES[xdt], N)
    ids = choices(T, n_exp, k, T * N, kind)
    weights = np.random.default_rng(T).uniform(-0.2, 1.0, (T, k)).astype(np.float32)
    gone = (ids.reshape(-1) < 0) | (ids.reshape(-1) >= n_exp)
    x[torch.from_numpy(gone)] = math.nan             # rows without an expert are not read into the result
    weights.reshape(-1)[gone] = np.nan
    y = awq.awq_w4a16_experts_down(gpu(x), gpu(torch.from_numpy(ids)), gpu(torch.from_numpy(weights)), *packed(w),
                                   out_dtype=DTYPES[ydt], group_size=g)
    check_down(x, ids, weights, w, g, DTYPES[ydt], y, case)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [
    # rows dealt to many blocks, an even share each or all on one expert
    (900, 2, 1, 192, 130, 64, "f16", "f32", "one"),
    (2000, 30, 2, 384, 34, 128, "bf16", "f32", "one"),
    (1500, 5, 2, 256, 18, 256, "f16", "bf16", "holes"),
    # tiles of 64 rows and of 128 rows
    (1100, 3, 2, 64, 4000, 64, "bf16", "f32", "holes"),
    (6500, 5, 2, 64, 4098, 64, "f16", "bf16", "holes"),
    # as many experts as there may be: few rows, and sorted in chunks for tiles
    (800, 1024, 3, 64, 18, 64, "f16", "f32", "holes"),
    (400, 1024, 20, 64, 18, 64, "bf16", "f32", "holes"),
    # more experts than slots, all on one
    (150, 300, 1, 192, 34, 64, "f16", "f32", "one"),
], ids=lambda c: "x".join(str(v) for v in c))
def test_experts_dealt_rows_and_tall_tiles(on_gpu, case):
    test_experts_up(on_gpu, case, "none")
    test_experts_up(on_gpu, case, "swiglu")
    test_experts_down(on_gpu, case)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [
    # one token; few rows; tiles of 32, 64 and 128 rows
    (1, 16, 2, 512, 96, 128, "bf16", "f32", ""),
    (20, 6, 2, 512, 96, 64, "f16", "f32", "holes"),
    (1500, 3, 3, 384, 96, 128, "f16", "f32", "holes"),
    (1100, 3, 2, 128, 4000, 64, "bf16", "f32", "holes"),
    (6500, 5, 2, 128, 4096, 128, "f16", "f32", "holes"),
], ids=lambda c: "x".join(str(v) for v in c))
def test_experts_steps_of_any_sign(on_gpu, case):
    """Steps of zero (some groups, whole rows), below zero, the smallest and far
    apart, and one that is not a number; activations that are not finite stay
    in their rows."""
    T, n_exp, k, K, N, g, xdt, ydt, kind = case
    q, step, zero = stack(n_exp, N, K, g, T + K)
    rng = np.random.default_rng(K)
    step[:, 0::8] *= rng.choice([-1, 1], step[:, 0::8].shape).astype(np.float16)
    step[:, 1::8] *= rng.integers(0, 2, step[:, 1::8].shape).astype(np.float16)
    step[:, 2::8] = 0
    step[:, 3::8] = 2.0 ** -24
    step[:, 4::8, ::2] = 2.0 ** -24
    step[:, 5::8, -1] = 0
    w = (q, step, zero)
    x = acts(T, K, DTYPES[xdt], N)
    ids = choices(T, n_exp, k, T * N, kind)
    p = packed(w)
    gi = gpu(torch.from_numpy(ids))
    y = awq.awq_w4a16_experts_up(gpu(x), gi, *p, out_dtype=DTYPES[ydt], group_size=g)
    check_up(x, ids, w, g, "none", DTYPES[ydt], y, case)
    h = acts(T * k, K, DTYPES[xdt], N)
    weights = rng.uniform(-0.2, 1.0, (T, k)).astype(np.float32)
    gw = gpu(torch.from_numpy(weights))
    d = awq.awq_w4a16_experts_down(gpu(h), gi, gw, *p, out_dtype=DTYPES[ydt], group_size=g)
    check_down(h, ids, weights, w, g, DTYPES[ydt], d, case)
    # one step that is not a number: its column, of its expert's slots
    p[1][n_exp - 1, 7, 0] = math.nan
    ok = (ids.reshape(-1) >= 0) & (ids.reshape(-1) < n_exp)
    hit = torch.from_numpy(ids.reshape(-1) == n_exp - 1)
    want = torch.zeros((T * k, N), dtype=torch.bool)
    want[hit, 7] = True
    got = awq.awq_w4a16_experts_up(gpu(x), gi, *p, out_dtype=DTYPES[ydt], group_size=g)
    assert torch.equal(got.view(T * k, N).isnan().cpu(), want)
    assert torch.equal(got.view(T * k, N).cpu()[~want], y.view(T * k, N).cpu()[~want])
    got = awq.awq_w4a16_experts_down(gpu(h), gi, gw, *p, out_dtype=DTYPES[ydt], group_size=g)
    assert torch.equal(got.isnan().cpu(), want.view(T, k, N).any(1))
    # rows that are not finite (no step of zero: 0 inf is not a number)
    p[1].copy_(gpu(torch.from_numpy(np.where(step == 0, np.float16(1e-3), step))))
    y = awq.awq_w4a16_experts_up(gpu(x), gi, *p, out_dtype=DTYPES[ydt], group_size=g).view(T, k, N)
    x[T // 3, 5], x[T // 2, 6] = math.inf, math.nan
    got = awq.awq_w4a16_experts_up(gpu(x), gi, *p, out_dtype=DTYPES[ydt], group_size=g).view(T, k, N)
    rows = torch.zeros(T, dtype=torch.bool)
    rows[[T // 3, T // 2]] = True
    assert torch.equal(got[gpu(~rows)], y[gpu(~rows)])
    assert not got[gpu(rows)].isfinite()[torch.from_numpy(ok).view(T, k)[rows].cuda()].any()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 8, 600])
def test_experts_infinite_step_stays_in_its_column(on_gpu, T):
    n_exp, k, K, N, g = 4, 2, 256, 1100, 128
    w = stack(n_exp, N, K, g, T)
    x = acts(T * k, K, torch.bfloat16, 2) * 8        # products past 4
    ids = choices(T, n_exp, k, 1, "")
    weights = np.random.default_rng(T).uniform(0.5, 1.0, (T, k)).astype(np.float32)
    p = packed(w)
    p[1][:, 7] = math.inf
    y = awq.awq_w4a16_experts_down(gpu(x), gpu(torch.from_numpy(ids)), gpu(torch.from_numpy(weights)), *p,
                                   out_dtype=torch.bfloat16, group_size=g).cpu()
    assert not y[:, 7].isfinite().any()
    w[1][:, 7] = 0
    y[:, 7] = 0
    check_down(x, ids, weights, w, g, torch.bfloat16, y, T)


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("xdt", ["f16", "bf16"])
@pytest.mark.parametrize("T,g", [(1, 128), (40, 64), (1500, 64), (1500, 128), (3000, 256)])
def test_down_terms_that_cancel(on_gpu, T, g, xdt, out):
    """Whole numbers, so that every sum is exact in fp32: two rows that differ in
    one channel, through one expert with weights 1 and -1, leave that
    channel's weight exactly."""
    n_exp, K, N = 3 if T > 1 else 16, 256, 203
    rng = np.random.default_rng(T + g)
    q = rng.integers(-2 ** 31, 2 ** 31, (n_exp, N, K // 8), dtype=np.int64).astype(np.int32)
    step, zero = np.ones((n_exp, N, K // g), np.float16), np.full((n_exp, N, K // g), 8, np.uint8)
    one = rng.integers(-127, 127, (T, 1, K)).astype(np.float32)
    x = np.repeat(one, 2, axis=1)
    at = rng.integers(0, K, T)
    x[np.arange(T), 0, at] += 1
    ids = np.repeat(rng.integers(0, n_exp, (T, 1)), 2, axis=1).astype(np.int32)
    weights = np.tile(np.array([[1.0, -1.0]], np.float32), (T, 1))
    y = awq.awq_w4a16_experts_down(gpu(torch.from_numpy(x.reshape(2 * T, K)).to(DTYPES[xdt])), gpu(torch.from_numpy(ids)),
                                   gpu(torch.from_numpy(weights)), *packed((q, step, zero)), out_dtype=DTYPES[out],
                                   group_size=g)
    codes = np.stack([O.unpack_codes(q[e]) for e in range(n_exp)]).astype(np.float64) - 8
    assert np.array_equal(f32(y).astype(np.float64), codes[ids[:, 0], :, at])


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("N", [201, 257, 258, 259])
def test_down_small_outputs_beside_a_huge_step(on_gpu, N, out):
    """The first column's step is the largest there is, the others' the smallest:
    what the tiles hold past the last column takes no part."""
    T, n_exp, k, K, g = 1500, 3, 2, 256, 128
    q, step, zero = stack(n_exp, N, K, g, N)
    step[:] = 2.0 ** -24
    step[:, :1] = 65504.0
    zero[:] = 15
    x = acts(T * k, K, torch.bfloat16, 3)
    ids = choices(T, n_exp, k, 4, "holes")
    weights = np.random.default_rng(T).uniform(0.5, 1.0, (T, k)).astype(np.float32)
    if out == "f16":                                 # within its range
        step[:, :1] = 2.0 ** -10
    y = awq.awq_w4a16_experts_down(gpu(x), gpu(torch.from_numpy(ids)), gpu(torch.from_numpy(weights)),
                                   *packed((q, step, zero)), out_dtype=DTYPES[out], group_size=g)
    check_down(x, ids, weights, (q, step, zero), g, DTYPES[out], y, N)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,g", [(1500, 256, 64), (1500, 8192, 64), (6500, 2048, 128), (1500, 2048, 256)])
def test_one_step_for_all_of_a_row(on_gpu, T, K, g):
    """Rows whose groups share one step, of whole-number sums: the step enters
    with one rounding, however many groups there are."""
    n_exp, k, N = 3, 1 if T < 2000 else 2, 400
    rng = np.random.default_rng(K)
    q = rng.integers(-2 ** 31, 2 ** 31, (n_exp, N, K // 8), dtype=np.int64).astype(np.int32)
    step = np.repeat(rng.uniform(2e-4, 4e-3, (n_exp, N, 1)).astype(np.float16), K // g, axis=2)
    zero = np.full((n_exp, N, K // g), 8, np.uint8)
    x = rng.integers(-31, 32, (T, K)).astype(np.float32)   # sums below 2^24
    ids = rng.integers(0, n_exp, (T, k)).astype(np.int32)
    y = awq.awq_w4a16_experts_up(gpu(torch.from_numpy(x).half()), gpu(torch.from_numpy(ids)), *packed((q, step, zero)),
                                 out_dtype=torch.float32, group_size=g)
    y = f32(y).reshape(T, k, N)
    for e in range(n_exp):
        z = x.astype(np.float64) @ (O.unpack_codes(q[e]).astype(np.float64) - 8).T * step[e, :, 0].astype(np.float64)
        for j in range(k):
            assert np.array_equal(y[ids[:, j] == e, j], z.astype(np.float32)[ids[:, j] == e]), (e, j)


@pytest.mark.gpu
@pytest.mark.parametrize("T,g", [(30, 128), (1500, 64), (1500, 256)])
@pytest.mark.parametrize("groups", [(0,), (1,), (0, 1), (1, 3), (3,), (2, 3)])
def test_infinite_steps_give_infinity(on_gpu, T, g, groups):
    """One or more groups of a row with an infinite step, of products above 0:
    the row's outputs are infinite, the others what they were."""
    n_exp, K, N = 3, 4 * g, 400
    q, step, zero = stack(n_exp, N, K, g, T + g)
    zero[:] = 0
    q |= 0x11111111
    x = torch.from_numpy(np.random.default_rng(T).uniform(0.5, 2.0, (T, K))).half()
    ids = choices(T, n_exp, 2, T, "")
    p, gi = packed((q, step, zero)), gpu(torch.from_numpy(ids))
    y = f32(awq.awq_w4a16_experts_up(gpu(x), gi, *p, out_dtype=torch.float32, group_size=g))
    for i in groups:
        p[1][:, 5::7, i] = math.inf
    got = f32(awq.awq_w4a16_experts_up(gpu(x), gi, *p, out_dtype=torch.float32, group_size=g))
    y[:, 5::7] = np.inf
    assert np.array_equal(got, y)


@pytest.mark.gpu
@pytest.mark.parametrize("xdt", ["f16", "bf16"])
@pytest.mark.parametrize("T,g", [(1, 128), (1, 64), (30, 128), (30, 64), (1500, 128), (1500, 64), (6500, 256)])
def test_experts_infinite_activations(on_gpu, T, g, xdt):
    """One infinite activation, whose weight is not 0, makes its rows' outputs
    infinite with the sign of the weight's step; the row's other activations
    are large and stay finite."""
    n_exp, k, K, N = 16 if T == 1 else 3, 2, 512, 262
    q, step, zero = stack(n_exp, N, K, g, T + g)
    rng = np.random.default_rng(T)
    step *= rng.choice([-1, 1], step.shape).astype(np.float16)
    zero[:] = 0
    q[:, :, 37 // 8] |= 1 << (4 * (37 % 8))          # the code of channel 37 is not 0
    sign = np.sign(step[:, :, 37 // g].astype(np.float64))
    ids = choices(T, n_exp, k, T, "")
    p, gi = packed((q, step, zero)), gpu(torch.from_numpy(ids))
    x = acts(T, K, DTYPES[xdt], 6) * 50
    hit = rng.random(T) < 0.2
    hit[0] = True
    x[torch.from_numpy(hit), 37] = math.inf
    y = f32(awq.awq_w4a16_experts_up(gpu(x), gi, *p, out_dtype=torch.float32, group_size=g)).reshape(T, k, N)
    assert np.array_equal(y[hit], sign[ids[hit]] * np.inf) and np.isfinite(y[~hit]).all()
    # down: one of the token's rows is infinite
    h = acts(T * k, K, DTYPES[xdt], 7) * 50
    h[::k][torch.from_numpy(hit), 37] = -math.inf
    weights = rng.uniform(0.5, 1.0, (T, k)).astype(np.float32)
    for out in ("f32", "bf16"):
        y = f32(awq.awq_w4a16_experts_down(gpu(h), gi, gpu(torch.from_numpy(weights)), *p, out_dtype=DTYPES[out],
                                           group_size=g))
        assert np.array_equal(y[hit], -sign[ids[hit, 0]] * np.inf) and np.isfinite(y[~hit]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 25, 1200])
def test_experts_of_part_of_a_stack(on_gpu, T):
    """Experts 1, 2, ... of a larger stack, whose steps and zero points start
    off 16 bytes, in inputs that are parts of larger ones; rows of tokens that
    have no expert may hold anything."""
    n_exp, k, K, N, g = 9, 2, 192, 35, 64
    w = stack(n_exp, N, K, g, T)
    p = tuple(t[1:] for t in packed(w))
    part = tuple(t[1:] for t in w)
    assert T > 1 or p[2].data_ptr() % 8
    ids = choices(T, n_exp - 1, k, 3, "holes")
    x = acts(T, K, torch.float16, 4)
    lost = ((ids < 0) | (ids >= n_exp - 1)).all(1)
    x[torch.from_numpy(lost)] = math.nan
    gi = gpu(torch.from_numpy(np.concatenate([ids[:1], ids])))[1:]
    y = awq.awq_w4a16_experts_up(gpu(x), gi, *p, out_dtype=torch.float32, group_size=g)
    x[torch.from_numpy(lost)] = 0
    check_up(x, ids, part, g, "none", torch.float32, y, T)
    h = acts(T * k, K, torch.bfloat16, 4)
    weights = np.random.default_rng(T).uniform(0, 1, (T, k)).astype(np.float32)
    d = awq.awq_w4a16_experts_down(gpu(h), gi, gpu(torch.from_numpy(weights)), *p, out_dtype=torch.bfloat16, group_size=g)
    check_down(h, ids, weights, part, g, torch.bfloat16, d, T)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 90, 400])
def test_experts_strides_and_neighbours(on_gpu, T):
    """Padded input and output rows: what lies beside the output stays."""
    n_exp, k, K, N, g = 4, 2, 256, 50, 128
    w = stack(n_exp, N, K, g, 3)
    ids = choices(T, n_exp, k, 8, "holes")
    wide = acts(T * k, K + 24, torch.float16, 4)
    weights = np.random.default_rng(4).uniform(0, 1, (T, k)).astype(np.float32)
    p = packed(w)
    gi = gpu(torch.from_numpy(ids))
    for col in (3, 4):                               # output rows off and on 16 bytes
        big = torch.full((T * k + 2, N + 14), 9.0, device="cuda")
        awq.awq_w4a16_experts_up(gpu(wide)[:T, 8:8 + K], gi, *p, y=big[1:T * k + 1, col:col + N])
        check_up(wide[:T, 8:8 + K], ids, w, g, "none", torch.float32, big[1:T * k + 1, col:col + N], "up")
        big[1:T * k + 1, col:col + N] = 9.0
        assert (big == 9.0).all()
        big = torch.full((T + 2, N + 14), 9.0, dtype=torch.bfloat16, device="cuda")
        awq.awq_w4a16_experts_down(gpu(wide)[:, 8:8 + K], gi, gpu(torch.from_numpy(weights)), *p,
                                   y=big[1:T + 1, col:col + N])
        check_down(wide[:, 8:8 + K], ids, weights, w, g, torch.bfloat16, big[1:T + 1, col:col + N], "down")
        big[1:T + 1, col:col + N] = 9.0
        assert (big == 9.0).all()


@pytest.mark.gpu
def test_experts_empty(on_gpu):
    w = packed(stack(2, 16, 128, 128, 1))
    x = gpu(acts(0, 128, torch.float16, 1))
    ids = torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    assert awq.awq_w4a16_experts_up(x, ids, *w).shape == (0, 16)
    assert awq.awq_w4a16_experts_down(x, ids, torch.zeros((0, 2), device="cuda"), *w).shape == (0, 16)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 30, 600])
def test_moe_layer(on_gpu, T):
    """Routing, both products and a shared expert on weights this library
    packed, one after another; then captured once and replayed on new inputs
    with eager work between."""
    n_exp, k, H, I = 8, 2, 512, 384
    rng = np.random.default_rng(T)
    dev = torch.device("cuda")
    w1 = gpu(torch.from_numpy(rng.normal(0, 0.04, (n_exp * 2 * I, H))).to(torch.float16))
    w2 = gpu(torch.from_numpy(rng.normal(0, 0.04, (n_exp * H, I))).to(torch.float16))
    p1 = tuple(t.view(n_exp, 2 * I, -1) for t in awq.awq_quantize_pack(w1))
    p2 = tuple(t.view(n_exp, H, -1) for t in awq.awq_quantize_pack(w2))
    gate = gpu(torch.from_numpy(rng.normal(0, 0.1, (H, n_exp))).float())
    n1, n2 = (tuple(t.cpu().numpy() for t in p) for p in (p1, p2))

    def layer(x, logits):
        ids, weights = awq.awq_route_experts(logits, k)
        h = awq.awq_w4a16_experts_up(x, ids, *p1, act="swiglu")
        return ids, weights, h, awq.awq_w4a16_experts_down(h, ids, weights, *p2)

    def verify(x, logits, outs, what):
        ids, weights, h, y = outs
        compare_route((ids, weights), O.route_experts(f32(logits), k), what)
        check_up(x, ids.cpu().numpy(), n1, 128, "swiglu", torch.float16, h, what)
        check_down(h, ids.cpu().numpy(), weights.cpu().numpy(), n2, 128, torch.float16, y, what)

    x = gpu(acts(T, H, torch.float16, 2))
    logits = x.float() @ gate
    eager = layer(x, logits)
    verify(x, logits, eager, "eager")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x, logits)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = layer(x, logits)
    for seed in range(3):
        x.copy_(gpu(acts(T, H, torch.float16, 10 + seed)))
        logits.copy_(x.float() @ gate)
        if T > 4:
            logits[T // 2:] = -math.inf              # the rest of the batch is padding now
        again = layer(x, logits)
        torch.cuda.synchronize(dev)
        for o in outs:
            o.fill_(55)
        graph.replay()
        torch.cuda.synchronize(dev)
        for a, b in zip(again, outs):
            assert torch.equal(a, b), seed
    verify(x, logits, outs, "replayed")


# ---- adapters ---------------------------------------------------------------------------


def check_lora(x, adapter, a, b, ranks, scaling, base, out, y, what):
    ref, size_h, size_x = O.lora(f32(x), adapter, f32(a), f32(b), ranks, scaling)
    # the first sum has K terms (and the parts' additions), the second 2 R; the
    # intermediate enters as two 16-bit values: 2^-17 of it for bf16 (half a
    # step each, the second of what the first left), 2^-23 for fp16; with an
    # fp32 output as three in bf16
    slack = size_x * (x.shape[1] + 160) * 2.0 ** -23
    kept = 2.0 ** -23 if out == torch.float32 else 2.0 ** -17
    slack += (size_h + slack) * (kept + (3 * a.shape[1] + 8) * 2.0 ** -23)
    if base is not None:
        ref = ref + f32(base).astype(np.float64)
        slack = slack + 2.0 ** -23 * (np.abs(ref) + slack)
    check(y, ref, slack, out, what)


LORAS = [
    # rows, adapters, R, K, N, type, y type, ranks, scaling, base, adapter choice
    (1, 1, 8, 8, 1, "f16", "f32", False, False, False, "mixed"),
    (1, 8, 16, 512, 70, "bf16", "bf16", False, True, True, "mixed"),
    (2, 3, 24, 136, 65, "f16", "f16", True, True, True, "mixed"),
    (3, 2, 48, 1000, 264, "bf16", "f32", True, True, True, "mixed"),
    (21, 3, 64, 4096, 130, "bf16", "f32", True, True, True, "mixed"),
    (130, 70, 32, 2056, 320, "f16", "f16", True, True, True, "mixed"),
    (48, 40, 128, 600, 192, "bf16", "bf16", True, False, True, "mixed"),
    (300, 12, 16, 4096, 96, "f16", "f32", False, True, True, "runs"),
    (1500, 5, 64, 328, 128, "bf16", "f32", True, True, True, "runs"),
    (700, 6, 200, 192, 320, "f16", "f16", True, True, True, "mixed"),
    (19, 5, 64, 264, 300, "bf16", "f32", True, True, False, "mixed"),
    (64, 32, 40, 1032, 130, "f16", "f32", True, False, True, "mixed"),
    (100, 2, 256, 64, 257, "bf16", "f32", True, True, True, "mixed"),
    (37, 4, 136, 72, 64, "f16", "bf16", False, True, True, "none"),
    (90, 0, 16, 64, 33, "f16", "f32", False, False, True, "mixed"),
    (700, 0, 16, 64, 33, "bf16", "bf16", False, False, False, "mixed"),
    (513, 9, 16, 200, 100, "bf16", "bf16", True, True, True, "mixed"),
    (900, 3, 32, 128, 259, "f16", "f32", True, True, True, "runs"),
    (1100, 600, 8, 64, 40, "f16", "f32", False, False, False, "mixed"),
    (600, 1, 72, 96, 64, "bf16", "f32", False, True, True, "none"),
    (9000, 7, 8, 64, 40, "f16", "f32", True, True, True, "mixed"),
    (5000, 1100, 16, 72, 24, "bf16", "f32", False, True, False, "runs"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", LORAS, ids=lambda c: "x".join(str(v) for v in c))
def test_lora(on_gpu, case):
    M, L, R, K, N, xdt, ydt, with_ranks, with_scaling, with_base, kind = case
    dtype, out = DTYPES[xdt], DTYPES[ydt]
    rng = np.random.default_rng(M + K + N)
    x = acts(M, K, dtype, M)
    a = torch.from_numpy(rng.normal(0, 1 / math.sqrt(K), (L, R, K))).to(dtype)
    b = torch.from_numpy(rng.normal(0, 1, (L, N, R))).to(dtype)
    adapter = rng.integers(-1, L + 1, M).astype(np.int32)
    if kind == "runs":
        adapter = np.sort(adapter)
    if kind == "none":
        adapter[:] = np.where(rng.random(M) < 0.5, -2 ** 31, L)
    ranks = rng.integers(-1, R + 2, L).astype(np.int32) if with_ranks else None
    if with_ranks:                                   # what lies past a rank is not used
        for i, r in enumerate(np.clip(ranks, 0, R)):
            a[i, r:] = math.nan
            b[i, :, r:] = math.inf
    scaling = rng.uniform(-2, 2, L).astype(np.float32) if with_scaling else None
    base = torch.from_numpy(rng.normal(0, 1, (M, N))).to(out) if with_base else None
    t = lambda v: None if v is None else gpu(torch.from_numpy(v))  # noqa: E731
    gb = None if base is None else gpu(base)
    y = awq.awq_lora_add(gpu(x), t(adapter), gpu(a), gpu(b), base=gb, scaling=t(scaling), ranks=t(ranks), out_dtype=out)
    check_lora(x, adapter, a, b, ranks, scaling, base, out, y, case)
    if base is not None:                             # in place
        awq.awq_lora_add(gpu(x), t(adapter), gpu(a), gpu(b), base=gb, scaling=t(scaling), ranks=t(ranks), y=gb)
        assert torch.equal(gb, y)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [40, 600, 5000])
def test_lora_as_many_adapters_as_there_may_be(on_gpu, M):
    test_lora(on_gpu, (M, 8192, 8, 16, 24, "f16", "f32", True, True, True, "mixed"))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [40, 200, 500])
@pytest.mark.parametrize("L", [1, 3, 600])
@pytest.mark.parametrize("one", [True, False])
def test_lora_all_rows_one_adapter(on_gpu, M, L, one):
    """Rows dealt to blocks (few adapters), or 16 from every 16th row's block
    (more adapters than rows), in one launch or two."""
    K, R, N = (256, 16, 70) if one else (2304, 72, 70)
    rng = np.random.default_rng(M + L)
    x = acts(M, K, torch.float16, M)
    a = torch.from_numpy(rng.normal(0, 1 / math.sqrt(K), (L, R, K))).to(torch.float16)
    b = torch.from_numpy(rng.normal(0, 1, (L, N, R))).to(torch.float16)
    adapter = np.full(M, L - 1, np.int32)
    adapter[M // 2:M // 2 + 3] = -1
    base = torch.from_numpy(rng.normal(0, 1, (M, N))).float()
    y = awq.awq_lora_add(gpu(x), gpu(torch.from_numpy(adapter)), gpu(a), gpu(b), base=gpu(base))
    check_lora(x, adapter, a, b, None, None, base, torch.float32, y, (M, L, one))
    adapter[:] = -1                                  # nobody's rows are dealt too
    y = awq.awq_lora_add(gpu(x), gpu(torch.from_numpy(adapter)), gpu(a), gpu(b), base=gpu(base))
    assert torch.equal(y.cpu(), base)


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("xdt", ["f16", "bf16"])
@pytest.mark.parametrize("M,R", [(1, 8), (40, 8), (40, 72), (300, 136), (700, 32), (700, 136)])
def test_lora_keeps_all_of_the_intermediate(on_gpu, M, R, xdt, out):
    """Whole numbers, so that every sum is exact in fp32, and a base that takes
    all but the last bits away: what is left of A x is right to the last bit."""
    K, N, L = 1024, 90, 3
    rng = np.random.default_rng(M + R)
    x = rng.integers(-100, 101, (M, K)).astype(np.float64)
    a = rng.integers(-100, 101, (L, R, K)).astype(np.float64)
    b = rng.integers(-1, 2, (L, N, R)).astype(np.float64)
    adapter = rng.integers(0, L, M).astype(np.int32)
    h = np.einsum("mk,mrk->mr", x, a[adapter])
    delta = np.einsum("mr,mnr->mn", h, b[adapter])
    assert np.abs(h).max() > 2 ** 16 and np.einsum("mr,mnr->mn", np.abs(h), np.abs(b[adapter])).max() < 2 ** 24
    scale = 2.0 ** -8                                # within fp16's range
    base = torch.from_numpy(-delta * scale).to(DTYPES[out])
    t = lambda v: gpu(torch.from_numpy(v).to(DTYPES[xdt]))  # noqa: E731
    y = awq.awq_lora_add(t(x), gpu(torch.from_numpy(adapter)), t(a), t(b), base=gpu(base),
                         scaling=torch.full((L,), scale, device="cuda"))
    want = torch.from_numpy(delta * scale + f32(base).astype(np.float64)).to(DTYPES[out])
    assert np.array_equal(f32(y), f32(want))


@pytest.mark.gpu
@pytest.mark.parametrize("xdt", ["f16", "bf16"])
@pytest.mark.parametrize("M,R", [(1, 8), (40, 24), (40, 72), (300, 136), (700, 32), (700, 136)])
def test_lora_infinite_activations(on_gpu, M, R, xdt):
    """An infinite activation makes A x infinite; B of the same signs makes the
    row's outputs infinite, and no other row's."""
    K, N, L = 264, 90, 3
    rng = np.random.default_rng(M + R)
    x = acts(M, K, DTYPES[xdt], M)
    a = torch.from_numpy(rng.normal(0, 1 / math.sqrt(K), (L, R, K))).to(DTYPES[xdt])
    b = torch.from_numpy(rng.uniform(0.5, 1.0, (L, N, R))).to(DTYPES[xdt])
    b *= torch.where(a[:, :, 100] < 0, -1.0, 1.0).to(b.dtype)[:, None, :]
    assert (a[:, :, 100] != 0).all()
    adapter = rng.integers(0, L, M).astype(np.int32)
    hit = rng.random(M) < 0.2
    hit[0] = True
    x[torch.from_numpy(hit), 100] = math.inf
    for out in (torch.float32, DTYPES[xdt]):
        y = f32(awq.awq_lora_add(gpu(x), gpu(torch.from_numpy(adapter)), gpu(a), gpu(b), out_dtype=out))
        assert (y[hit] == np.inf).all() and np.isfinite(y[~hit]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 20, 640])
def test_lora_strides_and_neighbours(on_gpu, M):
    L, R, K, N = 3, 16, 128, 50
    rng = np.random.default_rng(M)
    wide = acts(M, K + 24, torch.bfloat16, 1)
    a = torch.from_numpy(rng.normal(0, 0.1, (L, R, K))).to(torch.bfloat16)
    b = torch.from_numpy(rng.normal(0, 1, (L, N, R))).to(torch.bfloat16)
    adapter = rng.integers(-1, L, M).astype(np.int32)
    for col in (3, 8):
        base = torch.from_numpy(rng.normal(0, 1, (M, N + 30))).to(torch.bfloat16)
        big = torch.full((M + 2, N + 14), 9.0, dtype=torch.bfloat16, device="cuda")
        awq.awq_lora_add(gpu(wide)[:, 8:8 + K], gpu(torch.from_numpy(adapter)), gpu(a), gpu(b),
                         base=gpu(base)[:, 5:5 + N], y=big[1:M + 1, col:col + N])
        check_lora(wide[:, 8:8 + K], adapter, a, b, None, None, base[:, 5:5 + N], torch.bfloat16,
                   big[1:M + 1, col:col + N], col)
        big[1:M + 1, col:col + N] = 9.0
        assert (big == 9.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 48, 800])
def test_lora_beside_the_shared_product(on_gpu, M):
    """The packed product and the adapters of its rows, eager and captured."""
    N, K, L, R = 384, 512, 5, 16
    rng = np.random.default_rng(M)
    w = gpu(torch.from_numpy(rng.normal(0, 0.04, (N, K))).to(torch.float16))
    q, sc, z = awq.awq_quantize_pack(w)
    x = gpu(acts(M, K, torch.float16, 3))
    a = gpu(torch.from_numpy(rng.normal(0, 0.05, (L, R, K))).to(torch.float16))
    b = gpu(torch.from_numpy(rng.normal(0, 0.3, (L, N, R))).to(torch.float16))
    adapter = gpu(torch.from_numpy(rng.integers(-1, L, M).astype(np.int32)))

    def step():
        y = awq.awq_w4a16_gemm(x, q, sc, z, out_dtype=torch.float32)
        return y, awq.awq_lora_add(x, adapter, a, b, base=y)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in range(3):
        x.copy_(gpu(acts(M, K, torch.float16, 20 + seed)))
        adapter.copy_(torch.from_numpy(rng.integers(-1, L, M).astype(np.int32)))
        again = step()
        torch.cuda.synchronize()
        for o in outs:
            o.fill_(55)
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(again, outs):
            assert torch.equal(u, v), seed
        check_lora(x.cpu(), adapter.cpu().numpy(), a.cpu(), b.cpu(), None, None, again[0].cpu(), torch.float32,
                   again[1], seed)


@pytest.mark.gpu
def test_two_streams_at_once(on_gpu):
    """Calls on two streams with workspaces of their own do not meet."""
    jobs = []
    for i in range(2):
        w = stack(8, 128, 512, 128, i)
        x = acts(300, 512, torch.float16, i)
        ids = choices(300, 8, 2, i, "")
        jobs.append((w, x, ids, packed(w), gpu(x), gpu(torch.from_numpy(ids)), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for w, x, ids, p, gx, gi, st in jobs:
            with torch.cuda.stream(st):
                outs.append(awq.awq_w4a16_experts_up(gx, gi, *p, out_dtype=torch.float32))
    torch.cuda.synchronize()
    for n, y in enumerate(outs):
        w, x, ids = jobs[n % 2][:3]
        check_up(x, ids, w, 128, "none", torch.float32, y, n)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 20, 500])
def test_given_stream_workspace_and_output(on_gpu, T):
    """On a stream handed in, as an object or a handle, with memory handed in
    or made by the call; the memory the caller's own stream gets afterwards is
    not the call's."""
    n_exp, k, K, N = 16, 4, 512, 200
    w = stack(n_exp, N, K, 128, T)
    x = acts(T, K, torch.float16, 5)
    ids = choices(T, n_exp, k, 6, "holes")
    p, gx, gi = packed(w), gpu(x), gpu(torch.from_numpy(ids))
    need = awq.awq_workspace_bytes(awq.AWQ_OP_EXPERTS_UP, T, N, K, n_exp, k)
    own = torch.full((need + 256,), 7, dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    outs = []
    for stream in (st, st.cuda_stream, torch.cuda.default_stream(), 0):
        y = torch.empty((T * k, N), device="cuda")
        torch.cuda.synchronize()
        outs.append(awq.awq_w4a16_experts_up(gx, gi, *p, y=y, ws=own[:need] if need else None, stream=stream))
        torch.cuda.synchronize()
        outs.append(awq.awq_w4a16_experts_up(gx, gi, *p, out_dtype=torch.float32, stream=stream))
        noise = torch.full((need + 1,), 255, dtype=torch.uint8, device="cuda")   # noqa: F841
        torch.cuda.synchronize()
    for y in outs:
        check_up(x, ids, w, 128, "none", torch.float32, y, T)
    assert (own[need:] == 7).all()
    r = awq.awq_route_experts(gx, 3, stream=st)
    lo = awq.awq_lora_add(gx, gi[:, 0].contiguous(), torch.ones(16, 8, K, dtype=torch.float16, device="cuda"),
                          torch.ones(16, 8, 8, dtype=torch.float16, device="cuda"), stream=st)
    torch.cuda.synchronize()
    compare_route(r, O.route_experts(f32(x), 3), "stream")
    assert torch.equal(lo, awq.awq_lora_add(gx, gi[:, 0].contiguous(),
                                            torch.ones(16, 8, K, dtype=torch.float16, device="cuda"),
                                            torch.ones(16, 8, 8, dtype=torch.float16, device="cuda")))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 90, 2500])
def test_same_bits_every_time(on_gpu, T):
    """The order in which rows of one expert or adapter are taken up varies;
    the results do not."""
    w = packed(stack(6, 130, 384, 128, 1))
    x = gpu(acts(T, 384, torch.bfloat16, 2))
    ids = gpu(torch.from_numpy(choices(T, 6, 3, 3, "holes")))
    weights = torch.rand(T, 3, device="cuda")
    h = gpu(acts(T * 3, 384, torch.bfloat16, 4))
    a, b = torch.randn(6, 24, 384, device="cuda").bfloat16(), torch.randn(6, 100, 24, device="cuda").bfloat16()
    first = None
    for _ in range(6):
        outs = [awq.awq_w4a16_experts_up(x, ids, *w, act="swiglu"), awq.awq_w4a16_experts_down(h, ids, weights, *w),
                awq.awq_lora_add(x, ids[:, 0].contiguous(), a, b, out_dtype=torch.float32)]
        if first is None:
            first = outs
        assert all(torch.equal(u, v) for u, v in zip(first, outs))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 12, 300])
def test_experts_past_4_gigabytes(on_gpu, T):
    """The last expert's words lie past 2^32 bytes of the stack."""
    n_exp, N, K, k = 40, 8192, 28672, 2
    q = torch.zeros((n_exp, N, K // 8), dtype=torch.int32, device="cuda")
    sc = torch.zeros((n_exp, N, K // 256), dtype=torch.float16, device="cuda")
    z = torch.zeros((n_exp, N, K // 256), dtype=torch.uint8, device="cuda")
    rows = 96                                        # only these rows of the last expert are not zero
    w = stack(1, rows, K, 256, T)
    for big, part in zip((q, sc, z), packed(w)):
        big[-1, N - rows:] = part[0]
    sc[:-1] = 1.0                                    # the others' codes are zero points
    x = acts(T, K, torch.bfloat16, 8)
    ids = np.tile(np.array([[n_exp - 1, 3]], dtype=np.int32), (T, 1))
    y = awq.awq_w4a16_experts_up(gpu(x), gpu(torch.from_numpy(ids)), q, sc, z, out_dtype=torch.float32, group_size=256)
    assert (y[1::2] == 0).all() and (y[::2, :N - rows] == 0).all()
    check_up(x, np.zeros((T, 1), dtype=np.int32), w, 256, "none", torch.float32, y[::2, N - rows:], T)
    h = acts(T * k, K, torch.bfloat16, 9)
    weights = np.random.default_rng(1).uniform(0, 1, (T, k)).astype(np.float32)
    y = awq.awq_w4a16_experts_down(gpu(h), gpu(torch.from_numpy(ids)), gpu(torch.from_numpy(weights)), q, sc, z,
                                   out_dtype=torch.float32, group_size=256)
    assert (y[:, :N - rows] == 0).all()
    check_down(h[::2], np.zeros((T, 1), dtype=np.int32), weights[:, :1], w, 256, torch.float32, y[:, N - rows:], T)


@pytest.mark.gpu
def test_lora_past_4_gigabytes(on_gpu):
    """Rows of the output, and adapters, past 2^32 bytes."""
    M, N, K, R, L = 70000, 32768, 64, 8, 3
    x = gpu(acts(M, K, torch.bfloat16, 1))
    a, b = torch.randn(L, R, K, device="cuda").bfloat16(), torch.randn(L, N, R, device="cuda").bfloat16()
    adapter = torch.randint(-1, L, (M,), device="cuda", dtype=torch.int32)
    y = torch.full((M, N), 3.0, dtype=torch.bfloat16, device="cuda")
    awq.awq_lora_add(x, adapter, a, b, base=y, y=y)
    at = torch.tensor([0, 1, 32767, 65535, 65536, M - 2, M - 1], device="cuda")
    check_lora(x[at].cpu(), adapter[at].cpu().numpy(), a.cpu(), b.cpu(), None, None,
               torch.full((len(at), N), 3.0, dtype=torch.bfloat16), torch.bfloat16, y[at], "rows")
    del y
    M, N, K, R, L = 40, 16, 65536, 256, 140          # 140 adapters of 32 MiB
    x = gpu(acts(M, K, torch.float16, 2))
    a = torch.zeros((L, R, K), dtype=torch.float16, device="cuda")
    a[-1] = torch.randn(R, K, device="cuda").half() / 256
    b = torch.randn(L, N, R, device="cuda").half()
    adapter = torch.full((M,), L - 1, dtype=torch.int32, device="cuda")
    y = awq.awq_lora_add(x, adapter, a, b, out_dtype=torch.float32)
    check_lora(x[:3].cpu(), np.zeros(3, dtype=np.int32), a[-1:].cpu(), b[-1:].cpu(), None, None, None, torch.float32,
               y[:3], "adapters")


# ---- refusals (no launch, so no GPU) ----------------------------------------------------

A, B, C, D = (ctypes.c_void_p(v << 16) for v in (1, 2, 3, 4))
BAD = ctypes.c_void_p(0x10002)
ODD = ctypes.c_void_p(0x10001)


def test_route_refusals():
    f = awq.lib().awq_route_experts

    def call(**kw):
        a = dict(x=A, dt=0, T=4, E=64, ld=64, bias=None, score=0, ng=8, tg=4, gt=2, k=8, rn=1, sc=1.0, ids=B, w=C)
        a.update(kw)
        return f(a["x"], a["dt"], a["T"], a["E"], a["ld"], a["bias"], a["score"], a["ng"], a["tg"], a["gt"], a["k"],
                 a["rn"], a["sc"], a["ids"], a["w"], None)

    assert call(T=0, x=None) == 0
    assert call(x=None) == 1 and call(ids=None) == 1 and call(w=None) == 1
    for kw in (dict(T=-1), dict(E=0), dict(ld=63), dict(ng=0), dict(ng=7), dict(tg=0), dict(tg=9), dict(gt=0),
               dict(gt=3), dict(k=0), dict(k=33), dict(ng=1, tg=1, k=65)):
        assert call(**kw) == 2, kw
    assert call(dt=3) == 3
    assert call(x=ODD) == 4 and call(dt=2, x=BAD) == 4 and call(ids=BAD) == 4 and call(w=BAD) == 4 and call(bias=BAD) == 4
    assert call(score=2) == 5 and call(E=1032, ld=1032) == 5 and call(E=512, ld=512, ng=128) == 5
    assert call(E=512, ld=512, ng=1, tg=1, k=65) == 5 and call(T=1 << 31) == 5


@pytest.mark.parametrize("down", [False, True])
def test_experts_refusals(down):
    lib = awq.lib()

    def call(**kw):
        a = dict(x=A, dt=0, M=4, K=256, ld=256, ids=B, w=C, k=2, q=A, s=B, z=C, E=8, N=64, g=128, act=1, y=D, ydt=2,
                 ldy=64, ws=D, wsb=1 << 40)
        a.update(kw)
        head = (a["x"], a["dt"], a["M"], a["K"], a["ld"], a["ids"])
        mid = (a["q"], a["s"], a["z"], a["E"], a["N"], a["g"])
        tail = (a["y"], a["ydt"], a["ldy"], a["ws"], a["wsb"], None)
        if down:
            return lib.awq_w4a16_experts_down(*head, a["w"], a["k"], *mid, *tail)
        return lib.awq_w4a16_experts_up(*head, a["k"], *mid, a["act"], *tail)

    assert call(M=0, x=None) == 0 and call(N=0, y=None) == 0
    for name in ("x", "ids", "q", "s", "z", "y") + (("w",) if down else ()):
        assert call(**{name: None}) == 1, name
    for kw in (dict(M=-1), dict(N=-2), dict(E=0), dict(k=0), dict(K=0), dict(K=200, ld=256), dict(ld=128),
               dict(ldy=31)):
        assert call(**kw) == 2, kw
    assert call(dt=2) == 3 and call(ydt=5) == 3
    assert call(x=BAD) == 4 and call(q=BAD) == 4 and call(ids=BAD) == 4 and call(y=BAD) == 4 and call(ld=260) == 4
    assert call(s=ODD) == 4
    assert call(g=32) == 5 and call(E=1025) == 5 and call(k=65) == 5 and call(K=1 << 18, ld=1 << 18) == 5
    assert call(M=1 << 24) == 5                      # more than 2^24 slots
    assert call(N=1 << 24, ldy=1 << 24) == 5         # 2^31 bytes of words per expert
    assert call(M=1 << 22, K=4096, ld=4096, k=1) == 5  # activations past 32-bit offsets
    assert call(M=1 << 23, K=64, ld=64, g=64, N=1 << 16, ldy=1 << 16) == 5   # more threads than a launch has
    op = awq.AWQ_OP_EXPERTS_DOWN if down else awq.AWQ_OP_EXPERTS_UP
    need = awq.awq_workspace_bytes(op, 4000, 64, 256, 8, 2)
    assert need > 0
    big = dict(M=4000)
    assert call(**big, wsb=need - 1) == 6 and call(**big, ws=None) == 6 and call(**big, ws=BAD) == 6
    if down:
        assert call(w=BAD) == 4
    else:
        assert call(N=63) == 2 and call(act=2) == 5 and call(act=0, ldy=63) == 2
    assert awq.awq_workspace_bytes(op, -1, 64, 256, 8, 2) == 0


def test_lora_refusals():
    f = awq.lib().awq_lora_add

    def call(**kw):
        a = dict(x=A, dt=0, M=4, K=256, ld=256, ad=B, a=A, b=B, L=3, R=16, ranks=None, sc=None, base=None, ldb=0,
                 N=64, y=D, ydt=2, ldy=64, ws=D, wsb=1 << 40)
        a.update(kw)
        return f(a["x"], a["dt"], a["M"], a["K"], a["ld"], a["ad"], a["a"], a["b"], a["L"], a["R"], a["ranks"], a["sc"],
                 a["base"], a["ldb"], a["N"], a["y"], a["ydt"], a["ldy"], a["ws"], a["wsb"], None)

    assert call(M=0, x=None) == 0 and call(N=0, y=None) == 0
    for name in ("x", "ad", "a", "b", "y"):
        assert call(**{name: None}) == 1, name
    for kw in (dict(M=-1), dict(N=-1), dict(L=-1), dict(K=0), dict(R=0), dict(ld=128), dict(ldy=63),
               dict(base=A, ldb=63)):
        assert call(**kw) == 2, kw
    assert call(dt=2) == 3 and call(ydt=3) == 3
    for kw in (dict(K=252, ld=256), dict(R=12), dict(ld=260), dict(x=BAD), dict(a=BAD), dict(b=BAD), dict(ad=BAD),
               dict(ranks=BAD), dict(sc=BAD), dict(base=BAD, ldb=64), dict(y=BAD), dict(ydt=0, y=ODD)):
        assert call(**kw) == 4, kw
    assert call(R=264) == 5 and call(L=8193) == 5 and call(L=16385) == 5 and call(M=(1 << 24) + 1) == 5 and call(K=1 << 18, ld=1 << 18) == 5
    assert call(M=1 << 24, N=1 << 16, ldy=1 << 16) == 5  # more threads than a launch has
    big = dict(M=300, N=4096, ldy=4096, K=4096, ld=4096, L=30, R=64)
    need = awq.awq_workspace_bytes(awq.AWQ_OP_LORA, 300, 4096, 4096, 30, 64)
    assert need >= 300 * 64 * 4
    assert call(**big, wsb=need - 1) == 6 and call(**big, ws=None) == 6 and call(**big, ws=BAD) == 6
    assert awq.awq_workspace_bytes(awq.AWQ_OP_LORA, -1, 64, 256, 3, 16) == 0


@pytest.mark.parametrize("M,L", [(512, 1), (500, 0), (512, 40), (600, 2)])
def test_lora_refuses_more_threads_than_a_launch_has(M, L):
    """The most columns whose launch still fits are answered (up to the missing
    workspace), some more refused."""
    def call(N):
        return awq.lib().awq_lora_add(A, 0, M, 4096, 4096, B, A, B, L, 128, None, None, None, 0, N, D, 2, N, None, 0, None)

    # block rows of 256 threads and 256 columns: 16 rows of an adapter each, dealt twice over, or tiles of 64
    rows = (L + 1) * ((M // (L + 1) + 7) // 8) if M <= 512 else M // 64 + L + 1
    most = ((1 << 32) - 1) // (256 * rows) * 256
    if L:
        assert call(most) == 6
    assert call(most + 1) == 5 and call(most + (most >> 3)) == 5 and call(1 << 40) == 5


def test_experts_refuse_more_threads_than_a_launch_has():
    """The constants' layout takes a thread per weight row and eight groups."""
    def call(M, n_exp, K, N):
        return awq.lib().awq_w4a16_experts_up(A, 0, M, K, K, B, 2, A, B, C, n_exp, N, 64, 0, D, 2, N, None, 0, None)

    assert call(4000, 1024, 1024, 2_000_000) == 6    # answered up to the missing workspace
    assert call(4000, 1024, 1024, 3_000_000) == 5


@pytest.mark.parametrize("op,N,K,T,n", [
    ("LORA", 4096, 4096, 6, 64), ("LORA", 11008, 4096, 32, 64), ("LORA", 4096, 14336, 1, 128), ("LORA", 64, 96, 2, 8),
    ("LORA", 300, 131072, 8192, 256), ("LORA", 4096, 4096, 0, 16),
    ("EXPERTS_UP", 4096, 1024, 8, 2), ("EXPERTS_UP", 100, 64, 3, 1), ("EXPERTS_UP", 2048, 2048, 64, 64),
    ("EXPERTS_DOWN", 2049, 1024, 64, 8), ("EXPERTS_DOWN", 4096, 64, 6, 1), ("EXPERTS_DOWN", 30, 8192, 1024, 2),
])
def test_workspace_of_the_largest_batch_serves_all(op, N, K, T, n):
    """A program that makes its workspace once, for the most rows it takes."""
    rows = sorted(set(range(1, 3000)) | set(range(3000, 70000, 37)) | {int(1.1 ** i) for i in range(80, 174)})
    need = [awq.awq_workspace_bytes(getattr(awq._abi, "AWQ_OP_" + op), M, N, K, T, n) for M in rows]
    assert need == sorted(need)


@pytest.mark.parametrize("op", ["EXPERTS_UP", "EXPERTS_DOWN", "LORA"])
def test_workspace_of_sizes_past_the_limits(op):
    """Answers at once, with 0, whatever the sizes; a call with them is refused."""
    most = (1 << 63) - 1
    fine = (40, 64, 128, 8, 8)
    for at, values in enumerate(((most, (1 << 24) + 1), (most,), (most, (1 << 17) + 1), (most, 8193),
                                 ((1 << 31) - 1, 1 << 30, 257))):
        for v in values:
            args = list(fine)
            args[at] = v
            assert awq.awq_workspace_bytes(getattr(awq._abi, "AWQ_OP_" + op), *args) == 0, args


def test_lora_one_launch_only_where_it_reads_little():
    """A call without a workspace forms A x again in every block: not where many
    rows would read A and x a gigabyte over."""
    ws = lambda M, N, K, L, R: awq.awq_workspace_bytes(awq.AWQ_OP_LORA, M, N, K, L, R)  # noqa: E731
    for sizes in ((1, 4096, 4096, 8, 16), (8, 1024, 4096, 8, 16), (32, 4096, 1024, 1, 8), (1, 11008, 1024, 1, 64)):
        assert ws(*sizes) == 0, sizes
    for sizes in ((512, 16384, 4096, 1, 16), (512, 8192, 4096, 1, 32), (400, 4096, 4096, 3, 32), (512, 4096, 1024, 40, 8)):
        assert ws(*sizes) > 0, sizes


def test_outputs_over_inputs_are_refused():
    """Other blocks still read what one writes."""
    at = lambda n: ctypes.c_void_p((1 << 24) + n)  # noqa: E731
    far, far2 = ctypes.c_void_p(1 << 40), ctypes.c_void_p(1 << 41)
    lib = awq.lib()

    def lora(y, base=None, ldb=0, M=4, ldy=512, N=64):
        return lib.awq_lora_add(at(0), 0, M, 256, 512, far, far, far, 2, 16, None, None, base, ldb, N, y, 0, ldy, far, 1 << 40, None)

    def up(y, M=4, ldy=512):
        return lib.awq_w4a16_experts_up(at(0), 0, M, 256, 512, far, 1, far, far, far, 8, 64, 128, 0, y, 0, ldy, far, 1 << 40, None)

    def down(y, M=4, ldy=512):
        return lib.awq_w4a16_experts_down(at(0), 0, M, 256, 512, far, far, 1, far, far, far, 8, 64, 128, y, 0, ldy, far, 1 << 40, None)

    for f in (lora, up, down):
        # x: rows of 512 bytes every 1024; y: rows of 128 bytes
        for n in (0, 510, -126, 1024, 3 * 1024 + 510, -3 * 1024 - 126):
            assert f(at(n)) == 5, (f, n)
        assert f(at(600), ldy=64) == 5 and f(at(400), M=1, ldy=64) == 5
    # base: 64 columns every 512 elements at far2
    over = lambda n: ctypes.c_void_p((1 << 41) + n)  # noqa: E731
    for y, ldy in ((over(2), 512), (over(126), 512), (over(1024), 512), (over(-2), 512), (over(0), 520), (over(0), 64)):
        assert lora(y, far2, 512, ldy=ldy) == 5, (y, ldy)


@pytest.mark.gpu
def test_outputs_between_the_rows_of_inputs(on_gpu):
    """Columns of one buffer beside each other, and the rows before and after."""
    M, K, N, L = 40, 256, 72, 3
    rng = np.random.default_rng(1)
    buf = torch.zeros((M + 20, K + 2 * N + 8), dtype=torch.float16, device="cuda")
    x = acts(M, K, torch.float16, 5)
    xs = buf[10:M + 10, N:N + K]
    xs.copy_(gpu(x))
    w = stack(L, N, K, 128, 2)
    ids = choices(M, L, 1, 3, "")
    gi, weights = gpu(torch.from_numpy(ids)), rng.uniform(0, 1, (M, 1)).astype(np.float32)
    a = torch.from_numpy(rng.normal(0, 0.1, (L, 16, K))).half()
    b = torch.from_numpy(rng.normal(0, 1, (L, N, 16))).half()
    for y in (buf[10:M + 10, :N], buf[10:M + 10, N + K:2 * N + K], buf[:M, :N], buf[20:, N + K + 8:]):
        awq.awq_w4a16_experts_up(xs, gi, *packed(w), y=y)
        check_up(x, ids, w, 128, "none", torch.float16, y, "up")
        awq.awq_w4a16_experts_down(xs, gi, gpu(torch.from_numpy(weights)), *packed(w), y=y)
        check_down(x, ids, weights, w, 128, torch.float16, y, "down")
        base = y.cpu()
        awq.awq_lora_add(xs, gi[:, 0].contiguous(), gpu(a), gpu(b), base=y, y=y)
        check_lora(x, ids[:, 0], a, b, None, None, base, torch.float16, y, "adapters")
    assert torch.equal(xs.cpu(), x)
    for y in (xs[:, :N], buf[:M, N - 8:2 * N - 8], buf[:M, K:K + N]):
        with pytest.raises(awq.AwqError):
            awq.awq_w4a16_experts_up(xs, gi, *packed(w), y=y)
        with pytest.raises(awq.AwqError):
            awq.awq_lora_add(xs, gi[:, 0].contiguous(), gpu(a), gpu(b), y=y)
    with pytest.raises(awq.AwqError):
        awq.awq_lora_add(xs, gi[:, 0].contiguous(), gpu(a), gpu(b), base=buf[:M, :N], y=buf[1:M + 1, :N])


def test_binding_refuses_host_tensors_and_wrong_names():
    x = torch.zeros(2, 64)
    ids = torch.zeros(2, 1, dtype=torch.int32)
    w = (torch.zeros(1, 8, 8, dtype=torch.int32), torch.zeros(1, 8, 1, dtype=torch.float16),
         torch.zeros(1, 8, 1, dtype=torch.uint8))
    with pytest.raises(ValueError):
        awq.awq_route_experts(x, 1)
    with pytest.raises(ValueError):
        awq.awq_w4a16_experts_up(x.half(), ids, *w, group_size=64)
    with pytest.raises(ValueError):
        awq.awq_w4a16_experts_up(x.half(), ids, *w, group_size=64, act="gelu")
    with pytest.raises(ValueError):
        awq.awq_w4a16_experts_down(x.half(), ids, torch.zeros(2, 1), *w, group_size=64)
    with pytest.raises(ValueError):
        awq.awq_lora_add(x.half(), ids[:, 0], torch.zeros(1, 8, 64).half(), torch.zeros(1, 4, 8).half())


@pytest.mark.gpu
def test_a_stream_of_another_gpu_is_refused(on_gpu):
    """It would not order the call's work, which runs where its tensors are."""
    other = types.SimpleNamespace(cuda_stream=0, device=torch.device("cuda", 7))
    x = gpu(acts(3, 128, torch.float16, 1))
    ids = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    w = packed(stack(2, 16, 128, 128, 1))
    a, b = (torch.zeros(s, dtype=torch.float16, device="cuda") for s in ((2, 8, 128), (2, 16, 8)))
    for call in (lambda: awq.awq_route_experts(x, 2, stream=other), lambda: awq.awq_w4a16_experts_up(x, ids, *w, stream=other),
                 lambda: awq.awq_w4a16_experts_down(x, ids[:, :1].contiguous(), torch.ones((3, 1), device="cuda"), *w, stream=other),
                 lambda: awq.awq_lora_add(x, ids[:, 0].contiguous(), a, b, stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()
    awq.awq_route_experts(x, 2, stream=torch.cuda.Stream())


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors(on_gpu):
    w = packed(stack(2, 16, 128, 128, 1))
    x = gpu(acts(3, 128, torch.float16, 1))
    ids = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    up = awq.awq_w4a16_experts_up
    for args in ((x, ids.long(), *w), (x, ids.t(), *w), (x[:2], ids, *w), (x, ids[:, 0], *w), (x, ids, w[0][0], *w[1:]),
                 (x, ids, w[0], w[1].float(), w[2]), (x, ids, w[0], w[1], w[2][:1]), (x.t(), ids, *w),
                 (x, ids.cpu(), *w)):
        with pytest.raises(ValueError):
            up(*args)
    with pytest.raises(ValueError):
        up(x, ids, *w, y=torch.zeros((6, 15), device="cuda"))
    with pytest.raises(ValueError):
        awq.awq_w4a16_experts_down(x, ids, torch.zeros((3, 2), device="cuda"), *w)
    with pytest.raises(awq.AwqError):
        up(x.float(), ids, *w)
    with pytest.raises(ValueError):
        awq.awq_route_experts(x, 2, ids=torch.zeros((3, 2), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        awq.awq_route_experts(x, 2, bias=torch.zeros(127, device="cuda"))
    with pytest.raises(awq.AwqError):
        awq.awq_route_experts(x, 129)
    a = torch.zeros((2, 8, 128), dtype=torch.float16, device="cuda")
    b = torch.zeros((2, 16, 8), dtype=torch.float16, device="cuda")
    ad = torch.zeros(3, dtype=torch.int32, device="cuda")
    for kw in (dict(a=a.bfloat16()), dict(b=b[:1]), dict(adapter=ad.long()), dict(adapter=ad[:2]),
               dict(base=torch.zeros((3, 15), device="cuda")), dict(scaling=torch.zeros(3, device="cuda")),
               dict(ranks=torch.zeros(2, device="cuda")), dict(a=a[:, :, ::2])):
        args = dict(x=x, adapter=ad, a=a, b=b)
        args.update(kw)
        with pytest.raises(ValueError):
            awq.awq_lora_add(**args)
