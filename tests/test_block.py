"""The operators of a block around the packed linears (awq_w4a16_linear,
awq_bias_act_backward, awq_w4a16_gemm_dx, awq_layer_norm and its backward pass,
awq_balance_loss and its backward pass) against float64, and what they refuse."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import block as B
from tests.gpu_util import f32, gpu

awq = pytest.importorskip("weight_only_int4_stats_amd")
E = awq._abi

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
U = 2.0 ** -24                                       # half a step of fp32


@pytest.fixture
def on_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    awq.lib()


# ---- tolerances ----------------------------------------------------------------
# One output rounding is at most eps / 2 of the value (half the smallest
# subnormal near 0).  An fp32 sum of n terms is off by at most n units U of the
# sum of their sizes; a matrix-core sum by twice that (each addition is within
# one unit of the running size, whatever its rounding).


def rounding(ref, dtype):
    i = torch.finfo(dtype)
    return np.abs(ref) * (i.eps / 2) + (i.tiny * i.eps / 2 if dtype != torch.bfloat16 else i.tiny)


def check(got, ref, slack, dtype, what=""):
    """|got - ref| <= slack (what the computation may be off) + the rounding of
    a value that far from ref; NaN where the reference has NaN."""
    got = f32(got).astype(np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bound = slack + rounding(np.abs(ref) + slack, dtype)
    with np.errstate(invalid="ignore"):
        off = np.abs(got - ref)
        bad = ~((off <= bound) | (got == ref) | (np.isnan(got) & np.isnan(ref)))
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(off / np.maximum(bound, 1e-300))),
                           np.argwhere(bad)[:5].tolist())


def product_slack(x, w, step_sum):
    """What the product of x [M, n] and w [n, N] may be off.  The weights are
    rounded once to fp16 (half a step of fp16, 2^-11 of each), or stay exact and
    meet an offset of 1024 in each chunk of 32 (one token): sums of 17 additions
    and a subtraction of terms of at most 1040 |step x|.  Then an fp32 sum."""
    size = np.abs(x) @ np.abs(w)
    slack = size * (2.0 ** -11 + (w.shape[0] + 64) * 2 * U)
    if x.shape[0] == 1:
        slack = slack + 20 * 1040 * U * (np.abs(x) @ step_sum)
    # fp16 activations: what lies 2^-28 below the largest they share a power with
    return slack + 2.0 ** -24 * np.abs(x).max(axis=1, keepdims=True) * np.abs(w).max(axis=0) * 8


def act_slack(z, dz):
    """A slope of at most 1.13, and the activation's own: an exponential whose
    argument is rounded (|u| U, times a slope in u of at most |z| / 4 e^-|u| u
    <= 0.1 |z| per unit), its sum, quotient and product."""
    return 1.13 * dz + 16 * U * np.abs(z)


def packed(N, K, g, seed, signs=False):
    rng = np.random.default_rng(seed)
    words = rng.integers(-2 ** 31, 2 ** 31, (N, K // 8), dtype=np.int64).astype(np.int32)
    step = rng.uniform(2e-4, 4e-3, (N, K // g)).astype(np.float16)
    if signs:
        step = (step * rng.choice([-1, 1], step.shape)).astype(np.float16)
    zero = rng.integers(0, 16, (N, K // g)).astype(np.uint8)
    w = B.dequantized(words, step, zero, g)
    return tuple(gpu(torch.from_numpy(t)) for t in (words, step, zero)), w, np.repeat(np.abs(step.astype(np.float64)), g, axis=1)


def normal(shape, dtype, seed, size=1.0, outliers=True):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, size, shape)
    if outliers:
        x = x * np.where(rng.random(shape[-1]) < 0.02, 20.0, 1.0)
    return torch.from_numpy(x).to(dtype)


# ---- the product with an epilogue ---------------------------------------------------

LINEARS = [
    # M, N, K, group, xdt, out: every kernel the product has, both sides of its borders
    (1, 512, 512, 128, "f16", "f16"),
    (1, 1027, 1024, 64, "bf16", "bf16"),
    (1, 6200, 4096, 128, "bf16", "f16"),             # one block per compute unit
    (1, 100, 8192, 256, "f16", "bf16"),
    (1, 40, 26624, 128, "f16", "f16"),
    (2, 1, 64, 64, "bf16", "bf16"),
    (2, 300, 512, 128, "f16", "f32"),
    (7, 1025, 1024, 64, "f16", "bf16"),
    (16, 2048, 4096, 128, "bf16", "bf16"),
    (16, 4099, 2048, 256, "f16", "f16"),
    (16, 200, 11008, 128, "bf16", "f16"),
    (5, 9000, 8192, 64, "f16", "f16"),               # more steps than one launch stages
    (3, 7, 128, 128, "f16", "f16"),
    (9, 130, 192, 64, "bf16", "f32"),                # K no multiple of 128
    (17, 1040, 1024, 128, "f16", "f16"),
    (33, 100, 4096, 128, "bf16", "bf16"),            # split over K
    (24, 4100, 512, 64, "bf16", "f16"),
    (64, 333, 8192, 256, "f16", "bf16"),
    (50, 5000, 256, 128, "f16", "f16"),
    (65, 257, 256, 128, "f16", "f16"),
    (130, 1027, 576, 64, "bf16", "f16"),
    (519, 700, 1024, 256, "f16", "f16"),
    (300, 513, 512, 128, "bf16", "f32"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", LINEARS, ids=lambda c: "x".join(str(v) for v in c))
def test_linear(on_gpu, case):
    M, N, K, g, xdt, out = case
    dt, od = DTYPES[xdt], DTYPES[out]
    q, w, steps = packed(N, K, g, M + N, signs=M % 2 == 0)
    x = normal((M, K), dt, K)
    bias = normal((N,), dt, 1, outliers=False)
    res = normal((M, N), od, 2, outliers=False)
    xf = f32(x).astype(np.float64)
    z0, dz0 = xf @ w.T, product_slack(xf, w.T, steps.T)
    z1 = z0 + f32(bias)
    y = awq.awq_w4a16_linear(gpu(x), *q, out_dtype=od, group_size=g)
    check(y, z0, dz0, od, "plain")
    for act in ACTS:
        for with_res in (False, True):
            pre = torch.full((M, N), 7.0, dtype=od, device="cuda")
            y = awq.awq_w4a16_linear(gpu(x), *q, bias=gpu(bias), act=act, residual=gpu(res) if with_res else None, pre=pre,
                                     out_dtype=od, group_size=g)
            dz1 = dz0 + 2 * U * np.abs(z1)
            ref = B.act_value(act, z1)
            slack = act_slack(z1, dz1)
            if with_res:
                ref = ref + f32(res)
                slack = slack + 2 * U * np.abs(ref)
            check(pre, z1, dz1, od, (act, "pre"))
            check(y, ref, slack, od, (act, with_res))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 8, 40, 200])
def test_linear_strides_offsets_and_in_place(on_gpu, M):
    """Rows of larger tensors, outputs off 16 bytes, residual in place, bias of each type; what lies between stays."""
    N, K = 259, 512
    q, w, steps = packed(N, K, 128, 3)
    x = gpu(normal((M, K + 24), torch.bfloat16, 5))[:, 8:8 + K]
    xf = f32(x).astype(np.float64)
    z, dz = xf @ w.T, product_slack(xf, w.T, steps.T)
    for od in DTYPES.values():
        for bdt in DTYPES.values():
            big = torch.full((M + 2, N + 13), 3.0, dtype=od, device="cuda")
            wide = torch.full((M, N + 5), 5.0, dtype=od, device="cuda")
            y, pre = big[1:M + 1, 3:3 + N], wide[:, 1:1 + N]
            res = normal((M, N), od, 6)
            y.copy_(res)
            bias = normal((N + 1,), bdt, 8, outliers=False)
            awq.awq_w4a16_linear(x, *q, bias=gpu(bias)[1:], act="silu", residual=y, y=y, pre=pre)
            z1 = z + f32(bias)[1:]
            dz1 = dz + 2 * U * np.abs(z1)
            ref = B.act_value("silu", z1) + f32(res)
            check(y, ref, act_slack(z1, dz1) + 2 * U * np.abs(ref), od, (od, bdt))
            check(pre, z1, dz1, od, "pre")
            big[1:M + 1, 3:3 + N] = 3.0
            wide[:, 1:1 + N] = 5.0
            assert bool((big == 3.0).all()) and bool((wide == 5.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 5, 30, 100])
def test_linear_small_activations(on_gpu, M):
    """Activations of 1e-5: fp16's lower end, which every path scales up."""
    q, w, steps = packed(300, 1024, 128, 11)
    x = normal((M, 1024), torch.float16, 12, size=1e-5, outliers=False)
    xf = f32(x).astype(np.float64)
    y = awq.awq_w4a16_linear(gpu(x), *q, out_dtype=torch.float32)
    check(y, xf @ w.T, product_slack(xf, w.T, steps.T), torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 3, 20, 70])
@pytest.mark.parametrize("act", ACTS)
def test_linear_limits_of_the_activation(on_gpu, M, act):
    """A bias of +-inf, huge and tiny: the activation's limits, no NaN beside a NaN bias."""
    N, K = 64, 128
    q, w, steps = packed(N, K, 128, 1)
    x = normal((M, K), torch.float16, 2)
    bias = torch.zeros(N)
    bias[1], bias[2], bias[3], bias[4], bias[5] = math.inf, -math.inf, 1e30, -1e30, math.nan
    y = f32(awq.awq_w4a16_linear(gpu(x), *q, bias=gpu(bias), act=act, out_dtype=torch.float32))
    assert np.all(y[:, 1] == np.inf) and np.all(y[:, 3] > 9e29)
    assert np.all(y[:, 2] == (-np.inf if act == "none" else 0.0))
    assert np.all(y[:, 4] < -9e29 if act == "none" else y[:, 4] == 0.0)
    assert np.all(np.isnan(y[:, 5])) and np.isfinite(np.delete(y, [1, 2, 5], axis=1)).all()


BIG_LINEARS = [
    # M, N, K, group, xdt, out: each height of the tiles, slices, two heights in one launch, odd edges
    (80, 520, 2048, 128, "f16", "f16"),
    (519, 1027, 4096, 64, "f16", "f16"),
    (200, 11008, 1024, 128, "bf16", "bf16"),
    (1024, 4096, 4096, 128, "f16", "f16"),
    (1100, 900, 8192, 256, "bf16", "f16"),
    (2048, 9001, 256, 128, "f16", "f16"),
    (2300, 11008, 512, 64, "bf16", "bf16"),
    (4097, 4100, 256, 256, "f16", "bf16"),
]


def on_device(x, w):
    """The product in float64 on the device and what it may be off, as product_slack."""
    xd = x.double()
    ref, size = xd @ w, xd.abs() @ w.abs()
    slack = size * (2.0 ** -11 + (w.shape[0] + 64) * 2 * U)
    return ref, slack + 2.0 ** -24 * xd.abs().amax(1, keepdim=True) * w.abs().amax(0) * 8


def check_on_device(got, ref, slack, what):
    i = torch.finfo(got.dtype)
    tiny = i.tiny if got.dtype == torch.bfloat16 else i.tiny * i.eps / 2
    bound = slack + (ref.abs() + slack) * (i.eps / 2) + tiny
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:5].tolist())


@pytest.mark.gpu
@pytest.mark.parametrize("case", BIG_LINEARS, ids=lambda c: "x".join(str(v) for v in c))
def test_linear_tiles(on_gpu, case):
    M, N, K, g, xdt, out = case
    od = DTYPES[out]
    q, w, _ = packed(N, K, g, M + N, signs=True)
    x, bias = gpu(normal((M, K), DTYPES[xdt], K)), gpu(normal((N,), DTYPES[xdt], 1, outliers=False))
    res = gpu(normal((M, N), od, 2, outliers=False))
    z, dz = on_device(x, gpu(torch.from_numpy(w)).t())
    z, dz = z + bias.double(), dz + 2 * U * (z + bias.double()).abs()
    pre = torch.empty(M, N, dtype=od, device="cuda")
    y = awq.awq_w4a16_linear(x, *q, bias=bias, act="silu", residual=res, pre=pre, out_dtype=od, group_size=g)
    ref = z * torch.sigmoid(z) + res.double()
    check_on_device(pre, z, dz, "pre")
    check_on_device(y, ref, 1.13 * dz + 16 * U * z.abs() + 2 * U * ref.abs(), "y")
    y2 = awq.awq_w4a16_linear(x, *q, out_dtype=od, group_size=g)
    check_on_device(y2, z - bias.double(), dz, "plain")


@pytest.mark.gpu
def test_linear_empty(on_gpu):
    q, _, _ = packed(16, 128, 128, 1)
    x = torch.empty(0, 128, dtype=torch.float16, device="cuda")
    assert awq.awq_w4a16_linear(x, *q, act="gelu").shape == (0, 16)
    none = tuple(t[:0] for t in q)
    assert awq.awq_w4a16_linear(gpu(normal((3, 128), torch.float16, 1)), *none).shape == (3, 0)


# ---- the epilogue's backward pass ------------------------------------------------------

GRADS = [(1, 1), (1, 4096), (3, 7), (5, 511), (16, 513), (17, 1027), (130, 2048), (519, 300), (2100, 1100), (4099, 8)]


def bias_sum_slack(size, M):
    """The bias's gradient: rows of a block one after another, four waves, the blocks' partial sums 16 at a time."""
    return size * (M + 40) * U


@pytest.mark.gpu
@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("shape", GRADS, ids=lambda s: "x".join(map(str, s)))
def test_bias_act_backward(on_gpu, shape, dt):
    M, N = shape
    dtype = DTYPES[dt]
    dy, pre = normal((M, N), dtype, 1, size=0.1), normal((M, N), dtype, 2, size=2.0, outliers=False)
    g, z = f32(dy).astype(np.float64), f32(pre).astype(np.float64)
    for act in ACTS:
        dz, db = awq.awq_bias_act_backward(gpu(dy), None if act == "none" else gpu(pre), act=act)
        ref = g * B.act_slope(act, z)
        # slopes of size 1 formed of an exponential (its argument's rounding: up to z^2 U), a few sums and products
        slack = np.abs(g) * (20 + z * z + 2 * np.abs(z) ** 3) * U if act != "none" else np.zeros_like(g)
        check(dz, ref, slack, dtype, act)
        check(db, ref.sum(0), slack.sum(0) + bias_sum_slack(np.abs(ref).sum(0), M), torch.float32, (act, "dbias"))
    assert awq.awq_bias_act_backward(gpu(dy), gpu(pre), act="silu", dbias=False)[1] is None


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS[1:])
def test_act_slopes_against_differences(on_gpu, act):
    """The slope of the forward pass's own activation, by central differences in float64."""
    z = torch.linspace(-9, 9, 1801)
    dz, _ = awq.awq_bias_act_backward(gpu(torch.ones(1, 1801)), gpu(z[None]), act=act)
    zz, h = z.numpy().astype(np.float64), 1e-5
    diff = (B.act_value(act, zz + h) - B.act_value(act, zz - h)) / (2 * h)
    keep = np.abs(zz) > 1e-3 if act == "relu" else np.ones_like(zz, bool)
    # differences: h^2 f''' / 6 and 2^-53 |f| / h; the kernel's as above
    assert np.all(np.abs(f32(dz)[0] - diff)[keep] <= (1e-9 + (20 + zz * zz + 2 * np.abs(zz) ** 3) * U)[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS[1:])
def test_act_slopes_at_the_ends(on_gpu, act):
    pre = torch.tensor([[math.inf, -math.inf, 3e38, -3e38, 200.0, -200.0, 0.0, -0.0, math.nan]])
    dz, _ = awq.awq_bias_act_backward(gpu(torch.ones_like(pre)), gpu(pre), act=act)
    got = f32(dz)[0]
    assert got[:6].tolist() == [1, 0, 1, 0, 1, 0]
    assert got[6] == got[7] == (0.0 if act == "relu" else 0.5) and np.isnan(got[8])


@pytest.mark.gpu
def test_bias_act_backward_strides_and_in_place(on_gpu):
    for dtype in DTYPES.values():
        big = gpu(normal((70, 300), dtype, 1))
        wide = gpu(normal((70, 311), dtype, 2, outliers=False))
        dy, pre = big[:, 5:282], wide[:, 3:280]
        g, z = f32(dy).astype(np.float64), f32(pre).astype(np.float64)
        ref, slack = g * B.act_slope("gelu", z), np.abs(g) * (20 + z * z + 2 * np.abs(z) ** 3) * U
        keep = big.clone(), wide.clone()
        dz, db = awq.awq_bias_act_backward(dy, pre, act="gelu")
        check(dz, ref, slack, dtype)
        assert torch.equal(big, keep[0]) and torch.equal(wide, keep[1])
        for target in ("dy", "pre"):
            b, p = keep[0].clone(), keep[1].clone()
            t = b[:, 5:282] if target == "dy" else p[:, 3:280]
            again, db2 = awq.awq_bias_act_backward(b[:, 5:282], p[:, 3:280], act="gelu", dz=t)
            assert torch.equal(again, dz) and torch.equal(db2, db)
            assert torch.equal(b[:, :5], keep[0][:, :5]) and torch.equal(b[:, 282:], keep[0][:, 282:])
            assert torch.equal(p[:, :3], keep[1][:, :3]) and torch.equal(p[:, 280:], keep[1][:, 280:])


@pytest.mark.gpu
def test_bias_act_backward_empty(on_gpu):
    dz, db = awq.awq_bias_act_backward(torch.empty(0, 100, device="cuda"), torch.empty(0, 100, device="cuda"), act="gelu")
    assert dz.shape == (0, 100) and db.tolist() == [0.0] * 100
    dz, db = awq.awq_bias_act_backward(torch.empty(4, 0, device="cuda"))
    assert dz.shape == (4, 0) and db.shape == (0,)


# ---- the gradient of the product's input -------------------------------------------------

DXS = [
    # M, N, K, group, dzt, out
    (1, 1, 64, 64, "f16", "f16"),
    (1, 4096, 512, 128, "bf16", "bf16"),
    (1, 63, 256, 256, "f16", "f32"),
    (2, 65, 192, 64, "bf16", "f16"),
    (7, 1027, 1024, 64, "f16", "bf16"),
    (16, 2048, 2048, 128, "bf16", "bf16"),
    (31, 129, 320, 64, "f16", "f16"),
    (33, 500, 4096, 256, "f16", "f16"),
    (37, 4096, 1280, 128, "f16", "f16"),
    (64, 300, 128, 128, "bf16", "f16"),
    (100, 11008, 384, 128, "f16", "f16"),
    (130, 1000, 1024, 128, "bf16", "bf16"),
    (257, 128, 4096, 128, "f16", "f16"),
    (519, 1027, 512, 64, "bf16", "f32"),
    (1030, 512, 2304, 256, "f16", "f16"),
    (2048, 320, 1024, 128, "bf16", "bf16"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", DXS, ids=lambda c: "x".join(str(v) for v in c))
def test_gemm_dx(on_gpu, case):
    M, N, K, g, dzt, out = case
    dt, od = DTYPES[dzt], DTYPES[out]
    q, w, _ = packed(N, K, g, M + N, signs=M % 2 == 0)
    dz = normal((M, N), dt, K, size=1e-3 if dt == torch.bfloat16 else 0.1)
    z = f32(dz).astype(np.float64)
    dx = awq.awq_w4a16_gemm_dx(gpu(dz), *q, out_dtype=od, group_size=g)
    check(dx, z @ w, product_slack(np.concatenate([z, z]), w, None)[:M], od)


BIG_DXS = [
    (200, 11008, 1024, 128, "bf16", "bf16"),
    (512, 4096, 4096, 128, "f16", "f16"),
    (1024, 4096, 8192, 128, "f16", "bf16"),
    (2048, 2111, 4096, 64, "bf16", "f16"),
    (4097, 512, 4096, 256, "f16", "f16"),
    (3, 20000, 512, 128, "bf16", "f16"),             # rows read twice by the conversion
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", BIG_DXS, ids=lambda c: "x".join(str(v) for v in c))
def test_gemm_dx_tiles(on_gpu, case):
    M, N, K, g, dzt, out = case
    q, w, _ = packed(N, K, g, M + N, signs=True)
    dz = gpu(normal((M, N), DTYPES[dzt], K, size=0.1))
    ref, slack = on_device(dz, gpu(torch.from_numpy(w)))
    check_on_device(awq.awq_w4a16_gemm_dx(dz, *q, out_dtype=DTYPES[out], group_size=g), ref, slack, case)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 40, 300])
def test_gemm_dx_strides_and_offsets(on_gpu, M):
    """Rows of larger tensors, off 16 bytes; what lies between stays."""
    N, K = 515, 576
    q, w, _ = packed(N, K, 64, 9)
    big = gpu(normal((M, N + 11), torch.bfloat16, 4))
    dz = big[:, 3:3 + N]
    z = f32(dz).astype(np.float64)
    for od in DTYPES.values():
        wide = torch.full((M + 1, K + 7), 3.0, dtype=od, device="cuda")
        dx = wide[1:, 5:5 + K]
        awq.awq_w4a16_gemm_dx(dz, *q, dx=dx, group_size=64)
        check(dx, z @ w, product_slack(np.concatenate([z, z]), w, None)[:M], od)
        wide[1:, 5:5 + K] = 3.0
        assert bool((wide == 3.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 50, 400])
def test_gemm_dx_rows_of_very_different_steps(on_gpu, M):
    """Rows whose steps lie far apart: each carries a power of two of its own."""
    N, K, g = 192, 256, 64
    rng = np.random.default_rng(1)
    words = rng.integers(-2 ** 31, 2 ** 31, (N, K // 8), dtype=np.int64).astype(np.int32)
    step = (rng.uniform(1, 2, (N, K // g)) * 2.0 ** rng.integers(-14, 12, (N, 1))).astype(np.float16)
    step[5] = 0
    zero = rng.integers(0, 16, (N, K // g)).astype(np.uint8)
    w = B.dequantized(words, step, zero, g)
    dz = rng.normal(0, 1, (M, N))
    dz[:, np.abs(w).max(axis=1) > 1] = 0             # only rows of small weights count
    dz = torch.from_numpy(dz).half()
    q = tuple(gpu(torch.from_numpy(t)) for t in (words, step, zero))
    z = f32(dz).astype(np.float64)
    dx = awq.awq_w4a16_gemm_dx(gpu(dz), *q, out_dtype=torch.float32, group_size=g)
    check(dx, z @ w, product_slack(np.concatenate([z, z]), w, None)[:M], torch.float32)


@pytest.mark.gpu
def test_gemm_dx_empty(on_gpu):
    q, _, _ = packed(16, 128, 128, 1)
    assert awq.awq_w4a16_gemm_dx(torch.empty(0, 16, dtype=torch.float16, device="cuda"), *q).shape == (0, 128)
    none = tuple(t[:0] for t in q)
    for od in DTYPES.values():
        dx = awq.awq_w4a16_gemm_dx(torch.empty(3, 0, dtype=torch.float16, device="cuda"), *none, out_dtype=od)
        assert dx.shape == (3, 128) and bool((dx == 0).all())


# ---- norms ---------------------------------------------------------------------------

NORMS = [(1, 1), (1, 4096), (3, 7), (5, 64), (66, 511), (9, 512), (7, 513), (4, 1000), (5, 1030), (3, 2048), (6, 2049),
         (4, 4096), (2, 4097), (700, 96), (300, 1024), (3, 8192), (2, 8200), (3, 16384), (2, 20001), (2, 33000),
         (530, 5120), (2, 131072)]


def norm_slack(x, w, mean, rstd, y, rms):
    """Sums of K values as 8 or more per lane, 6 steps of a wave, up to 16 waves: under 160 additions for
    K <= 131072; the mean's error moves every value, the variance's half that of 1 / sigma."""
    d = np.abs(x - mean[:, None])
    e_mean = np.zeros((x.shape[0], 1)) if rms else 160 * U * np.abs(x).mean(axis=1, keepdims=True)
    e_d = e_mean + U * d
    return np.abs(w) * rstd[:, None] * (e_d + d * 90 * U) + 4 * U * np.abs(y) + np.abs(w) * d * rstd[:, None] ** 3 * (
        d * e_d).mean(axis=1, keepdims=True)


@pytest.mark.gpu
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("xdt,ydt", [("f16", "f16"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("shape", NORMS, ids=lambda s: "x".join(map(str, s)))
def test_layer_norm(on_gpu, shape, xdt, ydt, rms):
    M, K = shape
    x = normal(shape, DTYPES[xdt], K) + torch.arange(M).to(DTYPES[xdt])[:, None] % 5
    x[0] += 30.0                                     # a mean far from 0
    w, b = normal((K,), DTYPES[xdt], 2, outliers=False), normal((K,), torch.float32, 3, outliers=False)
    xf, wf, bf = (f32(t).astype(np.float64) for t in (x, w, b))
    stats = torch.full((2, M), 9.0, device="cuda")
    y = awq.awq_layer_norm(gpu(x), gpu(w), gpu(b), eps=1e-5, rms=rms, out_dtype=DTYPES[ydt], stats=stats)
    ref, mean, rstd = B.layer_norm(xf, wf, bf, 1e-5, rms)
    slack = norm_slack(xf, wf, mean, rstd, ref, rms)
    check(y, ref, slack + 2 * U * np.abs(bf), DTYPES[ydt])
    got = stats.double().cpu().numpy()
    assert np.all(np.abs(got[0] - mean) <= 160 * U * np.abs(xf).mean(axis=1) + U * np.abs(mean))
    d = np.abs(xf - mean[:, None])
    e_r = 90 * U + rstd ** 2 * (d * (0 if rms else 160 * U) * np.abs(xf).mean(axis=1, keepdims=True)).mean(axis=1)
    assert np.all(np.abs(got[1] / rstd - 1) <= e_r)
    # the same without a bias and without stats
    ref, _, _ = B.layer_norm(xf, wf, None, 1e-5, rms)
    y = awq.awq_layer_norm(gpu(x), gpu(w), eps=1e-5, rms=rms, out_dtype=DTYPES[ydt])
    check(y, ref, norm_slack(xf, wf, mean, rstd, ref, rms), DTYPES[ydt])


def sum_rows(M, K):
    """Additions of a column's sum over the rows: one after another in a block, then the blocks."""
    return M + 100


@pytest.mark.gpu
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("xdt,dyt", [(a, b) for a in DTYPES for b in DTYPES])
@pytest.mark.parametrize("shape", NORMS + [(2050, 40), (1100, 700), (600, 16400), (8, 5000), (9, 5000), (128, 300), (129, 300)], ids=lambda s: "x".join(map(str, s)))
def test_layer_norm_backward(on_gpu, shape, xdt, dyt, rms):
    M, K = shape
    x = normal(shape, DTYPES[xdt], K)
    w, dy = normal((K,), torch.float32, 2, outliers=False), normal(shape, DTYPES[dyt], 3, size=0.1, outliers=False)
    xf, wf, g = (f32(t).astype(np.float64) for t in (x, w, dy))
    _, mean, rstd = B.layer_norm(xf, wf, None, 1e-5, rms)
    stats = torch.from_numpy(np.stack([mean, rstd])).float()
    mean, rstd = stats.double().numpy()
    dx, dw, db = awq.awq_layer_norm_backward(gpu(dy), gpu(x), gpu(w), gpu(stats), rms=rms)
    ref, rw, rb = B.layer_norm_backward(g, xf, wf, mean, rstd, rms)
    a = np.abs(g * wf)
    xh = np.abs((xf if rms else xf - mean[:, None]) * rstd[:, None])
    # two sums over the row (as the norm's) and a few products
    slack = rstd[:, None] * (8 * U * a + 170 * U * ((0 if rms else 1) * a.mean(axis=1, keepdims=True) + xh * (a * xh).mean(
        axis=1, keepdims=True)))
    check(dx, ref, slack, DTYPES[xdt])
    check(dw, rw, (np.abs(g) * xh).sum(0) * (sum_rows(M, K) + 4) * U, torch.float32, "dweight")
    check(db, rb, np.abs(g).sum(0) * sum_rows(M, K) * U, torch.float32, "dbias")
    dx2, none, db2 = awq.awq_layer_norm_backward(gpu(dy), gpu(x), gpu(w), gpu(stats), rms=rms, dweight=False)
    assert none is None and torch.equal(dx2, dx) and torch.equal(db2, db)
    dx2, dw2, none = awq.awq_layer_norm_backward(gpu(dy), gpu(x), gpu(w), gpu(stats), rms=rms, bias=False)
    assert none is None and torch.equal(dx2, dx) and torch.equal(dw2, dw)
    dx2, a, b = awq.awq_layer_norm_backward(gpu(dy), gpu(x), gpu(w), gpu(stats), rms=rms, bias=False, dweight=False)
    assert a is None and b is None and torch.equal(dx2, dx)


@pytest.mark.gpu
@pytest.mark.parametrize("rms", [False, True])
def test_layer_norm_gradient_against_differences(on_gpu, rms):
    """The backward pass against central differences of the oracle's forward pass in float64."""
    rng = np.random.default_rng(4)
    M, K, h = 3, 24, 1e-5
    x, w, b, g = rng.normal(0, 1, (M, K)), rng.normal(1, 0.3, K), rng.normal(0, 1, K), rng.normal(0, 1, (M, K))
    x, w, g = (t.astype(np.float32).astype(np.float64) for t in (x, w, g))
    _, mean, rstd = B.layer_norm(x, w, b, 1e-5, rms)
    to = lambda t: gpu(torch.from_numpy(t).float())  # noqa: E731
    dx, dw, db = (f32(t) for t in awq.awq_layer_norm_backward(to(g), to(x), to(w), to(np.stack([mean, rstd])), rms=rms))
    loss = lambda x, w, b: float((B.layer_norm(x, w, b, 1e-5, rms)[0] * g).sum())  # noqa: E731

    def diff(args, i, at):
        hi, lo = [t.copy() for t in args], [t.copy() for t in args]
        hi[i][at] += h
        lo[i][at] -= h
        return (loss(*hi) - loss(*lo)) / (2 * h)

    args = [x, w, b]
    # differences: h^2 of the third derivative (size about 10) and 2^-53 of the loss over h; fp32 and the fp32 stats
    for i, got in ((0, dx), (1, dw), (2, db)):
        for at in np.ndindex(args[i].shape):
            assert abs(diff(args, i, at) - got[at]) < 2e-5, (i, at)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [37, 512, 4096, 9000, 33001])
def test_layer_norm_strides_offsets_and_in_place(on_gpu, K):
    """Rows off every alignment, in place, into rows of a larger tensor; what lies between stays."""
    M = 5
    for dtype in DTYPES.values():
        big = gpu(normal((M, K + 9), dtype, 1))
        w = gpu(normal((K + 1,), dtype, 2, outliers=False))[1:]
        x = big[:, 3:3 + K]
        keep = big.clone()
        stats = torch.empty(2, M, device="cuda")
        y = awq.awq_layer_norm(x, w, stats=stats)
        check(y, *(lambda r: (r[0], norm_slack(f32(x), f32(w), r[1], r[2], r[0], False)))(
            B.layer_norm(f32(x).astype(np.float64), f32(w), None, 1e-5, False)), dtype)
        wide = torch.full((M, K + 4), 2.0, dtype=dtype, device="cuda")
        awq.awq_layer_norm(x, w, y=wide[:, 1:1 + K])
        assert torch.equal(wide[:, 1:1 + K], y)
        assert bool((wide[:, 0] == 2).all()) and bool((wide[:, 1 + K:] == 2).all()) and torch.equal(big, keep)
        dy = gpu(normal((M, K + 2), dtype, 5, size=0.1))[:, 1:1 + K]
        dx, dw, db = awq.awq_layer_norm_backward(dy, x, w, stats)
        for target in ("x", "dy"):
            b2, d2 = big.clone(), dy.clone()
            xx = b2[:, 3:3 + K]
            again = awq.awq_layer_norm_backward(d2, xx, w, stats, dx=xx if target == "x" else d2)
            assert torch.equal(again[0], dx) and torch.equal(again[1], dw) and torch.equal(again[2], db)
            assert torch.equal(b2[:, :3], keep[:, :3]) and torch.equal(b2[:, 3 + K:], keep[:, 3 + K:])
        awq.awq_layer_norm(x, w, y=x)
        assert torch.equal(x, y) and torch.equal(big[:, :3], keep[:, :3]) and torch.equal(big[:, 3 + K:], keep[:, 3 + K:])


@pytest.mark.gpu
def test_layer_norm_one_bad_row_and_constant_rows(on_gpu):
    """A row with an infinity or NaN spoils itself alone; rows of one value have variance 0; eps 0."""
    x = torch.randn(6, 300)
    x[1, 7], x[2, 9] = math.inf, math.nan
    x[3], x[4] = 5.0, 0.0
    w = torch.ones(300)
    stats = torch.empty(2, 6, device="cuda")
    y = f32(awq.awq_layer_norm(gpu(x), gpu(w), stats=stats))
    assert np.isnan(y[1]).any() and np.isnan(y[2]).all()
    assert np.isfinite(y[[0, 3, 4, 5]]).all() and np.all(y[3] == 0) and np.all(y[4] == 0)
    assert abs(stats[1, 3].item() * math.sqrt(1e-5) - 1) < 1e-6
    z = f32(awq.awq_layer_norm(gpu(x[5:]), gpu(w), eps=0.0))
    assert np.isfinite(z).all()
    r = f32(awq.awq_layer_norm(gpu(x), gpu(w), rms=True))
    assert np.isfinite(r[[0, 3, 4, 5]]).all() and np.allclose(r[3], 1.0, atol=1e-6)


@pytest.mark.gpu
def test_layer_norm_empty(on_gpu):
    w = torch.ones(50, device="cuda")
    x = torch.empty(0, 50, device="cuda")
    assert awq.awq_layer_norm(x, w).shape == (0, 50)
    dx, dw, db = awq.awq_layer_norm_backward(x, x, w, torch.empty(2, 0, device="cuda"))
    assert dx.shape == (0, 50) and dw.tolist() == [0.0] * 50 and db.tolist() == [0.0] * 50


# ---- balance loss ------------------------------------------------------------------------

BALANCES = [
    # T, experts, top_k, score, dtype
    (1, 1, 1, "softmax", "f32"),
    (1, 64, 8, "softmax", "bf16"),
    (5, 3, 2, "sigmoid", "f16"),
    (130, 65, 4, "softmax", "f16"),
    (519, 60, 4, "softmax", "f32"),
    (257, 128, 6, "sigmoid", "bf16"),
    (300, 257, 16, "sigmoid", "f32"),
    (128, 512, 3, "softmax", "f32"),                 # the most that one block takes, and one more
    (129, 96, 3, "sigmoid", "bf16"),
    (40, 1024, 8, "sigmoid", "f16"),
    (1500, 512, 8, "softmax", "bf16"),
    (70, 1000, 64, "sigmoid", "f16"),
    (2100, 1024, 2, "softmax", "f32"),
]


def check_balance(logits, ids, coef, sig, mask, grad, what):
    x, m = f32(logits), None if mask is None else mask.numpy()
    loss, counts, slope, dl = B.balance_loss(x, ids.numpy(), coef, sig, m, 1.0 if grad is None else grad)
    score = "sigmoid" if sig else "softmax"
    lg, mk = gpu(logits), None if mask is None else gpu(mask)
    got = awq.awq_balance_loss(lg, gpu(ids), coef=coef, score=score, mask=mk)
    assert np.array_equal(got[1].cpu().numpy(), counts), what
    # an exponential of an argument of at most 104 in size (below, it is 0): 104 U, and under 60 more for the row's sum
    # and the quotient; sums over the tokens are rounded to fp32 at most T / 512 + 10 times
    T = logits.shape[0]
    assert abs(got[0].item() - loss) <= abs(loss) * (170 + T / 512) * U + 1e-30, (what, got[0].item(), loss)
    check(got[2], slope, np.zeros_like(slope), torch.float32, (what, "slope"))
    gt = None if grad is None else torch.tensor([grad], device="cuda")
    d = awq.awq_balance_loss_backward(lg, got[2], grad=gt, score=score, mask=mk)
    _, _, _, one = B.balance_loss(x, ids.numpy(), coef, sig, m, 1.0)
    # p (d - sum p d) with d the slopes about their mean, each held in fp32
    spread = np.abs(slope - slope.mean()).max() + 2 * U * np.abs(slope).max()
    p = np.zeros_like(one)
    for t in range(T):
        row = x[t].astype(np.float64)
        ok = ~np.isnan(row) & (row > -np.inf)
        if (m is None or m[t]) and ok.any():
            l = np.minimum(row[ok], float(np.finfo(np.float32).max))
            s = np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l))) if sig else l
            p[t, ok] = np.exp(s - s.max()) / np.exp(s - s.max()).sum()
    slack = abs(1.0 if grad is None else grad) * p * (2 * spread * 350 * U + 4 * U * np.abs(slope).max()) + 1e-37
    check(d, dl, slack, logits.dtype, (what, "dlogits"))
    assert np.all(f32(d)[p == 0] == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("case", BALANCES, ids=lambda c: "x".join(map(str, c)))
def test_balance(on_gpu, case):
    T, n, k, score, dt = case
    rng = np.random.default_rng(T + n)
    logits = torch.from_numpy(rng.normal(0, 1.5, (T, n)) + rng.normal(0, 0.7, n)).to(DTYPES[dt])
    ids = torch.from_numpy(np.argsort(-f32(logits), axis=1, kind="stable")[:, :k].astype(np.int32))
    check_balance(logits, ids, 0.01, score == "sigmoid", None, None, case)
    mask = torch.from_numpy(rng.random(T) < 0.6)
    check_balance(logits, ids, 1.0, score == "sigmoid", mask, -2.5, (case, "masked"))
    odd = ids.clone()
    odd[::3, 0] = -1
    odd[1::5, -1] = n
    odd[2::7] = odd[2::7, :1]                        # one expert for all of a token's choices
    check_balance(logits, odd, 3.0, score == "sigmoid", mask.to(torch.uint8), 0.5, (case, "odd ids"))


@pytest.mark.gpu
@pytest.mark.parametrize("sig", [False, True])
@pytest.mark.parametrize("dt", list(DTYPES))
def test_balance_masked_and_extreme_logits(on_gpu, sig, dt):
    """Rows of -inf, of NaN, of the type's lowest value, with +inf, far apart, very low, in counted and masked rows."""
    dtype = DTYPES[dt]
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.normal(0, 1, (24, 48))).to(dtype)
    low = torch.finfo(dtype).min
    x[0], x[1] = -math.inf, math.nan
    x[2, 3:] = -math.inf
    x[3] = low
    x[4, :45] = low
    x[5, 7] = math.inf
    x[6, 11], x[6, 29] = math.inf, math.inf
    x[7] = 60 * torch.arange(48).to(dtype)
    x[8, ::2] = math.nan
    x[9] -= 200
    x[10] = -300 + torch.arange(48).to(dtype)
    x[12:18] = x[:6]
    ids = torch.from_numpy(rng.integers(0, 48, (24, 5)).astype(np.int32))
    mask = torch.ones(24, dtype=torch.bool)
    mask[12:18] = False
    check_balance(x, ids, 1.0, sig, None, None, "all")
    check_balance(x, ids, 1.0, sig, mask, None, "masked")
    check_balance(x[:2], ids[:2], 1.0, sig, None, None, "none usable")
    check_balance(x, ids, 1.0, sig, torch.zeros(24, dtype=torch.bool), None, "none counted")
    check_balance(x, torch.full_like(ids, -1), 1.0, sig, None, None, "no ids")
    got = awq.awq_balance_loss_backward(gpu(x), torch.ones(48, device="cuda"), grad=torch.tensor([math.inf], device="cuda"),
                                        score="sigmoid" if sig else "softmax", mask=gpu(mask))
    assert np.all(f32(got)[[0, 1, 12, 13, 14, 15, 16, 17]] == 0)


@pytest.mark.gpu
def test_balance_even_routing_and_empty(on_gpu):
    logits = torch.zeros(64, 8, device="cuda")
    ids = torch.arange(128, dtype=torch.int32, device="cuda").view(64, 2) % 8
    loss, counts, slope = awq.awq_balance_loss(logits, ids, coef=0.25)
    assert loss.item() == 0.25 and counts.tolist() == [16] * 8
    assert bool((awq.awq_balance_loss_backward(logits, slope) == 0).all())
    loss, counts, slope = awq.awq_balance_loss(logits[:0], ids[:0])
    assert loss.item() == 0 and counts.tolist() == [0] * 8 and slope.tolist() == [0.0] * 8
    assert awq.awq_balance_loss_backward(logits[:0], slope).shape == (0, 8)


@pytest.mark.gpu
@pytest.mark.parametrize("experts", [1, 3, 5, 6, 7, 11, 29, 60, 64])
@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_of_experts_that_serve_alike_has_no_gradient(on_gpu, score, dt, experts):
    """Every token names every expert: the slopes are equal, and the gradient is 0 to the last bit."""
    rng = np.random.default_rng(experts)
    l = gpu(torch.from_numpy(1.5 * rng.standard_normal((333, experts))).to(DTYPES[dt]))
    ids = gpu(torch.arange(experts, dtype=torch.int32).repeat(333, 1))
    loss, counts, slope = awq.awq_balance_loss(l, ids, coef=0.01, score=score)
    assert torch.all(counts == 333) and torch.all(slope == slope[0]) and abs(loss.item() - 0.01) <= 0.01 * (experts + 16) * U
    assert torch.all(awq.awq_balance_loss_backward(l, slope, score=score) == 0)


@pytest.mark.gpu
def test_balance_strides_and_in_place(on_gpu):
    for dtype in DTYPES.values():
        big = gpu(normal((40, 77), dtype, 1, outliers=False))
        keep = big.clone()
        x = big[:, 3:70]
        ids = torch.topk(x.float(), 3, dim=1).indices.int().contiguous()
        loss, counts, slope = awq.awq_balance_loss(x, ids)
        again = awq.awq_balance_loss(x.contiguous(), ids)
        assert torch.equal(loss, again[0]) and torch.equal(counts, again[1]) and torch.equal(slope, again[2])
        d = awq.awq_balance_loss_backward(x, slope)
        wide = torch.full((40, 90), 3.0, dtype=dtype, device="cuda")
        awq.awq_balance_loss_backward(x, slope, dlogits=wide[:, 5:72])
        assert torch.equal(wide[:, 5:72], d) and bool((wide[:, :5] == 3).all()) and bool((wide[:, 72:] == 3).all())
        assert torch.equal(big, keep)
        awq.awq_balance_loss_backward(x, slope, dlogits=x)
        assert torch.equal(x, d) and torch.equal(big[:, :3], keep[:, :3]) and torch.equal(big[:, 70:], keep[:, 70:])


@pytest.mark.gpu
@pytest.mark.parametrize("sig", [False, True])
def test_balance_gradient_against_differences(on_gpu, sig):
    rng = np.random.default_rng(9)
    x = rng.normal(0, 1, (6, 12)).astype(np.float32)
    ids = rng.integers(0, 12, (6, 3)).astype(np.int32)
    score = "sigmoid" if sig else "softmax"
    lg = gpu(torch.from_numpy(x))
    _, _, slope = awq.awq_balance_loss(lg, gpu(torch.from_numpy(ids)), score=score)
    d = f32(awq.awq_balance_loss_backward(lg, slope, score=score))
    h = 1e-5
    for at in np.ndindex(x.shape):
        hi, lo = x.astype(np.float64), x.astype(np.float64)
        hi[at] += h
        lo[at] -= h
        want = (B.balance_loss(hi, ids, 1.0, sig)[0] - B.balance_loss(lo, ids, 1.0, sig)[0]) / (2 * h)
        # h^2 of a third derivative below 1, 2^-53 over h, and fp32
        assert abs(d[at] - want) < 1e-9 + 1e-6 * np.abs(d).max(), at


# ---- together ---------------------------------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 9, 40, 300])
@pytest.mark.parametrize("rms", [False, True])
def test_block_forward_and_backward(on_gpu, M, rms):
    """A pre-norm block as it is run and tuned: norm, up projection with bias and activation, down projection added to
    the stream; then back through both projections into the norm's weight, each step against the formula on the tensors
    that the step before it wrote."""
    H, F, g = 512, 1088, 64
    dt = torch.bfloat16
    q1, w1, s1 = packed(F, H, g, 1)
    q2, w2, s2 = packed(H, F, g, 2)
    h = gpu(normal((M, H), dt, 3))
    nw, nb = gpu(normal((H,), dt, 4, outliers=False)), gpu(normal((H,), dt, 5, outliers=False))
    b1 = gpu(normal((F,), dt, 6, outliers=False))
    stats = torch.empty(2, M, device="cuda")
    pre = torch.empty(M, F, dtype=dt, device="cuda")
    x = awq.awq_layer_norm(h, nw, nb, rms=rms, stats=stats)
    u = awq.awq_w4a16_linear(x, *q1, bias=b1, act="gelu_tanh", pre=pre, group_size=g)
    y = awq.awq_w4a16_linear(u, *q2, residual=h, group_size=g)
    d = lambda t: f32(t).astype(np.float64)  # noqa: E731
    xr, mean, rstd = B.layer_norm(d(h), d(nw), d(nb), 1e-5, rms)
    check(x, xr, norm_slack(d(h), d(nw), mean, rstd, xr, rms) + 2 * U * np.abs(d(nb)), dt, "norm")
    z = d(x) @ w1.T + d(b1)
    dz = product_slack(d(x), w1.T, s1.T) + 2 * U * np.abs(z)
    check(pre, z, dz, dt, "pre")
    check(u, B.act_value("gelu_tanh", z), act_slack(z, dz), dt, "up")
    yr = d(u) @ w2.T + d(h)
    check(y, yr, product_slack(d(u), w2.T, s2.T) + 2 * U * np.abs(yr), dt, "down")

    dy = gpu(normal((M, H), dt, 7, size=1e-2, outliers=False))
    du = awq.awq_w4a16_gemm_dx(dy, *q2, group_size=g)
    dpre, db1 = awq.awq_bias_act_backward(du, pre, act="gelu_tanh")
    dx = awq.awq_w4a16_gemm_dx(dpre, *q1, group_size=g)
    dh, dnw, dnb = awq.awq_layer_norm_backward(dx, h, nw, stats, rms=rms)
    two = lambda t: np.concatenate([t, t])  # noqa: E731
    check(du, d(dy) @ w2, product_slack(two(d(dy)), w2, None)[:M], dt, "du")
    p = d(pre)
    ref, slack = d(du) * B.act_slope("gelu_tanh", p), np.abs(d(du)) * (20 + p * p + 2 * np.abs(p) ** 3) * U
    check(dpre, ref, slack, dt, "dpre")
    check(db1, ref.sum(0), slack.sum(0) + bias_sum_slack(np.abs(ref).sum(0), M), torch.float32, "db1")
    check(dx, d(dpre) @ w1, product_slack(two(d(dpre)), w1, None)[:M], dt, "dx")
    st = stats.double().cpu().numpy()
    ref, rw, rb = B.layer_norm_backward(d(dx), d(h), d(nw), st[0], st[1], rms)
    xh = np.abs((d(h) if rms else d(h) - st[0][:, None]) * st[1][:, None])
    a = np.abs(d(dx) * d(nw))
    slack = st[1][:, None] * (8 * U * a + 170 * U * (a.mean(axis=1, keepdims=True) + xh * (a * xh).mean(axis=1, keepdims=True)))
    check(dh, ref, slack, dt, "dh")
    check(dnw, rw, (np.abs(d(dx)) * xh).sum(0) * (M + 110) * U, torch.float32, "dnw")
    check(dnb, rb, np.abs(d(dx)).sum(0) * (M + 110) * U, torch.float32, "dnb")


@pytest.mark.gpu
def test_router_step(on_gpu):
    """Logits to choices to the balance loss and its gradient, the padding masked by the ids and the mask alike."""
    T, n = 200, 64
    logits = gpu(normal((T, n), torch.bfloat16, 1, size=1.5, outliers=False))
    mask = torch.arange(T, device="cuda") % 50 < 37
    ids, weights = awq.awq_route_experts(logits, 6, score="sigmoid", n_group=8, topk_group=4, group_top=2)
    loss, counts, slope = awq.awq_balance_loss(logits, ids, coef=0.1, score="sigmoid", mask=mask)
    assert int(counts.sum()) == 6 * int(mask.sum())
    assert torch.equal(counts.long(), torch.bincount(ids[mask].flatten().long(), minlength=n))
    check_balance(logits.cpu(), ids.cpu(), 0.1, True, mask.cpu(), None, "router")


CALLS = ["linear1", "linear", "linear_mid", "linear_big", "dx1", "dx", "act", "norm", "norm_grad", "balance"]


def a_call(name, seed=0):
    """(function of keyword arguments that returns a tuple of tensors, its inputs made)."""
    M = {"linear1": 1, "linear": 7, "linear_mid": 40, "linear_big": 150, "dx1": 1, "dx": 150}.get(name, 90)
    N, K, g = 515, 512, 128
    if name.startswith("linear"):
        q, _, _ = packed(N, K, g, 1)
        x, b, r = gpu(normal((M, K), torch.bfloat16, seed)), gpu(normal((N,), torch.float32, 2)), gpu(normal((M, N), torch.bfloat16, 3))
        return lambda **k: (awq.awq_w4a16_linear(x, *q, bias=b, act="gelu", residual=r, **k),)
    if name.startswith("dx"):
        q, _, _ = packed(N, K, g, 1)
        dz = gpu(normal((M, N), torch.bfloat16, seed))
        return lambda **k: (awq.awq_w4a16_gemm_dx(dz, *q, **k),)
    if name == "act":
        dy, pre = gpu(normal((M, N), torch.float16, seed)), gpu(normal((M, N), torch.float16, 1))
        return lambda **k: awq.awq_bias_act_backward(dy, pre, act="silu", **k)
    if name == "balance":
        lg = gpu(normal((M, 96), torch.float16, seed, outliers=False))
        ids = torch.topk(lg.float(), 4, dim=1).indices.int().contiguous()

        def both(**k):
            s = {i: k[i] for i in k if i == "stream"}
            out = awq.awq_balance_loss(lg, ids, **k)
            return out + (awq.awq_balance_loss_backward(lg, out[2], **s),)
        return both
    x, w = gpu(normal((M, K), torch.float16, seed)), gpu(normal((K,), torch.float16, 1))
    if name == "norm":
        return lambda **k: (awq.awq_layer_norm(x, w, w, **k),)
    dy, stats = gpu(normal((M, K), torch.float16, 2)), torch.empty(2, M, device="cuda")
    awq.awq_layer_norm(x, w, stats=stats)
    return lambda **k: awq.awq_layer_norm_backward(dy, x, w, stats, **k)


def equal(a, b):
    return len(a) == len(b) and all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("name", CALLS)
def test_same_bits_every_time_and_on_streams(on_gpu, name):
    call, other = a_call(name), a_call(name, 5)
    first, second = call(), other()
    torch.cuda.synchronize()
    for _ in range(5):
        assert equal(call(), first)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(10):                              # two at once, each with its own workspace
        outs.append((call(stream=streams[0]), other(stream=streams[1])))
    torch.cuda.synchronize()
    for a, b in outs:
        assert equal(a, first) and equal(b, second)
    last = call(stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    assert equal(last, first)


@pytest.mark.gpu
@pytest.mark.parametrize("name", CALLS)
def test_captured_and_replayed(on_gpu, name):
    """Two graphs of one call on different inputs, replayed in turn with eager work between, each replay as the eager call."""
    calls = [a_call(name, s) for s in (0, 5)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    graphs = []
    for c in calls:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = c()
        graphs.append((graph, out))
    for _ in range(3):
        for (graph, out), ref in zip(graphs, want):
            for t in out:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert equal(out, ref)
        assert equal(calls[0](), want[0])


@pytest.mark.gpu
@pytest.mark.parametrize("op,args", [("AWQ_OP_LINEAR", ("linear1", "linear", "linear_mid", "linear_big")), ("AWQ_OP_GEMM_DX", ("dx1", "dx"))])
def test_one_workspace_for_every_number_of_rows(on_gpu, op, args):
    ws = torch.empty(awq.awq_workspace_bytes(getattr(E, op), 150, 515, 512), dtype=torch.uint8, device="cuda")
    for name in args:
        call = a_call(name)
        assert equal(call(ws=ws), call())


@pytest.mark.gpu
def test_a_call_reads_nothing_that_its_workspace_held(on_gpu):
    """Workspaces full of NaN bits give the same results."""
    sizes = {"linear1": ("AWQ_OP_LINEAR", (1, 515, 512)), "linear_mid": ("AWQ_OP_LINEAR", (40, 515, 512)),
             "linear_big": ("AWQ_OP_LINEAR", (150, 515, 512)), "dx1": ("AWQ_OP_GEMM_DX", (1, 515, 512)),
             "dx": ("AWQ_OP_GEMM_DX", (150, 515, 512)), "act": ("AWQ_OP_BIAS_ACT_BACKWARD", (90, 515)),
             "norm_grad": ("AWQ_OP_LAYER_NORM_BACKWARD", (90, 0, 512)), "balance": ("AWQ_OP_BALANCE_LOSS", (90, 0, 0, 96))}
    for name, (op, size) in sizes.items():
        call = a_call(name)
        need = awq.awq_workspace_bytes(getattr(E, op), *size)
        ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")[:need]
        assert equal(call(ws=ws), call()), name


@pytest.mark.gpu
def test_outputs_past_4_gigabytes(on_gpu):
    """Rows whose offsets pass 32 bits, against the same rows by themselves."""
    M, N, K = 70000, 32768, 64
    q, _, _ = packed(N, K, 64, 1)
    x = gpu(normal((M, K), torch.float16, 1))
    y = awq.awq_w4a16_linear(x, *q, act="relu", group_size=64)
    assert y.numel() * 2 > 1 << 32
    for rows in (slice(0, 300), slice(32700, 33000), slice(M - 300, M)):
        assert torch.allclose(y[rows].float(), awq.awq_w4a16_linear(x[rows], *q, act="relu", group_size=64).float(), rtol=2e-3,
                              atol=2e-4)
    dz, db = awq.awq_bias_act_backward(y, y, act="relu")
    assert torch.equal(dz[-5:], torch.where(y[-5:] > 0, y[-5:], 0))
    assert torch.allclose(db, y.sum(0, dtype=torch.float32), rtol=1e-3)
    del dz
    w = torch.ones(N, device="cuda")
    stats = torch.empty(2, M, device="cuda")
    n = awq.awq_layer_norm(y, w, stats=stats)
    last = awq.awq_layer_norm(y[-3:], w)
    assert torch.equal(n[-3:], last)
    dx, dw, _ = awq.awq_layer_norm_backward(n, y, w, stats, dx=n, bias=False)
    assert bool(torch.isfinite(dx[-3:]).all()) and bool(torch.isfinite(dw).all())
    del n, dx, y
    q, _, _ = packed(64, N, 64, 2)
    dz = gpu(normal((M, 64), torch.float16, 3))
    dx = awq.awq_w4a16_gemm_dx(dz, *q, group_size=64)
    for rows in (slice(0, 300), slice(M - 300, M)):
        assert torch.allclose(dx[rows].float(), awq.awq_w4a16_gemm_dx(dz[rows], *q, group_size=64).float(), rtol=2e-3, atol=2e-4)


@pytest.mark.gpu
def test_balance_past_4_gigabytes(on_gpu):
    T, n = 2200000, 1024
    lg = torch.zeros(T, n, dtype=torch.bfloat16, device="cuda")
    lg[-1, 5] = 3.0
    ids = (torch.arange(2 * T, dtype=torch.int32, device="cuda") % n).view(T, 2)
    loss, counts, slope = awq.awq_balance_loss(lg, ids)
    assert int(counts.sum()) == 2 * T and abs(loss.item() - 1) < 1e-3
    d = awq.awq_balance_loss_backward(lg, slope, dlogits=lg)
    assert bool(torch.isfinite(d[-1]).all())


# ---- refusals (no GPU) ---------------------------------------------------------------------

A, A2, A3, A4, A5 = (ctypes.c_void_p(i << 32) for i in range(1, 6))
BAD = ctypes.c_void_p((1 << 32) + 2)
ODD = ctypes.c_void_p((1 << 32) + 1)
WS = ctypes.c_void_p(9 << 32)
BIG = 1 << 40


def refuses(fn, names, base):
    """call(code, key=value, ...): the entry point with these arguments in place of base's returns code."""
    f = getattr(awq.lib(), fn)

    def call(want, **kw):
        a = dict(base, **kw)
        assert set(kw) <= set(names), kw
        got = f(*(a[n] for n in names), None)
        assert got == want, (fn, kw, got)
    return call


def test_linear_refusals():
    c = refuses("awq_w4a16_linear", ["x", "xdt", "M", "K", "ldx", "q", "s", "z", "N", "g", "bias", "bdt", "act", "res", "ldr", "pre",
                                     "ldp", "y", "ydt", "ldy", "ws", "wsb"],
                dict(x=A, xdt=0, M=100, K=512, ldx=512, q=A2, s=A3, z=A3, N=256, g=128, bias=None, bdt=0, act=0, res=None, ldr=0,
                     pre=None, ldp=0, y=A4, ydt=0, ldy=256, ws=WS, wsb=BIG))
    c(5, g=32), c(5, act=1), c(5, act=6), c(5, act=-1)
    c(3, xdt=2), c(3, ydt=3), c(3, xdt=-1), c(3, bias=A3, bdt=7)
    c(2, M=-1), c(2, N=-1), c(2, K=0), c(2, K=500), c(2, ldx=504), c(2, ldy=255), c(2, res=A5, ldr=255), c(2, pre=A5, ldp=3)
    c(0, M=0), c(0, N=0, ldy=0), c(0, M=0, x=None, y=None)
    for n in ("x", "q", "s", "z", "y"):
        c(1, **{n: None})
    c(4, x=BAD), c(4, ldx=516), c(4, q=BAD), c(4, s=ODD), c(4, y=ODD), c(4, y=BAD, ydt=2), c(4, bias=BAD, bdt=2)
    c(4, res=ODD, ldr=256), c(4, pre=ODD, ldp=256)
    c(6, ws=None), c(6, wsb=8), c(6, ws=ctypes.c_void_p((9 << 32) + 128))
    c(5, K=131072 + 128, ldx=131072 + 128), c(5, M=(1 << 24) + 1), c(5, N=(1 << 22) + 1, ldy=1 << 23)
    c(5, N=1 << 22, ldy=1 << 22, K=4096, ldx=4096)
    c(5, M=1 << 24, N=1 << 22, ldy=1 << 22)          # tiles for more than 2^32 threads
    # rows that share memory
    c(5, y=A, ldy=512), c(5, pre=A, ldp=512), c(5, pre=A4, ldp=256), c(5, res=A4, ldr=264), c(5, res=A5, ldr=256, pre=A5, ldp=256)
    c(5, res=ctypes.c_void_p((4 << 32) + 2), ldr=256)


def test_bias_act_backward_refusals():
    c = refuses("awq_bias_act_backward", ["dy", "dt", "M", "N", "lddy", "pre", "ldp", "act", "dz", "lddz", "db", "ws", "wsb"],
                dict(dy=A, dt=0, M=100, N=256, lddy=256, pre=A2, ldp=256, act=3, dz=A3, lddz=256, db=A4, ws=WS, wsb=BIG))
    c(5, act=1), c(5, act=9), c(3, dt=3)
    c(2, M=-1), c(2, N=-1), c(2, lddy=255), c(2, ldp=255), c(2, lddz=255)
    c(0, N=0)
    c(1, dy=None), c(1, pre=None), c(1, dz=None)
    c(4, dy=ODD), c(4, pre=ODD), c(4, dz=ODD), c(4, db=BAD), c(4, dy=BAD, dt=2)
    c(6, ws=None), c(6, wsb=8)
    c(5, M=(1 << 24) + 1), c(5, N=(1 << 22) + 1, lddy=1 << 23, ldp=1 << 23, lddz=1 << 23)
    c(5, dz=ctypes.c_void_p((1 << 32) + 2)), c(5, dz=A, lddz=264), c(5, dz=A2, lddz=264)


def test_gemm_dx_refusals():
    c = refuses("awq_w4a16_gemm_dx", ["dz", "dzt", "M", "N", "lddz", "q", "s", "z", "K", "g", "dx", "dxt", "lddx", "ws", "wsb"],
                dict(dz=A, dzt=0, M=100, N=256, lddz=256, q=A2, s=A3, z=A3, K=512, g=128, dx=A4, dxt=0, lddx=512, ws=WS, wsb=BIG))
    c(5, g=0), c(3, dzt=2), c(3, dxt=4)
    c(2, M=-1), c(2, N=-1), c(2, K=0), c(2, K=448), c(2, lddz=255), c(2, lddx=511)
    c(0, M=0)
    for n in ("dz", "q", "s", "z", "dx"):
        c(1, **{n: None})
    c(4, dz=ODD), c(4, q=BAD), c(4, s=ODD), c(4, dx=ODD), c(4, dx=BAD, dxt=2)
    c(6, ws=None), c(6, wsb=8)
    c(5, K=131072 + 128, lddx=1 << 20), c(5, M=(1 << 24) + 1), c(5, N=(1 << 22) + 1, lddz=1 << 23)
    c(5, dx=A), c(5, dx=ctypes.c_void_p((1 << 32) + 256))


def test_layer_norm_refusals():
    c = refuses("awq_layer_norm", ["x", "xdt", "M", "K", "ldx", "w", "wdt", "b", "bdt", "eps", "rms", "y", "ydt", "ldy", "mean", "rstd"],
                dict(x=A, xdt=0, M=100, K=500, ldx=500, w=A2, wdt=0, b=None, bdt=0, eps=1e-5, rms=0, y=A3, ydt=0, ldy=500, mean=None,
                     rstd=None))
    c(3, xdt=3), c(3, wdt=-1), c(3, ydt=5), c(3, b=A4, bdt=3)
    c(2, M=-1), c(2, K=0), c(2, ldx=499), c(2, ldy=499)
    c(5, K=131073, ldx=1 << 20, ldy=1 << 20), c(5, eps=-1.0), c(5, eps=math.nan), c(5, eps=math.inf)
    c(0, M=0)
    c(1, x=None), c(1, w=None), c(1, y=None)
    c(5, M=(1 << 24) + 1), c(5, M=1 << 22, K=9000, ldx=9000, ldy=9000)
    c(4, x=ODD), c(4, w=ODD), c(4, b=ODD), c(4, y=ODD), c(4, mean=BAD), c(4, rstd=BAD), c(4, x=BAD, xdt=2)
    c(5, y=A, ldy=501), c(5, y=A, ydt=2), c(5, y=ctypes.c_void_p((1 << 32) + 2))


def test_layer_norm_backward_refusals():
    c = refuses("awq_layer_norm_backward", ["dy", "dyt", "M", "K", "lddy", "x", "xdt", "ldx", "w", "wdt", "mean", "rstd", "rms", "dx",
                                            "lddx", "dw", "db", "ws", "wsb"],
                dict(dy=A, dyt=0, M=1000, K=500, lddy=500, x=A2, xdt=0, ldx=500, w=A3, wdt=0, mean=A3, rstd=A3, rms=0, dx=A4, lddx=500,
                     dw=A5, db=A5, ws=WS, wsb=BIG))
    c(3, dyt=3), c(3, xdt=3), c(3, wdt=3)
    c(2, M=-1), c(2, K=0), c(2, lddy=499), c(2, ldx=499), c(2, lddx=499)
    c(5, K=131073, lddy=1 << 20, ldx=1 << 20, lddx=1 << 20), c(5, M=(1 << 24) + 1)
    for n in ("dy", "x", "w", "mean", "rstd", "dx"):
        c(1, **{n: None})
    c(4, dy=ODD), c(4, x=ODD), c(4, w=ODD), c(4, mean=BAD), c(4, rstd=BAD), c(4, dx=ODD), c(4, dw=BAD), c(4, db=BAD)
    c(6, ws=None), c(6, wsb=8)
    c(5, dx=A, lddx=501), c(5, dx=A2, lddx=501), c(5, dx=A, dyt=2)


def test_balance_refusals():
    c = refuses("awq_balance_loss", ["l", "dt", "T", "E", "ldl", "ids", "k", "mask", "score", "coef", "loss", "counts", "slope", "ws", "wsb"],
                dict(l=A, dt=0, T=1000, E=64, ldl=64, ids=A2, k=4, mask=None, score=0, coef=1.0, loss=A3, counts=A3, slope=A3, ws=WS,
                     wsb=BIG))
    c(3, dt=3), c(5, score=2), c(2, T=-1), c(2, E=0), c(2, ldl=63), c(2, k=0)
    c(5, E=1025, ldl=2000), c(5, k=65), c(5, T=(1 << 24) + 1)
    for n in ("l", "ids", "loss", "counts", "slope"):
        c(1, **{n: None})
    c(4, l=ODD), c(4, ids=BAD), c(4, loss=BAD), c(4, counts=BAD), c(4, slope=BAD), c(6, ws=None), c(6, wsb=8)
    c = refuses("awq_balance_loss_backward", ["l", "dt", "T", "E", "ldl", "slope", "grad", "mask", "score", "dl", "ldd"],
                dict(l=A, dt=0, T=100, E=64, ldl=64, slope=A2, grad=None, mask=None, score=0, dl=A3, ldd=64))
    c(3, dt=3), c(5, score=2), c(2, T=-1), c(2, E=0), c(2, ldl=63), c(2, ldd=63), c(5, E=1025, ldl=2000, ldd=2000)
    c(5, T=(1 << 24) + 1), c(0, T=0), c(1, l=None), c(1, slope=None), c(1, dl=None)
    c(4, l=ODD), c(4, slope=BAD), c(4, grad=BAD), c(4, dl=ODD), c(5, dl=A, ldd=65), c(5, dl=ctypes.c_void_p((1 << 32) + 2))


@pytest.mark.parametrize("N,K", [(4096, 4096), (4096, 11008), (515, 512), (100, 8192), (64, 131072)])
def test_workspace_of_the_largest_batch_serves_all(N, K):
    for op in (E.AWQ_OP_LINEAR, E.AWQ_OP_GEMM_DX, E.AWQ_OP_BIAS_ACT_BACKWARD, E.AWQ_OP_LAYER_NORM_BACKWARD):
        last = 0
        for M in (1, 2, 16, 17, 33, 63, 64, 65, 100, 257, 1000, 2048, 5000, 40000, 1 << 20):
            b = awq.awq_workspace_bytes(op, M, N, K)
            assert b >= last, (op, M)
            last = b
    for op in (E.AWQ_OP_LINEAR, E.AWQ_OP_GEMM_DX):
        assert awq.awq_workspace_bytes(op, (1 << 24) + 1, N, K) == awq.awq_workspace_bytes(op, 4, (1 << 22) + 1, K) == 0
        assert awq.awq_workspace_bytes(op, 4, N, 131073) == awq.awq_workspace_bytes(op, -1, N, K) == 0
    assert awq.awq_workspace_bytes(E.AWQ_OP_BALANCE_LOSS, 4, 0, 0, 1025) == 0
    assert awq.awq_workspace_bytes(E.AWQ_OP_BALANCE_LOSS, 1000, 0, 0, 1024) > 0


@pytest.mark.parametrize("N,K", [(4096, 4096), (515, 512), (64, 8192), (2048, 16384), (11008, 256)])
def test_the_workspace_asked_for_is_enough_for_every_smaller_batch(N, K):
    # x and y overlap, which is refused after the workspace was found large enough
    A, V = ctypes.c_void_p(1 << 32), ctypes.c_void_p(1 << 40)
    for most in (64, 300, 5000):
        need = {op: awq.awq_workspace_bytes(getattr(E, op), most, N, K) for op in ("AWQ_OP_LINEAR", "AWQ_OP_GEMM_DX")}
        for M in [m for m in (1, 2, 7, 16, 17, 24, 32, 33, 48, 64, 65, 80, 100, 129, 256, 300, 519, 1000, 2048, 2500, 4097, 5000) if m <= most]:
            for g in (64, 128, 256):
                r = awq.lib().awq_w4a16_linear(A, 0, M, K, K, V, V, V, N, g, None, 0, 0, None, 0, None, 0, A, 0, N, V,
                                               need["AWQ_OP_LINEAR"], None)
                assert r == 5, ("linear", most, M, g)
                r = awq.lib().awq_w4a16_gemm_dx(A, 0, M, N, N, V, V, V, K, g, A, 0, K, V, need["AWQ_OP_GEMM_DX"], None)
                assert r == 5, ("dx", most, M, g)


def test_binding_refuses_host_tensors_and_wrong_names():
    x = torch.zeros(2, 128, dtype=torch.float16)
    q = torch.zeros(8, 16, dtype=torch.int32), torch.zeros(8, 1, dtype=torch.float16), torch.zeros(8, 1, dtype=torch.uint8)
    v = torch.ones(128)
    for call in (lambda: awq.awq_w4a16_linear(x, *q), lambda: awq.awq_w4a16_linear(x, *q, act="swiglu"),
                 lambda: awq.awq_bias_act_backward(x), lambda: awq.awq_bias_act_backward(x, x, act="tanh"),
                 lambda: awq.awq_w4a16_gemm_dx(x[:, :8], *q), lambda: awq.awq_layer_norm(x, v),
                 lambda: awq.awq_layer_norm_backward(x, x, v, torch.zeros(2, 2)),
                 lambda: awq.awq_balance_loss(x, torch.zeros(2, 1, dtype=torch.int32)),
                 lambda: awq.awq_balance_loss(x, torch.zeros(2, 1, dtype=torch.int32), score="tanh"),
                 lambda: awq.awq_balance_loss_backward(x, v)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors(on_gpu):
    q, _, _ = packed(64, 256, 128, 1)
    x = gpu(normal((4, 256), torch.float16, 1))
    dz = gpu(normal((4, 64), torch.float16, 1))
    v = torch.ones(256, device="cuda")
    st = torch.zeros(2, 4, device="cuda")
    lg, ids = torch.zeros(4, 16, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    bad = [
        lambda: awq.awq_w4a16_linear(x[:, :128], *q),
        lambda: awq.awq_w4a16_linear(x, q[0], q[1][:, :1], q[2]),
        lambda: awq.awq_w4a16_linear(x, q[0], q[1].float(), q[2]),
        lambda: awq.awq_w4a16_linear(x, *q, group_size=100),
        lambda: awq.awq_w4a16_linear(x, *q, bias=v),
        lambda: awq.awq_w4a16_linear(x, *q, bias=torch.ones(64, dtype=torch.float64, device="cuda")),
        lambda: awq.awq_w4a16_linear(x, *q, residual=dz.float(), out_dtype=torch.float16),
        lambda: awq.awq_w4a16_linear(x, *q, pre=torch.empty(4, 63, dtype=torch.float16, device="cuda")),
        lambda: awq.awq_w4a16_linear(x, *q, y=torch.empty(5, 64, dtype=torch.float16, device="cuda")),
        lambda: awq.awq_bias_act_backward(dz, act="gelu"),
        lambda: awq.awq_bias_act_backward(dz, dz.float(), act="gelu"),
        lambda: awq.awq_bias_act_backward(dz, dz=torch.empty_like(dz)),
        lambda: awq.awq_bias_act_backward(dz, dbias=torch.empty(63, device="cuda")),
        lambda: awq.awq_w4a16_gemm_dx(x, *q),
        lambda: awq.awq_w4a16_gemm_dx(dz, *q, dx=torch.empty(4, 255, device="cuda")),
        lambda: awq.awq_layer_norm(x, v[:255]),
        lambda: awq.awq_layer_norm(x, None),
        lambda: awq.awq_layer_norm(x, v, stats=st.t()),
        lambda: awq.awq_layer_norm(x.t(), v[:4]),
        lambda: awq.awq_layer_norm_backward(x, x[:3], v, st),
        lambda: awq.awq_layer_norm_backward(x, x, v, st.half()),
        lambda: awq.awq_balance_loss(lg, ids.long()),
        lambda: awq.awq_balance_loss(lg, ids[:3]),
        lambda: awq.awq_balance_loss(lg, ids, mask=torch.ones(3, dtype=torch.bool, device="cuda")),
        lambda: awq.awq_balance_loss(lg, ids, mask=torch.ones(4, device="cuda")),
        lambda: awq.awq_balance_loss_backward(lg, v),
        lambda: awq.awq_balance_loss_backward(lg, v[:16].contiguous(), grad=torch.tensor(1.0, device="cuda")),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    with pytest.raises(awq.AwqError):
        awq.awq_layer_norm(x, v, eps=-1.0)
    with pytest.raises(awq.AwqError):
        awq.awq_w4a16_linear(x.float(), *q)
