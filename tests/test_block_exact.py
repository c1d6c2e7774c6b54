"""The products with the packed weights of awq_w4a16_linear and awq_w4a16_gemm_dx where their results are known to the
last bit: infinite gradients, and inputs whose sums fp32 holds exactly."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_util import f32, gpu
from tests.test_block import DTYPES, awq, check, normal, on_gpu, packed, product_slack  # noqa: F401


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 200, 512), (5, 200, 512), (16, 200, 512), (17, 200, 512), (40, 200, 512), (300, 200, 512),
                                   (40, 1000, 4096), (130, 1000, 4096), (519, 1000, 4096)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_gemm_dx_of_infinite_gradients(on_gpu, M, N, K, dt):
    """An infinite dz gives what its products are, whatever the number of rows: infinities of the weight's sign, NaN where
    the weight is 0 or two of them meet with both signs; other rows keep their values."""
    g = 64
    q, w, _ = packed(N, K, g, 3, signs=True)
    dz = normal((M, N), DTYPES[dt], 4, size=0.1)
    dz[0, 7] = math.inf
    if M > 3:
        dz[1, 190] = -math.inf
        dz[2, 3], dz[2, 70] = math.inf, -math.inf
        dz[4, 11] = math.nan
    z = f32(dz).astype(np.float64)
    fin = np.where(np.isfinite(z), z, 0.0)
    ref = fin @ w
    with np.errstate(invalid="ignore"):
        for m, n in np.argwhere(~np.isfinite(z)):
            ref[m] += z[m, n] * w[n]
    got = f32(awq.awq_w4a16_gemm_dx(gpu(dz), *q, out_dtype=torch.float32, group_size=g))
    for kind in (np.isnan, np.isposinf, np.isneginf):
        assert np.array_equal(kind(got), kind(ref)), (kind, int((kind(got) != kind(ref)).sum()))
    keep = np.isfinite(ref)
    slack = product_slack(np.concatenate([fin, fin]), w, None)[:M]
    check(torch.from_numpy(np.where(keep, got, 0.0)), np.where(keep, ref, 0.0), slack, torch.float32)


# ---- weights of all their bits --------------------------------------------------------
# Steps m 2^-20 with m odd in 1025 .. 2047 (the 11 bits of an fp16 value), codes less their zero points up to 15 in
# size, and rows of 60 whole numbers up to 8 in size, the rest 0: every product is a whole number of 2^-20, and any sum of
# a row's is below 60 * 8 * 15 * 2047 < 2^24 of them, so fp32 holds each partial sum exactly in any order, and the result
# is the exact one, rounded once to the output's type.  Weights rounded to 11 bits miss most of them.


def whole_weights(N, K, g, seed):
    gen = torch.Generator().manual_seed(seed)
    words = torch.randint(-2 ** 31, 2 ** 31, (N, K // 8), generator=gen, dtype=torch.int32).cuda()
    m = 2 * torch.randint(512, 1024, (N, K // g), generator=gen) + 1
    sign = 2 * torch.randint(0, 2, (N, K // g), generator=gen) - 1
    step = (m * sign * 2.0 ** -20).to(torch.float16).cuda()
    zero = torch.randint(0, 16, (N, K // g), generator=gen, dtype=torch.uint8).cuda()
    codes = ((words.unsqueeze(-1) >> torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)) & 15).flatten(1).double()
    w = (codes.unflatten(1, (-1, g)) - zero.double().unsqueeze(-1)) * step.double().unsqueeze(-1)
    return (words, step, zero), w.flatten(1)


def whole_rows(M, n, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.zeros(M, n)
    at = torch.randint(0, n, (M, min(60, n)), generator=gen)
    v = (torch.randint(1, 9, at.shape, generator=gen) * (2 * torch.randint(0, 2, at.shape, generator=gen) - 1)).float()
    return x.scatter_(1, at, v).to(dtype).cuda()


def rounded(ref, dtype):
    """Exact values that fp32 holds, rounded once."""
    assert torch.equal(ref.float().double(), ref)
    return ref.float().to(dtype)


WHOLE_DXS = [
    # M, N, K, group: each height of the tiles, alone and with the contraction in slices
    (1, 453, 64, 64), (3, 8, 64, 64), (16, 1000, 512, 128), (17, 130, 1024, 64), (40, 4096, 4096, 128), (100, 2000, 2048, 256),
    (4266, 8, 64, 64), (1098, 472, 128, 64), (4201, 8, 320, 64), (519, 1000, 4096, 128), (1130, 990, 64, 64),
    (2858, 8, 1408, 128), (1051, 2004, 192, 64), (1100, 700, 4096, 256), (1635, 8, 5248, 128), (4095, 1027, 4096, 128),
    (4435, 1296, 64, 64), (733, 9430, 6912, 128), (2208, 982, 64, 64), (300, 4096, 4096, 128),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", WHOLE_DXS, ids=lambda c: "x".join(str(v) for v in c))
def test_gemm_dx_to_the_last_bit(on_gpu, case):
    M, N, K, g = case
    q, w = whole_weights(N, K, g, M)
    for dt in (torch.float16, torch.bfloat16):
        dz = whole_rows(M, N, dt, N)
        ref = dz.double() @ w
        for out in DTYPES.values():
            dx = awq.awq_w4a16_gemm_dx(dz, *q, out_dtype=out, group_size=g)
            wrong = int((dx != rounded(ref, out)).sum())
            assert wrong == 0, (dt, out, wrong)


WHOLE_LINEARS = [
    # M, N, K, group: one token, up to 16, 17 to 64, and each height of the tiles, alone, in slices, two in one launch
    (1, 515, 1024, 64), (1, 6200, 4096, 128), (2, 300, 512, 128), (9, 130, 192, 64), (16, 2048, 4096, 128),
    (17, 1040, 1024, 128), (24, 4096, 2048, 256), (33, 100, 4096, 128), (50, 5000, 256, 64), (64, 333, 8192, 256),
    (80, 520, 2048, 128), (300, 16, 64, 64), (635, 28, 2048, 128), (1246, 3163, 1024, 64), (510, 8465, 128, 128),
    (519, 1027, 4096, 64), (1024, 4096, 4096, 128), (1100, 900, 8192, 256), (2048, 9001, 256, 128), (2300, 11008, 512, 64),
    (4097, 4100, 256, 256), (4110, 260, 64, 64), (1050, 8, 512, 128), (200, 515, 2048, 256),
]


def one_step_a_row(q, w, g):
    """The same with each row's first step and zero point's sign kept for all of its groups."""
    words, step, zero = q
    n = step.shape[0]
    units = w.unflatten(1, (-1, g)) / step.double().unsqueeze(-1)
    step = step[:, :1].expand(n, step.shape[1]).contiguous()
    return (words, step, zero), (units * step.double().unsqueeze(-1)).flatten(1)


@pytest.mark.gpu
@pytest.mark.parametrize("case", WHOLE_LINEARS, ids=lambda c: "x".join(str(v) for v in c))
def test_linear_to_the_last_bit(on_gpu, case):
    M, N, K, g = case
    q, w = one_step_a_row(*whole_weights(N, K, g, M), g)
    for dt in (torch.float16, torch.bfloat16):
        x = whole_rows(M, K, dt, N)
        ref = x.double() @ w.t()
        for out in DTYPES.values():
            pre = torch.empty(M, N, dtype=out, device="cuda")
            y = awq.awq_w4a16_linear(x, *q, act="relu", pre=pre, out_dtype=out, group_size=g)
            wrong = int((pre != rounded(ref, out)).sum()), int((y != rounded(ref.clamp_min(0), out)).sum())
            assert wrong == (0, 0), (dt, out, wrong)


@pytest.mark.gpu
@pytest.mark.parametrize("case", WHOLE_LINEARS, ids=lambda c: "x".join(str(v) for v in c))
def test_linear_with_a_step_for_each_group(on_gpu, case):
    """Steps that differ: what fp32 loses at each group (a quotient of steps, a product with it or a multiply-add, three
    half steps of the running sum) and at each of the 60 sums, each at most the sum of all terms' sizes in size."""
    M, N, K, g = case
    q, w = whole_weights(N, K, g, M)
    x = whole_rows(M, K, torch.bfloat16, N)
    ref, size = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    y = awq.awq_w4a16_linear(x, *q, out_dtype=torch.float32, group_size=g)
    off = (y.double() - ref).abs()
    assert bool((off <= (3 * (K // g) + 2 * 60 + 4) * 2.0 ** -24 * size).all()), float((off / size.clamp_min(1e-30)).max() * 2 ** 24)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 5, 16, 17, 40, 100, 519, 1300])
@pytest.mark.parametrize("N,K,g", [(520, 1024, 64), (300, 2048, 256)])
def test_linear_of_steps_far_apart(on_gpu, M, N, K, g):
    """Steps of a row up to 2^18 apart, some 0, tokens that meet one group each: no group costs another its bits.  In the
    tiles a step of 0 beside others counts as 2^-80 (its codes' sum, in units of the step, joins a sum whose unit has to
    be other than 0): a token that meets such a group alone has 2^-80 of the sum of its codes' sizes in place of 0."""
    gen = torch.Generator().manual_seed(M)
    q, w = whole_weights(N, K, g, M)
    G = K // g
    shift = 2.0 ** -torch.randint(0, 19, (N, G), generator=gen).double()
    shift[torch.rand(N, G, generator=gen) < 0.1] = 0.0
    shift[3], shift[7, 1:] = 0.0, 0.0
    base = q[1].double() * 2.0 ** 14
    step = (base * shift.cuda()).to(torch.float16)
    assert bool((step.double() == base * shift.cuda()).all())
    units = w.unflatten(1, (-1, g)) / q[1].double().unsqueeze(-1)
    w = (units * step.double().unsqueeze(-1)).flatten(1)
    at = torch.randint(0, G, (M,), generator=gen)
    x = torch.zeros(M, G, g)
    x[torch.arange(M), at] = torch.randint(-8, 9, (M, g), generator=gen).float()
    x = x.flatten(1).half().cuda()
    ref, size = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    y = awq.awq_w4a16_linear(x, q[0], step, q[2], out_dtype=torch.float32, group_size=g)
    assert bool((y[:, 3] == 0).all())
    off = (y.double() - ref).abs()
    none = x.double().abs() @ torch.where(step.repeat_interleave(g, 1) == 0, units.abs().flatten(1), 0.0).t()
    assert bool((off <= (3 * G + 2 * g + 4) * 2.0 ** -24 * size + 2.0 ** -80 * none * 1.001).all()), float((off / size.clamp_min(1e-30)).max() * 2 ** 24)


# ---- norms of rows far from 0 ---------------------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("K", [9, 512, 1000, 4096, 8192, 20001, 40000, 131072])
@pytest.mark.parametrize("mean", [0.0, 1e3, -1e4, 1e5])
def test_layer_norm_of_rows_far_from_zero(on_gpu, K, mean):
    """A mean of many times the spread costs no more than its own rounding where it is stored: the values themselves are off
    by what a norm of centred values is, sums of under 160 additions (K values as 8 or more per lane, 6 steps of a wave,
    up to 16 waves) of values the size of the spread."""
    gen = torch.Generator().manual_seed(K)
    x = (torch.randn(5, K, generator=gen) + mean).cuda()
    w = torch.randn(K, generator=gen).cuda()
    stats = torch.empty(2, 5, device="cuda")
    y = awq.awq_layer_norm(x, w, stats=stats, eps=1e-5)
    xd = x.double()
    mu = xd.mean(1, keepdim=True)
    d = xd - mu
    rstd = 1.0 / torch.sqrt(d.square().mean(1, keepdim=True) + 1e-5)
    u = 2.0 ** -24
    # a centred value: the first subtraction (exact from 2 spreads on, else half a step of the value and the mean) and the
    # second one, half a step of the spread each; the mean of what is left, 160 additions; 1 / sigma: as many again, halved
    e_d = 2 * u * d.abs() + (160 * u + 2 * u) * d.abs().mean(1, keepdim=True)
    ref = d * rstd * w.double()
    e = w.double().abs() * rstd * (e_d + d.abs() * 90 * u) + w.double().abs() * d.abs() * rstd ** 3 * (d.abs() * e_d).mean(1, keepdim=True)
    e = e + 4 * u * ref.abs()
    assert bool(((y.double() - ref).abs() <= e).all()), float(((y.double() - ref).abs() / e).max())
    assert bool(((stats[0].double() - mu[:, 0]).abs() <= u * mu[:, 0].abs() + 164 * u * d.abs().mean(1)).all())
    assert bool(((stats[1].double() / rstd[:, 0] - 1).abs() <= 90 * u + 164 * u).all())


@pytest.mark.gpu
@pytest.mark.parametrize("K", [7, 300, 4096, 9000, 40000])
def test_layer_norm_of_equal_values(on_gpu, K):
    """Rounding leaves no negative variance: finite with the smallest eps."""
    x = torch.tensor([0.1, 1e4 / 3, -7e-3, 1e20], device="cuda")[:, None].expand(4, K).contiguous()
    stats = torch.empty(2, 4, device="cuda")
    y = awq.awq_layer_norm(x, torch.ones(K, device="cuda"), stats=stats, eps=1e-30)
    assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(stats[:, :3]).all())


# ---- workspaces -------------------------------------------------------------------------------


def test_workspace_sizes_are_asked_of_the_tensors_gpu(monkeypatch):
    """Two GPUs with different numbers of compute units: each call's bytes are those of the GPU its tensors are on, whichever
    is the current one and whichever was asked first."""
    import contextlib

    import weight_only_int4_stats_amd as pkg

    current = [0]

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d
        yield
        current[0] = before

    class Stub:
        @staticmethod
        def awq_workspace_bytes_exact(op, M, N, K, T, n):
            return M * (256, 304)[current[0]]

    monkeypatch.setattr(pkg, "lib", lambda: Stub)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    pkg._ws_need.cache_clear()
    try:
        for _ in range(2):
            for now in (0, 1):
                current[0] = now
                assert pkg._ws_need(pkg.AWQ_OP_LINEAR, 10, 1, 1, 0, 0, 0) == 2560
                assert pkg._ws_need(pkg.AWQ_OP_LINEAR, 10, 1, 1, 0, 0, 1) == 3040
                assert current[0] == now
    finally:
        pkg._ws_need.cache_clear()


@pytest.mark.parametrize("N,K", [(11008, 4096), (4096, 11008), (515, 512), (64, 8192), (2048, 16384)])
def test_exact_workspaces_are_what_a_call_asks_for(N, K):
    """A byte less is refused, as many are taken (x and y overlap: refused after the workspace), and the query that serves
    every smaller batch gives no less."""
    lib, A, V = awq.lib(), 1 << 32, 1 << 40
    for M in (1, 2, 16, 17, 33, 64, 65, 130, 519, 1000, 2048, 4097):
        for op in (awq._abi.AWQ_OP_LINEAR, awq._abi.AWQ_OP_GEMM_DX):
            need = lib.awq_workspace_bytes_exact(op, M, N, K, 0, 0)
            assert 0 <= need <= lib.awq_workspace_bytes(op, M, N, K, 0, 0)

            def status(bytes_, g):
                if op == awq._abi.AWQ_OP_LINEAR:
                    return lib.awq_w4a16_linear(A, 0, M, K, K, V, V, V, N, g, None, 0, 0, None, 0, None, 0, A, 0, N, V, bytes_, None)
                return lib.awq_w4a16_gemm_dx(A, 0, M, N, N, V, V, V, K, g, A, 0, K, V, bytes_, None)

            groups = [g for g in (64, 128, 256) if K % g == 0]
            assert all(status(need, g) == 5 for g in groups)
            assert need == 0 or any(status(need - 1, g) == 6 for g in groups)
    assert lib.awq_workspace_bytes_exact(awq._abi.AWQ_OP_LINEAR, 2048, 11008, 4096, 0, 0) < 24e6
    for op, size in ((awq._abi.AWQ_OP_BALANCE_LOSS, (1000, 0, 0, 64)), (awq._abi.AWQ_OP_LAYER_NORM_BACKWARD, (1000, 0, 512, 0)),
                     (awq._abi.AWQ_OP_GEMM, (100, 512, 512, 0)), (awq._abi.AWQ_OP_LINEAR, (-1, 512, 512, 0)),
                     (awq._abi.AWQ_OP_LINEAR, (0, 512, 512, 0)), (awq._abi.AWQ_OP_GEMM_DX, (1 << 25, 512, 512, 0))):
        assert lib.awq_workspace_bytes_exact(op, *size, 0) == lib.awq_workspace_bytes(op, *size, 0)
