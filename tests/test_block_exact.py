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
