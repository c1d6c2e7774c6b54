"""Operators of a block on arrays past 4 GB: rows beyond offsets of 2^31 and 2^32 bytes against the same rows by themselves,
and sums over all rows against chunks of them in float64."""
import pytest
import torch

from tests.test_block import awq, on_gpu  # noqa: F401

U = 2.0 ** -24


def spots(rows, row_bytes):
    """Slices of 200 rows: the first, around 2^31 and 2^32 bytes, the last."""
    at = [100, (1 << 31) // row_bytes, (1 << 32) // row_bytes, rows - 100]
    assert at[2] < rows - 100
    return [slice(a - 100, a + 100) for a in at]


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance(on_gpu, score):
    T, E, k = 2200000, 1024, 2
    gen = torch.Generator(device="cuda").manual_seed(1)
    lg = torch.empty(T, E, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    ids = (torch.rand(T, k, generator=gen, device="cuda") ** 3 * E).int()
    # only the last rows count: what they give alone
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    mask[-500:] = True
    loss, counts, slope = awq.awq_balance_loss(lg, ids, score=score, mask=mask)
    want = awq.awq_balance_loss(lg[-500:].clone(), ids[-500:].clone(), score=score)
    assert torch.equal(counts, want[1]) and torch.equal(slope, want[2])
    # either sum of p: an exponential, the row's sum and the quotient, and the order of its rows
    assert abs(loss.item() - want[0].item()) <= 2 * 171 * U * abs(want[0].item())
    loss, counts, slope = awq.awq_balance_loss(lg, ids, score=score)
    assert torch.equal(counts, torch.bincount(ids.flatten().long(), minlength=E).int())
    d = awq.awq_balance_loss_backward(lg, slope, score=score)
    rows = [(s, awq.awq_balance_loss_backward(lg[s].clone(), slope, score=score)) for s in spots(T, E * 2)]
    assert all(bool((r != 0).any()) for _, r in rows)
    assert all(torch.equal(d[s], r) for s, r in rows)
    del d
    awq.awq_balance_loss_backward(lg, slope, score=score, dlogits=lg)
    assert all(torch.equal(lg[s], r) for s, r in rows)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [(290000, 8192), (150000, 16384), (72000, 32768)])
def test_layer_norm_and_its_gradients(on_gpu, M, K):
    gen = torch.Generator(device="cuda").manual_seed(K)
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_(0.5, 1.5, generator=gen)
    w = torch.empty(K, device="cuda").normal_(1.0, 0.3, generator=gen)
    stats = torch.empty(2, M, device="cuda")
    y = awq.awq_layer_norm(x, w, w, stats=stats)
    dy = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    dw = torch.zeros(K, dtype=torch.float64, device="cuda")
    db, size_w, size_b = torch.zeros_like(dw), torch.zeros_like(dw), torch.zeros_like(dw)
    step = (1 << 27) // K
    for i in range(0, M, step):
        g = dy[i:i + step].double()
        p = (x[i:i + step].double() - stats[0, i:i + step, None]) * stats[1, i:i + step, None] * g
        dw += p.sum(0)
        db += g.sum(0)
        size_w += p.abs().sum(0)
        size_b += g.abs().sum(0)
    rows = []
    for s in spots(M, K * 2):
        part = stats[:, s].clone()
        assert torch.equal(awq.awq_layer_norm(x[s].clone(), w, w), y[s])
        rows.append((s, awq.awq_layer_norm_backward(dy[s].clone(), x[s].clone(), w, part)[0]))
    del y
    # in place, so that rows left alone would hold dy
    dx, gw, gb = awq.awq_layer_norm_backward(dy, x, w, stats, dx=dy)
    assert all(torch.equal(dx[s], r) for s, r in rows)
    # a block's rows one after another, its row groups, then the blocks' partial rows 16 at a time; a product's roundings
    n = M / 256 + 1 + 16 + 16 + 16
    assert bool(((gw.double() - dw).abs() <= (n + 4) * U * size_w).all())
    assert bool(((gb.double() - db).abs() <= n * U * size_b).all())
