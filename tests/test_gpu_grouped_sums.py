"""Long sums with 16-bit results: the grouped product and its gradients."""

import pytest
import torch

import grouped_helpers as gh

pytestmark = pytest.mark.gpu

F16 = torch.float16
K = 65536
# Values of one sign, which the tensor core's additions all cut off to the same side.  Sums of
# 1024 products do so 1024 times at most, by a step of 2^-23 of their own size so far, which
# is half of what it becomes on average; their sum, of K / 1024 of them, rounds to nearest.
# Then half a step of the result's own binade.  In one go K / 16 additions would cut half a
# step of half the sum each: 1.2e-4, where 6.5e-5 are allowed.
ALLOWED = 1024 * gh.STEP / 2 + K // 1024 * 2.0 ** -24


@pytest.fixture(scope="module")
def mq():
    import weight_quantized_moe_gb300 as m
    return m


def values(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ((torch.rand(*shape, generator=g, device="cuda") + 0.5) * scale).to(F16)


def check_rounded(got, ref):
    assert got.dtype == F16 and got.isfinite().all()
    half_step = torch.exp2(torch.floor(torch.log2(ref)) - 11)
    assert ((got.double() - ref).abs() <= half_step + ALLOWED * ref).all()


@pytest.mark.parametrize("transposed", [False, True])
def test_product(mq, transposed):
    """(So many outputs that K is not split.)"""
    R, N = 40, 10240
    a, w = values(R, K, seed=1, scale=2.0 ** -4), values(N, K, seed=2)
    ref = a.double() @ w.double().T
    if transposed:
        w = w.T.contiguous().T
    out = mq.moe_grouped_product(a, w)
    torch.cuda.synchronize()
    assert mq.mq_device_status() == 0
    check_rounded(out, ref)


@pytest.mark.parametrize("transposed", [False, True])
def test_gradient_of_rows(mq, transposed):
    R, n = 40, 10240
    dy, w = values(R, K, seed=1, scale=2.0 ** -4), values(K, n, seed=2)
    ref = dy.double() @ w.double()
    if transposed:
        w = w.T.contiguous().T
    da, _ = mq.moe_grouped_product_grad(dy, torch.zeros(R, n, dtype=F16, device="cuda"), w, need_w=False)
    torch.cuda.synchronize()
    assert mq.mq_device_status() == 0
    check_rounded(da, ref)


def test_gradient_of_weights(mq):
    """Two experts, one of whose sums is short."""
    n = 2048
    rows = [K, 300]
    a, dy = values(sum(rows), n, seed=1, scale=2.0 ** -4), values(sum(rows), n, seed=2)
    off = gh.offsets_of(rows).cuda()
    w = torch.zeros(2, n, n, dtype=F16, device="cuda")
    _, dw = mq.moe_grouped_product_grad(dy, a, w, off, need_a=False)
    torch.cuda.synchronize()
    assert mq.mq_device_status() == 0
    for e, s in enumerate(gh.rows_of(off)):
        check_rounded(dw[e], dy[s].double().T @ a[s].double())


def test_both_gradients_with_long_and_short_sums(mq):
    """Side by side (many experts), one with more rows than a segment has."""
    counts = [3, 2500, 0, 17] + [20] * 60
    kk, n = 1408, 1536
    a, dy = (gh.randn(sum(counts), c, seed=s, dtype=F16, scale=0.1) for c, s in ((kk, 1), (n, 2)))
    w = gh.randn(len(counts), n, kk, seed=3, dtype=F16, scale=0.1)
    off = gh.offsets_of(counts)
    da, dw = mq.moe_grouped_product_grad(dy.cuda(), a.cuda(), w.cuda(), off.cuda())
    da1, _ = mq.moe_grouped_product_grad(dy.cuda(), a.cuda(), w.cuda(), off.cuda(), need_w=False)
    _, dw1 = mq.moe_grouped_product_grad(dy.cuda(), a.cuda(), w.cuda(), off.cuda(), need_a=False)
    torch.cuda.synchronize()
    assert mq.mq_device_status() == 0
    assert torch.equal(da, da1) and torch.equal(dw, dw1)
    gh.check(da, *gh.product64(dy, w.transpose(1, 2), off), n, "da")
    gh.check(dw, *gh.weights_grad64(dy, a, off, len(counts)), max(counts), "dw")
