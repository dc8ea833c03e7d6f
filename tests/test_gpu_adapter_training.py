"""Adapters trained as two recorded grouped products over rows that are sorted by adapter."""

import pytest
import torch

import grouped_helpers as gh

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("R,K,N,r,L", [(7, 64, 72, 8, 3), (300, 264, 136, 16, 5), (900, 512, 520, 64, 40)])
def test_gradients_of_adapters(R, K, N, r, L, dtype):
    """out = base + s B (A x) for rows with an adapter, some adapters without rows: each product
    and each gradient against its 64-bit formula on what went into it.  The forward agrees with
    moe_lora_product's up to the roundings of A x and of the delta."""
    import weight_quantized_moe_gb300 as mq
    g = torch.Generator().manual_seed(R)
    ids = torch.randint(-1, L - 1, (R,), generator=g, dtype=torch.int32)   # (the last one has none)
    x = gh.randn(R, K, seed=1, dtype=dtype)
    a, b = gh.randn(L, r, K, seed=2, dtype=dtype, scale=K ** -0.5), gh.randn(L, N, r, seed=3, dtype=dtype, scale=r ** -0.5)
    dy, base = gh.randn(R, N, seed=4, dtype=dtype), gh.randn(R, N, seed=5, dtype=dtype)

    leaves = [t.cuda().requires_grad_() for t in (x, a, b)]
    dx, da, db = leaves
    order = torch.argsort(ids, stable=True)
    live = order[int((ids == -1).sum()):]                  # rows with an adapter, by adapter
    off = gh.offsets_of(torch.bincount(ids[live].long(), minlength=L).tolist())
    xs = dx[live.cuda()]
    xs.retain_grad()
    h = mq.moe_grouped_product(xs, da, off.cuda())
    h.retain_grad()
    delta = mq.moe_grouped_product(h, db, off.cuda())
    out = base.cuda().index_add(0, live.cuda(), delta)
    out.backward(dy.cuda())
    torch.cuda.synchronize()
    assert mq.mq_device_status() == 0

    x0, dy0, h0, dh0 = x[live], dy[live], h.detach().cpu(), h.grad.cpu()
    most = int(torch.bincount(ids[live].long()).max())
    gh.check(h.detach(), *gh.product64(x0, a, off), K, "A x")
    gh.check(delta.detach(), *gh.product64(h0, b, off), r, "B h")
    gh.check(db.grad, *gh.weights_grad64(dy0, h0, off, L), most, "dB")
    gh.check(h.grad, *gh.product64(dy0, b.transpose(1, 2), off), N, "dh")
    gh.check(da.grad, *gh.weights_grad64(dh0, x0, off, L), most, "dA")
    gh.check(xs.grad, *gh.product64(dh0, a.transpose(1, 2), off), r, "dx")
    assert (dx.grad[(ids == -1).cuda()] == 0).all() and torch.equal(dx.grad[live.cuda()], xs.grad)
    assert (da.grad[-1] == 0).all() and (db.grad[-1] == 0).all()

    with torch.no_grad():
        served = mq.moe_lora_product(*[t.detach() for t in leaves], ids.cuda(), base=base.cuda())
    want, slack = gh.lora64(x, a[:, None], b[:, None], ids.tolist(), [0] * R, None, base, dtype)
    step = gh.HALF_STEP[dtype]
    size = torch.zeros(R, N, dtype=torch.float64)          # of what is rounded on the way
    size[live] = gh.product64(h0.abs(), b.abs(), off)[0] + delta.detach().cpu().double().abs()
    assert ((served.cpu().double() - out.detach().cpu().double()).abs()
            <= 2 * slack + step * (1.01 * size + 2.01 * want.abs()) + 2 * step * step * size).all()
