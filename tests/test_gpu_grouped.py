"""The 16-bit grouped product and its gradients against their 64-bit definitions, at
the sizes where tiles, splits and steps end."""

import pytest
import torch

import grouped_helpers as gh

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def mq():
    import weight_quantized_moe_gb300 as m
    return m


def clean(mq):
    torch.cuda.synchronize()
    assert mq.mq_device_status() == 0


def storage(w, transposed):
    """w on the device, stored as it is or the other way round."""
    if not transposed:
        return w.cuda()
    return w.transpose(-1, -2).contiguous().cuda().transpose(-1, -2)


# (rows of each expert, rows before and behind them, K, N)
SHAPES = [
    ([1], 0, 0, 64, 128),                       # one row
    ([1], 0, 0, 4096, 256),                     # one row, K split
    ([20], 0, 0, 4096, 256),
    ([3, 0, 1], 0, 0, 72, 40),                  # an empty expert, K and N that fill no tile
    ([0, 2, 4, 0, 1], 1, 0, 264, 33 * 8),       # eight rows with one of no expert
    ([8], 0, 0, 8200, 24),
    ([0, 1, 3], 2, 2, 2056, 40),
    ([40] * 24, 1, 2, 136, 264),                # both gradients in one launch
    ([0, 130, 7, 0, 33, 64], 0, 0, 520, 392),
    ([0, 5, 0, 16, 17], 2, 3, 200, 136),        # rows of no expert on both sides
    ([31, 32, 33], 0, 1, 64, 264),
    ([63, 64, 65, 0], 5, 0, 136, 128),
    ([100, 128, 129], 0, 0, 8, 8),              # K and N of eight
    ([255, 256, 257, 300], 1, 2, 192, 520),     # CTA pairs
    ([700], 0, 0, 2048, 256),                   # pairs, one expert
    ([40] * 24, 0, 0, 64, 96),
    ([1, 0, 0, 2, 0, 0, 0, 1], 1, 1, 264, 48),  # more experts than rows
    ([3], 0, 0, 72, 8200),                      # few rows, more outputs than CTAs at a time
    ([2, 0, 5], 1, 2, 296, 8200),
    ([1500], 3, 2, 1024, 264),                  # many rows, K split
    ([900, 0, 700], 1, 4, 2056, 136),
    ([0, 0, 0], 4, 4, 64, 64),                  # no rows at all
]


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, BF16)])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_product(mq, shape, transposed, dtype, out_dtype):
    counts, before, behind, K, N = shape
    E, R = len(counts), sum(counts) + before + behind
    off = gh.offsets_of(counts, before)
    a, w = gh.randn(R, K, seed=1, dtype=dtype), gh.randn(E, N, K, seed=2, dtype=dtype, scale=0.1)
    live = slice(before, R - behind)
    ref, mag = gh.product64(a, w, off)
    a[:before] = float("nan")                   # rows of no expert reach nothing
    a[R - behind:] = float("inf")
    out = torch.full((R, N), 7.0, dtype=out_dtype, device="cuda")
    got = mq.moe_grouped_product(a.cuda(), storage(w, transposed), off.cuda(), out=out)
    clean(mq)
    assert got is out
    gh.check(out[live], ref[live], mag[live], K)
    assert (out[:before] == 7).all() and (out[R - behind:] == 7).all()


@pytest.mark.parametrize("dtype,dw_dtype", [(BF16, BF16), (F16, F16), (BF16, F32)])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradients(mq, shape, transposed, dtype, dw_dtype):
    counts, before, behind, K, N = shape
    E, R = len(counts), sum(counts) + before + behind
    off = gh.offsets_of(counts, before)
    a, w = gh.randn(R, K, seed=1, dtype=dtype), gh.randn(E, N, K, seed=2, dtype=dtype, scale=0.1)
    dy = gh.randn(R, N, seed=3, dtype=dtype)
    live = slice(before, R - behind)
    da64, da_mag = gh.product64(dy, w.transpose(1, 2), off)
    dw64, dw_mag = gh.weights_grad64(dy, a, off, E)
    for t in (a, dy):                           # rows of no expert are not read
        t[:before] = float("nan")
        t[R - behind:] = float("inf")
    da, dw = mq.moe_grouped_product_grad(dy.cuda(), a.cuda(), storage(w, transposed), off.cuda(),
                                         dw_dtype=dw_dtype)
    clean(mq)
    assert da.dtype == dtype and dw.dtype == dw_dtype and dw.shape == w.shape
    gh.check(da[live], da64[live], da_mag[live], N, "da")
    assert (da[:before] == 0).all() and (da[R - behind:] == 0).all()
    gh.check(dw, dw64, dw_mag, max(counts), "dw")
    for e, n in enumerate(counts):
        assert n or (dw[e] == 0).all()


@pytest.mark.parametrize("n", [1, 15, 16, 17, 48, 63, 64, 65, 130])
def test_infinities_of_the_next_expert_stay_there(mq, n):
    """The last rows of an expert share a stage with the next one's, which here are
    infinities and NaN: only that expert's gradient has them."""
    R, K, N = n + 70, 256, 264
    off = gh.offsets_of([n, 70])
    a, dy = gh.randn(R, K, seed=1, dtype=BF16), gh.randn(R, N, seed=2, dtype=BF16)
    ref, mag = gh.weights_grad64(dy[:n], a[:n], off[:2], 1)
    a[n:], dy[n:] = float("inf"), float("nan")
    w = torch.zeros(2, N, K, dtype=BF16, device="cuda")
    _, dw = mq.moe_grouped_product_grad(dy.cuda(), a.cuda(), w, off.cuda(), need_a=False)
    clean(mq)
    gh.check(dw[:1], ref, mag, n)
    assert dw[1].isnan().all()


def test_infinities_in_an_expert_stay_there(mq):
    """An expert whose weights or rows hold infinities and NaN changes no other's rows."""
    counts, K, N = [20, 3, 40, 300], 136, 200
    off = gh.offsets_of(counts)
    a, w = gh.randn(sum(counts), K, seed=1, dtype=F16), gh.randn(4, N, K, seed=2, dtype=F16)
    ref, mag = gh.product64(a, w, off)
    w[1] = float("nan")
    a[23:63] = float("inf")
    out = mq.moe_grouped_product(a.cuda(), w.cuda(), off.cuda())
    clean(mq)
    for rows in (slice(0, 20), slice(63, 363)):
        gh.check(out[rows], ref[rows], mag[rows], K)
    assert out[20:23].isnan().all() and not out[23:63].isfinite().any()


@pytest.mark.parametrize("R", [1, 2, 7, 300])
@pytest.mark.parametrize("N", [1, 7, 33, 257])
def test_dense_odd_sizes(mq, R, N):
    """A dense product (no offsets), odd K out of wider buffers, odd N."""
    K = 67
    a = gh.randn(R, 88, seed=1, dtype=BF16).cuda()[:, 8:8 + K]
    w = gh.randn(N, 72, seed=2, dtype=BF16).cuda()[:, :K]
    ref, mag = gh.product64(a.cpu(), w.cpu()[None], gh.offsets_of([R]))
    gh.check(mq.moe_grouped_product(a, w), ref, mag, K)
    dy = gh.randn(R, 264, seed=3, dtype=BF16).cuda()[:, :N]
    da, dw = mq.moe_grouped_product_grad(dy, a, w)
    clean(mq)
    ref, mag = gh.product64(dy.cpu(), w.cpu().T[None], gh.offsets_of([R]))
    gh.check(da, ref, mag, N, "da")
    ref, mag = gh.weights_grad64(dy.cpu(), a.cpu(), gh.offsets_of([R]), 1)
    gh.check(dw, ref[0], mag[0], R, "dw")


def test_halves_and_interleaved_experts(mq):
    """Weights that are part of a wider tensor: the gate rows of [E, 2I, H], and
    experts interleaved row by row."""
    E, I, H, counts = 3, 72, 136, [9, 0, 40]
    off = gh.offsets_of(counts)
    a = gh.randn(49, H, seed=1, dtype=BF16)
    w13 = gh.randn(E, 2 * I, H, seed=2, dtype=BF16, scale=0.1)
    wide, mixed = w13.cuda(), w13.transpose(0, 1).contiguous().cuda()
    for w, dev in ((w13[:, :I], wide[:, :I]), (w13[:, I:], wide[:, I:]), (w13, mixed.transpose(0, 1))):
        assert not dev.is_contiguous()
        ref, mag = gh.product64(a, w, off)
        gh.check(mq.moe_grouped_product(a.cuda(), dev, off.cuda()), ref, mag, H)
        dy = gh.randn(49, w.shape[1], seed=3, dtype=BF16)
        da, dw = mq.moe_grouped_product_grad(dy.cuda(), a.cuda(), dev, off.cuda())
        gh.check(da, *gh.product64(dy, w.transpose(1, 2), off), w.shape[1], "da")
        gh.check(dw, *gh.weights_grad64(dy, a, off, E), max(counts), "dw")
    clean(mq)


def test_bad_offsets_set_the_status(mq):
    a = gh.randn(40, 64, seed=1, dtype=BF16).cuda()
    w = gh.randn(3, 64, 64, seed=2, dtype=BF16).cuda()
    for o in ([0, 20, 10, 40], [-1, 3, 4, 40], [0, 10, 20, 41], [2 ** 31 - 1, -2 ** 31, 0, 1]):
        off = torch.tensor(o, dtype=torch.int32, device="cuda")
        mq.moe_grouped_product(a, w, off)
        assert mq.mq_device_status() == mq.MQ_DEV_BAD_OFFSETS
        mq.moe_grouped_product_grad(a, a, w, off)
        assert mq.mq_device_status() == mq.MQ_DEV_BAD_OFFSETS
    assert mq.mq_device_status() == 0


def test_no_rows(mq):
    w = gh.randn(3, 64, 72, seed=2, dtype=F16).cuda()
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    a = torch.empty(0, 72, dtype=F16, device="cuda")
    assert mq.moe_grouped_product(a, w, off).shape == (0, 64)
    da, dw = mq.moe_grouped_product_grad(torch.empty(0, 64, dtype=F16, device="cuda"), a, w, off)
    assert da.shape == (0, 72) and (dw == 0).all() and dw.shape == w.shape
    clean(mq)


def test_gradients_alone_and_together(mq):
    """Each gradient by itself has the bits that both together have, where they run side
    by side (many experts, few rows) and where they do not."""
    for counts, K, N in (([40] * 24, 136, 264), ([900, 300], 256, 392), ([5, 3], 64, 64)):
        off = gh.offsets_of(counts).cuda()
        a, dy = gh.randn(sum(counts), K, seed=1, dtype=BF16).cuda(), gh.randn(sum(counts), N, seed=2, dtype=BF16).cuda()
        w = gh.randn(len(counts), N, K, seed=3, dtype=BF16).cuda()
        da, dw = mq.moe_grouped_product_grad(dy, a, w, off)
        da1, none = mq.moe_grouped_product_grad(dy, a, w, off, need_w=False)
        assert none is None and torch.equal(da, da1)
        none, dw1 = mq.moe_grouped_product_grad(dy, a, w, off, need_a=False)
        assert none is None and torch.equal(dw, dw1)
        clean(mq)


@pytest.mark.parametrize("R,K,N", [(1, 65536, 128), (40, 65536, 72), (1040, 65536, 128)])
@pytest.mark.parametrize("transposed", [False, True])
def test_long_sums_with_float32_results(mq, R, K, N, transposed):
    """The tensor core cuts off where it adds.  Sums of 256 products do so 256 times at most,
    by a step of 2^-23 of their own size; their sum, of K / 256 of them, rounds to nearest.
    In one go values of one sign, which are all cut off to the same side, would be out by
    about K / 16 times half a step of half the sum: 1.2e-4 here, where 4.6e-5 are allowed."""
    g = torch.Generator().manual_seed(R)
    a = (torch.rand(R, K, generator=g) + 0.5).to(BF16).cuda()
    w = (torch.rand(N, K, generator=g) + 0.5).to(BF16)
    out = mq.moe_grouped_product(a, storage(w, transposed)[None], out_dtype=F32)
    clean(mq)
    ref = a.double() @ w.cuda().double().T
    assert ((out.double() - ref).abs() <= (256 * gh.STEP + K // 256 * 2.0 ** -24 + 2.0 ** -24) * ref).all()


def test_long_sums_of_weight_gradients(mq):
    """The same over an expert's rows."""
    R, K, N = 16384, 2048, 2048
    g = torch.Generator().manual_seed(3)
    a = (torch.rand(R, K, generator=g) + 0.5).to(F16).cuda()
    dy = (torch.rand(R, N, generator=g) + 0.5).to(F16).cuda()
    w = torch.zeros(1, N, K, dtype=F16, device="cuda")
    _, dw = mq.moe_grouped_product_grad(dy, a, w, need_a=False, dw_dtype=F32)
    clean(mq)
    ref = dy.double().T @ a.double()
    assert ((dw[0].double() - ref).abs() <= (256 * gh.STEP + R // 256 * 2.0 ** -24 + 2.0 ** -24) * ref).all()


@pytest.mark.parametrize("counts,K,N", [([1], 4096, 512), ([700, 300], 512, 512), ([3, 1, 0, 2], 2048, 136)])
def test_same_result_every_time(mq, counts, K, N):
    off = gh.offsets_of(counts).cuda()
    a, w = gh.randn(sum(counts), K, seed=1, dtype=BF16).cuda(), gh.randn(len(counts), N, K, seed=2, dtype=BF16).cuda()
    dy = gh.randn(sum(counts), N, seed=3, dtype=BF16).cuda()
    first = [mq.moe_grouped_product(a, w, off), *mq.moe_grouped_product_grad(dy, a, w, off)]
    for _ in range(3):
        for x, y in zip(first, [mq.moe_grouped_product(a, w, off), *mq.moe_grouped_product_grad(dy, a, w, off)]):
            assert torch.equal(x, y)
    clean(mq)


def test_replayed_graph_and_another_stream(mq):
    """Captured calls replayed on new inputs; offsets change between replays."""
    E, K, N, R = 4, 512, 264, 96
    w = gh.randn(E, N, K, seed=2, dtype=BF16).cuda()
    a, dy = torch.zeros(R, K, dtype=BF16, device="cuda"), torch.zeros(R, N, dtype=BF16, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mq.moe_grouped_product(a, w, off, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mq.moe_grouped_product(a, w, off)
        da, dw = mq.moe_grouped_product_grad(dy, a, w, off)
    for seed, counts in ((5, [10, 0, 80, 6]), (6, [96, 0, 0, 0]), (7, [1, 2, 3, 90])):
        a.copy_(gh.randn(R, K, seed=seed, dtype=BF16))
        dy.copy_(gh.randn(R, N, seed=seed + 10, dtype=BF16))
        off.copy_(gh.offsets_of(counts))
        graph.replay()
        clean(mq)
        o = off.cpu()
        gh.check(out, *gh.product64(a.cpu(), w.cpu(), o), K, "out")
        gh.check(da, *gh.product64(dy.cpu(), w.cpu().transpose(1, 2), o), N, "da")
        gh.check(dw, *gh.weights_grad64(dy.cpu(), a.cpu(), o, E), max(counts), "dw")


def leaves(E, N, K, R, dtype, seed=1):
    a = gh.randn(R, K, seed=seed, dtype=dtype).cuda().requires_grad_()
    w = gh.randn(E, N, K, seed=seed + 1, dtype=dtype, scale=0.1).cuda().requires_grad_()
    return a, w


@pytest.mark.parametrize("N", [72, 33])
@pytest.mark.parametrize("out_dtype", [None, F32])
def test_autograd_against_the_formulas(mq, N, out_dtype):
    """The recorded call's gradients, with rows of no expert; odd N too, whose
    gradient comes in with rows on odd boundaries."""
    counts, K = [5, 0, 20], 64
    off = gh.offsets_of(counts, 1)
    R = sum(counts) + 3
    a, w = leaves(3, N, K, R, BF16)
    y = mq.moe_grouped_product(a, w, off.cuda(), out_dtype=out_dtype)
    assert y.requires_grad and y.dtype == (out_dtype or BF16)
    gy = gh.randn(R, N, seed=9, dtype=BF16)
    y.backward(gy.cuda().to(y.dtype))
    clean(mq)
    gh.check(a.grad, *gh.product64(gy, w.detach().cpu().transpose(1, 2), off), N, "da")
    gh.check(w.grad, *gh.weights_grad64(gy, a.detach().cpu(), off, 3), max(counts), "dw")
    assert (a.grad[0] == 0).all() and (a.grad[-2:] == 0).all()


def test_autograd_against_differences(mq):
    """A float32 result is linear in each operand: the difference quotient over a step
    is the derivative, but for what the steps' rounding to the operands' type does,
    which is none here (small whole numbers)."""
    off = gh.offsets_of([4, 3]).cuda()
    g = torch.Generator().manual_seed(1)
    a = torch.randint(-3, 4, (7, 16), generator=g).to(F16).cuda().requires_grad_()
    w = torch.randint(-3, 4, (2, 8, 16), generator=g).to(F16).cuda().requires_grad_()
    c = torch.randint(-3, 4, (7, 8), generator=g).float().cuda()

    def loss(a, w):
        return (mq.moe_grouped_product(a, w, off, out_dtype=F32) * c).sum()
    loss(a, w).backward()
    with torch.no_grad():
        for leaf in (a, w):
            flat, base = leaf.view(-1), loss(a, w)
            for i in range(0, flat.numel(), 5):
                flat[i] += 1
                diff = loss(a, w) - base
                flat[i] -= 1
                assert diff == leaf.grad.view(-1)[i]


def test_autograd_only_where_it_is_asked_for(mq):
    off = gh.offsets_of([4, 4]).cuda()
    a, w = leaves(2, 64, 64, 8, BF16)
    with torch.no_grad():
        assert not mq.moe_grouped_product(a, w, off).requires_grad
    y = mq.moe_grouped_product(a.detach(), w, off)
    y.sum().backward()
    assert a.grad is None and w.grad is not None
    w.grad = None
    mq.moe_grouped_product(a, w.detach(), off).sum().backward()   # (an expanded gradient)
    assert w.grad is None and a.grad is not None
    with pytest.raises(ValueError, match="out"):
        mq.moe_grouped_product(a, w, off, out=torch.empty(8, 64, dtype=BF16, device="cuda"))
    clean(mq)


def test_training_step_in_a_graph(mq):
    """Forward and backward captured together, replayed on new rows."""
    off = gh.offsets_of([30, 2, 32]).cuda()
    a, w = leaves(3, 72, 64, 64, BF16)
    gy = gh.randn(64, 72, seed=3, dtype=BF16).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(mq.moe_grouped_product(a, w, off), (a, w), gy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        da, dw = torch.autograd.grad(mq.moe_grouped_product(a, w, off), (a, w), gy)
    with torch.no_grad():
        a.copy_(gh.randn(64, 64, seed=8, dtype=BF16))
    graph.replay()
    clean(mq)
    gh.check(dw, *gh.weights_grad64(gy.cpu(), a.detach().cpu(), off.cpu(), 3), 32, "dw")
    gh.check(da, *gh.product64(gy.cpu(), w.detach().cpu().transpose(1, 2), off.cpu()), 72, "da")


def test_operands_and_results_side_by_side_in_one_allocation(mq):
    """Results that begin where an input ends, and the other way round."""
    R, K, N, E = 64, 64, 128, 2
    buf = torch.zeros(R * N + R * K + E * N * K + R * N + R * K + E * N * K, dtype=BF16, device="cuda")
    parts, at = [], 0
    for shape in ((R, N), (R, K), (E, N, K), (R, N), (R, K), (E, N, K)):
        n = torch.Size(shape).numel()
        parts.append(buf[at:at + n].view(shape))
        at += n
    out, a, w, dy, da, dw = parts
    for t, seed in ((a, 1), (w, 2), (dy, 3)):
        t.copy_(gh.randn(*t.shape, seed=seed, dtype=BF16))
    off = gh.offsets_of([24, 40])
    mq.moe_grouped_product(a, w, off.cuda(), out=out)
    mq.moe_grouped_product_grad(dy, a, w, off.cuda(), da=da, dw=dw)
    clean(mq)
    gh.check(out, *gh.product64(a.cpu(), w.cpu(), off), K, "out")
    gh.check(da, *gh.product64(dy.cpu(), w.cpu().transpose(1, 2), off), N, "da")
    gh.check(dw, *gh.weights_grad64(dy.cpu(), a.cpu(), off, E), 40, "dw")
    with pytest.raises(mq.MoeqError, match="share"):
        mq.moe_grouped_product(a, w, off.cuda(), out=buf[R * N - 64:2 * R * N - 64].view(R, N))


def test_call_from_a_new_thread(mq):
    """A thread whose first CUDA work is the call."""
    import threading
    off = gh.offsets_of([5, 6]).cuda()
    a, w = gh.randn(11, 64, seed=1, dtype=BF16).cuda(), gh.randn(2, 40, 64, seed=2, dtype=BF16).cuda()
    want = mq.moe_grouped_product(a, w, off)
    torch.cuda.synchronize()
    got = []
    stream = torch.cuda.current_stream()

    def work():
        got.append(mq.moe_grouped_product(a, w, off, stream=stream))
    t = threading.Thread(target=work)
    t.start()
    t.join()
    clean(mq)
    assert torch.equal(got[0], want)
