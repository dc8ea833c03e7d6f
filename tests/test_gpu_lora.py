"""Low-rank adapters of many requests against their 64-bit definition, in both forms
(clusters of single rows, tiles of 128 rows) and at their borders."""

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


class Case:
    """Inputs on the host, the call on the device."""

    def __init__(self, R, K, N, r, L, ids, dtype=BF16, out_dtype=None, counts=None, before=0, seed=0, base=True,
                 scaled=True):
        self.dtype, self.out_dtype = dtype, out_dtype or dtype
        E = len(counts) if counts else 1
        self.off = gh.offsets_of(counts, before) if counts else None
        self.experts = [0] * R
        if counts:
            self.experts = [-1] * R
            for e, rows in enumerate(gh.rows_of(self.off)):
                for t in range(rows.start, rows.stop):
                    self.experts[t] = e
        g = torch.Generator().manual_seed(seed)
        self.x = gh.randn(R, K, seed=seed + 1, dtype=dtype)
        self.a = gh.randn(L, E, r, K, seed=seed + 2, dtype=dtype, scale=K ** -0.5)
        self.b = gh.randn(L, E, N, r, seed=seed + 3, dtype=dtype, scale=r ** -0.5)
        self.ids = torch.tensor(ids(R, L, g) if callable(ids) else ids, dtype=torch.int32)
        self.scaling = torch.rand(L, generator=g) + 0.5 if scaled else None
        self.base = gh.randn(R, N, seed=seed + 4, dtype=self.out_dtype) if base else None
        self.flat = E == 1 and counts is None

    def ref(self):
        return gh.lora64(self.x, self.a, self.b, self.ids.tolist(), self.experts, self.scaling, self.base, self.dtype)

    def call(self, mq, **k):
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        a, b = (self.a[:, 0], self.b[:, 0]) if self.flat else (self.a, self.b)
        args = dict(base=c(self.base), expert_offsets=c(self.off), scaling=c(self.scaling), out_dtype=self.out_dtype)
        args.update(k)
        return mq.moe_lora_product(c(self.x), c(a.contiguous()), c(b.contiguous()), c(self.ids), **args)

    def check(self, got, what=""):
        ref, off = self.ref()
        inside = [t for t in range(len(self.experts)) if self.experts[t] >= 0]
        gh.check_lora(got[inside], ref[inside], off[inside], what)


def runs(length):
    """Requests of about this many rows each, a fifth of them without an adapter."""
    def make(R, L, g):
        ids = []
        while len(ids) < R:
            l = int(torch.randint(L, (1,), generator=g))
            n = 1 + int(torch.randint(2 * length, (1,), generator=g))
            ids += [l if torch.rand(1, generator=g) > 0.2 else -1] * n
        return ids[:R]
    return make


def mixed(R, L, g):
    return torch.randint(-1, L, (R,), generator=g).tolist()


SMALL = [  # (R, K, N, r, L): rows
    (1, 64, 64, 8, 1), (1, 4096, 512, 16, 3), (2, 8, 1, 8, 2), (5, 72, 33, 24, 4), (17, 264, 1000, 32, 2),
    (64, 512, 520, 64, 48), (130, 136, 257, 72, 7), (3, 2048, 40, 128, 5),
]
LARGE = [  # tiles: more than 1024 rows
    (1025, 64, 128, 8, 1), (1100, 72, 136, 16, 5), (1153, 200, 264, 24, 9), (1280, 128, 72, 32, 3),
    (1031, 320, 33, 64, 4), (1200, 64, 384, 72, 6), (1100, 136, 200, 128, 3),
]


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, BF16)])
@pytest.mark.parametrize("ids", [runs(60), mixed], ids=["runs", "mixed"])
@pytest.mark.parametrize("sizes", SMALL + LARGE)
def test_adapters(mq, sizes, ids, dtype, out_dtype):
    c = Case(*sizes, ids, dtype=dtype, out_dtype=out_dtype, seed=sizes[0])
    got = c.call(mq)
    clean(mq)
    assert got.dtype == out_dtype
    c.check(got)


def test_both_forms_are_tested(mq):
    """(Only the tiles have a workspace.)"""
    for R, K, N, r, L in SMALL:
        assert mq.moe_lora_product_workspace(R, K, N, r, L) == 0
    for R, K, N, r, L in LARGE:
        assert mq.moe_lora_product_workspace(R, K, N, r, L) > 0


@pytest.mark.parametrize("R", [1, 3, 17, 129])
@pytest.mark.parametrize("r", [96, 128])
def test_few_rows_of_high_rank(mq, R, r):
    """Tiles that are mostly empty."""
    K, N = 4096, 4104
    assert r == 96 or mq.moe_lora_product_workspace(R, K, N, r, 5) > 0
    for ids in (mixed, runs(2), [0] * R):
        for dtype, out_dtype in ((BF16, BF16), (F16, F32)):
            c = Case(R, K, N, r, 5, ids, dtype=dtype, out_dtype=out_dtype, seed=R)
            got = c.call(mq)
            clean(mq)
            c.check(got)


@pytest.mark.parametrize("r,L", [(128, 40), (64, 100), (16, 300)])
def test_many_large_adapters_on_few_tiles(mq, r, L):
    """Few rows whose adapters are large: a tile's groups are divided among CTAs."""
    K, N = (2048, 2040) if r == 128 else (2560, 2560) if r == 64 else (4096, 4096)
    R = 700 if r == 16 else 300
    assert mq.moe_lora_product_workspace(R, K, N, r, L) > 0
    for ids in (mixed, runs(30)):
        c = Case(R, K, N, r, L, ids, seed=r)
        got = c.call(mq)
        clean(mq)
        c.check(got)


@pytest.mark.parametrize("base", [True, False])
@pytest.mark.parametrize("N", [136, 33])
@pytest.mark.parametrize("counts,before,behind", [([3, 0, 1], 0, 0), ([0, 40, 7, 0], 2, 3),
                                                  ([500, 0, 300, 260], 3, 2), ([20] * 64, 0, 1), ([0, 0], 5, 4),
                                                  ([0, 0], 700, 700)])
def test_experts(mq, counts, before, behind, N, base):
    R = before + sum(counts) + behind
    c = Case(R, 72, N, 16, 3, runs(9), counts=counts, before=before, seed=R, base=base)
    c.x[:before] = float("nan")                  # rows of no expert reach nothing
    c.x[R - behind:] = float("inf")
    out = torch.full((R, N), 7.0, dtype=BF16, device="cuda")
    assert c.call(mq, out=out) is out
    clean(mq)
    c.check(out)
    assert (out[:before] == 7).all() and (out[R - behind:] == 7).all()


@pytest.mark.parametrize("R", [40, 1300])
@pytest.mark.parametrize("N", [264, 65])
def test_in_place_and_strided(mq, R, N):
    c = Case(R, 64, N, 16, 4, runs(50), seed=R)
    ref, off = c.ref()
    base = c.base.cuda()
    assert c.call(mq, base=base, out=base) is base
    gh.check_lora(base, ref, off, "in place")
    for pad in (8, 3):                           # slices of one wider buffer
        wide = torch.full((R, 2 * N + 3 * pad), 7.0, dtype=BF16, device="cuda")
        b, o = wide[:, pad:pad + N], wide[:, 2 * pad + N:2 * pad + 2 * N]
        b.copy_(c.base)
        c.call(mq, base=b, out=o)
        gh.check_lora(o, ref, off, "strided")
        assert torch.equal(b, c.base.cuda())
        c.call(mq, base=b, out=b)
        gh.check_lora(b, ref, off, "strided in place")
        rest = torch.ones(wide.shape[1], dtype=torch.bool)
        rest[pad:pad + N] = rest[2 * pad + N:2 * pad + 2 * N] = False
        assert (wide[:, rest.cuda()] == 7).all()
    x = gh.randn(R, 88, seed=5, dtype=BF16)
    c.x = x[:, 8:72]
    xs = x.cuda()[:, 8:72]
    got = mq.moe_lora_product(xs, c.a[:, 0].cuda(), c.b[:, 0].cuda(), c.ids.cuda(), base=c.base.cuda(),
                              scaling=c.scaling.cuda())
    clean(mq)
    c.check(got)


@pytest.mark.parametrize("R", [60, 1100])
def test_without_base_and_scaling(mq, R):
    c = Case(R, 128, 72, 32, 3, mixed, seed=1, base=False, scaled=False)
    got = c.call(mq)
    clean(mq)
    c.check(got)
    assert (got[(c.ids == -1).cuda()] == 0).all()


@pytest.mark.parametrize("R", [50, 1100])
def test_rows_without_adapters_keep_base(mq, R):
    c = Case(R, 64, 72, 16, 3, [-1] * R, seed=1)
    c.base[1] = float("nan")
    c.base[2] = float("-inf")
    got = c.call(mq)
    clean(mq)
    assert torch.equal(got.view(torch.int16), c.base.cuda().view(torch.int16))


@pytest.mark.parametrize("R", [50, 1100])
def test_another_request_infinities_stay_there(mq, R):
    """Adapter 1 holds NaN, row 3 infinities: no other adapter's rows change."""
    c = Case(R, 136, 200, 16, 3, [0, 1, 2, 0, -1] * (R // 5), seed=2)
    ref, off = c.ref()
    c.a[1], c.b[1] = float("nan"), float("inf")
    c.x[3] = float("inf")
    got = c.call(mq)
    clean(mq)
    rows = [t for t in range(R) if c.ids[t] != 1 and t != 3]
    gh.check_lora(got[rows], ref[rows], off[rows])
    assert got[[t for t in range(R) if c.ids[t] == 1]].isnan().all() and not got[3].isfinite().any()


@pytest.mark.parametrize("R", [30, 1100])
@pytest.mark.parametrize("scale", [1e5, 1e-6])
def test_sums_outside_f16(mq, R, scale):
    """A x beyond f16's range, or among its subnormals, is not cut: the scaling brings
    the result back."""
    c = Case(R, 64, 72, 16, 2, runs(20), dtype=F16, seed=4, out_dtype=F32)
    c.x = (c.x * 100).to(F16)
    c.scaling = torch.tensor([scale, scale * 1.5])
    got = c.call(mq)
    clean(mq)
    c.check(got)


@pytest.mark.parametrize("R", [30, 1100])
def test_infinite_sums(mq, R):
    """An infinite A x gives what the formula gives: infinities of the second factor's
    signs."""
    c = Case(R, 64, 72, 8, 1, [0] * R, seed=4, base=False, scaled=False)
    c.a[0, 0, 1:] = 0
    c.a[0, 0, 0] = 1
    c.x[:] = 1
    c.x[7, 3] = float("inf")
    c.a[0, 0, 1:, 3] = 0.5
    c.a[0, 0, 1:] = c.a[0, 0, 0]      # every rank sums to infinity
    c.b[0, 0] = c.b[0, 0].abs()
    c.b[0, 0, 5] = -c.b[0, 0, 5]
    got = c.call(mq)
    clean(mq)
    want = torch.full((72,), float("inf"))
    want[5] = float("-inf")
    assert torch.equal(got[7].float().cpu(), want)
    assert got[:7].isfinite().all() and got[8:].isfinite().all()


@pytest.mark.parametrize("R", [40, 1100])
def test_bad_ids_and_offsets_set_the_status(mq, R):
    c = Case(R, 64, 72, 16, 3, [0, 1, 3, -2] * (R // 4) , seed=2)
    got = c.call(mq)
    torch.cuda.synchronize()
    assert mq.mq_device_status() == mq.MQ_DEV_BAD_ADAPTER_ID
    bad = ((c.ids > 2) | (c.ids < 0)).cuda()
    assert torch.equal(got[bad], c.base.cuda()[bad])
    c.ids[bad.cpu()] = -1
    c.check(got)
    for o in ([0, R + 1], [-1, R], [5, 4], [2 ** 31 - 1, -2 ** 31]):
        out = torch.full((R, 72), 7.0, dtype=BF16, device="cuda")
        c.call(mq, expert_offsets=torch.tensor(o, dtype=torch.int32, device="cuda"), out=out)
        torch.cuda.synchronize()
        assert mq.mq_device_status() == mq.MQ_DEV_BAD_OFFSETS
        assert (out == 7).all()
    c.ids[:] = 2 ** 31 - 1
    c.call(mq)
    torch.cuda.synchronize()
    assert mq.mq_device_status() == mq.MQ_DEV_BAD_ADAPTER_ID


def test_no_rows(mq):
    c = Case(0, 64, 72, 16, 3, [], seed=2)
    assert c.call(mq).shape == (0, 72)
    clean(mq)


@pytest.mark.parametrize("R", [64, 1500])
def test_a_row_does_not_depend_on_its_neighbours(mq, R):
    """The same rows in another order give the same bits (within one form)."""
    c = Case(R, 512, 264, 32, 5, mixed, seed=3)
    got = c.call(mq)
    for _ in range(2):
        assert torch.equal(got, c.call(mq))
    p = torch.randperm(R, generator=torch.Generator().manual_seed(1))
    c.x, c.ids, c.base = c.x[p], c.ids[p], c.base[p]
    assert torch.equal(c.call(mq), got[p.cuda()])
    clean(mq)


@pytest.mark.parametrize("R", [24, 1200])
def test_replayed_graphs_that_share_a_workspace(mq, R):
    """Two captured calls with one workspace, replayed in turn on new inputs."""
    c = Case(R, 256, 136, 16, 4, runs(40), seed=1)
    need = mq.moe_lora_product_workspace(R, 256, 136, 16, 4)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    x, ids, base = c.x.cuda(), c.ids.cuda(), c.base.cuda()
    a, b, s = c.a[:, 0].cuda(), c.b[:, 0].cuda(), c.scaling.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mq.moe_lora_product(x, a, b, ids, base=base, scaling=s, workspace=ws, stream=side)
    side.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(mq.moe_lora_product(x, a, b, ids, base=base, scaling=s, workspace=ws))
        graphs.append(g)
    for seed in (5, 6):
        d = Case(R, 256, 136, 16, 4, mixed, seed=seed)
        c.x, c.ids = d.x, d.ids
        x.copy_(d.x)
        ids.copy_(d.ids)
        for g, out in zip(graphs, outs):
            g.replay()
            clean(mq)
            c.check(out)


def test_gradients_are_refused(mq):
    c = Case(8, 64, 72, 16, 2, mixed, seed=1)
    c.a.requires_grad_()
    with pytest.raises(ValueError, match="moe_grouped_product"):
        c.call(mq)
    with torch.no_grad():
        c.call(mq)
    clean(mq)


@pytest.mark.parametrize("r", [16, 32, 64, 128])
def test_many_calls_in_a_queue(mq, r):
    """Thousands of calls without a wait between them, on inputs in turn: tiles with two
    and more groups, whose loads come in any order.  (Two warps consume them: each has to
    have slots of its own.)"""
    R, K, N = 1100, 512, 1024
    cases = [Case(R, K, N, r, 6, runs(40), seed=s) for s in (1, 2, 3)]
    dev = [tuple(t.cuda() for t in (c.x, c.a[:, 0].contiguous(), c.b[:, 0].contiguous(), c.ids, c.base, c.scaling))
           for c in cases]

    def call(i):
        x, a, b, ids, base, s = dev[i % 3]
        return mq.moe_lora_product(x, a, b, ids, base=base, scaling=s)
    first = [call(i) for i in range(3)]
    for c, got in zip(cases, first):
        c.check(got)
    for rounds in range(3):
        last = [call(i) for i in range(999)][-3:]
        clean(mq)
        for got, want in zip(last, first):
            assert torch.equal(got, want)
