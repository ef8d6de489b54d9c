"""Layer norm, embedding and the head's cross entropy on the GPU, against their definitions in
64 bits.  Bounds count roundings: u = 2^-24 per fp32 operation, half a step of the output's type
for the one rounding of a 16-bit output."""
import math

import pytest
import torch

import zero_partitioned_optimizer_shard_gb300 as z

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
# half a step, relative (finfo.eps / 2); and for the smallest values half of the subnormal step
HALF = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
TINY = {BF16: 2.0 ** -134, F16: 2.0 ** -25, F32: 2.0 ** -150}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def gen(seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, sigma=1.0, dtype=F32):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, sigma, generator=g)


def rows_of(g, n, d, dtype, pad=0, sigma=1.0):
    return normal(g, n, d + pad, sigma=sigma, dtype=dtype)[:, :d]


def check(name, got, want, err):
    """|got - want| <= err + the output's rounding, element by element; the same NaN places."""
    got64, want = got.double(), want.double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got64), nan), f"{name}: NaN places differ"
    # before its one rounding the value is within err of the definition's
    lim = err * (1 + HALF[got.dtype]) + HALF[got.dtype] * want.abs() + TINY[got.dtype]
    bad = ((got64 - want).abs() > lim) & ~nan
    if bad.any():
        i = int(torch.argmax(((got64 - want).abs() / lim).nan_to_num(0).flatten()))
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, worst at {i}: {got64.flatten()[i]} "
                             f"against {want.flatten()[i]}, bound {lim.flatten()[i] if lim.dim() else lim}")


def work_bytes(n):
    return torch.full((max(n, 1),), 0xA5, dtype=torch.uint8, device="cuda")  # needs no initialisation


# ------------------------------------------------------------------------------------------
# layer norm
# ------------------------------------------------------------------------------------------
SHAPES = [(1, 1), (1, 8), (3, 17), (5, 64), (257, 641), (64, 1600), (33, 2048), (9, 2056), (7, 4096), (5, 4104),
          (3, 8192), (6, 8200), (2, 12001), (3, 16384), (1000, 40), (4099, 96)]
TYPES = [(BF16, BF16), (F16, F16), (F32, F32), (BF16, F32), (F16, F32)]


def norm_forward(x, w, b, eps):
    x, w = x.double(), w.double()
    mean = x.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    return (x - mean) * rstd * w + (0.0 if b is None else b.double()), mean[..., 0], rstd[..., 0]


def norm_bounds(x, w, mean, rstd, y):
    """Sums of a row go through at most 8 x 8 + 8 + 10 additions: 96 roundings of the largest
    magnitude bound the mean's, and (twice halved) the deviation's, relative error."""
    top = x.double().abs().amax(-1, keepdim=True)
    r, xh = rstd[..., None], ((x.double() - mean[..., None]) * rstd[..., None]).abs()
    return 96 * U * (top * r * w.double().abs() * (1 + xh) + y.abs()), 96 * U * top[..., 0]


@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("n,d", SHAPES)
def test_layernorm(n, d, dtype, ptype):
    g = gen(n * 7 + d)
    for pad, bias in ((0, True), (7, False)):
        x = rows_of(g, n, d, dtype, pad) + 0.5
        if pad:
            x = torch.nn.functional.pad(x, (0, pad))[:, :d]
        w, b = normal(g, d, dtype=ptype) + 1.0, normal(g, d, dtype=ptype) if bias else None
        y = torch.full((n, d + pad), 7.0, dtype=dtype, device="cuda")
        mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        z.zero_layernorm(x, w, b, y[:, :d], mean, rstd, eps=1e-5)
        want, m64, r64 = norm_forward(x, w, b, 1e-5)
        ey, em = norm_bounds(x, w, m64, r64, want)
        check("y", y[:, :d], want, ey)
        check("mean", mean, m64, em)
        check("rstd", rstd, r64, 96 * U * r64 * (1 + (x.double().abs().amax(-1) * r64)))
        assert (y[:, d:] == 7.0).all()
        z.zero_layernorm(x, w, b, y[:, :d], eps=1e-5)   # without statistics: the same
        check("y", y[:, :d], want, ey)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,d", [(40000, 64), (20011, 128), (30001, 10), (30001, 34), (10007, 135), (10007, 256), (157, 200)])
def test_short_rows(n, d, dtype):
    """Heads' norms: many rows of at most 256 elements, several to a warp."""
    g = gen(n + d)
    x, dy = rows_of(g, n, d, dtype, 0 if d % 8 == 0 else 3), rows_of(g, n, d, dtype)
    w, b = normal(g, d, dtype=dtype) + 1.0, normal(g, d, dtype=dtype)
    y, mean, rstd = torch.empty(n, d, dtype=dtype, device="cuda"), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    z.zero_layernorm(x, w, b, y, mean, rstd)
    want, m64, r64 = norm_forward(x, w, b, 1e-5)
    check("y", y, want, norm_bounds(x, w, m64, r64, want)[0])
    dx, dw, db = torch.empty_like(y), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    z.zero_layernorm_backward(x, w, mean, rstd, dy, dx, dw, db, work_bytes(z.zero_layernorm_workspace_bytes(n, d)))
    wx, ex, ww, ew, wb, eb = norm_backward(x, w, mean, rstd, dy)
    check("dx", dx, wx, ex)
    check("dweight", dw, ww, ew)
    check("dbias", db, wb, eb)


def test_layernorm_far_mean_constant_rows_and_nan():
    g = gen(5)
    x = normal(g, 64, 1600) + 4096.0
    x[3] = 17.0
    x[5, 100] = float("nan")
    x[9, 7] = float("inf")
    w, b = normal(g, 1600) + 1.0, normal(g, 1600)
    y, mean, rstd = torch.empty_like(x), torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    z.zero_layernorm(x, w, b, y, mean, rstd)
    want, m64, r64 = norm_forward(x, w, b, 1e-5)
    ok = torch.tensor([i not in (3, 5, 9) for i in range(64)], device="cuda")
    ey, _ = norm_bounds(x, w, m64, r64, want)
    check("y", y[ok], want[ok], ey[ok])
    # a constant row: the mean is the value but for 96 roundings; times rstd = eps^-1/2
    check("constant", y[3], b.double(), 96 * U * 17.0 * 1e-5 ** -0.5 * w.double().abs() + U * b.double().abs())
    assert torch.isnan(y[5]).all() and torch.isnan(y[9]).any()


def norm_backward(x, w, mean, rstd, dy):
    x, w, dy, mean, rstd = x.double(), w.double(), dy.double(), mean.double()[:, None], rstd.double()[:, None]
    xh = (x - mean) * rstd
    gg = dy * w
    dx = rstd * (gg - gg.mean(1, keepdim=True) - xh * (gg * xh).mean(1, keepdim=True))
    # every operation of an element, and 96 additions of a row's sums, at the terms' magnitudes
    ex = 96 * U * rstd * (gg.abs() + gg.abs().mean(1, keepdim=True) + xh.abs() * (gg * xh).abs().mean(1, keepdim=True) * 2)
    # a column's sum: a block's rows one after another, then the blocks': below 200 additions
    return dx, ex, (dy * xh).sum(0), 200 * U * (dy * xh).abs().sum(0), dy.sum(0), 200 * U * dy.abs().sum(0)


@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("n,d", SHAPES)
def test_layernorm_backward(n, d, dtype, ptype):
    g = gen(n * 11 + d)
    for pad, acc, gt in ((0, False, dtype), (7, True, F32), (0, True, dtype), (8, False, F32)):
        x, dy = rows_of(g, n, d, dtype, pad), rows_of(g, n, d, dtype, pad)
        w = normal(g, d, dtype=ptype) + 1.0
        mean, rstd = x.float().mean(1), torch.rand(n, device="cuda", generator=g) + 0.5
        dx = torch.full((n, d + pad), 7.0, dtype=dtype, device="cuda")
        dw, db = normal(g, d, dtype=gt), normal(g, d, dtype=gt)
        dw0, db0 = (dw.double(), db.double()) if acc else (0.0, 0.0)
        work = work_bytes(z.zero_layernorm_workspace_bytes(n, d))
        z.zero_layernorm_backward(x, w, mean, rstd, dy, dx[:, :d], dw, db, work, accumulate=acc)
        rx, ex, rw, ew, rb, eb = norm_backward(x, w, mean, rstd, dy)
        check("dx", dx[:, :d], rx, ex)
        check("dweight", dw, rw + dw0, ew)
        check("dbias", db, rb + db0, eb)
        assert (dx[:, d:] == 7.0).all()


@pytest.mark.parametrize("d", [24, 17, 1600, 8200, 12001])
def test_layernorm_backward_of_a_large_constant_row(d):
    """mean * rstd is more than fp32 holds, the row's own differences are 0: its gradient is finite."""
    g = gen(d)
    x, dy, w = normal(g, 9, d), normal(g, 9, d), normal(g, d)
    x[4] = 2.0 ** 120
    mean, rstd = x.mean(1), torch.full((9,), 2.0, device="cuda")
    mean[4], rstd[4] = 2.0 ** 120, 2.0 ** 10
    dx, dw, db = torch.empty_like(x), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    z.zero_layernorm_backward(x, w, mean, rstd, dy, dx, dw, db, work_bytes(z.zero_layernorm_workspace_bytes(9, d)))
    wx, ex, ww, ew, wb, eb = norm_backward(x, w, mean, rstd, dy)
    check("dx", dx, wx, ex)
    check("dweight", dw, ww, ew)
    check("dbias", db, wb, eb)


def test_layernorm_backward_without_some_outputs_and_without_rows():
    g = gen(2)
    x, dy, w = normal(g, 50, 96), normal(g, 50, 96), normal(g, 96)
    mean, rstd = x.mean(1), torch.ones(50, device="cuda")
    work = work_bytes(z.zero_layernorm_workspace_bytes(50, 96))
    rx, ex, rw, ew, rb, eb = norm_backward(x, w, mean, rstd, dy)
    for dw, db in ((torch.empty(96, device="cuda"), None), (None, torch.empty(96, device="cuda")), (None, None)):
        dx = torch.empty_like(x)
        z.zero_layernorm_backward(x, w, mean, rstd, dy, dx, dw, db, work)
        check("dx", dx, rx, ex)
        if dw is not None:
            check("dweight", dw, rw, ew)
        if db is not None:
            check("dbias", db, rb, eb)
    dw, db = torch.ones(96, device="cuda"), torch.ones(96, device="cuda")
    none = x[:0]
    z.zero_layernorm_backward(none, w, mean[:0], rstd[:0], none, none.clone(), dw, db, work, accumulate=True)
    assert (dw == 1).all() and (db == 1).all()
    z.zero_layernorm_backward(none, w, mean[:0], rstd[:0], none, none.clone(), dw, db, work)
    assert (dw == 0).all() and (db == 0).all()


def test_layernorm_gradients_against_differences():
    """The directional derivative of sum(y * c) by differences of the definition in 64 bits."""
    g = gen(8)
    x, w, b, c = normal(g, 40, 200), normal(g, 200) + 1.0, normal(g, 200), normal(g, 40, 200)
    y, mean, rstd = torch.empty_like(x), torch.empty(40, device="cuda"), torch.empty(40, device="cuda")
    z.zero_layernorm(x, w, b, y, mean, rstd)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    z.zero_layernorm_backward(x, w, mean, rstd, c, dx, dw, db, work_bytes(z.zero_layernorm_workspace_bytes(40, 200)))
    vx, vw, vb = (normal(g, *t.shape).double() for t in (x, w, b))
    f = lambda h: (norm_forward(x.double() + h * vx, w.double() + h * vw, b.double() + h * vb, 1e-5)[0] * c).sum()  # noqa: E731
    h = 1e-4
    want = (f(h) - f(-h)) / (2 * h)
    terms = ((dx * vx).sum(), (dw * vw).sum(), (db * vb).sum())
    size = (dx * vx).abs().sum() + (dw * vw).abs().sum() + (db * vb).abs().sum()
    # central differences: h^2 of the third derivative, below 1e-6 of the terms
    assert abs(float(sum(terms) - want)) <= 2e-6 * float(size)


# ------------------------------------------------------------------------------------------
# embedding
# ------------------------------------------------------------------------------------------
EMBED = [(1, 8, 17), (1, 1, 1), (5, 17, 3), (16, 1600, 50), (100, 64, 100000), (257, 641, 10007), (4096, 72, 31),
         (8192, 40, 300), (8193, 48, 70000), (20000, 8, 1000), (33, 4096, 8), (40, 2056, 257), (1000, 24, 1)]


def ids(g, n, v, dtype, missing=0.1):
    t = torch.randint(0, v, (n,), device="cuda", generator=g, dtype=torch.int64)
    t = torch.where(torch.rand(n, device="cuda", generator=g) < 0.3, t % max(1, v // 50), t)  # some often
    m = torch.rand(n, device="cuda", generator=g) < missing
    odd = torch.tensor([-1, v, -100, 2 ** 31 - 1], device="cuda")[torch.arange(n, device="cuda") % 4]
    return torch.where(m, odd, t).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("n,d,v", EMBED)
def test_embedding(n, d, v, dtype):
    g = gen(n + d)
    for it, scale, pad in ((torch.int64, 1.0, 0), (torch.int32, 3.7, 5)):
        t, table = ids(g, n, v, it), normal(g, v, d, dtype=dtype)
        out = torch.full((n, d + pad), 7.0, dtype=dtype, device="cuda")
        z.zero_embedding(t, table, out[:, :d], scale=scale)
        there = (t >= 0) & (t < v)
        rows = (table[t.clamp(0, v - 1).long()].float() * torch.tensor(scale, device="cuda")).to(dtype)
        want = torch.where(there[:, None], rows, torch.zeros_like(rows))
        assert torch.equal(out[:, :d], want)       # one product, one rounding: the same bits
        assert (out[:, d:] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("n,d,v", EMBED)
def test_embedding_backward(n, d, v, dtype):
    g = gen(n * 3 + d)
    for it, scale, pad, acc, gt in ((torch.int64, 1.0, 0, False, dtype), (torch.int32, 3.7, 5, True, F32),
                                    (torch.int64, 0.5, 8, True, dtype)):
        t, dout = ids(g, n, v, it), rows_of(g, n, d, dtype, pad)
        dtable = normal(g, v, d, dtype=gt)
        old = dtable.clone()
        work = work_bytes(z.zero_embedding_workspace_bytes(n, d, v))
        z.zero_embedding_backward(t, dout, dtable, work, scale=scale, accumulate=acc)
        s32 = float(torch.tensor(scale))
        there = (t >= 0) & (t < v)
        at, rows = t[there].long(), dout[there].double()
        want = torch.zeros(v, d, dtype=torch.float64, device="cuda").index_add_(0, at, rows * s32)
        size = torch.zeros(v, d, dtype=torch.float64, device="cuda").index_add_(0, at, rows.abs() * s32)
        count = torch.zeros(v, dtype=torch.float64, device="cuda").index_add_(0, at, torch.ones_like(rows[:, 0]))
        if acc:
            want = want + old.double()
        check("dtable", dtable, want, (count[:, None] + 4) * U * size + (2 * U * old.double().abs() if acc else 0.0))
        if acc:
            assert torch.equal(dtable[count == 0], old[count == 0])
        again = old.clone()
        work.fill_(0x5A)
        z.zero_embedding_backward(t, dout, again, work, scale=scale, accumulate=acc)
        assert torch.equal(again.view(torch.uint8), dtable.view(torch.uint8))  # the same bits


@pytest.mark.parametrize("n,d,v,gt", [(3000, 1600, 33000, BF16), (8192, 64, 400_000, F32), (9000, 1600, 33000, BF16),
                                      (1, 4096, 40000, BF16)])
def test_embedding_backward_of_large_tables(n, d, v, gt):
    """Tables whose zeros are written in two parts, the second beside the sums: every row is
    written, once."""
    g = gen(n)
    t = ids(g, n, v, torch.int64, 0.05)
    t[:1] = v - 1
    t[1:2] = 0
    dout = normal(g, n, d, dtype=BF16)
    dtable = torch.full((v, d), float("nan"), dtype=gt, device="cuda")
    z.zero_embedding_backward(t, dout, dtable, work_bytes(z.zero_embedding_workspace_bytes(n, d, v)))
    there = (t >= 0) & (t < v)
    want = torch.zeros(v, d, dtype=torch.float64, device="cuda").index_add_(0, t[there], dout[there].double())
    size = torch.zeros(v, d, dtype=torch.float64, device="cuda").index_add_(0, t[there], dout[there].double().abs())
    check("dtable", dtable, want, (n + 4) * U * size)


@pytest.mark.parametrize("v", [200, 50257, 70000])
@pytest.mark.parametrize("n", [1024, 1025, 2048, 2049, 8192, 8193, 16384, 16385, 32769, 65536, 65537])
def test_embedding_backward_around_the_sorts_sizes(n, v):
    """One block with 1 and 2 tokens to a thread, a cluster with 1, 2, 4 and 8 tokens to a thread, several launches; 1 to 3 passes.
    Whole numbers: every sum is exact, whatever its order."""
    g = gen(n + v)
    d = 8
    t = ids(g, n, v, torch.int64)
    t[-3:] = v - 1
    dout = torch.randint(-3, 4, (n, d), device="cuda", generator=g).to(F32)
    dt = torch.full((v, d), 7.0, device="cuda")
    z.zero_embedding_backward(t, dout, dt, work_bytes(z.zero_embedding_workspace_bytes(n, d, v)))
    there = (t >= 0) & (t < v)
    want = torch.zeros(v, d, device="cuda").index_add_(0, t[there], dout[there])
    assert torch.equal(dt, want)


def test_embedding_backward_edges():
    d, v = 40, 9
    table = torch.full((v, d), 3.0, device="cuda")
    work = work_bytes(z.zero_embedding_workspace_bytes(4096, d, v))
    dout = torch.ones(4096, d, device="cuda")
    z.zero_embedding_backward(torch.full((4096,), 4, device="cuda"), dout, table, work)     # one token alone
    want = torch.zeros(v, d, device="cuda")
    want[4] = 4096.0
    assert torch.equal(table, want)
    z.zero_embedding_backward(torch.full((4096,), -1, device="cuda"), dout * float("nan"), table, work, accumulate=True)
    assert torch.equal(table, want)                                                          # padding alone
    z.zero_embedding_backward(torch.full((4096,), 9, device="cuda"), dout * float("nan"), table, work)
    assert (table == 0).all()
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    table.fill_(3.0)
    z.zero_embedding_backward(none, dout[:0], table, work, accumulate=True)
    assert (table == 3.0).all()
    z.zero_embedding_backward(none, dout[:0], table, work)
    assert (table == 0).all()


# ------------------------------------------------------------------------------------------
# the head
# ------------------------------------------------------------------------------------------
HEAD = [(1, 8, 17), (1, 64, 256), (5, 1, 1), (130, 64, 257), (128, 128, 300), (300, 72, 1000), (5, 641, 1003),
        (257, 1600, 5000), (64, 24, 40000), (1000, 200, 129), (3000, 40, 70)]


def head_case(g, n, d, v, dtype, pad=0, missing=0.2, it=torch.int64):
    h, w = rows_of(g, n, d, dtype, pad), normal(g, v, d, sigma=2.0 / math.sqrt(d), dtype=dtype)
    t = ids(g, n, v, torch.int64, missing).to(it)
    return h, w, t, (t >= 0) & (t < v)


def head_reference(h, w, t, there):
    """loss and lse in 64 bits, the logits, and a bound of what the matrix unit's fp32 sums are off:
    one instruction per 16 of the sum, each off by at most 2^-21 of the terms' magnitudes."""
    h64, w64 = torch.where(there[:, None], h.double(), 0.0), w.double()
    l = h64 @ w64.T
    el = (h.shape[1] / 16 + 1) * 2.0 ** -21 * (h64.abs() @ w64.abs().T).amax(1)
    lse = torch.logsumexp(l, 1)
    at = torch.where(there, t, 0).long()
    loss = lse - l.gather(1, at[:, None])[:, 0]
    zero = torch.zeros_like(lse)
    return l, torch.where(there, loss, zero), torch.where(there, lse, zero), el, at


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n,d,v", HEAD)
def test_head_loss(n, d, v, dtype):
    g = gen(n + d + v)
    for pad, missing, it in ((0, 0.0, torch.int64), (0, 0.3, torch.int32), (5, 0.1, torch.int64), (8, 1.0, torch.int64)):
        h, w, t, there = head_case(g, n, d, v, dtype, pad, missing, it)
        loss, lse = torch.full((n,), 7.0, device="cuda"), torch.full((n,), 7.0, device="cuda")
        z.zero_head_loss(h, w, t, loss, lse, work_bytes(z.zero_head_workspace_bytes(n, d, v)))
        _, rl, re, el, _ = head_reference(h, w, t, there)
        # exponentials within 2^-22 and their argument's rounding (|l| below 64: 2^-18), sums, log
        e = el + 2.0 ** -17 + 16 * U * re.abs()
        check("lse", lse, re, e)
        check("loss", loss, rl, e + el)


def head_gradients(h, w, t, there, f, dtype):
    """Both gradients in 64 bits with bounds: each D is off by its rounding to 16 bits, the logits'
    and the exponential's error; then the products' own fp32 sums."""
    l, _, lse, el, at = head_reference(h, w, t, there)
    p = torch.exp(l - lse[:, None])
    d = p.clone()
    d[torch.arange(len(at), device="cuda"), at] -= 1.0
    f = torch.where(there, f, 0.0)
    d = torch.where(there[:, None], d * f[:, None], 0.0)
    ed = HALF[dtype] * d.abs() + f.abs()[:, None] * p * (2 * el[:, None] + 2.0 ** -16)
    ed = torch.where(there[:, None], ed, 0.0)
    if dtype == F16:
        ed += 2.0 ** -25 * f.abs().max() * 2.0 ** -14   # below fp16's normal numbers: D's unit is 2^14
    hh, ww = torch.where(there[:, None], h.double(), 0.0), w.double()
    n, v = d.shape
    eh = ed @ ww.abs() + (v / 16 + 8) * 2.0 ** -21 * (d.abs() @ ww.abs())
    ew = ed.T @ hh.abs() + (n / 16 + 8) * 2.0 ** -21 * (d.T.abs() @ hh.abs())
    return d @ ww, eh, d.T @ hh, ew


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n,d,v", HEAD)
def test_head_loss_backward(n, d, v, dtype):
    g = gen(n * 5 + d + v)
    cases = ((0, 0.0, False, dtype, False, None), (0, 0.3, True, F32, True, 1024.0), (5, 0.1, True, dtype, True, None),
             (8, 1.0, False, dtype, False, 64.0), (8, 0.0, False, F32, False, None))
    for pad, missing, weighted, gt, acc, scale in cases:
        h, w, t, there = head_case(g, n, d, v, dtype, pad, missing)
        _, _, re, _, _ = head_reference(h, w, t, there)
        lse = re.float()
        row = torch.rand(n, device="cuda", generator=g) + 0.5 if weighted else None
        st = None
        if scale:
            st = torch.empty(z.STATE_BYTES, dtype=torch.uint8, device="cuda")
            z.zero_tensors_state_init(1, scale, True, 100, st)
        dh = torch.full((n, d + pad), 7.0, dtype=dtype, device="cuda")
        dw = normal(g, v, d, sigma=0.1, dtype=gt)
        old = dw.double() if acc else 0.0
        work = work_bytes(z.zero_head_workspace_bytes(n, d, v))
        z.zero_head_loss_backward(h, w, t, lse, dh[:, :d], dw, work, scale=1.0 / n, row_scale=row, st=st, accumulate=acc)
        f = torch.full((n,), (scale or 1.0) / n, dtype=torch.float64, device="cuda") * (row.double() if weighted else 1.0)
        rh, eh, rw, ew = head_gradients(h, w, t, there, f, dtype)
        check("dhidden", dh[:, :d], rh, eh)
        check("dweight", dw, rw + old, ew + (2 * U * old.abs() if acc else 0.0))
        assert (dh[:, d:] == 7.0).all()
        if acc:
            continue
        only = torch.empty_like(dw)
        z.zero_head_loss_backward(h, w, t, lse, None, only, work, scale=1.0 / n, row_scale=row, st=st)
        assert torch.equal(only, dw)
        only = torch.empty(n, d, dtype=dtype, device="cuda")
        z.zero_head_loss_backward(h, w, t, lse, only, None, work, scale=1.0 / n, row_scale=row, st=st)
        assert torch.equal(only, dh[:, :d])


@pytest.mark.parametrize("n,d,v,gt,acc", [(2100, 200, 3000, BF16, False), (2100, 200, 3000, F32, True), (2100, 203, 3000, BF16, True),
                                          (2048, 320, 2500, BF16, False), (300, 203, 3000, F32, True)])
def test_head_rows_off_the_128_byte_grid(n, d, v, gt, acc):
    """Calls of many rows move to 128-byte boundaries first; odd rows of the gradient are added to."""
    g = gen(n + d + v)
    for pad in (0, 8):
        h, w, t, there = head_case(g, n, d, v, BF16, pad)
        work = work_bytes(z.zero_head_workspace_bytes(n, d, v))
        loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        z.zero_head_loss(h, w, t, loss, lse, work)
        _, rl, re, el, _ = head_reference(h, w, t, there)
        e = el + 2.0 ** -17 + 16 * U * re.abs()   # as in test_head_loss
        check("lse", lse, re, e)
        check("loss", loss, rl, e + el)
        dh, dw = torch.empty(n, d, dtype=BF16, device="cuda"), normal(g, v, d, sigma=0.1, dtype=gt)
        old = dw.double() if acc else 0.0
        z.zero_head_loss_backward(h, w, t, re.float(), dh, dw, work, scale=1.0 / n, accumulate=acc)
        rh, eh, rw, ew = head_gradients(h, w, t, there, torch.full((n,), 1.0 / n, dtype=torch.float64, device="cuda"), BF16)
        check("dhidden", dh, rh, eh)
        check("dweight", dw, rw + old, ew + (2 * U * old.abs() if acc else 0.0))


@pytest.mark.parametrize("n,d,v", [(8200, 64, 20000), (16500, 24, 9000)])
def test_head_in_several_pieces(n, d, v):
    g = gen(3)
    h, w, t, there = head_case(g, n, d, v, BF16, 0, 0.05)
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    work = work_bytes(z.zero_head_workspace_bytes(n, d, v))
    z.zero_head_loss(h, w, t, loss, lse, work)
    _, rl, re, el, _ = head_reference(h, w, t, there)
    check("loss", loss, rl, 2 * el + 2.0 ** -17 + 16 * U * re.abs())
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    z.zero_head_loss_backward(h, w, t, lse, dh, dw, work, scale=1.0 / n)
    f = torch.full((n,), 1.0 / n, dtype=torch.float64, device="cuda")
    rh, eh, rw, ew = head_gradients(h, w, t, there, f, BF16)
    check("dhidden", dh, rh, eh)
    check("dweight", dw, rw, ew)


def test_head_masked_rows_may_hold_anything():
    g = gen(4)
    for dtype, d in ((BF16, 64), (F16, 96), (BF16, 33)):
        h, w, t, there = head_case(g, 200, d, 777, dtype, 0, 0.5)
        clean = torch.where(there[:, None], h, torch.zeros_like(h))
        h[~there] = float("nan")
        h[torch.nonzero(~there)[0, 0]] = float("inf")
        out = []
        for x in (h, clean):
            work = work_bytes(z.zero_head_workspace_bytes(200, d, 777))
            loss, lse, dh, dw = torch.empty(200, device="cuda"), torch.empty(200, device="cuda"), torch.empty_like(h), torch.empty_like(w)
            z.zero_head_loss(x, w, t, loss, lse, work)
            z.zero_head_loss_backward(x, w, t, lse, dh, dw, work, scale=0.01)
            out.append((loss, lse, dh, dw))
        for a, b in zip(*out):
            assert torch.isfinite(a).all() and torch.equal(a, b)
        assert (out[0][2][~there] == 0).all()


def test_head_loss_with_infinite_and_nan_logits():
    g = gen(6)
    h, w, t, _ = head_case(g, 70, 64, 300, BF16, 0, 0.0)
    t = t.clamp(max=250)
    h[3, 5] = float("nan")
    w[280] = 0.0
    w[280, 7] = float("inf")      # logits of +-inf at 280, NaN where the row's element 7 is 0
    h[4, 7] = -h[4, 7].abs() - 1  # -inf there: the row stays finite
    h[5, 7] = h[5, 7].abs() + 1   # +inf: no finite loss
    loss, lse = torch.empty(70, device="cuda"), torch.empty(70, device="cuda")
    z.zero_head_loss(h, w, t, loss, lse, work_bytes(z.zero_head_workspace_bytes(70, 64, 300)))
    assert torch.isnan(loss[3]) and not torch.isfinite(loss[5])
    l = h[4].double() @ w.double().T
    assert abs(float(loss[4]) - float(torch.logsumexp(l, 0) - l[t[4]])) < 1e-4


def test_head_gradients_against_differences():
    g = gen(9)
    n, d, v = 96, 64, 400
    h, w, t, there = head_case(g, n, d, v, BF16, 0, 0.1)
    row = torch.rand(n, device="cuda", generator=g) + 0.5
    work = work_bytes(z.zero_head_workspace_bytes(n, d, v))
    loss, lse, dh, dw = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(h), torch.empty(v, d, device="cuda")
    z.zero_head_loss(h, w, t, loss, lse, work)
    z.zero_head_loss_backward(h, w, t, lse, dh, dw, work, scale=0.25, row_scale=row)
    vh, vw = normal(g, n, d).double(), normal(g, v, d).double()

    def f(s):
        l = (h.double() + s * vh) @ (w.double() + s * vw).T
        x = torch.logsumexp(l, 1) - l.gather(1, torch.where(there, t, 0)[:, None])[:, 0]
        return (torch.where(there, x, 0.0) * row.double() * 0.25).sum()

    s = 1e-5
    want = (f(s) - f(-s)) / (2 * s)
    got = (dh.double() * vh).sum() + (dw.double() * vw).sum()
    # 16-bit D and dhidden: each 2^-8 of its terms at most, and rounded either way; half of that is
    # 2^-8 of all terms
    size = (dh.double() * vh).abs().sum() + (dw.double() * vw).abs().sum()
    assert abs(float(got - want)) <= 2.0 ** -8 * float(size)


# ------------------------------------------------------------------------------------------
# together, and how they are called
# ------------------------------------------------------------------------------------------
class Tied:
    """Embedding, layer norm and tied head with their gradients in one TensorList."""

    def __init__(self, n=512, d=64, v=1000, dtype=BF16, loss_scale=1.0):
        g = gen(1)
        self.n, self.d, self.v = n, d, v
        self.tokens = ids(g, n, v, torch.int64, 0.05)
        self.targets = ids(g, n, v, torch.int64, 0.1)
        self.master = [normal(g, v, d, sigma=0.3), torch.ones(d, device="cuda"), torch.zeros(d, device="cuda")]
        self.params = [m.to(dtype) for m in self.master]
        self.grads = [torch.empty_like(p) for p in self.params]
        zeros = lambda: [torch.zeros_like(m) for m in self.master]  # noqa: E731
        self.list = z.TensorList(grad=self.grads, master=self.master, m=zeros(), v=zeros(), params=self.params, weight_decay=0.0)
        self.hp = z.hparams(lr=1e-2, max_grad_norm=1.0)
        new = lambda *s, t=dtype: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        self.x, self.y, self.dy, self.dx = new(n, d), new(n, d), new(n, d), new(n, d)
        self.mean, self.rstd, self.loss, self.lse = new(n, t=F32), new(n, t=F32), new(n, t=F32), new(n, t=F32)
        self.st = new(z.STATE_BYTES, t=torch.uint8)
        z.zero_tensors_state_init(1, loss_scale, True, 1000, self.st)
        self.work = new(max(z.zero_head_workspace_bytes(n, d, v), z.zero_layernorm_workspace_bytes(n, d),
                            z.zero_embedding_workspace_bytes(n, d, v)), t=torch.uint8)
        self.norm_work = new(z.zero_tensors_workspace_bytes(3), t=torch.uint8)

    def backward(self):
        (table, w, b), (dtable, dw, db) = self.params, self.grads
        z.zero_embedding(self.tokens, table, self.x, scale=8.0)
        z.zero_layernorm(self.x, w, b, self.y, self.mean, self.rstd)
        z.zero_head_loss(self.y, table, self.targets, self.loss, self.lse, self.work)
        z.zero_head_loss_backward(self.y, table, self.targets, self.lse, self.dy, dtable, self.work, scale=1.0 / self.n, st=self.st)
        z.zero_layernorm_backward(self.x, w, self.mean, self.rstd, self.dy, self.dx, dw, db, self.work)
        z.zero_embedding_backward(self.tokens, self.dx, dtable, self.work, scale=8.0, accumulate=True)

    def step(self):
        self.backward()
        z.zero_tensors_grad_norm(self.list, self.hp, self.norm_work, self.st)
        z.zero_tensors_adamw(self.list, self.hp, self.st)


@pytest.mark.parametrize("dtype,scale", [(BF16, 1.0), (F16, 1024.0)])
def test_a_step_with_a_tied_table(dtype, scale):
    """Against autograd in 64 bits through the same rounded intermediate results' formulas."""
    m = Tied(dtype=dtype, loss_scale=scale)
    m.backward()
    table, w, b = (p.double().requires_grad_() for p in m.params)
    there = (m.tokens >= 0) & (m.tokens < m.v)
    x = torch.where(there[:, None], table[m.tokens.clamp(0, m.v - 1)] * 8.0, 0.0)
    mean = x.mean(1, keepdim=True)
    y = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + 1e-5) * w + b
    l = y @ table.T
    has = (m.targets >= 0) & (m.targets < m.v)
    loss = torch.logsumexp(l, 1) - l.gather(1, m.targets.clamp(0, m.v - 1)[:, None])[:, 0]
    (torch.where(has, loss, 0.0).sum() * scale / m.n).backward()
    # three roundings to 16 bits stand between the loss and the table (y, dy, dx), and D's and the
    # logits' shift by y's; 8 half steps of the whole gradient's norm
    for got, p in zip(m.grads, (table, w, b)):
        off = float((got.double() - p.grad).norm() / p.grad.norm())
        assert off <= 8 * HALF[dtype], off
    before = [x.clone() for x in m.master]
    m.step()
    s = z.zero_step_state_read(m.st)
    assert s.skip == 0 and s.t == 1 and s.error == 0
    assert all(not torch.equal(a, c) for a, c in zip(before, m.master))
    total = math.sqrt(sum(float((x.double() / scale).square().sum()) for x in m.grads))
    assert abs(s.norm - total) <= 1e-5 * total


def test_an_overflow_of_the_scaled_loss_skips_the_step():
    m = Tied(dtype=F16, loss_scale=float(2 ** 24))
    m.params[0].mul_(64.0)
    before = [x.clone() for x in m.master]
    m.step()
    s = z.zero_step_state_read(m.st)
    assert s.skip == 1 and s.loss_scale == 2.0 ** 23
    assert all(torch.equal(a, c) for a, c in zip(before, m.master))


def test_a_captured_step_follows_its_inputs_and_its_loss_scale():
    a, b = Tied(), Tied()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        a.step()                       # warm up on the stream
    torch.cuda.synchronize()
    a = Tied()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    a, saved = a, graph
    for k in range(3):
        new = ids(gen(50 + k), a.n, a.v, torch.int64, 0.05 * k)
        for m in (a, b):
            m.tokens.copy_(new)
            m.targets.copy_(new.roll(1))
        saved.replay()
        b.step()
        torch.cuda.synchronize()
        for x, y in zip(a.master + a.grads + [a.loss, a.lse, a.dx], b.master + b.grads + [b.loss, b.lse, b.dx]):
            assert torch.equal(x, y)


def test_a_capture_as_the_first_call_of_a_process():
    """No call needs one before it: everything that is looked up once is allowed in a capture."""
    import os
    import subprocess
    import sys
    code = """
import torch, zero_partitioned_optimizer_shard_gb300 as z
from tests import test_gpu_layers as T
m = T.Tied(); torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    m.step()
graph.replay(); torch.cuda.synchronize()
other = T.Tied(); other.step(); torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(m.master + m.grads + [m.loss], other.master + other.grads + [other.loss]))
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=240)
    assert done.returncode == 0 and "same" in done.stdout, done.stderr[-2000:]


def every_shape():
    """One call of each of the operators' shapes that a small model does not reach: short and long rows of
    layer norm, a cluster's sort and the one beyond it, rows of the head off the 128-byte grid."""
    g = gen(7)
    out = []
    for n, d in ((20000, 64), (20000, 1600), (300, 5000), (40, 9000)):
        x, w = normal(g, n, d, dtype=BF16), normal(g, d, dtype=BF16)
        out.append([x, w, torch.empty_like(x), torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(x),
                    torch.empty(d, device="cuda"), torch.empty(d, device="cuda"),
                    work_bytes(z.zero_layernorm_workspace_bytes(n, d))])
    for n, d, v in ((3000, 64, 40000), (20000, 16, 70000), (66000, 8, 300)):
        out.append([ids(g, n, v, torch.int64), normal(g, n, d), torch.empty(v, d, device="cuda"),
                    work_bytes(z.zero_embedding_workspace_bytes(n, d, v))])
    n, d, v = 2100, 200, 3000
    out.append([normal(g, n, d, dtype=BF16), normal(g, v, d, sigma=0.1, dtype=BF16), ids(g, n, v, torch.int64),
                torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty(n, d, dtype=BF16, device="cuda"),
                torch.empty(v, d, dtype=BF16, device="cuda"), work_bytes(z.zero_head_workspace_bytes(n, d, v))])

    def run():
        for x, w, y, mean, rstd, dx, dw, db, work in out[:4]:
            z.zero_layernorm(x, w, w, y, mean, rstd)
            z.zero_layernorm_backward(x, w, mean, rstd, y, dx, dw, db, work)
        for t, dout, dt, work in out[4:7]:
            z.zero_embedding_backward(t, dout, dt, work)
        h, w, t, loss, lse, dh, dw, work = out[7]
        z.zero_head_loss(h, w, t, loss, lse, work)
        z.zero_head_loss_backward(h, w, t, lse, dh, dw, work)

    return run, [t for part in out for t in part[:-1]]


def test_every_shape_captured_as_the_first_call_of_a_process():
    import os
    import subprocess
    import sys
    code = """
import torch
from tests import test_gpu_layers as T
run, tensors = T.every_shape(); torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run()
graph.replay(); graph.replay(); torch.cuda.synchronize()
other, others = T.every_shape(); other(); torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(tensors, others))
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=240)
    assert done.returncode == 0 and "same" in done.stdout, done.stderr[-2000:]


def test_two_captured_graphs_share_a_workspace():
    a, b = Tied(), Tied()
    b.work = a.work
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        Tied().step()
    torch.cuda.synchronize()
    graphs = []
    for m in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            m.step()
    alone = Tied()
    for k in range(3):
        for graph in graphs:        # one after another on one stream
            graph.replay()
        alone.step()
    torch.cuda.synchronize()
    for m in (a, b):
        for x, y in zip(m.master + m.grads + [m.loss], alone.master + alone.grads + [alone.loss]):
            assert torch.equal(x, y)


def test_two_streams_with_a_workspace_each():
    a, b = Tied(n=700), Tied(n=700)
    alone = Tied(n=700)
    for _ in range(3):
        alone.backward()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            a.backward()
        with torch.cuda.stream(s2):
            b.backward()
    torch.cuda.synchronize()
    for m in (a, b):
        for x, y in zip(m.grads + [m.loss, m.dx], alone.grads + [alone.loss, alone.dx]):
            assert torch.equal(x, y)


def test_leading_dimensions_and_empty_calls():
    g = gen(12)
    x = normal(g, 4, 6, 80, dtype=BF16)
    w, b = normal(g, 80, dtype=BF16), normal(g, 80, dtype=BF16)
    y, flat = torch.empty_like(x), torch.empty(24, 80, dtype=BF16, device="cuda")
    z.zero_layernorm(x, w, b, y)
    z.zero_layernorm(x.view(24, 80), w, b, flat)
    assert torch.equal(y.view(24, 80), flat)
    z.zero_layernorm(x[:, 2], w, b, flat[:4])           # one row of each sequence
    assert torch.equal(flat[:4], y[:, 2])
    z.zero_layernorm(x[:0], w, b, y[:0])
    tokens = torch.randint(0, 50, (4, 6), device="cuda", generator=g)
    table, out = normal(g, 50, 80, dtype=BF16), torch.empty_like(x)
    z.zero_embedding(tokens, table, out)
    assert torch.equal(out, table[tokens])
    z.zero_embedding(tokens[:0], table, out[:0])
    loss, lse = torch.empty(4, 6, device="cuda"), torch.empty(4, 6, device="cuda")
    work = work_bytes(z.zero_head_workspace_bytes(24, 80, 50))
    z.zero_head_loss(x, table, tokens, loss, lse, work)
    want = torch.nn.functional.cross_entropy((x.double() @ table.double().T).view(24, 50), tokens.view(24), reduction="none")
    assert torch.allclose(loss.view(24).double(), want, rtol=0, atol=1e-4)
    z.zero_head_loss(x[:0], table, tokens[:0], loss[:0], lse[:0], work)
    dw = torch.ones(50, 80, device="cuda")
    z.zero_head_loss_backward(x[:0], table, tokens[:0], lse[:0], x[:0].clone(), dw, work, accumulate=True)
    assert (dw == 1).all()
    z.zero_head_loss_backward(x[:0], table, tokens[:0], lse[:0], x[:0].clone(), dw, work)
    assert (dw == 0).all()


def test_views_off_the_16_byte_grid():
    """Every tensor one element past an aligned address, rows at odd distances."""
    g = gen(21)
    n, d, v = 300, 72, 500
    for dtype in (BF16, F16):
        off = lambda *s: normal(g, math.prod(s) + 1, dtype=dtype)[1:].view(*s)  # noqa: E731
        rows = lambda: normal(g, n, d + 3, dtype=dtype)[:, 1:1 + d]             # noqa: E731
        x, dy, y, dx, w, b = rows(), rows(), rows(), rows(), off(d), off(d)
        mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        z.zero_layernorm(x, w, b, y, mean, rstd)
        want, m64, r64 = norm_forward(x, w, b, 1e-5)
        check("y", y, want, norm_bounds(x, w, m64, r64, want)[0])
        dw, db = off(d), off(d)
        z.zero_layernorm_backward(x, w, mean, rstd, dy, dx, dw, db, work_bytes(z.zero_layernorm_workspace_bytes(n, d)))
        rx, ex, rw, ew, rb, eb = norm_backward(x, w, mean, rstd, dy)
        check("dx", dx, rx, ex)
        check("dweight", dw, rw, ew)
        check("dbias", db, rb, eb)
        t, table, out, dtable = ids(g, n, v, torch.int32), off(v, d), rows(), off(v, d)
        z.zero_embedding(t, table, out, scale=2.0)
        there = (t >= 0) & (t < v)
        assert torch.equal(out, torch.where(there[:, None], table[t.clamp(0, v - 1).long()] * 2.0, torch.zeros_like(out)))
        z.zero_embedding_backward(t, dy, dtable, work_bytes(z.zero_embedding_workspace_bytes(n, d, v)))
        want = torch.zeros(v, d, dtype=torch.float64, device="cuda").index_add_(0, t[there].long(), dy[there].double())
        size = torch.zeros(v, d, dtype=torch.float64, device="cuda").index_add_(0, t[there].long(), dy[there].double().abs())
        check("dtable", dtable, want, (n + 4) * U * size)
        # the head: hidden and its gradient anywhere, weight on 16 bytes (rows of whole groups)
        h, dh, hw = rows(), rows(), normal(g, v, d, sigma=0.2, dtype=dtype)
        head_check(h, hw, t.long(), dh, normal(g, v * d + 1)[1:].view(v, d))
        hw = normal(g, v * (d - 1) + 1, sigma=0.2, dtype=dtype)[1:].view(v, d - 1)  # odd rows: anywhere
        head_check(h[:, :d - 1], hw, t.long(), dh[:, :d - 1], normal(g, v * (d - 1) + 1, dtype=dtype)[1:].view(v, d - 1))


def test_a_captured_gradient_of_a_table_off_the_16_byte_grid():
    g = gen(47)
    n, d, v = 300, 24, 500
    buf = torch.full((v * d + 3,), 7.0, dtype=BF16, device="cuda")
    t, dout = ids(g, n, v, torch.int64), normal(g, n, d, dtype=BF16)
    work = work_bytes(z.zero_embedding_workspace_bytes(n, d, v))
    want = torch.empty(v, d, dtype=BF16, device="cuda")
    z.zero_embedding_backward(t, dout, want, work)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z.zero_embedding_backward(t, dout, buf[1:1 + v * d].view(v, d), work)
    for _ in range(2):
        buf.fill_(7.0)
        graph.replay()
        assert torch.equal(buf[1:1 + v * d].view(v, d), want)
        assert (buf[:1] == 7.0).all() and (buf[1 + v * d:] == 7.0).all()


def test_rows_of_no_elements_are_refused():
    e = torch.empty(4, 0, device="cuda")
    with pytest.raises(ValueError):
        z.zero_layernorm(e, torch.empty(0, device="cuda"), None, e.clone())
    with pytest.raises(ValueError):
        z.zero_embedding(torch.zeros(4, dtype=torch.int64, device="cuda"), torch.empty(5, 0, device="cuda"), e)


def test_columns_of_one_buffer():
    """Inputs and outputs as columns of the same rows, side by side."""
    g = gen(22)
    buf = normal(g, 50, 256, dtype=BF16)
    x, y, dx = buf[:, :64], buf[:, 64:128], buf[:, 192:]
    w, b = normal(g, 64, dtype=BF16), normal(g, 64, dtype=BF16)
    old, mean, rstd = buf.clone(), torch.empty(50, device="cuda"), torch.empty(50, device="cuda")
    z.zero_layernorm(x, w, b, y, mean, rstd)
    want, m64, r64 = norm_forward(old[:, :64], w, b, 1e-5)
    check("y", y, want, norm_bounds(old[:, :64], w, m64, r64, want)[0])
    z.zero_layernorm_backward(x, w, mean, rstd, y, dx, None, None, work_bytes(z.zero_layernorm_workspace_bytes(50, 64)))
    rx, ex = norm_backward(x, w, mean, rstd, y)[:2]
    check("dx", dx, rx, ex)
    assert torch.equal(buf[:, :64], old[:, :64]) and torch.equal(buf[:, 128:192], old[:, 128:192])
    with pytest.raises(z.ZeroError):
        z.zero_layernorm(x, w, b, buf[:, 63:127])


def head_check(h, w, t, dh, dw):
    n, (v, d), dtype = h.shape[0], w.shape, h.dtype
    there = (t >= 0) & (t < v)
    work = work_bytes(z.zero_head_workspace_bytes(n, d, v))
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    z.zero_head_loss(h, w, t, loss, lse, work)
    _, rl, re, el, _ = head_reference(h, w, t, there)
    check("loss", loss, rl, 2 * el + 2.0 ** -17 + 16 * U * re.abs())
    z.zero_head_loss_backward(h, w, t, lse, dh, dw, work, scale=1.0 / n)
    f = torch.full((n,), 1.0 / n, dtype=torch.float64, device="cuda")
    rh, eh, rw, ew = head_gradients(h, w, t, there, f, dtype)
    check("dhidden", dh, rh, eh)
    check("dweight", dw, rw, ew)


def test_offsets_past_32_bits():
    """Tables and activations of more than 2^32 bytes (and 2^31 elements)."""
    g = gen(31)
    v, d = 540_000, 4096
    table = torch.zeros(v, d, dtype=BF16, device="cuda")
    t = torch.tensor([0, v - 1, 530_000, 7, v - 1], device="cuda")
    table[t] = normal(g, 5, d, dtype=BF16)
    out = torch.empty(5, d, dtype=BF16, device="cuda")
    z.zero_embedding(t, table, out)
    assert torch.equal(out, table[t])
    grad = torch.full((v, d), 3.0, dtype=BF16, device="cuda")
    z.zero_embedding_backward(t, out, grad, work_bytes(z.zero_embedding_workspace_bytes(5, d, v)))
    assert torch.equal(grad[v - 1], (out[1].float() + out[4].float()).bfloat16()) and torch.equal(grad[530_000], out[2])
    assert int((grad != 0).any(1).sum()) == 4
    del grad
    # the head's forward pass over the same table, and dweight's last rows
    h = normal(g, 70, d, dtype=BF16)
    h[:, 1::2] = 0
    table *= 0.02
    targets = torch.full((70,), v - 1, device="cuda")
    loss, lse = torch.empty(70, device="cuda"), torch.empty(70, device="cuda")
    work = work_bytes(z.zero_head_workspace_bytes(70, d, v))
    z.zero_head_loss(h, table, targets, loss, lse, work)
    some = h.double() @ table[t[:4]].double().T
    want = torch.log(torch.exp(some).sum(1) + (v - 4))
    assert torch.allclose(lse.double(), want, rtol=0, atol=1e-4)
    assert torch.allclose(loss.double(), want - some[:, 1], rtol=0, atol=1e-4)
    dw = torch.empty_like(table)
    z.zero_head_loss_backward(h, table, targets, lse, None, dw, work, scale=1.0)
    p = torch.exp(some[:, 1] - want) - 1.0
    want = (p[:, None] * h.double()).sum(0)
    assert float((dw[v - 1].double() - want).norm() / want.norm()) < 2.0 ** -7
    del table, dw, work
    n, d = 1_100_000, 2048
    x = torch.empty(n, d, dtype=BF16, device="cuda").normal_(generator=g)
    w = normal(g, d, dtype=BF16) + 1.0
    y, mean, rstd = torch.empty_like(x), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    z.zero_layernorm(x, w, w, y, mean, rstd)
    for s in (slice(0, 40), slice(n - 40, n)):
        want, m64, r64 = norm_forward(x[s], w, w, 1e-5)
        check("y", y[s], want, norm_bounds(x[s], w, m64, r64, want)[0])
    dx, dw, db = torch.empty_like(x), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    z.zero_layernorm_backward(x, w, mean, rstd, y, dx, dw, db, work_bytes(z.zero_layernorm_workspace_bytes(n, d)))
    for s in (slice(0, 40), slice(n - 40, n)):
        want, err = norm_backward(x[s], w, mean[s], rstd[s], y[s])[:2]
        check("dx", dx[s], want, err)
    want = torch.zeros(d, dtype=torch.float64, device="cuda")
    for part in y.split(1 << 17):
        want += part.double().sum(0)
    # a block's 1,800 turns of 2 rows, then the blocks: below 5,000 additions of |y| below 1 on average
    assert float((db.double() - want).abs().max()) <= 5000 * U * n


def test_waits_that_run_out_are_told(hooked):
    """A copy that never comes (test build only): the kernels leave after ~2 s, say so, and the
    GPU stays usable."""
    import ctypes as C
    import time
    L, ref, never = hooked, z.lib(), 0xFFFFFFFFFFFFFFFF
    for name in ("zero_layernorm", "zero_layernorm_backward", "zero_head_loss", "zero_head_loss_backward"):
        getattr(L, name).argtypes, getattr(L, name).restype = getattr(ref, name).argtypes, C.c_int
    for name in ("zero_test_withhold_head_stage", "zero_test_withhold_norm_turn"):
        getattr(L, name).argtypes, getattr(L, name).restype = [C.c_ulonglong], C.c_int
    g = gen(41)
    s = torch.cuda.current_stream().cuda_stream

    def timed(f):
        t0 = time.time()
        assert f() == 0
        torch.cuda.synchronize()
        waited = time.time() - t0
        assert 1.0 < waited < 60.0, waited

    n, d = 20000, 1600
    x, w = normal(g, n, d, dtype=BF16), normal(g, d, dtype=BF16)
    y, mean, rstd = torch.zeros_like(x), torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    assert L.zero_test_withhold_norm_turn(1) == 0
    p = lambda t: t.data_ptr()  # noqa: E731
    timed(lambda: L.zero_layernorm(z.ZERO_BF16, n, d, p(x), d, p(w), p(w), z.ZERO_BF16, 1e-5, p(y), d, p(mean), p(rstd), s))
    lost = torch.isnan(y).any(1)
    assert 0 < int(lost.sum()) < n and not torch.isnan(y[~lost]).any()
    mean.zero_(), rstd.fill_(1.0)
    dx, dw, db = torch.zeros_like(x), torch.zeros(d, device="cuda"), torch.zeros(d, device="cuda")
    work = work_bytes(z.zero_layernorm_workspace_bytes(n, d))
    timed(lambda: L.zero_layernorm_backward(z.ZERO_BF16, n, d, p(x), d, p(w), z.ZERO_BF16, p(mean), p(rstd), p(x), d, p(dx), d,
                                            p(dw), p(db), z.ZERO_F32, 0, p(work), s))
    assert torch.isnan(dw).any() and torch.isnan(db).any()
    lost = torch.isnan(dx).all(1)
    assert 0 < int(lost.sum()) < n and not torch.isnan(dx[~lost]).any()
    assert L.zero_test_withhold_norm_turn(never) == 0
    n, d, v = 600, 640, 5000
    h, w, t = normal(g, n, d, dtype=BF16), normal(g, v, d, sigma=0.05, dtype=BF16), torch.randint(0, v, (n,), device="cuda")
    loss, lse = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    work = work_bytes(z.zero_head_workspace_bytes(n, d, v))
    dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    st = torch.empty(z.STATE_BYTES, dtype=torch.uint8, device="cuda")
    z.zero_tensors_state_init(1, 1.0, False, 0, st)
    assert L.zero_test_withhold_head_stage(3) == 0
    timed(lambda: L.zero_head_loss(z.ZERO_BF16, n, d, v, p(h), d, p(w), p(t), 8, p(loss), p(lse), p(work), s))
    assert torch.isnan(loss).all()
    assert int(work[4:8].view(torch.int32)) == 1
    timed(lambda: L.zero_head_loss_backward(z.ZERO_BF16, n, d, v, p(h), d, p(w), p(t), 8, p(lse), 1.0, None, p(st), p(dh), d,
                                            p(dw), z.ZERO_BF16, 0, p(work), s))
    assert z.zero_step_state_read(st).error == 1 and torch.isnan(dh).all()
    assert L.zero_test_withhold_head_stage(never) == 0
    # the context is still good
    head_check(h, w, t, dh, dw)


# ------------------------------------------------------------------------------------------
# the example's token model
# ------------------------------------------------------------------------------------------
@pytest.fixture(scope="module")
def example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_tensors.py")
    spec = importlib.util.spec_from_file_location("train_tensors", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs_on_tokens(example):
    losses, opt = example.train_tokens(8, 8, vocab=503, dim=64)
    s = z.zero_step_state_read(opt.st)
    assert len(losses) == 8 and all(math.isfinite(x) for x in losses)
    assert s.t == 8 and s.skip == 0 and s.error == 0 and opt.bits == 8


def test_example_gradients(example):
    """The token model's gradients at a loss scale, against torch's in 64 bits."""
    vocab, dim, scale = 503, 64, 256.0
    model, opt = example.token_model(vocab, dim, loss_scale=scale)
    tokens, targets = example.sequence(1, vocab)
    n = int((targets >= 0).sum())
    (model(tokens, targets, opt.st).sum() / n).backward()
    ref = example.TokenModel(vocab, dim, 5).double().cuda()
    ref.load_state_dict({k: p.double() for k, p in model.state_dict().items()})
    x = ref.table[tokens] * dim ** 0.5
    f, (a, b) = torch.nn.functional, ref.norms
    x = x + ref.down(f.gelu(ref.up(f.layer_norm(x, (dim,), a.weight, a.bias))))
    logits = f.layer_norm(x, (dim,), b.weight, b.bias) @ ref.table.T
    loss = f.cross_entropy(logits.view(-1, vocab), targets.view(-1), reduction="sum", ignore_index=-100) / n
    (loss * scale).backward()
    # seven roundings to bf16 on the way to the logits (up to 8 in size), the gradients' seven on the
    # way back; each at most half a step, 2^-8, of what it rounds
    for (name, p), q in zip(model.named_parameters(), ref.parameters()):
        off = float((p.grad.double() - q.grad).norm() / q.grad.norm())
        assert off <= 14 * 2.0 ** -8, (name, off)
