"""The operators beside the matrix products at the largest sizes that they take, against definitions
in 64 bits or whole numbers that add exactly."""
import math

import pytest
import torch

import zero_partitioned_optimizer_shard_gb300 as z
from tests.test_gpu_layers import BF16, F16, F32, U, check, gen, head_gradients, head_reference, normal, work_bytes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def whole(shape, lo, hi, g, dtype):
    return torch.randint(lo, hi, shape, device="cuda", generator=g, dtype=torch.int8).to(dtype)


def test_layernorm_of_2_to_the_30_rows():
    """Rows of one element: y is the bias, dx is 0, dbias counts."""
    g, n = gen(1), 1 << 30
    x = torch.empty(n, 1, dtype=BF16, device="cuda").normal_(generator=g)
    w, b = torch.full((1,), 3.0, dtype=BF16, device="cuda"), torch.full((1,), 0.5, dtype=BF16, device="cuda")
    y, mean, rstd = torch.empty_like(x), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    z.zero_layernorm(x, w, b, y, mean, rstd)
    assert bool((y == 0.5).all()) and torch.equal(mean.bfloat16(), x[:, 0])
    dy, dx, dw, db = torch.ones_like(x), x.clone(), torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    z.zero_layernorm_backward(x, w, mean, rstd, dy, dx, dw, db, work_bytes(z.zero_layernorm_workspace_bytes(n, 1)))
    # a thread's and a block's counts stay below 2^24; at most 1,000 blocks' are then added
    assert bool((dx == 0).all()) and float(dw) == 0.0 and abs(float(db) - n) <= 1000 * U * n


def test_embedding_of_2_to_the_28_tokens():
    g, n, v = gen(2), 1 << 28, 1000
    t = torch.randint(-1, v + 1, (n,), device="cuda", generator=g, dtype=torch.int32)
    table = torch.arange(v, device="cuda").view(v, 1).to(F32)
    out = torch.empty(n, 1, device="cuda")
    z.zero_embedding(t, table, out)
    there = (t >= 0) & (t < v)
    assert torch.equal(out[:, 0], torch.where(there, t, 0).float())
    dout, dt = torch.ones(n, 1, dtype=BF16, device="cuda"), torch.empty(v, 1, device="cuda")
    z.zero_embedding_backward(t, dout, dt, work_bytes(z.zero_embedding_workspace_bytes(n, 1, v)))
    assert torch.equal(dt[:, 0].double(), torch.bincount(t[there], minlength=v).double())  # below 2^24 each


def test_embedding_table_of_2_to_the_30_rows():
    g, v, n = gen(3), 1 << 30, 5000
    table = torch.empty(v, 1, dtype=F16, device="cuda").normal_(generator=g)
    t = torch.randint(0, v, (n,), device="cuda", generator=g)
    t[:3] = torch.tensor([v - 1, 0, v - 1], device="cuda")
    out = torch.empty(n, 1, dtype=F16, device="cuda")
    z.zero_embedding(t, table, out)
    assert torch.equal(out, table[t])
    dout = whole((n, 1), -3, 4, g, F16)
    z.zero_embedding_backward(t, dout, table, work_bytes(z.zero_embedding_workspace_bytes(n, 1, v)))
    at, back = torch.unique(t, return_inverse=True)
    want = torch.zeros(len(at), device="cuda").index_add_(0, back, dout[:, 0].float())
    assert torch.equal(table[at, 0].float(), want)
    assert int(torch.count_nonzero(table)) == int(torch.count_nonzero(want))


@pytest.mark.parametrize("n,d,v", [(5, 65536, 300), (300, 65535, 40), (70, 20000, 1000)])
def test_head_of_wide_rows(n, d, v):
    g = gen(d)
    h, w = normal(g, n, d, dtype=BF16), normal(g, v, d, sigma=2.0 / math.sqrt(d), dtype=BF16)
    t = torch.randint(-1, v, (n,), device="cuda", generator=g)
    there = t >= 0
    work = work_bytes(z.zero_head_workspace_bytes(n, d, v))
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    z.zero_head_loss(h, w, t, loss, lse, work)
    _, rl, re, el, _ = head_reference(h, w, t, there)
    check("lse", lse, re, el + 2.0 ** -17 + 16 * U * re.abs())
    check("loss", loss, rl, 2 * el + 2.0 ** -17 + 16 * U * re.abs())
    dh, dw = torch.empty_like(h), torch.empty(v, d, device="cuda")
    z.zero_head_loss_backward(h, w, t, lse, dh, dw, work, scale=1.0 / n)
    rh, eh, rw, ew = head_gradients(h, w, t, there, torch.full((n,), 1.0 / n, dtype=torch.float64, device="cuda"), BF16)
    check("dhidden", dh, rh, eh)
    check("dweight", dw, rw, ew)


def test_head_of_a_vocabulary_of_2_to_the_24():
    n, d, v = 10, 8, 1 << 24
    g = gen(5)
    h, w = normal(g, n, d, dtype=BF16), normal(g, v, d, dtype=BF16)
    t = torch.tensor([v - 1, 0, 5, -1, v, v // 2, 77, v - 256, 1, 2], device="cuda")
    there = (t >= 0) & (t < v)
    work = work_bytes(z.zero_head_workspace_bytes(n, d, v))
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    z.zero_head_loss(h, w, t, loss, lse, work)
    _, rl, re, el, _ = head_reference(h, w, t, there)
    # k_head_loss: 4,096 turns of a lane over the tiles, each at most 4 roundings of the sum
    e = el + 2.0 ** -17 + 16 * U * re.abs() + 4 * 4096 * U
    check("lse", lse, re, e)
    check("loss", loss, rl, e + el)
    dh, dw = torch.empty_like(h), torch.empty(v, d, device="cuda")
    z.zero_head_loss_backward(h, w, t, re.float(), dh, dw, work)
    rh, eh, rw, ew = head_gradients(h, w, t, there, torch.ones(n, dtype=torch.float64, device="cuda"), BF16)
    check("dhidden", dh, rh, eh)
    check("dweight", dw, rw, ew)


def test_head_of_2_to_the_24_tokens():
    n, d, v = 1 << 24, 8, 17
    g = gen(6)
    h, w = torch.empty(n, d, dtype=BF16, device="cuda").normal_(generator=g), normal(g, v, d, dtype=BF16)
    t = torch.randint(-1, v, (n,), device="cuda", generator=g, dtype=torch.int32)
    work = work_bytes(z.zero_head_workspace_bytes(n, d, v))
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty(v, d, device="cuda")
    z.zero_head_loss(h, w, t, loss, lse, work)
    z.zero_head_loss_backward(h, w, t, lse, dh, dw, work)
    rw, size = (torch.zeros(v, d, dtype=torch.float64, device="cuda") for _ in range(2))
    for at in range(0, n, 1 << 20):
        s = slice(at, at + (1 << 20))
        ts, there = t[s].long(), t[s] >= 0
        _, rl, re, el, _ = head_reference(h[s], w, ts, there)
        check("loss", loss[s], rl, 2 * el + 2.0 ** -17 + 16 * U * re.abs())
        f = torch.ones(1 << 20, dtype=torch.float64, device="cuda")
        rh, eh, part, ew = head_gradients(h[s], w, ts, there, f, BF16)
        check("dhidden", dh[s], rh, eh)
        rw += part
        size += ew
    # a split's steps of 16 tokens, 1/76 of all, each cut off by 2^-23 of the sum so far at most
    check("dweight", dw, rw, size + n / 76 / 16 * 2.0 ** -23 * rw.abs())
