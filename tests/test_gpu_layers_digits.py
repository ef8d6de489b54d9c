"""Digits that the operators beside the matrix products keep where a looser bound would hide a loss:
confident tokens, logits far from 0, sums of many terms of one sign, weights' gradients over many
rows; and that the same call gives the same bits.  Definitions in 64 bits."""
import math

import pytest
import torch

import zero_partitioned_optimizer_shard_gb300 as z
from tests.test_gpu_layers import BF16, F16, F32, HALF, U, check, gen, ids, normal, work_bytes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


def head_loss(h, w, t):
    n, (v, d) = h.shape[0], w.shape
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    z.zero_head_loss(h, w, t, loss, lse, work_bytes(z.zero_head_workspace_bytes(n, d, v)))
    return loss, lse


# ------------------------------------------------------------------------------------------
# the loss
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("size", [20.0, 64.0, 200.0])
def test_the_loss_of_a_confident_token_is_not_negative(size, dtype):
    """Target logits between 1 and 2 times `size`, all others 0: the loss is log(1 + (v - 1) exp(-top)).
    A logit is one product, exact in fp32 (2 x 8 or 2 x 11 bits)."""
    n, d, v = 512, 16, 300
    h, w = torch.zeros(n, d, dtype=dtype, device="cuda"), torch.zeros(v, d, dtype=dtype, device="cuda")
    h[:, 3] = (1.0 + torch.arange(n, device="cuda") / n).to(dtype)
    w[17, 3] = size * 1.03
    t = torch.full((n,), 17, device="cuda")
    loss, lse = head_loss(h, w, t)
    top = h[:, 3].double() * w[17, 3].double()
    want = torch.log1p((v - 1) * torch.exp(-top))
    assert (loss >= 0).all()
    # a sum near 1: its last additions' and the logarithm's roundings, at a magnitude of 1
    check("loss", loss, want, torch.full_like(want, 2.0 ** -21))
    check("lse", lse, top + want, torch.full_like(want, 2.0 ** -21))


def test_logits_far_from_0_over_a_large_vocabulary():
    """Logits around 64 to 128, a few apart: every one exact in fp32 (a product in halves plus a
    multiple of 1/64), so only the sums' own errors are left."""
    n, d, v = 300, 16, 50257
    g = gen(3)
    h, w = torch.zeros(n, d, dtype=BF16, device="cuda"), torch.zeros(v, d, dtype=BF16, device="cuda")
    h[:, 0] = (1.0 + torch.arange(n, device="cuda") % 128 / 128).bfloat16()
    h[:, 1] = 1.0
    w[:, 0] = 64.0
    w[:, 1] = (torch.randint(-128, 129, (v,), device="cuda", generator=g) / 64.0).bfloat16()
    t = torch.randint(0, v, (n,), device="cuda", generator=g)
    loss, lse = head_loss(h, w, t)
    l = h.double() @ w.double().T
    want = torch.logsumexp(l, 1)
    # each exponential: its argument within 2 roundings of at most 6 (2^-21), ex2 2^-22; 128 terms by 4
    # chains of 32 and their join (34 roundings), then tiles by lanes: 25 turns and 5 exchanges of at
    # most 8 roundings (an exponential of 0 is 1).  All relative to the sum, so to lse as they are
    err = 2.0 ** -21 + 2.0 ** -22 + (34 + 30 * 8) * U + 4 * U
    check("lse", lse, want, torch.full_like(want, err))
    rows = torch.arange(n, device="cuda")
    check("loss", loss, want - l[rows, t], torch.full_like(want, err))


def one_sign(n, d, v, seed):
    """Tokens and weights whose logits' terms have one sign each: around +8 at row 0, -8 elsewhere."""
    g = gen(seed)
    h = (normal(g, n, d).abs() + 0.25).bfloat16()
    w = normal(g, v, d).abs() + 0.25
    w = w * (8.0 / (h.float().mean() * w.mean() * d))
    w[1:].neg_()
    return h, w.bfloat16()


# A sum of d terms of one sign by the matrix unit: d/16 steps, each cut off by less than one unit
# (2^-23) of what the sum is then.  In parts of 1,024 terms, 64 steps, whose sums grow evenly up to
# a part of the logit, that is less than 2^-23 * 33 of the logit; in one part of 4,096 terms 4 times that.
CUT = 33 * 2.0 ** -23


def test_logits_of_many_terms_of_one_sign():
    n, d, v = 512, 4096, 64
    h, w = one_sign(n, d, v, 5)
    _, lse = head_loss(h, w, torch.zeros(n, dtype=torch.int64, device="cuda"))
    want = torch.logsumexp(h.double() @ w.double().T, 1)
    assert float((lse.double() - want).mean().abs()) <= CUT * float(want.abs().mean())


# ------------------------------------------------------------------------------------------
# the loss's gradients
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [640, 4096])
def test_gradients_of_confident_tokens(d, dtype):
    """Targets that take all but 1e-4 of the softmax: D there is the small difference of two numbers
    near 1, of which the logit in the backward pass and the lse of the forward pass must agree."""
    n, v = 256, 1000
    h, w = (x.to(dtype) for x in one_sign(n, d, v, 7))
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    _, lse = head_loss(h, w, t)
    dh, dw = torch.empty_like(h), torch.empty(v, d, device="cuda")
    z.zero_head_loss_backward(h, w, t, lse, dh, dw, work_bytes(z.zero_head_workspace_bytes(n, d, v)))
    h64, w64 = h.double(), w.double()
    l = h64 @ w64.T
    lse64 = torch.logsumexp(l, 1)
    p = torch.exp(l - lse64[:, None])
    less = p[:, 1:].sum(1)              # 1 - p at the target, without cancellation
    assert 1e-6 < float(less.min()) and float(less.max()) < 1e-2
    D = p.clone()
    D[:, 0] = -less
    # logits off by CUT of their size (the same in both passes) change p by its own share of that.
    # p - 1 takes in ex2's 2^-22 and what lse is off: half a unit of its own, and the roundings of its
    # sum, which is 1 and a little.  The additions to a partial sum that holds the target's 1 round by
    # half a unit of [1, 2), 2^-24, each: 31 in its chain of 32 columns, 2 where 4 chains join, then
    # 1 turn over the 8 half tiles and 5 exchanges of k_head_loss: 64 at most.  Then D's rounding
    el = CUT * (l.abs() + l[:, :1].abs())
    ed = p * (el + 2.0 ** -21)
    ed[:, 0] = less * el.amax(1) + 2.0 ** -24 * lse64.abs() + 2.0 ** -21 + 64 * 2.0 ** -24
    ed += HALF[dtype] * D.abs() + (2.0 ** -39 if dtype == F16 else 0.0)
    eh = ed @ w64.abs() + (v / 16 + 8) * 2.0 ** -21 * (D.abs() @ w64.abs())
    ew = ed.T @ h64.abs() + (n / 16 + 8) * 2.0 ** -21 * (D.T.abs() @ h64.abs())
    check("dhidden", dh, D @ w64, eh)
    check("dweight", dw, D.T @ h64, ew)
    # the target's row as a whole: nearly all of its bound is one-sided errors' room
    want = (D.T @ h64)[0]
    assert float((dw[0].double() - want).norm() / want.norm()) <= HALF[dtype] + float((ed[:, 0] / less).mean())


def test_the_heads_calls_repeat_their_bits():
    """Pieces of the vocabulary, sums cut into splits, and tokens without a target: the same bits."""
    for n, d, v, dtype, gt, acc in ((8192, 320, 20000, BF16, BF16, False), (1024, 640, 32000, F16, F32, True),
                                    (40, 96, 700, BF16, F32, False), (500, 203, 3000, F16, F16, True)):
        g = gen(n + v)
        h, w, t = normal(g, n, d, dtype=dtype), normal(g, v, d, sigma=2.0 / math.sqrt(d), dtype=dtype), ids(g, n, v, torch.int64)
        row, old, first = torch.rand(n, device="cuda", generator=g), normal(g, v, d, dtype=gt), None
        for fill in (0xA5, 0x00, 0x5A, 0xFF):
            work = work_bytes(z.zero_head_workspace_bytes(n, d, v)).fill_(fill)
            loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
            dh, dw = torch.empty_like(h), old.clone()
            z.zero_head_loss(h, w, t, loss, lse, work)
            z.zero_head_loss_backward(h, w, t, lse, dh, dw, work, scale=1.0 / n, row_scale=row, accumulate=acc)
            out = (loss, lse, dh, dw)
            first = first or out
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(out, first))


# ------------------------------------------------------------------------------------------
# layer norm's sums over rows
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("n,d,dtype", [(1_100_000, 2048, BF16), (300_000, 641, F16), (900_000, 64, BF16)])
def test_the_weights_gradients_take_in_every_row(n, d, dtype):
    """Sums over so many rows, as exact as their additions allow: in fp32 whole numbers below 2^24
    add exactly, so a row left out or taken twice shows."""
    g = gen(n)
    x = torch.randint(0, 2, (n, d), device="cuda", generator=g, dtype=torch.int8).to(dtype)
    dy = torch.empty_like(x)
    for part in dy.split(1 << 18):
        part.copy_(torch.randint(-2, 3, part.shape, device="cuda", generator=g, dtype=torch.int8))
    w, mean, rstd = torch.ones(d, dtype=dtype, device="cuda"), torch.full((n,), -1.0, device="cuda"), torch.full((n,), 2.0, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    z.zero_layernorm_backward(x, w, mean, rstd, dy, dx, dw, db, work_bytes(z.zero_layernorm_workspace_bytes(n, d)))
    ww, wb = (torch.zeros(d, dtype=torch.float64, device="cuda") for _ in range(2))
    for px, pd in zip(x.split(1 << 16), dy.split(1 << 16)):
        ww += (pd.double() * (px.double() + 1.0) * 2.0).sum(0)
        wb += pd.double().sum(0)
    assert torch.equal(dw.double(), ww) and torch.equal(db.double(), wb)
