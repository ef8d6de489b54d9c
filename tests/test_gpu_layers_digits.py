"""Digits that the operators beside the matrix products keep where a looser bound would hide a loss:
confident tokens, logits far from 0.  Definitions in 64 bits."""
import pytest
import torch

import zero_partitioned_optimizer_shard_gb300 as z
from tests.test_gpu_layers import BF16, F16, U, check, gen, work_bytes

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
