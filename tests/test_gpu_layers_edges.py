"""Edges of the operators beside the matrix products: rows that end inside a warp's columns with
further tiles behind them.  Definitions in 64 bits."""
import math

import pytest
import torch

import zero_partitioned_optimizer_shard_gb300 as z
from tests.test_gpu_layers import BF16, F32, U, check, gen, head_gradients, normal, work_bytes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("d", [33, 63, 129, 161, 223, 255])
@pytest.mark.parametrize("gt,acc", [(BF16, False), (F32, True)])
def test_tiles_behind_a_rows_end(d, gt, acc):
    """Weights whose rows the TMA does not take: lanes past a row's end have nothing to store, and
    the warp goes on to the next of more tiles than there are pairs of SMs."""
    n, v = 40, 256 * 160 + 7
    g = gen(d)
    h, w = normal(g, n, d, dtype=BF16), normal(g, v, d, sigma=2.0 / math.sqrt(d), dtype=BF16)
    t = torch.randint(0, v, (n,), device="cuda", generator=g)
    there = t >= 0
    lse = torch.logsumexp(h.double() @ w.double().T, 1).float()
    dh, dw = torch.empty_like(h), normal(g, v, d, sigma=0.1, dtype=gt)
    old = dw.double() if acc else 0.0
    z.zero_head_loss_backward(h, w, t, lse, dh, dw, work_bytes(z.zero_head_workspace_bytes(n, d, v)), scale=1.0 / n, accumulate=acc)
    rh, eh, rw, ew = head_gradients(h, w, t, there, torch.full((n,), 1.0 / n, dtype=torch.float64, device="cuda"), BF16)
    check("dhidden", dh, rh, eh)
    check("dweight", dw, rw + old, ew + (2 * U * old.abs() if acc else 0.0))
