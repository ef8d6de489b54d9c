"""Edges of the operators beside the matrix products: rows that end inside a warp's columns with
further tiles behind them, short rows in turns, factors that are not finite, and what waits that run
out leave.  Definitions in 64 bits."""
import math

import pytest
import torch

import zero_partitioned_optimizer_shard_gb300 as z
from tests.test_gpu_layers import BF16, F16, F32, U, check, gen, head_gradients, norm_bounds, norm_forward, normal, work_bytes

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


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("n,d,pad", [(200_003, 33, 0), (100_001, 65, 3), (60_007, 255, 0), (300_000, 9, 1), (150_001, 64, 1)])
def test_many_short_rows_off_the_16_byte_grid(n, d, pad, dtype):
    """More rows than as many blocks as fit take at a time: 16-bit ones go on in turns."""
    g = gen(n + d)
    x = normal(g, n, d + pad, dtype=dtype)[:, :d]
    w, b = normal(g, d, dtype=dtype) + 1.0, normal(g, d, dtype=dtype)
    y, mean, rstd = torch.full((n, d + 2), 7.0, dtype=dtype, device="cuda"), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    z.zero_layernorm(x, w, b, y[:, :d], mean, rstd)
    want, m64, r64 = norm_forward(x, w, b, 1e-5)
    check("y", y[:, :d], want, norm_bounds(x, w, m64, r64, want)[0])
    check("mean", mean, m64, norm_bounds(x, w, m64, r64, want)[1])
    assert (y[:, d:] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_a_factor_that_is_not_finite_is_its_own_tokens(value, dtype):
    """What arrives at one token's loss is not finite (a weight, an overflow): the other tokens'
    gradients keep their digits, small as their factors are."""
    n, d, v, bad = 200, 64, 3000, 77
    g = gen(8)
    h, w = normal(g, n, d, dtype=dtype), normal(g, v, d, sigma=0.25, dtype=dtype)
    t = torch.randint(0, v, (n,), device="cuda", generator=g)
    lse = torch.logsumexp(h.double() @ w.double().T, 1).float()
    row = torch.rand(n, device="cuda", generator=g) + 0.5
    row[0], row[bad] = 2.0, 1.0         # the largest is another's
    out = []
    for x in (1.0, value):
        row[bad] = x
        dh = torch.empty_like(h)
        z.zero_head_loss_backward(h, w, t, lse, dh, None, work_bytes(z.zero_head_workspace_bytes(n, d, v)), scale=2.0 ** -6, row_scale=row)
        out.append(dh)
    others = torch.arange(n, device="cuda") != bad
    assert not torch.isfinite(out[1][bad]).any()
    assert torch.equal(out[0][others], out[1][others])


# ------------------------------------------------------------------------------------------
# waits that run out
# ------------------------------------------------------------------------------------------
def prototypes(L):
    import ctypes as C
    ref = z.lib()
    for name in ("zero_layernorm", "zero_layernorm_backward", "zero_head_loss", "zero_head_loss_backward"):
        getattr(L, name).argtypes, getattr(L, name).restype = getattr(ref, name).argtypes, C.c_int
    for name in ("zero_test_withhold_head_stage", "zero_test_withhold_norm_turn"):
        getattr(L, name).argtypes, getattr(L, name).restype = [C.c_ulonglong], C.c_int
    return L


NEVER = 0xFFFFFFFFFFFFFFFF


@pytest.mark.parametrize("d,gt,acc", [(64, BF16, False), (64, BF16, True), (64, F32, True), (63, BF16, False), (63, F32, True)])
def test_weights_gradients_that_a_wait_left_undone_are_nan(hooked, d, gt, acc):
    """dweight alone, without a step state.  79 tiles of 256 rows over 76 pairs of SMs: the first pair has
    tiles 0 and 76.  A copy of D's launch that never comes leaves nothing of dweight; one of the
    second tile (stages 5 to 9 of the gradients' launch; D's has 4) that tile's rows."""
    L, g = prototypes(hooked), gen(d)
    n, v, s = 600, 20000, torch.cuda.current_stream().cuda_stream
    h, w, t = normal(g, n, d, dtype=BF16), normal(g, v, d, sigma=0.1, dtype=BF16), torch.randint(0, v, (n,), device="cuda", generator=g)
    lse = torch.logsumexp(h.double() @ w.double().T, 1).float()
    work = work_bytes(z.zero_head_workspace_bytes(n, d, v))
    old = normal(g, v, d, sigma=0.1, dtype=gt)
    code = z.ZERO_F32 if gt == F32 else z.ZERO_BF16

    def run(stage):
        dw = old.clone()
        assert L.zero_test_withhold_head_stage(stage) == 0
        assert L.zero_head_loss_backward(z.ZERO_BF16, n, d, v, h.data_ptr(), d, w.data_ptr(), t.data_ptr(), 8, lse.data_ptr(), 1.0,
                                         None, None, None, 0, dw.data_ptr(), code, acc, work.data_ptr(), s) == 0
        torch.cuda.synchronize()
        assert L.zero_test_withhold_head_stage(NEVER) == 0
        return dw, int(work[4:8].view(torch.int32))

    good, error = run(NEVER)
    assert error == 0 and torch.isfinite(good).all()
    lost, error = run(2)
    assert error == 1 and torch.isnan(lost).all()
    lost, error = run(5)
    assert error == 1
    undone = slice(76 * 256, 77 * 256)
    assert torch.isnan(lost[undone]).all()
    rest = torch.cat([lost[:undone.start], lost[undone.stop:]])
    want = torch.cat([good[:undone.start], good[undone.stop:]])
    told = torch.isnan(rest)            # a tile that ended after the wait gave up may be NaN as well
    assert torch.equal(rest[~told], want[~told]) and not told.all()
    again, error = run(NEVER)
    assert error == 0 and torch.equal(again, good)


def test_rows_that_a_wait_left_undone_have_no_statistics(hooked):
    L, g = prototypes(hooked), gen(4)
    n, d, s = 20000, 1600, torch.cuda.current_stream().cuda_stream
    x, w = normal(g, n, d, dtype=BF16), normal(g, d, dtype=BF16)
    y, mean, rstd = torch.zeros_like(x), torch.full((n,), 7.0, device="cuda"), torch.full((n,), 7.0, device="cuda")
    assert L.zero_test_withhold_norm_turn(1) == 0
    assert L.zero_layernorm(z.ZERO_BF16, n, d, x.data_ptr(), d, w.data_ptr(), w.data_ptr(), z.ZERO_BF16, 1e-5, y.data_ptr(), d,
                            mean.data_ptr(), rstd.data_ptr(), s) == 0
    torch.cuda.synchronize()
    assert L.zero_test_withhold_norm_turn(NEVER) == 0
    lost = torch.isnan(y).all(1)
    assert 0 < int(lost.sum()) < n
    assert torch.equal(torch.isnan(mean), lost) and torch.equal(torch.isnan(rstd), lost)
