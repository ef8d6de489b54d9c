"""The steps over lists of tensors on the GPU, against their formulas in 64 bits (the 8-bit
codes against the fp32 definition bit for bit), at the sizes, alignments and values where
they can go wrong.  Every array lies between guard zones that the calls must not touch.

Tolerances, from the arithmetic (u = 2^-24, one rounding): the norm's groups of 8 squares
round at most 9 times, so its square is within 9u and the norm within 4.5u < 3e-7; m takes
5 roundings of terms below |b1 m| + |(1-b1) gc|, v 8 of positive terms; the parameter adds
3 roundings of p and at most 12 of the update (the divisions and the square root may be
within 2 ulp), besides m's own error over the denominator."""
import ctypes as C
import time

import numpy as np
import pytest
import torch

import zero_partitioned_optimizer_shard_gb300 as z
from tests import state8_oracle as S

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
GUARD = 512
CANARY = 0xA5
NP = {torch.float32: np.float32, torch.uint8: np.uint8}
GRAD = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EDGES = [0, 1, 7, 8, 9, 31, 32, 255, 256, 257, 300, 1000, 2047, 2048, 2049, 4096, 5003, 8191, 8192, 8193, 20_011]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()


class Arena:
    """Arrays between guard zones, `shift` elements off a 256-byte boundary."""

    def __init__(self):
        self.raw = []

    def put(self, x: torch.Tensor, shift: int = 0) -> torch.Tensor:
        n, esz = x.numel() * x.element_size(), x.element_size()
        raw = torch.full((2 * GUARD + n + 256,), CANARY, dtype=torch.uint8, device="cuda")
        lo = GUARD + shift * esz
        view = raw[lo:lo + n].view(x.dtype) if n else torch.empty(0, dtype=x.dtype, device="cuda")
        view.copy_(x.reshape(-1))
        self.raw.append((raw, lo, n))
        return view

    def check(self):
        torch.cuda.synchronize()
        for raw, lo, n in self.raw:
            assert bool((raw[:lo] == CANARY).all()) and bool((raw[lo + n:] == CANARY).all())


def host(x):
    return (x.float() if x.dtype in (torch.bfloat16, torch.float16) else x).cpu().numpy()


def rand(n, seed, sigma, dtype=torch.float32, square=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, generator=g) * sigma
    return (x * x if square else x).to(dtype)


class Case:
    """A list with every array guarded; per-tensor gradient types and shifts cycle."""

    def __init__(self, sizes, grads=("bf16",), shifts=(0,), state="f32", params=("bf16",), scales=(1.0,),
                 decays=(0.01,), seed=1, sigma=1e-3, apart=False):
        """apart: every array of a tensor at an offset of its own, drawn from `shifts`."""
        self.arena, self.sizes = Arena(), list(sizes)
        pick = lambda xs, k: xs[k % len(xs)]  # noqa: E731
        draw = np.random.RandomState(seed)
        put = lambda x, sh: self.arena.put(x, int(draw.choice(shifts)) if apart else sh)  # noqa: E731
        self.scales = [pick(scales, k) for k in range(len(self.sizes))]
        self.decays = [pick(decays, k) for k in range(len(self.sizes))]
        self.grad, self.master, self.m, self.v, self.exps, self.params = [], [], [], [], [], []
        for k, n in enumerate(self.sizes):
            sh = pick(shifts, k)
            self.grad.append(put(rand(n, seed * 1000 + k, sigma, GRAD[pick(grads, k)]), sh))
            self.master.append(put(rand(n, seed * 1000 + 300 + k, 0.02), sh))
            m, v = rand(n, seed * 1000 + 500 + k, sigma), rand(n, seed * 1000 + 700 + k, sigma, square=True)
            if state == "u8":
                (cm, bm), (cv, bv) = S.encode(m.numpy(), "m", S.NEAREST), S.encode(v.numpy(), "v", S.NEAREST)
                m, v = torch.from_numpy(cm), torch.from_numpy(cv)
                self.exps.append(put(torch.from_numpy(np.stack([bm, bv], 1).astype(np.uint8)), sh))
            self.m.append(put(m, sh))
            self.v.append(put(v, sh))
            dt = pick(params, k)
            self.params.append(put(torch.zeros(n, dtype=GRAD[dt]), sh))
        self.list = z.TensorList(grad=self.grad, master=self.master, m=self.m, v=self.v,
                                 exps=self.exps or None, params=self.params, lr_scale=self.scales,
                                 weight_decay=self.decays)
        self.st = torch.empty(z.STATE_BYTES, dtype=torch.uint8, device="cuda")
        self.work = torch.empty(z.zero_tensors_workspace_bytes(len(self.sizes)), dtype=torch.uint8, device="cuda")
        self.hp = z.hparams()
        z.zero_tensors_state_init(1, 1.0, False, 0, self.st)

    def set(self, **kw):
        st = z.zero_step_state_read(self.st)
        for k, x in kw.items():
            setattr(st, k, x)
        z.zero_step_state_write(self.st, st)

    def state(self):
        return z.zero_step_state_read(self.st)

    def norm(self):
        z.zero_tensors_grad_norm(self.list, self.hp, self.work, self.st)
        self.arena.check()
        return self.state()

    def arrays(self):
        return {k: [host(x).copy() for x in getattr(self, k)] for k in ("master", "m", "v", "params", "exps")}


STEP = dict(t=7, clip_coef=0.731, inv_scale_used=0.5, step_size=2.3e-3, rbc2=0.41)


# ------------------------------------------------------------------------------------------
# gradient norm
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("shifts", [(0,), (1,), (0, 3, 8, 1)])
@pytest.mark.parametrize("grads", [("bf16",), ("f16",), ("f32",), ("f32", "bf16", "f16")])
def test_norm_over_edges(grads, shifts):
    c = Case(EDGES, grads, shifts)
    c.set(inv_scale=0.25)
    want = np.sqrt(sum(np.sum((host(g).astype(np.float64) * 0.25) ** 2) for g in c.grad))
    s = c.norm()
    assert abs(s.norm - want) <= 3e-7 * want and s.sumsq == pytest.approx(s.norm ** 2, rel=1e-14)
    assert (s.skip, s.t, s.n_steps, s.overflow, s.arrivals, s.error) == (0, 1, 1, 0, 0, 0)
    assert s.clip_coef == np.float32(min(1.0, 1.0 / (s.norm + 1e-6)))
    assert s.inv_scale_used == 0.25
    again = Case(EDGES, grads, shifts)
    again.set(inv_scale=0.25)
    assert bytes(again.norm()) == bytes(s)  # the same bits each time


@pytest.mark.parametrize("n", [0, 1, 3, 384, 385, 768, 769, 1500])
def test_norm_list_lengths(n):
    """Lists of one launch and of several, empty tensors among them."""
    c = Case([k % 5 * 37 for k in range(n)], grads=("f32", "bf16"), shifts=(0, 1))
    want = np.sqrt(sum(np.sum(host(g).astype(np.float64) ** 2) for g in c.grad))
    s = c.norm()
    assert abs(s.norm - want) <= 3e-7 * want and s.n_steps == 1


def test_norm_agrees_with_the_flat_path_on_the_scalars():
    """Everything but the sum's last bits is zero_grad_norm's, over steps with an overflow."""
    n = 50_000
    lay = z.zero_partition(n, 1)
    reps = torch.zeros(lay.psi_padded, dtype=torch.float16, device="cuda")
    c = Case([n], grads=("f16",))
    g = torch.empty(lay.psi_padded, device="cuda")
    part = torch.empty(z.zero_workspace_bytes(lay) // 8, dtype=torch.float64, device="cuda")
    st = torch.empty(z.STATE_BYTES, dtype=torch.uint8, device="cuda")
    z.zero_step_state_init(lay, 1024.0, True, 2, st, part)
    z.zero_tensors_state_init(1, 1024.0, True, 2, c.st)
    for step in range(6):
        x = rand(n, step, 1e-2 * 1024, torch.float16).cuda()
        if step == 3:
            x[n - 1] = float("inf")
        reps[:n] = x
        c.grad[0].copy_(x)
        z.zero_reduce_shard_unscale(lay, z.ZERO_F16, [reps], 0, lay.psi_padded, g, part, st)
        z.zero_grad_norm(lay, c.hp, part, st)
        a, b = z.zero_step_state_read(st), c.norm()
        for f, _ in z.StepState._fields_:
            if f in ("sumsq", "norm", "clip_coef", "applied_c"):
                if step != 3:
                    assert getattr(b, f) == pytest.approx(getattr(a, f), rel=9 * U), f
            elif f != "reserved":
                assert getattr(a, f) == getattr(b, f), (step, f)
        assert b.skip == (step == 3)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_one_nonfinite_gradient_skips_the_step(value, dtype):
    sizes = [5, 9000, 300]
    for tensor, at in ((0, 0), (1, 0), (1, 4097), (1, 8192), (1, 8999), (2, 299)):
        c = Case(sizes, (dtype,), (0, 1))
        c.grad[tensor][at] = value
        before = c.arrays()
        s = c.norm()
        assert (s.skip, s.t, s.n_skipped, s.clip_coef, s.applied_c) == (1, 0, 1, 1.0, -1.0)
        assert not np.isfinite(s.norm)
        z.zero_tensors_adamw(c.list, c.hp, c.st)
        c.arena.check()
        for k, xs in c.arrays().items():
            assert all(np.array_equal(a, b) for a, b in zip(xs, before[k])), k


@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e-22, 2e-19, 1e-18, 3e-18, 1e-15, 1e17, 1e18, 1e19, 1e30, 3e38])
@pytest.mark.parametrize("shift", [0, 1])
def test_norm_of_extreme_magnitudes(scale, shift):
    """Squares outside fp32's range, whole or only in one group."""
    c = Case([10_001, 77], ("f32",), (shift,), sigma=1.0)
    signs = torch.sign(rand(10_001, 5, 1.0)).cuda()
    c.grad[0].copy_(signs * scale)
    c.grad[1].zero_()
    want = np.sqrt(np.sum(host(c.grad[0]).astype(np.float64) ** 2))
    s = c.norm()
    assert abs(s.norm - want) <= 3e-7 * want and s.skip == 0
    c.grad[0].zero_()
    c.grad[0][1234] = scale
    assert abs(c.norm().norm - float(np.float32(scale))) <= 3e-7 * scale


@pytest.mark.parametrize("grads,n,value", [(("bf16",), 300_000_000, 4e17), (("f32",), 130_000_000, 5.7e17),
                                           (("bf16", "f32"), 160_000_000, 4e17)])
def test_norm_of_long_lists_of_large_gradients(grads, n, value):
    """Finite gradients whose squares fp32 can hold one granule at a time, but not a whole
    share's sum of them (over 256 granules a thread): the norm is finite, the clip bites."""
    xs = [torch.full((n,), value, dtype=GRAD[d], device="cuda") for d in grads]
    st = torch.empty(z.STATE_BYTES, dtype=torch.uint8, device="cuda")
    work = torch.empty(z.zero_tensors_workspace_bytes(len(xs)), dtype=torch.uint8, device="cuda")
    z.zero_tensors_state_init(1, 1.0, False, 0, st)
    z.zero_tensors_grad_norm(z.TensorList(grad=xs), z.hparams(), work, st)
    s = z.zero_step_state_read(st)
    want = np.sqrt(sum(n * float(x[0].double()) ** 2 for x in xs))
    assert (s.skip, s.t, s.n_skipped) == (0, 1, 0)
    assert abs(s.norm - want) <= 3e-7 * want
    assert s.clip_coef == np.float32(1.0 / (s.norm + 1e-6)) and s.applied_c == s.clip_coef


def test_norm_of_zero_and_of_a_gradient_that_unscaling_overflows():
    c = Case([5000, 3], ("f32",))
    c.grad[0].zero_()
    c.grad[1].zero_()
    s = c.norm()
    assert (s.norm, s.clip_coef, s.skip, s.t) == (0.0, 1.0, 0, 1)
    c.grad[0][17] = 1e30
    c.set(inv_scale=1e20)   # 1/L for L = 1e-20: x is finite, g is not
    s = c.norm()
    assert s.skip == 1
    c.set(inv_scale=1e20)
    c.grad[0][17] = 1e10
    assert c.norm().norm == pytest.approx(1e30, rel=3e-7)


def test_clipping_off_and_the_count_of_copies():
    c = Case([3000], ("f32",))
    z.zero_tensors_state_init(8, 4.0, False, 0, c.st)
    c.hp = z.hparams(max_grad_norm=0.0)
    s = c.norm()
    want = np.sqrt(np.sum(host(c.grad[0]).astype(np.float64) ** 2)) / 32
    assert abs(s.norm - want) <= 3e-7 * want and s.clip_coef == 1.0 and s.inv_scale == np.float32(1 / 32)


# ------------------------------------------------------------------------------------------
# AdamW, 32-bit states
# ------------------------------------------------------------------------------------------
def expected(c, before, k, hp, sc, m, v):
    """The 64-bit update of tensor k and its tolerances."""
    x = host(c.grad[k])
    m1, v1 = S.moments(x, m, v, sc["clip_coef"], sc["inv_scale_used"], hp.beta1, hp.beta2, np.float64)
    gc = np.abs(x.astype(np.float64)) * np.float32(sc["clip_coef"]) * np.float32(sc["inv_scale_used"])
    size = hp.beta1 * np.abs(m.astype(np.float64)) + (1 - hp.beta1) * gc
    step = np.float32(np.float32(sc["step_size"]) * np.float32(c.scales[k]))
    decay = np.float32(1.0 - float(np.float32(hp.lr)) * float(np.float32(c.scales[k])) * float(np.float32(c.decays[k])))
    p1 = S.update(before["master"][k], m1, v1, step, sc["rbc2"], decay, hp.eps)
    denom = np.sqrt(v1) / np.float64(np.float32(sc["rbc2"])) + hp.eps
    tol_m = 5 * U * size + 1e-44
    tol_p = 3 * U * np.abs(before["master"][k]) + float(step) * (tol_m + 20 * U * np.abs(m1)) / denom + U * np.abs(p1)
    return m1, v1, p1, tol_m, 8 * U * v1 + 1e-44, tol_p


@pytest.mark.parametrize("shifts", [(0,), (1,), (3, 0, 8, 5)])
@pytest.mark.parametrize("grads", [("bf16",), ("f16",), ("f32", "bf16", "f16")])
def test_adamw_over_edges(grads, shifts):
    c = Case(EDGES, grads, shifts, params=("bf16", "f16"), scales=(1.0, 0.5, 0.0), decays=(0.01, 0.0))
    c.set(**STEP)
    before = c.arrays()
    z.zero_tensors_adamw(c.list, c.hp, c.st)
    c.arena.check()
    after = c.arrays()
    for k in range(len(EDGES)):
        m1, v1, p1, tm, tv, tp = expected(c, before, k, c.hp, STEP, before["m"][k], before["v"][k])
        assert np.all(np.abs(after["m"][k] - m1) <= tm) and np.all(np.abs(after["v"][k] - v1) <= tv)
        assert np.all(np.abs(after["master"][k] - p1) <= tp)
        rounded = torch.from_numpy(after["master"][k]).to(c.params[k].dtype).float().numpy()
        assert np.array_equal(after["params"][k], rounded)
    assert c.state().adamw_next_chunk == 0 and c.state().adamw_done == 0


@pytest.mark.parametrize("state", ["f32", "u8"])
@pytest.mark.parametrize("seed", [3, 4, 5, 6])
def test_every_array_at_an_offset_of_its_own(state, seed):
    """Random sizes, types and offsets, in the direct and in the staged form."""
    draw = np.random.RandomState(seed)
    sizes = [int(np.exp(draw.uniform(0, np.log(40_000)))) for _ in range(40)]
    if seed % 2:
        sizes[7] = 6_400_000 + int(draw.randint(9000))
    c = Case(sizes, ("f32", "bf16", "f16"), (0, 0, 1, 2, 3, 4, 5, 7, 8, 16), state, ("bf16", "f16"),
             (1.0, 0.5, 0.0, 2.0), (0.01, 0.0, 0.1), seed, apart=True)
    c.set(**STEP)
    s = c.norm()
    want = np.sqrt(sum(np.sum(host(g).astype(np.float64) ** 2) for g in c.grad))
    assert abs(s.norm - want) <= 3e-7 * want
    c.set(**STEP)
    before = c.arrays()
    if state == "u8":
        z.zero_tensors_adamw8(c.list, c.hp, seed, c.st)
        c.arena.check()
        check8(c, before, STEP, seed)
        return
    z.zero_tensors_adamw(c.list, c.hp, c.st)
    c.arena.check()
    after = c.arrays()
    for k in range(len(sizes)):
        m1, v1, p1, tm, tv, tp = expected(c, before, k, c.hp, STEP, before["m"][k], before["v"][k])
        assert np.all(np.abs(after["m"][k] - m1) <= tm) and np.all(np.abs(after["v"][k] - v1) <= tv)
        assert np.all(np.abs(after["master"][k] - p1) <= tp)
        assert np.array_equal(after["params"][k], torch.from_numpy(after["master"][k]).to(c.params[k].dtype).float().numpy())


def test_the_pieces_of_the_ranks_shards():
    """The pieces that zero_segment_map lists for each rank, every rank's state in its own
    shard, the gradients in the model's tensors: the same bits as the whole tensors at once."""
    sizes = [50_003, 77, 4801, 0, 12_288, 1, 30_000]
    psi, ranks = sum(sizes), 4
    lay = z.zero_partition(psi, ranks, 2)
    grads = [rand(n, 20 + k, 1e-3, torch.bfloat16).cuda() for k, n in enumerate(sizes)]
    flat = {"master": rand(lay.psi_padded, 1, 0.02).cuda(), "m": rand(lay.psi_padded, 2, 1e-3).cuda(),
            "v": rand(lay.psi_padded, 3, 1e-3, square=True).cuda()}
    decay = [0.1 if n > 5000 else 0.0 for n in sizes]
    c = Case([1])
    c.set(**STEP)
    cuts = np.cumsum([0, *sizes])
    whole = {k: x.clone() for k, x in flat.items()}
    z.zero_tensors_adamw(z.TensorList(grad=grads, weight_decay=decay, **{
        k: [x[a:b] for a, b in zip(cuts, cuts[1:])] for k, x in whole.items()}), c.hp, c.st)
    shards = [{k: x[r * lay.shard:(r + 1) * lay.shard].clone() for k, x in flat.items()} for r in range(ranks)]
    for r in range(ranks):
        mine = [s for s in z.zero_segment_map(lay, sizes) if s.rank == r]
        lst = z.TensorList(
            grad=[grads[s.tensor][s.tensor_offset:s.tensor_offset + s.count] for s in mine],
            weight_decay=[decay[s.tensor] for s in mine],
            **{k: [x[s.shard_offset:s.shard_offset + s.count] for s in mine] for k, x in shards[r].items()})
        z.zero_tensors_adamw(lst, c.hp, c.st)
    for k, x in whole.items():
        got = torch.cat([s[k] for s in shards])
        assert torch.equal(got.view(torch.int32), x.view(torch.int32)), k


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("psi", [1, 8191, 100_003, 6_500_017])
def test_adamw_gives_the_flat_steps_bits(psi, dtype):
    """The flat buffer cut into pieces (at odd places, so most are misaligned) and as one
    tensor: zero_step's master, m, v and parameters, bit for bit, over three steps."""
    lay = z.zero_partition(psi, 1)
    code = z.ZERO_F16 if dtype == "f16" else z.ZERO_BF16
    hp = z.hparams()
    cuts = sorted({0, psi, *(int(x) for x in np.linspace(0, psi, 9)), min(5, psi), min(8, psi), min(300, psi)})
    spans = list(zip(cuts[:-1], cuts[1:]))
    runs = {"flat": None, "pieces": spans, "whole": [(0, psi)]}
    got = {}
    for name, cut in runs.items():
        bufs = {k: torch.zeros(lay.psi_padded, device="cuda") for k in ("g", "m", "v")}
        bufs["master"] = rand(lay.psi_padded, 3, 0.02).cuda()
        out = torch.zeros(lay.psi_padded, dtype=GRAD[dtype], device="cuda")
        part = torch.empty(z.zero_workspace_bytes(lay) // 8, dtype=torch.float64, device="cuda")
        st = torch.empty(z.STATE_BYTES, dtype=torch.uint8, device="cuda")
        hp.params_dtype = code
        z.zero_step_state_init(lay, 64.0, False, 0, st, part)
        for step in range(3):
            x = rand(lay.psi_padded, 10 + step, 64e-4, GRAD[dtype]).cuda()
            if name == "flat":
                z.zero_step(lay, hp, code, [x], bufs["g"], part, bufs["master"], bufs["m"], bufs["v"], out, st)
                continue
            # the flat step's scalars, so that the sum's last bits cannot matter
            z.zero_step_state_write(st, got["flat"][1][step])
            lst = z.TensorList(grad=[x[a:b] for a, b in cut], params=[out[a:b] for a, b in cut], weight_decay=0.01,
                               **{k: [bufs[k][a:b] for a, b in cut] for k in ("master", "m", "v")})
            z.zero_tensors_adamw(lst, hp, st)
        if name == "flat":
            states = []
            st2 = torch.empty_like(st)
            z.zero_step_state_init(lay, 64.0, False, 0, st2, part)
            for step in range(3):   # the scalars after each step, recomputed
                x = rand(lay.psi_padded, 10 + step, 64e-4, GRAD[dtype]).cuda()
                z.zero_reduce_shard_unscale(lay, code, [x], 0, lay.psi_padded, bufs["g"], part, st2)
                z.zero_grad_norm(lay, hp, part, st2)
                states.append(z.zero_step_state_read(st2))
            got["flat"] = ({k: b[:psi].clone() for k, b in bufs.items() if k != "g"} | {"out": out[:psi].clone()}, states)
        else:
            for k, want in got["flat"][0].items():
                have = out if k == "out" else bufs[k]
                bits = torch.int16 if k == "out" else torch.int32
                assert torch.equal(have[:psi].view(bits), want.view(bits)), (name, k)


@pytest.mark.parametrize("eps,lr", [(1e-8, 1e-3), (1e-30, 1e-3), (1e-8, 1e30), (1e-12, 0.0)])
@pytest.mark.parametrize("n", [300_000, 6_400_000])
def test_adamw_gives_the_flat_steps_bits_on_any_values(n, eps, lr):
    """zero_adamw_cast_gather's bits where division and square root have their special cases:
    zeros of both signs, subnormals, every exponent, infinities and NaN in each operand."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    u = lambda: torch.rand(n, device="cuda", generator=gen)  # noqa: E731

    def values(special, lo=-149.0, hi=60.0, signed=True):
        x = torch.exp2(u() * (hi - lo) + lo) * (1 + u())
        if signed:
            x = torch.where(u() < 0.5, -x, x)
        pick = torch.tensor(special, device="cuda")
        return torch.where(u() < 0.4, pick[(u() * len(special)).long().clamp(max=len(special) - 1)], x)

    inf, nan = float("inf"), float("nan")
    g = values([0.0, -0.0, 1e-4, -1e-3, 1e-30, 1e-45], -149, 40)
    m = values([0.0, -0.0, 1e-40, -1.4e-45, 1e-34, nan, inf], -149, 40)
    v = values([0.0, 1e-44, 1e-38, 1e-31, 1e-8, inf, nan], -149, 60, signed=False)
    p = values([0.0, -0.0, 0.02, -0.02, 1e-42, 1e-13, 2.0 ** -40, nan], -149, 20)
    lay = z.zero_partition(n, 1)
    hp = z.hparams(eps=eps, lr=lr)
    st = torch.empty(z.STATE_BYTES, dtype=torch.uint8, device="cuda")
    z.zero_tensors_state_init(1, 1.0, False, 0, st)
    s = z.zero_step_state_read(st)
    s.t, s.clip_coef, s.inv_scale_used, s.step_size, s.rbc2, s.decay = 7, 0.731, 1.0, lr * 2, 0.41, 1.0 - lr * 0.01 if lr < 1 else 0.5
    z.zero_step_state_write(st, s)
    flat = [x.clone() for x in (p, m, v)]
    out = torch.zeros(lay.psi_padded, dtype=torch.bfloat16, device="cuda")
    assert lay.psi_padded == n
    z.zero_adamw_cast_gather(lay, hp, g, *flat, out, st)
    params = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    wd = 0.01 if lr < 1 else 0.5 / lr
    z.zero_tensors_adamw(z.TensorList(grad=[g], master=[p], m=[m], v=[v], params=[params], weight_decay=wd), hp, st)
    for name, a, b in (("master", p, flat[0]), ("m", m, flat[1]), ("v", v, flat[2])):
        same = (a.view(torch.int32) == b.view(torch.int32)) | (a.isnan() & b.isnan())
        assert bool(same.all()), (name, int((~same).sum()), [(x[~same][:3].tolist()) for x in (a, b, m, v, p, g)])
    assert bool(((params.view(torch.int16) == out[:n].view(torch.int16)) | (params.isnan() & out[:n].isnan())).all())


@pytest.mark.parametrize("n", [300_000, 6_400_000])
def test_adamw_shows_a_negative_second_moment(n):
    """A v that has gone negative (a damaged state) gives NaN, as zero_adamw_cast_gather does,
    and no finite update, however small it is and whatever lies beside it."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    u = lambda: torch.rand(n, device="cuda", generator=gen)  # noqa: E731
    g = torch.where(u() < 0.5, 0.0, 1e-4 * (u() - 0.5))
    m, p = 1e-3 * (u() - 0.5), 0.02 * (u() - 0.5)
    m[u() < 0.3] = 0.0
    v = torch.exp2(-149 + 150 * u())
    v = torch.where(u() < 0.3, -v, torch.where(u() < 0.3, 0.0, v))
    lay, hp = z.zero_partition(n, 1), z.hparams()
    assert lay.psi_padded == n
    st = torch.empty(z.STATE_BYTES, dtype=torch.uint8, device="cuda")
    z.zero_tensors_state_init(1, 1.0, False, 0, st)
    s = z.zero_step_state_read(st)
    s.t, s.clip_coef, s.inv_scale_used, s.step_size, s.rbc2 = 7, 0.731, 1.0, 2e-3, 0.41
    s.decay = 1.0 - float(np.float32(hp.lr)) * float(np.float32(0.01))
    z.zero_step_state_write(st, s)
    flat = [x.clone() for x in (p, m, v)]
    out = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    z.zero_adamw_cast_gather(lay, hp, g, *flat, out, st)
    params = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    z.zero_tensors_adamw(z.TensorList(grad=[g], master=[p], m=[m], v=[v], params=[params], weight_decay=0.01), hp, st)
    assert int((flat[2] < 0).sum()) > n // 10
    assert bool(params[flat[2] < 0].isnan().all()) and bool(p[flat[2] < 0].isnan().all())
    for name, a, b in (("master", p, flat[0]), ("m", m, flat[1]), ("v", v, flat[2])):
        same = (a.view(torch.int32) == b.view(torch.int32)) | (a.isnan() & b.isnan())
        assert bool(same.all()), (name, int((~same).sum()))


@pytest.mark.parametrize("state", ["f32", "u8"])
@pytest.mark.parametrize("sizes", [[40 + 13 * (k % 11) for k in range(450)], [6_900_000, 300, 77]],
                         ids=["450 tensors", "staged"])
def test_whole_step_as_a_user_runs_it(sizes, state):
    """Norm, then AdamW, for a list longer than one launch and for one in the staged form, on a
    stream of its own, captured into a graph and replayed; the eager run gives the same bits."""
    eager, graphed = (Case(sizes, ("bf16", "f32"), (0, 1), state) for _ in range(2))

    def step(c):
        z.zero_tensors_grad_norm(c.list, c.hp, c.work, c.st)
        if state == "u8":
            z.zero_tensors_adamw8(c.list, c.hp, 6, c.st)
        else:
            z.zero_tensors_adamw(c.list, c.hp, c.st)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(4):
            step(eager)
    torch.cuda.current_stream().wait_stream(side)
    warm = Case(sizes, ("bf16", "f32"), (0, 1), state)
    step(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(graphed)
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    assert bytes(eager.state()) == bytes(graphed.state()) and eager.state().t == 4
    for k, xs in eager.arrays().items():
        assert all(np.array_equal(a, b) for a, b in zip(xs, graphed.arrays()[k])), k
    eager.arena.check()
    graphed.arena.check()


@pytest.mark.parametrize("state", ["f32", "u8"])
def test_tensors_dense_in_another_order(state):
    """A channels-last weight and a transposed one, every array in that order: the same update
    as on the elements in memory order."""
    c = Case([4 * 6 * 5 * 7, 60 * 33], ("f32",), state=state)
    c.set(**STEP)
    before = c.arrays()

    def shaped(xs):
        return [xs[0].view(4, 5, 7, 6).permute(0, 3, 1, 2), xs[1].view(60, 33).t()]

    kw = dict(exps=c.exps) if state == "u8" else {}
    lst = z.TensorList(grad=shaped(c.grad), master=shaped(c.master), m=shaped(c.m), v=shaped(c.v),
                       params=shaped(c.params), weight_decay=0.01, **kw)
    assert not lst.tensors["grad"][0].is_contiguous() and not lst.tensors["m"][1].is_contiguous()
    if state == "u8":
        z.zero_tensors_adamw8(lst, c.hp, 4, c.st)
        check8(c, before, STEP, 4)
    else:
        z.zero_tensors_adamw(lst, c.hp, c.st)
        for k in range(2):
            p1, tp = expected(c, before, k, c.hp, STEP, before["m"][k], before["v"][k])[2::3]
            assert np.all(np.abs(c.arrays()["master"][k] - p1) <= tp)
    c.arena.check()


def test_params_may_be_absent_and_integers():
    c = Case([3000, 77])
    c.set(**STEP)
    before = c.arrays()
    bits = [p.view(torch.int16) for p in c.params]
    hp = z.hparams(params_dtype=z.ZERO_F16)
    lst = z.TensorList(grad=c.grad, master=c.master, m=c.m, v=c.v, params=bits, weight_decay=0.01)
    z.zero_tensors_adamw(lst, hp, c.st)
    for p, b in zip(c.master, bits):
        assert torch.equal(b.view(torch.float16), p.half())
    lst = z.TensorList(grad=c.grad, master=c.master, m=c.m, v=c.v, weight_decay=0.01)
    kept = [b.clone() for b in bits]
    z.zero_tensors_adamw(lst, hp, c.st)
    c.arena.check()
    assert all(torch.equal(a, b) for a, b in zip(bits, kept))
    assert not np.array_equal(c.arrays()["master"][0], before["master"][0])


# ------------------------------------------------------------------------------------------
# AdamW, 8-bit states
# ------------------------------------------------------------------------------------------
def check8(c, before, sc, seed):
    after, block = c.arrays(), 0
    for k, n in enumerate(c.sizes):
        bm, bv = before["exps"][k].reshape(-1, 2).T if n else (np.zeros(0), np.zeros(0))
        m, v = S.decode(before["m"][k], bm, "m"), S.decode(before["v"][k], bv, "v")
        m32, v32 = S.moments(host(c.grad[k]), m, v, sc["clip_coef"], sc["inv_scale_used"], c.hp.beta1, c.hp.beta2)
        blocks = -(-n // 256)
        for name, x, codes, col in (("m", m32, after["m"][k], 0), ("v", v32, after["v"][k], 1)):
            want, b = S.encode(x, name, S.random20(blocks, seed, sc["t"], block, name))
            assert np.array_equal(after["exps"][k].reshape(-1, 2)[:, col], b), (k, name)
            assert np.array_equal(codes, want), (k, name, np.flatnonzero(codes != want)[:5])
        _, _, p1, _, _, tp = expected(c, before, k, c.hp, sc, m, v)
        assert np.all(np.abs(after["master"][k] - p1) <= tp), k
        rounded = torch.from_numpy(after["master"][k]).to(c.params[k].dtype).float().numpy()
        assert np.array_equal(after["params"][k], rounded)
        block += blocks


@pytest.mark.parametrize("shifts", [(0,), (1,), (3, 0, 8, 5)])
@pytest.mark.parametrize("grads", [("bf16",), ("f16",), ("f32", "bf16", "f16")])
def test_adamw8_over_edges(grads, shifts):
    c = Case(EDGES, grads, shifts, "u8", ("bf16", "f16"), (1.0, 0.5, 0.0), (0.01, 0.0))
    c.set(**STEP)
    for seed in (0, 0xFEDCBA9876543210):
        before = c.arrays()
        z.zero_tensors_adamw8(c.list, c.hp, seed, c.st)
        c.arena.check()
        check8(c, before, STEP, seed)


@pytest.mark.parametrize("n", [384, 385, 900])
def test_adamw8_long_lists(n):
    """The blocks are counted over the whole list, whatever launches it takes."""
    c = Case([(k * 97) % 700 for k in range(n)], ("f32", "bf16"), (0, 0, 1), "u8")
    c.set(**STEP)
    before = c.arrays()
    z.zero_tensors_adamw8(c.list, c.hp, 99, c.st)
    c.arena.check()
    check8(c, before, STEP, 99)


@pytest.mark.parametrize("shift", [0, 1])
def test_adamw8_values_at_the_ends_of_the_range(shift):
    """Fresh states, blocks of zeros, spreads wider than the codes, magnitudes that
    saturate, fp32 subnormals."""
    n = 256 * 9 + 100
    c = Case([n], ("f32",), (shift,), "u8")
    for x in (c.m[0], c.v[0], c.exps[0]):
        x.zero_()
    g = torch.zeros(n)
    g[256:512] = torch.logspace(-40, 3, 256)              # 43 decades in one block
    g[512:768] = rand(256, 1, 1e-30)
    g[768:1024] = 1e-38
    g[1024:1280] = rand(256, 2, 1e18)
    g[1280:1536] = torch.where(rand(256, 3, 1.0) > 0, 3e38, -3e38)
    g[1536] = 1.0                                         # one element in a block of zeros
    g[1792:2048] = 1.875 * 2.0 ** -5
    g[2048:2304] = 1.8751 * 2.0 ** -5
    c.grad[0].copy_(g)
    sc = dict(STEP, clip_coef=1.0, inv_scale_used=1.0)
    c.set(**sc)
    for step in range(3):
        before = c.arrays()
        with np.errstate(over="ignore", invalid="ignore"):
            z.zero_tensors_adamw8(c.list, c.hp, 5, c.st)
            c.arena.check()
            after = c.arrays()
            bm, bv = before["exps"][0].reshape(-1, 2).T
            m, v = S.decode(before["m"][0], bm, "m"), S.decode(before["v"][0], bv, "v")
            m1, v1 = S.moments(g.numpy(), m, v, 1.0, 1.0, c.hp.beta1, c.hp.beta2)
            for name, x, col in (("m", m1, 0), ("v", v1, 1)):
                want, b = S.encode(x, name, S.random20(-(-n // 256), 5, sc["t"], 0, name))
                assert np.array_equal(after["exps"][0].reshape(-1, 2)[:, col], b)
                assert np.array_equal(after[name][0], want), (name, np.flatnonzero(after[name][0] != want)[:5])
        assert np.all(after["v"][0][v1 > 0] > 0)
        assert np.all(after["m"][0][:256] == 0) and np.all(after["exps"][0][:2] == 0)
        fits = np.isfinite(v1)      # else the denominator is infinite in fp32, and the update 0
        with np.errstate(over="ignore"):
            _, _, p1, _, _, tp = expected(c, before, 0, c.hp, sc, m, v)
        assert np.all(np.abs(after["master"][0] - p1)[fits] <= tp[fits])
        assert np.all(np.isfinite(after["master"][0]))


@pytest.mark.parametrize("eps", [1e-8, 1e-30, 1e-35, 1e-40])
def test_adamw8_with_a_small_eps(eps):
    """An eps down to fp32's subnormals, with gradients and states of zero among the others."""
    c = Case([5000, 300], ("f32",), (0, 1), "u8")
    c.hp = z.hparams(eps=eps)
    c.set(**STEP)
    for x in (*c.grad, *c.m, *c.v):
        x[::3] = 0
    before = c.arrays()
    z.zero_tensors_adamw8(c.list, c.hp, 8, c.st)
    c.arena.check()
    check8(c, before, STEP, 8)


@pytest.mark.parametrize("eps", [1e-8, 1e-20, 1e-29])
@pytest.mark.parametrize("n", [3000, 6_300_000])
def test_adamw8_updates_from_gradients_near_the_smallest(n, eps):
    """Moments of 1e-37 over a small eps: the update is an ordinary number (1e-11 for the
    smallest eps) and as precise as any other, though step * m is subnormal."""
    c = Case([n], ("f32",), (0,), "u8")
    for x in (c.m[0], c.v[0], c.exps[0], c.master[0]):
        x.zero_()
    gen = torch.Generator(device="cuda").manual_seed(n)
    c.grad[0].copy_((1 + 3 * torch.rand(n, device="cuda", generator=gen)) * 1e-36)
    c.hp = z.hparams(eps=eps)
    c.set(**STEP)
    before = c.arrays()
    z.zero_tensors_adamw8(c.list, c.hp, 5, c.st)
    c.arena.check()
    zeros = np.zeros(n, np.float32)
    _, _, p1, _, _, tp = expected(c, before, 0, c.hp, STEP, zeros, zeros)
    got = c.arrays()["master"][0]
    assert np.all(np.abs(got - p1) <= tp), np.max(np.abs(got / p1 - 1))
    assert np.all(np.abs(p1) > 20 * tp)     # the tolerance says something of the update


def test_adamw8_follows_the_32_bit_moments():
    """Over 300 steps with gradients whose size drops by 10 after the first 100, v's mean
    follows the 32-bit run's (rounding to nearest would hold it where it was), and the
    parameters stay near the 32-bit run's: the noise of one rounding is at most 1/8 of v,
    its sum over the ~1/(1-b2) steps that v remembers about 1/4 per element, so 3% on a
    mean over 65,536 elements is over 25 standard errors."""
    n, hp = 65_536, z.hparams(lr=1e-3, beta2=0.99, weight_decay=0.0, max_grad_norm=0.0)
    master = torch.zeros(n, device="cuda")
    runs = {}
    for name in ("f32", "u8"):
        zeros = lambda dt, k=n: [torch.zeros(k, dtype=dt, device="cuda")]  # noqa: E731
        dt = torch.float32 if name == "f32" else torch.uint8
        kw = dict(exps=zeros(torch.uint8, 2 * n // 256)) if name == "u8" else {}
        lst = z.TensorList(grad=zeros(torch.float32), master=[master.clone()], m=zeros(dt), v=zeros(dt), **kw)
        st = torch.empty(z.STATE_BYTES, dtype=torch.uint8, device="cuda")
        work = torch.empty(z.zero_tensors_workspace_bytes(1), dtype=torch.uint8, device="cuda")
        z.zero_tensors_state_init(1, 1.0, False, 0, st)
        gen = torch.Generator(device="cuda").manual_seed(4)
        means = []
        for step in range(300):
            lst.tensors["grad"][0].normal_(0.0, 1e-3 if step < 100 else 1e-4, generator=gen)
            z.zero_tensors_grad_norm(lst, hp, work, st)
            if name == "u8":
                z.zero_tensors_adamw8(lst, hp, 77, st)
            else:
                z.zero_tensors_adamw(lst, hp, st)
            if step % 50 == 49:
                v = lst.tensors["v"][0]
                if name == "u8":
                    out = z.TensorList(m=zeros(torch.float32), v=zeros(torch.float32))
                    z.zero_tensors_state8_read(lst, out)
                    v = out.tensors["v"][0]
                means.append(float(v.double().mean()))
        runs[name] = (means, lst.tensors["master"][0].double())
    for a, b in zip(runs["u8"][0], runs["f32"][0]):
        assert abs(a - b) <= 0.03 * b, runs
    p8, p32 = runs["u8"][1], runs["f32"][1]
    assert float((p8 - p32).norm() / p32.norm()) < 0.5   # independent runs would give 1.4
    assert float(torch.dot(p8, p32) / p8.norm() / p32.norm()) > 0.9


def test_adamw8_repeats_and_its_seed_and_step_matter():
    def once(seed, t):
        c = Case([5000], state="u8")
        c.set(**dict(STEP, t=t))
        z.zero_tensors_adamw8(c.list, c.hp, seed, c.st)
        return c.arrays()

    base = once(5, 7)
    same = once(5, 7)
    assert all(np.array_equal(a, b) for k in base for a, b in zip(base[k], same[k]))
    for other in (once(6, 7), once(5, 8), once(5 + (1 << 32), 7)):
        assert np.array_equal(other["master"][0], base["master"][0])   # no rounding of p depends on it
        assert not np.array_equal(other["m"][0], base["m"][0])
        assert not np.array_equal(other["v"][0], base["v"][0])


# ------------------------------------------------------------------------------------------
# lists long enough for the staged form
# ------------------------------------------------------------------------------------------
LONG = EDGES + [6_300_003, 4095, 4097, 5887, 5889, 8200, 12_288, 1]


@pytest.mark.parametrize("grads,shifts", [(("bf16",), (0,)), (("f32", "bf16", "f16"), (1,)),
                                          (("f16", "f32", "bf16"), (3, 0, 8, 5))])
@pytest.mark.parametrize("state", ["f32", "u8"])
def test_adamw_on_long_lists(state, grads, shifts):
    """The same checks on a list of 6.4 million elements."""
    c = Case(LONG, grads, shifts, state, ("bf16", "f16"), (1.0, 0.5, 0.0), (0.01, 0.0))
    c.set(**STEP)
    for seed in (1,):
        before = c.arrays()
        if state == "u8":
            z.zero_tensors_adamw8(c.list, c.hp, seed, c.st)
            c.arena.check()
            check8(c, before, STEP, seed)
        else:
            z.zero_tensors_adamw(c.list, c.hp, c.st)
            c.arena.check()
            after = c.arrays()
            for k in range(len(LONG)):
                m1, v1, p1, tm, tv, tp = expected(c, before, k, c.hp, STEP, before["m"][k], before["v"][k])
                assert np.all(np.abs(after["m"][k] - m1) <= tm) and np.all(np.abs(after["v"][k] - v1) <= tv)
                assert np.all(np.abs(after["master"][k] - p1) <= tp)
                rounded = torch.from_numpy(after["master"][k]).to(c.params[k].dtype).float().numpy()
                assert np.array_equal(after["params"][k], rounded)
        s = c.state()
        assert (s.adamw_next_chunk, s.adamw_done, s.error) == (0, 0, 0)


@pytest.mark.parametrize("state", ["f32", "u8"])
def test_long_lists_of_several_launches(state):
    """430 tensors, 14 million elements, in the staged form: the blocks and the queue go on
    over the launches; a skipped step leaves everything."""
    sizes = [1 + (k * 7919) % 300 for k in range(424)] + [7_000_001, 2, 4096, 7_100_003, 300, 5889]
    assert sum(sizes) >= len(sizes) << 15
    c = Case(sizes, ("f32", "bf16"), (0, 0, 1), state)
    c.set(**STEP)
    before = c.arrays()
    call = z.zero_tensors_adamw if state == "f32" else lambda *a: z.zero_tensors_adamw8(a[0], a[1], 99, a[2])
    c.set(skip=1)
    call(c.list, c.hp, c.st)
    for k, xs in c.arrays().items():
        assert all(np.array_equal(a, b) for a, b in zip(xs, before[k])), k
    c.set(skip=0)
    call(c.list, c.hp, c.st)
    c.arena.check()
    if state == "u8":
        check8(c, before, STEP, 99)
    else:
        after = c.arrays()
        for k in range(len(sizes)):
            m1, v1, p1, tm, tv, tp = expected(c, before, k, c.hp, STEP, before["m"][k], before["v"][k])
            assert np.all(np.abs(after["m"][k] - m1) <= tm) and np.all(np.abs(after["v"][k] - v1) <= tv)
            assert np.all(np.abs(after["master"][k] - p1) <= tp)
    s = c.state()
    assert (s.adamw_next_chunk, s.adamw_done, s.error) == (0, 0, 0)


@pytest.mark.parametrize("state", ["f32", "u8"])
def test_a_wait_that_runs_out_reports_an_error(hooked, state):
    """With one chunk's copies withheld (test build only) the staged kernel gives up after
    ~2 s, records 1 in the error word, puts the queue back and ends; the GPU stays usable."""
    sizes = [6_500_017, 300]
    c = Case(sizes, state=state)
    c.set(**STEP)
    hooked.zero_test_withhold_tensors_chunk.argtypes = [C.c_ulonglong]
    hooked.zero_tensors_adamw.argtypes = z.lib().zero_tensors_adamw.argtypes
    hooked.zero_tensors_adamw8.argtypes = z.lib().zero_tensors_adamw8.argtypes
    stream = torch.cuda.current_stream().cuda_stream
    assert hooked.zero_test_withhold_tensors_chunk(200) == 0
    t0 = time.time()
    if state == "u8":
        rc = hooked.zero_tensors_adamw8(c.list.array, 2, C.byref(c.hp), 1, c.st.data_ptr(), stream)
    else:
        rc = hooked.zero_tensors_adamw(c.list.array, 2, C.byref(c.hp), c.st.data_ptr(), stream)
    assert rc == 0
    torch.cuda.synchronize()  # completes: the waits gave up, no fault
    waited = time.time() - t0
    assert hooked.zero_test_withhold_tensors_chunk(~0 & 0xFFFFFFFFFFFFFFFF) == 0
    s = c.state()
    assert (s.error, s.adamw_next_chunk, s.adamw_done) == (1, 0, 0) and 1.0 < waited < 60.0
    c.arena.check()
    # the context is still good: the product library's step on fresh buffers
    c = Case(sizes, state=state)
    c.set(**STEP)
    before = c.arrays()
    if state == "u8":
        z.zero_tensors_adamw8(c.list, c.hp, 1, c.st)
        check8(c, before, STEP, 1)
    else:
        z.zero_tensors_adamw(c.list, c.hp, c.st)
        p1, tp = expected(c, before, 0, c.hp, STEP, before["m"][0], before["v"][0])[2::3]
        assert np.all(np.abs(c.arrays()["master"][0] - p1) <= tp)
    c.arena.check()


# ------------------------------------------------------------------------------------------
# the 8-bit states read and written
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shifts", [(0,), (1,), (3, 0, 8, 5)])
def test_write_and_read(shifts, dtype):
    sizes = EDGES + [300_003]
    c = Case(sizes, state="u8", shifts=shifts)
    a = Arena()
    src = [[a.put(rand(n, 40 + k, 1e-3 * 10.0 ** (k % 7 - 3), square=sq), shifts[k % len(shifts)])
            for k, n in enumerate(sizes)] for sq in (False, True)]
    out = [[a.put(torch.zeros(n, dtype=dtype), shifts[k % len(shifts)]) for k, n in enumerate(sizes)] for _ in "mv"]
    z.zero_tensors_state8_write(c.list, z.TensorList(m=src[0], v=src[1]))
    z.zero_tensors_state8_read(c.list, z.TensorList(m=out[0], v=out[1]))
    c.arena.check()
    a.check()
    got = c.arrays()
    for k, n in enumerate(sizes):
        for name, x, y, col in (("m", src[0][k], out[0][k], 0), ("v", src[1][k], out[1][k], 1)):
            x, y = host(x), host(y)
            codes, b = S.encode(x, name, S.NEAREST)
            assert np.array_equal(got[name][k], codes) and np.array_equal(got["exps"][k].reshape(-1, 2)[:, col], b)
            assert np.array_equal(y, S.decode(codes, b, name))
            unit = np.exp2(np.repeat(b, 256)[:n] - 127.0) * 2.0 ** (-14 if name == "m" else -30)
            assert np.all(np.abs(y - x.astype(np.float64)) <= np.maximum(np.abs(x) / 16, unit / 8 * (1 if name == "v" else 0.5)))
    # writing what was read keeps every value
    if dtype == torch.float32:
        z.zero_tensors_state8_write(c.list, z.TensorList(m=out[0], v=out[1]))
        second = [[torch.empty_like(x) for x in xs] for xs in out]
        z.zero_tensors_state8_read(c.list, z.TensorList(m=second[0], v=second[1]))
        assert all(torch.equal(x, y) for xs, ys in zip(out, second) for x, y in zip(xs, ys))


def test_nan_and_infinity_are_stored_as_the_largest_code():
    x = torch.tensor([float("nan"), float("inf"), -float("inf"), 1.0, 3e38, 0.0], device="cuda")
    n = x.numel()
    lst = z.TensorList(m=[torch.zeros(n, dtype=torch.uint8, device="cuda")], v=[torch.zeros(n, dtype=torch.uint8, device="cuda")],
                       exps=[torch.zeros(2, dtype=torch.uint8, device="cuda")])
    out = z.TensorList(m=[torch.empty(n, device="cuda")], v=[torch.empty(n, device="cuda")])
    z.zero_tensors_state8_write(lst, z.TensorList(m=[x], v=[x.abs()]))
    z.zero_tensors_state8_read(lst, out)
    top = 1.875 * 2.0 ** 126
    assert out.tensors["m"][0].abs().tolist() == [top, top, top, 0.0, top, 0.0]
    assert out.tensors["v"][0].tolist()[:3] == [top] * 3 and out.tensors["v"][0].tolist()[3] > 0


# ------------------------------------------------------------------------------------------
# offsets past 32 bits
# ------------------------------------------------------------------------------------------
def test_norm_past_32_bit_offsets():
    n = (1 << 32) + 4101
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    at = [0, (1 << 31) - 1, 1 << 31, (1 << 32) - 1, 1 << 32, n - 1]
    g[at] = torch.arange(1, 7, dtype=torch.bfloat16, device="cuda")
    st = torch.empty(z.STATE_BYTES, dtype=torch.uint8, device="cuda")
    work = torch.empty(z.zero_tensors_workspace_bytes(1), dtype=torch.uint8, device="cuda")
    z.zero_tensors_state_init(1, 1.0, False, 0, st)
    z.zero_tensors_grad_norm(z.TensorList(grad=[g]), z.hparams(), work, st)
    assert z.zero_step_state_read(st).sumsq == 91.0
    del g
    torch.cuda.empty_cache()


def test_adamw_past_32_bit_offsets():
    """2^31 + 300 elements: 8 GB arrays, element and byte offsets past 32 bits."""
    n = (1 << 31) + 300
    near = [0, (1 << 30) - 128, (1 << 31) - 128]
    grad = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    master, m, v = (torch.zeros(n, device="cuda") for _ in "pmv")
    for k, i in enumerate(near):
        grad[i:i + 256] = (k + 1) * 1e-3
        master[i:i + 256] = 0.1 * (k + 1)
    grad[n - 1] = master[n - 1] = 1.0
    st = torch.empty(z.STATE_BYTES, dtype=torch.uint8, device="cuda")
    z.zero_tensors_state_init(1, 1.0, False, 0, st)
    s = z.zero_step_state_read(st)
    for k, x in dict(STEP, inv_scale_used=1.0, clip_coef=1.0).items():
        setattr(s, k, x)
    z.zero_step_state_write(st, s)
    z.zero_tensors_adamw(z.TensorList(grad=[grad], master=[master], m=[m], v=[v], weight_decay=0.01), z.hparams(), st)
    for k, i in enumerate(near + [n - 1]):
        g, p = grad[i].double().item(), 0.1 * (k + 1) if i < n - 1 else 1.0
        want = p * (1 - 1e-5) - 2.3e-3 * 0.1 * g / (np.sqrt(0.001) * g / 0.41 + 1e-8)
        got = master[i:min(n, i + 256)]
        assert torch.allclose(got, torch.full_like(got, want), rtol=1e-5), i
        assert torch.allclose(m[i:min(n, i + 256)], torch.full_like(got, 0.1 * g), rtol=1e-5)
    assert int((master != 0).sum()) == int((m != 0).sum()) == int((v != 0).sum()) == 3 * 256 + 1
    del grad, master, m, v, got
    torch.cuda.empty_cache()


def test_adamw8_and_read_past_32_bit_offsets():
    """A tensor of 2^32 + 300 elements: the elements around each power of two take the
    update that a short tensor with the same values takes (but for the random bits, which
    a gradient of zero and states on the codes' grid leave without effect on p)."""
    n = (1 << 32) + 300
    near = [0, (1 << 31) - 256, 1 << 31, (1 << 32) - 256, 1 << 32]
    grad = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    master = torch.zeros(n, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in "mv")
    exps = torch.zeros(2 * -(-n // 256), dtype=torch.uint8, device="cuda")
    for k, i in enumerate(near):
        grad[i:i + 256] = (k + 1) * 1e-3
        master[i:i + 256] = 0.1 * (k + 1)
    grad[n - 1] = master[n - 1] = 1.0
    st = torch.empty(z.STATE_BYTES, dtype=torch.uint8, device="cuda")
    z.zero_tensors_state_init(1, 1.0, False, 0, st)
    s = z.zero_step_state_read(st)
    for k, x in dict(STEP, inv_scale_used=1.0, clip_coef=1.0).items():
        setattr(s, k, x)
    z.zero_step_state_write(st, s)
    hp = z.hparams()
    z.zero_tensors_adamw8(z.TensorList(grad=[grad], master=[master], m=[m], v=[v], exps=[exps], weight_decay=0.01), hp, 3, st)
    def want(g, p):
        g, m1 = float(g), 0.1 * float(g)
        return p * (1 - 1e-5) - 2.3e-3 * m1 / (np.sqrt(0.001) * g / 0.41 + 1e-8)
    for k, i in enumerate(near[:4]):
        g = grad[i].item()
        got = master[i:i + 256]
        assert torch.allclose(got, torch.full_like(got, want(g, 0.1 * (k + 1))), rtol=1e-5)
    assert abs(master[n - 1].item() - want(1.0, 1.0)) < 1e-5
    assert int((master != 0).sum()) == 5 * 256 + 1 and bool((m[near[4]:near[4] + 256] > 0).all())
    out = z.TensorList(m=[torch.empty(n, dtype=torch.bfloat16, device="cuda")], v=[torch.empty(n, dtype=torch.bfloat16, device="cuda")])
    z.zero_tensors_state8_read(z.TensorList(m=[m], v=[v], exps=[exps]), out)
    got = out.tensors["m"][0]
    assert int((got != 0).sum()) == 5 * 256 + 1
    for k, i in enumerate(near):
        g = grad[i].item()
        assert bool(((got[i:i + 256].float() - 0.1 * g).abs() <= 0.125 * 0.1 * g).all())
    del grad, master, m, v, exps, out, got
    torch.cuda.empty_cache()


def test_lists_refuse_what_the_kernels_cannot_take():
    x = torch.zeros(64, device="cuda")
    u = torch.zeros(64, dtype=torch.uint8, device="cuda")
    square = torch.zeros(8, 8, device="cuda")
    for kw, match in ((dict(grad=[x[::2]]), "contiguous"), (dict(grad=[square.t()], master=[square]), "order"),
                      (dict(grad=[square], master=[square.t()]), "order"), (dict(grad=[x.double()]), "type"),
                      (dict(master=[x.half()]), "type"), (dict(grad=[x], master=[x[:63]]), "elements"),
                      (dict(m=[u], v=[x]), "differ"), (dict(m=[x]), "together"),
                      (dict(m=[u], v=[u], exps=[u]), "elements"), (dict(grad=[x], lr_scale=[1.0, 2.0]), "one per tensor"),
                      (dict(grad=[x], params=[x]), "type"), (dict(grad=[x.cpu()], master=[x]), "CUDA")):
        with pytest.raises(ValueError, match=match):
            z.TensorList(**kw)
    lst = z.TensorList(grad=[x], master=[x], m=[x], v=[x])
    with pytest.raises(z.ZeroError) as e:
        z.zero_tensors_adamw8(lst, z.hparams(), 0, x)
    assert e.value.status == z.ZERO_EINVAL
    with pytest.raises(ValueError, match="lists of"):
        z.zero_tensors_state8_read(lst, z.TensorList(m=[x, x], v=[x, x]))
    with pytest.raises(ValueError, match="elements"):
        lst.set_grad([x[:3]])
    moved = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    lst.set_grad([moved])
    assert lst.array[0].grad == moved.data_ptr() and lst.array[0].grad_dtype == z.ZERO_BF16
