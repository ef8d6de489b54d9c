"""The list-of-tensors entry points without a GPU: struct layout, workspace, host-side
refusals (every call here is invalid or empty, so nothing reaches the device), and the 8-bit
form's definition on the host: unbiased rounding, round trips, the generator's quality."""
import ctypes as C
import os
import re

import numpy as np
import pytest
import torch

import zero_partitioned_optimizer_shard_gb300 as z
from tests import state8_oracle as S
from zero_partitioned_optimizer_shard_gb300 import _build

A = 0x100000  # an aligned fake address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return z.lib()


def _tensor(**kw):
    t = dict(elems=1000, grad=A, master=A, m=A, v=A, exps=A, params=A, grad_dtype=z.ZERO_BF16,
             state_dtype=z.ZERO_F32, lr_scale=1.0, weight_decay=0.01)
    t.update(kw)
    a = (z.Tensor * 1)()
    for k, x in t.items():
        setattr(a[0], k, x)
    return a


def _call(lib, op, tensors, n=1, hp=None, st=A, work=A, other=None):
    hp = C.byref(hp) if hp is not None else C.byref(z.hparams())
    if op == "norm":
        return lib.zero_tensors_grad_norm(tensors, n, hp, work, st, None)
    if op == "adamw":
        return lib.zero_tensors_adamw(tensors, n, hp, st, None)
    if op == "adamw8":
        return lib.zero_tensors_adamw8(tensors, n, hp, 0, st, None)
    f = lib.zero_tensors_state8_read if op == "read" else lib.zero_tensors_state8_write
    return f(tensors, other if other is not None else _tensor(), n, None)


NEEDS = {"norm": ("grad",), "adamw": ("grad", "master", "m", "v"),
         "adamw8": ("grad", "master", "m", "v", "exps"), "read": ("m", "v", "exps"),
         "write": ("m", "v", "exps")}
STATE = {"norm": z.ZERO_F32, "adamw": z.ZERO_F32, "adamw8": z.ZERO_U8, "read": z.ZERO_U8, "write": z.ZERO_U8}


@pytest.mark.parametrize("op", list(NEEDS))
def test_null_pointers_are_refused(lib, op):
    for name in NEEDS[op]:
        assert _call(lib, op, _tensor(state_dtype=STATE[op], **{name: None})) == z.ZERO_EINVAL, name
    assert _call(lib, op, None) == z.ZERO_EINVAL
    if op in ("norm", "adamw", "adamw8"):
        assert _call(lib, op, _tensor(state_dtype=STATE[op]), st=None) == z.ZERO_EINVAL
        assert _call(lib, op, _tensor(state_dtype=STATE[op]), st=A + 4) == z.ZERO_EALIGN
    if op == "norm":
        assert _call(lib, op, _tensor(), work=None) == z.ZERO_EINVAL
        assert _call(lib, op, _tensor(), work=A + 8) == z.ZERO_EALIGN


@pytest.mark.parametrize("op,name,value,status", [
    ("norm", "grad", A + 1, z.ZERO_EALIGN), ("adamw", "grad", A + 1, z.ZERO_EALIGN),
    ("adamw", "master", A + 2, z.ZERO_EALIGN), ("adamw", "m", A + 2, z.ZERO_EALIGN),
    ("adamw", "v", A + 1, z.ZERO_EALIGN), ("adamw", "params", A + 1, z.ZERO_EALIGN),
    ("adamw8", "master", A + 2, z.ZERO_EALIGN), ("adamw8", "params", A + 1, z.ZERO_EALIGN),
    ("norm", "grad_dtype", 0, z.ZERO_EINVAL), ("norm", "grad_dtype", z.ZERO_U8, z.ZERO_EINVAL),
    ("adamw", "grad_dtype", 7, z.ZERO_EINVAL), ("adamw", "state_dtype", z.ZERO_U8, z.ZERO_EINVAL),
    ("adamw", "state_dtype", z.ZERO_BF16, z.ZERO_EINVAL), ("adamw8", "state_dtype", z.ZERO_F32, z.ZERO_EINVAL),
    ("read", "state_dtype", z.ZERO_F32, z.ZERO_EINVAL), ("write", "state_dtype", 0, z.ZERO_EINVAL),
    ("adamw", "params_dtype", z.ZERO_F32, z.ZERO_EINVAL), ("adamw8", "params_dtype", 9, z.ZERO_EINVAL),
    ("adamw", "lr_scale", -1.0, z.ZERO_EINVAL), ("adamw", "lr_scale", float("nan"), z.ZERO_EINVAL),
    ("adamw8", "lr_scale", float("inf"), z.ZERO_EINVAL), ("adamw", "weight_decay", float("nan"), z.ZERO_EINVAL),
    ("norm", "elems", 1 << 60, z.ZERO_EINVAL), ("adamw8", "elems", (1 << 42) + 1, z.ZERO_EINVAL),
])
def test_bad_fields_are_refused(lib, op, name, value, status):
    fields = {"state_dtype": STATE[op], name: value}
    assert _call(lib, op, _tensor(**fields)) == status


def test_fp32_gradients_need_four_byte_alignment(lib):
    assert _call(lib, "norm", _tensor(grad_dtype=z.ZERO_F32, grad=A + 2)) == z.ZERO_EALIGN


@pytest.mark.parametrize("field,value", [("beta1", 1.0), ("beta2", -0.1), ("eps", 0.0), ("lr", float("nan")),
                                         ("params_dtype", z.ZERO_F32)])
def test_bad_hyperparameters_are_refused(lib, field, value):
    hp = z.hparams()
    setattr(hp, field, value)
    for op in ("norm", "adamw", "adamw8"):
        assert _call(lib, op, _tensor(state_dtype=STATE[op]), hp=hp) == z.ZERO_EINVAL


@pytest.mark.parametrize("op,fields,status", [
    ("read", dict(elems=999), z.ZERO_EINVAL), ("read", dict(m=None), z.ZERO_EINVAL),
    ("read", dict(state_dtype=z.ZERO_U8), z.ZERO_EINVAL), ("read", dict(state_dtype=z.ZERO_F16), z.ZERO_EINVAL),
    ("read", dict(m=A + 2), z.ZERO_EALIGN), ("read", dict(state_dtype=z.ZERO_BF16, v=A + 1), z.ZERO_EALIGN),
    ("write", dict(state_dtype=z.ZERO_BF16), z.ZERO_EINVAL), ("write", dict(v=A + 1), z.ZERO_EALIGN),
    ("write", dict(elems=0), z.ZERO_EINVAL),
])
def test_codec_partner_is_checked(lib, op, fields, status):
    assert _call(lib, op, _tensor(state_dtype=z.ZERO_U8), other=_tensor(**fields)) == status


def test_empty_lists_and_counts(lib):
    for op in ("adamw", "adamw8", "read", "write"):   # nothing to do: no launch
        assert _call(lib, op, None, n=0) == z.ZERO_OK
        assert _call(lib, op, _tensor(elems=0, state_dtype=99), n=1, other=_tensor(elems=0)) == z.ZERO_OK
        assert _call(lib, op, _tensor(state_dtype=STATE[op]), n=1 << 40) == z.ZERO_EINVAL


def test_state_init_refusals(lib):
    f = lib.zero_tensors_state_init
    assert f(0, 1.0, 0, 0, A, None) == z.ZERO_EINVAL
    assert f(1, 0.0, 0, 0, A, None) == z.ZERO_EINVAL
    assert f(1, float("inf"), 0, 0, A, None) == z.ZERO_EINVAL
    assert f(1, 1.0, 0, 0, None, None) == z.ZERO_EINVAL
    assert f(1, 1.0, 0, 0, A + 8, None) == z.ZERO_EALIGN


def test_struct_and_workspace(lib):
    assert C.sizeof(z.Tensor) == 80
    sizes = [z.zero_tensors_workspace_bytes(n) for n in (0, 1, 384, 385, 10_000)]
    assert sizes == sorted(sizes) and sizes[0] > 0 and all(s % 16 == 0 for s in sizes)


def test_tensor_list_refusals():
    f = torch.zeros(8)
    with pytest.raises(ValueError, match="at least one"):
        z.TensorList()
    with pytest.raises(ValueError, match="CUDA"):
        z.TensorList(grad=[f])
    with pytest.raises(ValueError, match="the list 1"):
        z.TensorList(master=[f], grad=[f, f])
    assert len(z.TensorList(grad=[])) == 0


def test_loads_of_the_list_kernels_stay_behind_their_waits():
    """The kernels over lists know their first addresses before they wait for the launch
    before them.  A load that the compiler may move (an asm that is not volatile, an intrinsic
    that may be one) or that the hardware may take through the read-only path is not theirs:
    it could read what that launch has yet to write."""
    names = ("tensors.cuh", "tensors_norm.cu", "tensors_adamw.cu", "tensors_codec.cu")
    for name in names:
        with open(os.path.join(_build.CSRC, name)) as f:
            code = re.sub(r"/\*.*?\*/|//[^\n]*", "", f.read(), flags=re.S)
        assert not re.findall(r"\b(?:ld_stream_\w+|__ld\w+)\s*\(", code), name
        loads = re.findall(r"\basm\b(\s+volatile)?\s*\(\s*\"[^\"]*\bld\.global([\w.:]*)", code)
        assert all(volatile and ".nc" not in kind for volatile, kind in loads), (name, loads)
        assert loads or name in ("tensors_adamw.cu", "tensors_codec.cu")


class OnGpu(torch.Tensor):
    """A host tensor that passes for one of device 0: lists are built, nothing is launched."""
    is_cuda = True

    def get_device(self):
        return 0


def on_gpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


def weight(order, dtype=torch.float32):
    """A 4-dimensional weight of 4 x 3 x 5 x 2, contiguous or dense in another order."""
    return on_gpu(4, 5, 2, 3, dtype=dtype).permute(0, 3, 1, 2) if order == "channels last" else on_gpu(4, 3, 5, 2, dtype=dtype)


@pytest.mark.parametrize("order,other", [("contiguous", "channels last"), ("channels last", "contiguous")])
@pytest.mark.parametrize("first_grad", [False, True])
@pytest.mark.parametrize("state", [torch.float32, torch.uint8])
def test_set_grad_refuses_gradients_in_another_order(order, other, first_grad, state):
    """As the constructor does: element i of the gradient is then not element i of the master.
    The list stays as it was, the tensors it keeps alive included."""
    arrays = dict(master=[on_gpu(7), weight(order)], m=[on_gpu(7, dtype=state), weight(order, state)],
                  v=[on_gpu(7, dtype=state), weight(order, state)])
    if state == torch.uint8:
        arrays["exps"] = [on_gpu(2, dtype=state), on_gpu(2, dtype=state)]
    kw = dict(grad=[on_gpu(7), weight(order)]) if first_grad else {}
    with pytest.raises(ValueError, match="differ in order"):
        z.TensorList(grad=[on_gpu(7), weight(other)], **arrays)
    lst = z.TensorList(**arrays, **kw)
    before, kept = bytes(lst.array), lst.tensors.get("grad")
    with pytest.raises(ValueError, match="differ in order"):
        lst.set_grad([on_gpu(7), weight(other)])
    assert bytes(lst.array) == before and lst.tensors.get("grad") is kept
    moved = [on_gpu(7, dtype=torch.bfloat16), weight(order, torch.bfloat16)]
    lst.set_grad(moved)
    assert [a.grad for a in lst.array] == [g.data_ptr() for g in moved]
    assert [a.grad_dtype for a in lst.array] == [z.ZERO_BF16] * 2 and lst.tensors["grad"] == moved


def test_set_grad_keeps_the_old_gradients_whatever_the_new_ones_lack():
    """A gradient that is None (a parameter that took no part) raises; the list still holds the
    tensors that its addresses point to."""
    lst = z.TensorList(grad=[on_gpu(8), on_gpu(9)], master=[on_gpu(8), on_gpu(9)])
    kept, before = lst.tensors["grad"], bytes(lst.array)
    for bad in ([on_gpu(8), None], [on_gpu(8), on_gpu(8)], [on_gpu(8)], [on_gpu(8), on_gpu(9, dtype=torch.float64)]):
        with pytest.raises((ValueError, AttributeError)):
            lst.set_grad(bad)
        assert lst.tensors["grad"] is kept and bytes(lst.array) == before


def test_dimensions_of_one_element_do_not_count_as_an_order():
    """The strides of such dimensions say nothing of where the elements lie."""
    a = on_gpu(4, 1, 5, 2).permute(0, 3, 1, 2)          # 4 x 2 x 1 x 5
    b = torch.as_strided(a, a.shape, (10, 1, 77, 2)).as_subclass(OnGpu)
    assert not a.is_contiguous() and a.stride() != b.stride()
    lst = z.TensorList(grad=[a], master=[b])
    lst.set_grad([b])
    with pytest.raises(ValueError, match="differ in order"):
        lst.set_grad([on_gpu(4, 2, 1, 5)])


@pytest.mark.parametrize("call", ["zero_tensors_state8_read", "zero_tensors_state8_write"])
@pytest.mark.parametrize("order,other", [("contiguous", "channels last"), ("channels last", "contiguous"),
                                         ("channels last", "flat")])
def test_codec_refuses_lists_in_different_orders(monkeypatch, call, order, other):
    """The two lists of a state8 call lie alike, tensor by tensor; nothing reaches the library
    otherwise."""
    calls = []
    monkeypatch.setattr(z, "_lib", lambda: type("L", (), {call: staticmethod(lambda *a: calls.append(a) or 0)}))
    def flat(kind, dtype):
        return on_gpu(120, dtype=dtype) if kind == "flat" else weight(kind, dtype)

    def lists(a, b):
        code = dict(m=[on_gpu(7, dtype=torch.uint8), flat(a, torch.uint8)], exps=[on_gpu(2, dtype=torch.uint8)] * 2)
        return (z.TensorList(v=code["m"], **code), z.TensorList(**{k: [on_gpu(7), flat(b, torch.float32)] for k in "mv"}))

    for a, b in ((order, other), (other, order)):
        with pytest.raises(ValueError, match="differ in order"):
            getattr(z, call)(*lists(a, b), stream=0)
    assert not calls
    getattr(z, call)(*lists(order, order), stream=0)
    assert len(calls) == 1


def test_codec_refuses_lists_of_two_devices(monkeypatch):
    class Second(OnGpu):
        def get_device(self):
            return 1

    calls = []
    monkeypatch.setattr(z, "_lib", lambda: type("L", (), {"zero_tensors_state8_read": staticmethod(lambda *a: calls.append(a) or 0)}))
    code = [on_gpu(7, dtype=torch.uint8)]
    source = z.TensorList(m=code, v=code, exps=[on_gpu(2, dtype=torch.uint8)])
    there = [torch.zeros(7).as_subclass(Second)]
    with pytest.raises(ValueError, match="devices"):
        z.zero_tensors_state8_read(source, z.TensorList(m=there, v=there), stream=0)
    assert not calls


@pytest.mark.parametrize("n", [0, 1, 40, 999, 1000, 2500])
def test_a_workspace_that_is_too_small_is_refused(lib, monkeypatch, n):
    """Before the library is called: the norm's kernels write the workspace without knowing
    its size, which grows with the list."""
    calls = []

    class Library:
        zero_tensors_grad_norm = staticmethod(lambda *a: calls.append(a) or 0)

        def __getattr__(self, name):
            return getattr(lib, name)

    monkeypatch.setattr(z, "_lib", lambda: Library())
    tensors, hp, st = z.TensorList(grad=[on_gpu(3)] * n), z.hparams(), on_gpu(128, dtype=torch.uint8)
    need = z.zero_tensors_workspace_bytes(n)
    for small in (on_gpu(need - 1, dtype=torch.uint8), on_gpu(need // 8 - 1, dtype=torch.float64),
                  on_gpu(0, dtype=torch.uint8)):
        with pytest.raises(z.ZeroError) as e:
            z.zero_tensors_grad_norm(tensors, hp, small, st, stream=0)
        assert e.value.status == z.ZERO_ENOMEM and not calls
    for enough in (on_gpu(need, dtype=torch.uint8), on_gpu(need // 8, dtype=torch.float64), A):
        z.zero_tensors_grad_norm(tensors, hp, enough, st, stream=0)
    assert len(calls) == 3


@pytest.mark.parametrize("call", ["zero_tensors_adamw", "zero_tensors_adamw8"])
def test_a_list_without_a_decay_takes_the_hyperparameters(monkeypatch, call):
    """A list that names no weight decay trains with that of the call's hyperparameters, and
    follows it; a list that names one, zero among them, keeps its own."""
    seen = []
    monkeypatch.setattr(z, "_lib", lambda: type("L", (), {call: staticmethod(
        lambda array, n, *a: seen.append([array[i].weight_decay for i in range(n)]) or 0)}))
    arrays = dict(master=[on_gpu(3), on_gpu(4)])
    plain, zero, own = z.TensorList(**arrays), z.TensorList(weight_decay=0.0, **arrays), z.TensorList(weight_decay=[0.5, 0.0], **arrays)
    args = (7,) if call.endswith("8") else ()
    want = []
    for decay in (0.125, 0.125, 0.25, 0.0):
        for lst, w in ((plain, [decay] * 2), (zero, [0.0] * 2), (own, [0.5, 0.0])):
            getattr(z, call)(lst, z.hparams(weight_decay=decay), *args, A, stream=0)
            want.append(w)
    assert seen == want


# ------------------------------------------------------------------------------------------
# the 8-bit form on the host
# ------------------------------------------------------------------------------------------
def test_every_code_survives_a_round_trip():
    for name, n in (("m", 256), ("v", 256)):
        for b in (27, 64, 127, 200, 253):
            codes = np.arange(n, dtype=np.uint8)
            x = S.decode(codes, np.full(1, b), name)
            again, e = S.encode(x, name, S.NEAREST)
            assert np.array_equal(S.decode(again, e, name), x), (name, b)


def test_codes_stand_for_the_header_formula():
    for c in range(256):
        e, man = (c >> 3) & 15, c & 7
        want = (-1) ** (c >> 7) * ((1 + man / 8) * 2.0 ** (e - 15) if e else man / 8 * 2.0 ** -14)
        assert S.decode(np.array([c] + [0] * 255, np.uint8), np.array([127]), "m")[0] == want
        e = c >> 3
        want = (1 + man / 8) * 2.0 ** (e - 31) if e else man / 8 * 2.0 ** -30
        assert S.decode(np.array([c] + [0] * 255, np.uint8), np.array([127]), "v")[0] == want


def test_stochastic_rounding_is_unbiased():
    """The mean of many roundings of x: its standard error is spacing / sqrt(4 n) at most."""
    n = 1 << 16
    for name, values in (("m", (0.7e-4, -3.3e-9, 1.61e-4)), ("v", (3.7e-9, 1.3e-12, 7.3e-9))):
        for x in values:
            block = np.full((n // 255, 256), np.float32(x))
            block[:, 0] = 2e-4 if name == "m" else 9e-9   # the block's scale
            r = S.random20(block.size // 256, 7, 123, 0, name)
            codes, b = S.encode(block.reshape(-1), name, r)
            got = S.decode(codes, b, name).reshape(block.shape)[:, 1:].astype(np.float64)
            spacing = max(np.ptp(got), abs(x) / 16)
            assert abs(got.mean() - np.float64(np.float32(x))) < 5 * spacing / np.sqrt(4 * got.size), (name, x)


def test_random_bits_spread():
    """5 standard errors of n fair bits or of n independent numbers: every bit is set half the
    time, also against the next step's, the next group's and the next block's; and as
    numbers (what the rounding uses) neighbours and the m and v of one element are
    uncorrelated too.  (Their lowest bits alone are not: a linear congruence's are weak.)"""
    n = 1 << 11
    a, b = (S.random20(n, 3, t, 0, "m").astype(np.int64) for t in (10, 11))
    v = S.random20(n, 3, 10, 0, "v").astype(np.int64)
    tol = 5 * 0.5 / np.sqrt(a.size)
    for k in range(20):
        for other in (np.zeros_like(a), b, np.roll(a, 8), np.roll(a, 256)):
            assert abs(np.mean(((a ^ other) >> k) & 1) - 0.5) < tol, k
    for other in [b, v] + [np.roll(a, lag) for lag in (1, 2, 3, 4, 5, 6, 7, 8, 256)]:
        assert abs(np.corrcoef(a, other)[0, 1]) < 5 / np.sqrt(a.size)
    counts = np.bincount(a >> 12, minlength=256)
    assert np.sum((counts - a.size / 256) ** 2 / (a.size / 256)) < 255 + 5 * np.sqrt(2 * 255)
