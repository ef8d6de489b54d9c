"""Layer norm, embedding and the head's cross entropy without a GPU: workspaces and the refusals
of the C entry points (every call here is invalid or empty, so nothing reaches the device)."""
import ctypes as C

import pytest
import torch

import zero_partitioned_optimizer_shard_gb300 as z
from zero_partitioned_optimizer_shard_gb300 import _build

BF16, F16, F32, U8 = z.ZERO_BF16, z.ZERO_F16, z.ZERO_F32, z.ZERO_U8
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return z.lib()


def addr(k):
    """Aligned fake addresses, 1 GB apart; never dereferenced."""
    return (k + 1) << 30


CALLS = {
    "zero_layernorm": dict(dtype=BF16, rows=100, dim=64, x=addr(0), x_stride=64, weight=addr(1), bias=addr(2),
                           param_dtype=BF16, eps=1e-5, y=addr(3), y_stride=64, mean=addr(4), rstd=addr(5), stream=None),
    "zero_layernorm_backward": dict(dtype=BF16, rows=100, dim=64, x=addr(0), x_stride=64, weight=addr(1),
                                    param_dtype=BF16, mean=addr(2), rstd=addr(3), dy=addr(4), dy_stride=64, dx=addr(5),
                                    dx_stride=64, dweight=addr(6), dbias=addr(7), grad_dtype=F32, accumulate=0,
                                    workspace=addr(8), stream=None),
    "zero_embedding": dict(dtype=BF16, n_tokens=100, dim=64, vocab=1000, tokens=addr(0), token_bytes=8, table=addr(1),
                           scale=1.0, out=addr(2), out_stride=64, stream=None),
    "zero_embedding_backward": dict(dtype=BF16, n_tokens=100, dim=64, vocab=1000, tokens=addr(0), token_bytes=8,
                                    dout=addr(1), dout_stride=64, scale=1.0, dtable=addr(2), grad_dtype=F32,
                                    accumulate=0, workspace=addr(3), stream=None),
    "zero_head_loss": dict(dtype=BF16, rows=100, dim=64, vocab=1000, hidden=addr(0), hidden_stride=64, weight=addr(1),
                           targets=addr(2), target_bytes=8, loss=addr(3), lse=addr(4), workspace=addr(5), stream=None),
    "zero_head_loss_backward": dict(dtype=BF16, rows=100, dim=64, vocab=1000, hidden=addr(0), hidden_stride=64,
                                    weight=addr(1), targets=addr(2), target_bytes=8, lse=addr(3), scale=1.0,
                                    row_scale=addr(4), st=addr(5), dhidden=addr(6), dhidden_stride=64, dweight=addr(7),
                                    grad_dtype=F32, accumulate=0, workspace=addr(8), stream=None),
}

INVALID = {
    "zero_layernorm": [dict(dtype=U8), dict(dtype=0), dict(param_dtype=F16), dict(param_dtype=0), dict(rows=(1 << 30) + 1),
                       dict(dim=0), dict(dim=16385), dict(x=None), dict(weight=None), dict(y=None), dict(x_stride=63),
                       dict(y_stride=0), dict(x_stride=1 << 33), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF),
                       dict(y=addr(0)), dict(y=addr(0) + 100 * 128 - 16), dict(y=addr(1)), dict(y=addr(2) + 16),
                       dict(mean=addr(3) + 32), dict(rstd=addr(4))],
    "zero_layernorm_backward": [dict(dtype=9), dict(param_dtype=F16), dict(grad_dtype=F16), dict(grad_dtype=U8),
                                dict(accumulate=2), dict(workspace=None), dict(mean=None), dict(rstd=None), dict(dy=None),
                                dict(dx=None), dict(x=None), dict(weight=None), dict(dy_stride=1), dict(dx_stride=63),
                                dict(dim=0), dict(dim=20000), dict(dx=addr(4)), dict(dx=addr(0)), dict(dweight=addr(7)),
                                dict(dweight=addr(1)), dict(workspace=addr(5)), dict(workspace=addr(4) + 64),
                                dict(dbias=addr(8) + 16)],
    "zero_embedding": [dict(dtype=U8), dict(dim=0), dict(dim=65537), dict(vocab=0), dict(vocab=(1 << 30) + 1),
                       dict(n_tokens=(1 << 28) + 1), dict(token_bytes=2), dict(token_bytes=0), dict(tokens=None),
                       dict(table=None), dict(out=None), dict(out_stride=63), dict(scale=NAN), dict(scale=INF),
                       dict(out=addr(1) + 64), dict(out=addr(0))],
    "zero_embedding_backward": [dict(dtype=0), dict(grad_dtype=F16), dict(grad_dtype=U8), dict(dim=0), dict(vocab=0),
                                dict(token_bytes=3), dict(tokens=None), dict(dout=None), dict(dtable=None),
                                dict(workspace=None), dict(dout_stride=60), dict(scale=NAN), dict(accumulate=7),
                                dict(dtable=addr(1)), dict(dtable=addr(0) + 16), dict(workspace=addr(2) + 1024),
                                dict(workspace=addr(1)), dict(workspace=addr(0))],
    "zero_head_loss": [dict(dtype=F32), dict(dtype=U8), dict(rows=(1 << 24) + 1), dict(dim=0), dict(dim=65537),
                       dict(vocab=0), dict(vocab=(1 << 24) + 1), dict(hidden=None), dict(weight=None), dict(targets=None),
                       dict(target_bytes=1), dict(loss=None), dict(lse=None), dict(workspace=None), dict(hidden_stride=63),
                       dict(loss=addr(4)), dict(loss=addr(0) + 16), dict(lse=addr(1)), dict(lse=addr(2)),
                       dict(lse=addr(5) + 256), dict(workspace=addr(0)), dict(workspace=addr(1) + 256)],
    "zero_head_loss_backward": [dict(dtype=F32), dict(grad_dtype=F16), dict(grad_dtype=U8), dict(hidden=None),
                                dict(weight=None), dict(targets=None), dict(lse=None), dict(workspace=None),
                                dict(dhidden=None, dweight=None), dict(dhidden_stride=1), dict(scale=NAN), dict(scale=INF),
                                dict(accumulate=2), dict(target_bytes=5), dict(dhidden=addr(0)), dict(dhidden=addr(1)),
                                dict(dweight=addr(1)), dict(dweight=addr(6)), dict(dweight=addr(8) + 256),
                                dict(workspace=addr(3)), dict(workspace=addr(5)), dict(dhidden=addr(5))],
}

MISALIGNED = {
    "zero_layernorm": [dict(x=addr(0) + 1), dict(y=addr(3) + 1), dict(weight=addr(1) + 1), dict(bias=addr(2) + 1),
                       dict(mean=addr(4) + 2), dict(rstd=addr(5) + 1), dict(dtype=F32, param_dtype=F32, x=addr(0) + 2)],
    "zero_layernorm_backward": [dict(x=addr(0) + 1), dict(dy=addr(4) + 1), dict(dx=addr(5) + 1), dict(dweight=addr(6) + 2),
                                dict(dbias=addr(7) + 2), dict(mean=addr(2) + 2), dict(workspace=addr(8) + 8)],
    "zero_embedding": [dict(tokens=addr(0) + 4), dict(table=addr(1) + 1), dict(out=addr(2) + 1)],
    "zero_embedding_backward": [dict(tokens=addr(0) + 4), dict(dout=addr(1) + 1), dict(dtable=addr(2) + 2),
                                dict(workspace=addr(3) + 8)],
    "zero_head_loss": [dict(hidden=addr(0) + 1), dict(weight=addr(1) + 8), dict(targets=addr(2) + 4), dict(loss=addr(3) + 2),
                       dict(lse=addr(4) + 1), dict(workspace=addr(5) + 128)],
    "zero_head_loss_backward": [dict(hidden=addr(0) + 1), dict(weight=addr(1) + 2), dict(targets=addr(2) + 4),
                                dict(lse=addr(3) + 2), dict(row_scale=addr(4) + 2), dict(st=addr(5) + 8),
                                dict(dhidden=addr(6) + 1), dict(dweight=addr(7) + 2), dict(workspace=addr(8) + 16)],
}


def call(lib, name, change):
    a = {**CALLS[name], **change}
    return getattr(lib, name)(*a.values())


@pytest.mark.parametrize("name", list(CALLS))
def test_refusals(lib, name):
    for change in INVALID[name]:
        assert call(lib, name, change) == z.ZERO_EINVAL, change
    for change in MISALIGNED[name]:
        assert call(lib, name, change) == z.ZERO_EALIGN, change


def test_columns_of_one_buffer_that_overlap(lib):
    """Rows of 64 in buffers of 256 a row: y one element into x's columns, from either side, at any
    row, is refused (that y beside them is taken, the GPU tests show)."""
    for y in (addr(0) + 126, addr(0) - 126, addr(0) + 7 * 512 + 2, addr(0) + 8 * 512 - 126, addr(0) + 99 * 512):
        assert call(z.lib(), "zero_layernorm", dict(x_stride=256, y_stride=256, y=y)) == z.ZERO_EINVAL, y - addr(0)


def test_calls_without_rows_do_nothing(lib):
    nothing = dict(x=None, y=None, weight=None)
    assert call(lib, "zero_layernorm", dict(rows=0, **nothing)) == z.ZERO_OK
    assert call(lib, "zero_layernorm_backward", dict(rows=0, dweight=None, dbias=None)) == z.ZERO_OK
    assert call(lib, "zero_embedding", dict(n_tokens=0, tokens=None, out=None)) == z.ZERO_OK
    assert call(lib, "zero_embedding_backward", dict(n_tokens=0, tokens=None, dout=None, accumulate=1)) == z.ZERO_OK
    assert call(lib, "zero_head_loss", dict(rows=0, hidden=None, targets=None, loss=None, lse=None)) == z.ZERO_OK
    assert call(lib, "zero_head_loss_backward", dict(rows=0, hidden=None, targets=None, lse=None, accumulate=1)) == z.ZERO_OK


def test_workspaces():
    assert z.zero_layernorm_workspace_bytes(1, 0) == z.zero_layernorm_workspace_bytes(1, 16385) == 0
    assert z.zero_layernorm_workspace_bytes(0, 8) > 0
    assert z.zero_embedding_workspace_bytes(0, 8, 5) > 0 and z.zero_embedding_workspace_bytes(5, 8, 0) == 0
    assert z.zero_head_workspace_bytes(0, 8, 5) > 0 and z.zero_head_workspace_bytes(5, 8, 0) == 0
    sizes = [z.zero_head_workspace_bytes(n, 1600, 50257) for n in (1, 128, 1024, 8192, 65536)]
    assert sizes == sorted(sizes)
    # far below the logits of 65,536 tokens (13 GB in fp32): D's piece and the sums
    assert sizes[-1] < 65536 * 50257 * 4 / 5


def test_python_refuses_what_is_not_on_the_gpu():
    refused = (ValueError, RuntimeError)  # without a GPU it is torch that refuses
    x, w = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(refused):
        z.zero_layernorm(x, w, None, x.clone())
    with pytest.raises(refused):
        z.zero_embedding(torch.zeros(4, dtype=torch.int64), torch.zeros(5, 8), x)
    with pytest.raises(refused):
        z.zero_head_loss(x.bfloat16(), torch.zeros(5, 8).bfloat16(), torch.zeros(4, dtype=torch.int64), w[:4], w[:4], w)


def test_ctypes_signatures_match_the_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "zero.h"),
                encoding="utf-8").read()
    kinds = {"uint64_t": C.c_uint64, "uint32_t": C.c_uint32, "float": C.c_float, "zero_dtype_t": C.c_int}
    for name, given in CALLS.items():
        body = re.search(rf"int {name}\((.*?)\);", text, re.S).group(1)
        params = [p.split() for p in body.replace("\n", " ").split(",")]
        want = [C.c_void_p if "*" in " ".join(p) or p[0] == "zero_stream_t" else kinds[p[0]] for p in params]
        assert getattr(z.lib(), name).argtypes == want, name
        assert [p[-1].lstrip("*") for p in params] == list(given), name
