"""The training example end to end: the loss falls with either form of the states, the run
that changes over to 8 bits stays with the 32-bit one, and its parameters are the masters'
bf16 roundings."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_tensors.py")


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("train_tensors", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_training_with_either_states(example):
    steps, tail = 200, 20
    runs = {bits: example.train(steps, bits) for bits in (32, 8)}
    # the same arithmetic until the change-over (but for what autograd's own sums may vary)
    assert runs[8][0][:steps // 2] == pytest.approx(runs[32][0][:steps // 2], rel=0.05)
    mean = {b: sum(r[0][-tail:]) / tail for b, r in runs.items()}
    for b, (losses, opt) in runs.items():
        assert mean[b] < 0.25 * losses[0], (b, losses[0], mean[b])
        for p, master in zip(opt.params, opt.master):
            assert torch.equal(p.detach().view(-1), master.bfloat16())
        ck = opt.checkpoint()
        assert all(torch.isfinite(t).all() for k in ("master", "m", "v") for t in ck[k])
    assert mean[8] < 1.2 * mean[32], mean
    assert runs[8][1].bits == 8 and runs[32][1].bits == 32
