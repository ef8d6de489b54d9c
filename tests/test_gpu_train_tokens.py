"""The example's token model as programs use it around its backward pass: micro-batches,
gradients let go between steps."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_tensors.py")
VOCAB, DIM = 503, 64


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("train_tensors", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def backward(example, model, opt, step):
    tokens, targets = example.sequence(step, VOCAB)
    (model(tokens, targets, opt.st).sum() / (targets >= 0).sum()).backward()


def gradients(model):
    return {name: p.grad.double().clone() for name, p in model.named_parameters()}


def test_micro_batches_add_up(example):
    model, opt = example.token_model(VOCAB, DIM)
    alone = []
    for k in (1, 2):
        for p in opt.params:
            p.grad.zero_()
        backward(example, model, opt, k)
        alone.append(gradients(model))
    for p in opt.params:
        p.grad.zero_()
    for k in (1, 2):
        backward(example, model, opt, k)
    # bf16 sums: the table's is rounded with each of the two ends' gradients of both batches, 4 times,
    # and each part 2 times when alone; half a step (2^-8) each, of no more than both batches' norms
    for name, got in gradients(model).items():
        a, b = alone[0][name], alone[1][name]
        assert float((got - a - b).norm()) <= 6 * 2.0 ** -8 * float(a.norm() + b.norm()), name


def test_gradients_that_were_let_go_come_back(example):
    model, opt = example.token_model(VOCAB, DIM)
    backward(example, model, opt, 1)
    want = gradients(model)
    model.zero_grad(set_to_none=True)
    backward(example, model, opt, 1)
    got = gradients(model)
    assert set(got) == set(want)
    for name in want:                   # the sums that torch makes may vary in their last bits
        assert float((got[name] - want[name]).norm()) <= 2.0 ** -8 * float(want[name].norm()), name
    opt.list.set_grad(opt.grads())
    before = [x.clone() for x in opt.master]
    opt.step()
    assert all(not torch.equal(a, b) for a, b in zip(before, opt.master))
