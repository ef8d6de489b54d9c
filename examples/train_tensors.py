"""Trains a small bf16 model with the list-of-tensors step: gradients where autograd leaves
them, fp32 master weights, per-tensor weight decay, optimizer states of 32 or of 8 bits.

  python examples/train_tensors.py [--task network|tokens] [--steps 300] [--states 32|8|both]

The task is regression onto a fixed random network, or (tokens) the next token of a sequence: a
model with a tied embedding, whose embedding, layer norms and loss are this library's, with their
gradients written where the list reads them and the loss at the step state's scale.  With 8-bit
states the run changes over
from 32 bits half way (zero_tensors_state8_write), and at the end its states are read out as
a checkpoint would hold them (zero_tensors_state8_read).  Needs a GB300 and the built library
(python -c "import __graft_entry__ as g; g.build()").
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_partitioned_optimizer_shard_gb300 as z  # noqa: E402


def network(width: int, seed: int) -> torch.nn.Module:
    torch.manual_seed(seed)
    return torch.nn.Sequential(torch.nn.Linear(64, width), torch.nn.GELU(), torch.nn.LayerNorm(width),
                               torch.nn.Linear(width, width), torch.nn.GELU(), torch.nn.Linear(width, 16))


class Optimizer:
    """The lists, the step state and the workspace that a training program keeps."""

    def __init__(self, params: list, hp, weight_decay: float, seed: int = 1, loss_scale: float = 1.0):
        self.params, self.hp, self.seed = params, hp, seed
        dev = params[0].device
        self.master = [p.detach().float().clone().view(-1) for p in params]
        self.m = [torch.zeros_like(x) for x in self.master]
        self.v = [torch.zeros_like(x) for x in self.master]
        # matrices decay, biases and norms do not
        self.common = dict(master=self.master, params=[p.detach().view(-1) for p in params],
                           weight_decay=[weight_decay if p.dim() > 1 else 0.0 for p in params])
        self.list = z.TensorList(grad=self.grads(), m=self.m, v=self.v, **self.common)
        self.bits = 32
        self.st = torch.empty(z.STATE_BYTES, dtype=torch.uint8, device=dev)
        self.work = torch.empty(z.zero_tensors_workspace_bytes(len(params)), dtype=torch.uint8, device=dev)
        z.zero_tensors_state_init(1, loss_scale, loss_scale != 1.0, 1000, self.st)

    def grads(self) -> list:
        return [p.grad.view(-1) for p in self.params]

    def to_8_bits(self) -> None:
        """The states so far into the 8-bit form; the 32-bit ones are let go."""
        codes = lambda: [torch.zeros(x.numel(), dtype=torch.uint8, device=x.device) for x in self.master]  # noqa: E731
        exps = [torch.zeros(2 * -(-x.numel() // z.ZERO_STATE8_BLOCK), dtype=torch.uint8, device=x.device)
                for x in self.master]
        old, self.list = self.list, z.TensorList(grad=self.grads(), m=codes(), v=codes(), exps=exps, **self.common)
        z.zero_tensors_state8_write(self.list, old)
        self.m = self.v = None
        self.bits = 8

    def step(self) -> None:
        z.zero_tensors_grad_norm(self.list, self.hp, self.work, self.st)
        if self.bits == 8:
            z.zero_tensors_adamw8(self.list, self.hp, self.seed, self.st)
        else:
            z.zero_tensors_adamw(self.list, self.hp, self.st)

    def checkpoint(self) -> dict:
        """master, m and v in fp32, whatever form the states have."""
        if self.bits == 8:
            values = z.TensorList(m=[torch.empty_like(x) for x in self.master],
                                  v=[torch.empty_like(x) for x in self.master])
            z.zero_tensors_state8_read(self.list, values)
            m, v = values.tensors["m"], values.tensors["v"]
        else:
            m, v = self.m, self.v
        return {"master": self.master, "m": m, "v": v, "state": bytes(z.zero_step_state_read(self.st))}


def train(steps: int, bits: int, width: int = 512, batch: int = 256, log=None) -> tuple[list, Optimizer]:
    dev = torch.device("cuda")
    teacher, model = network(width, 1).to(dev), network(width, 2).to(dev, torch.bfloat16)
    params = list(model.parameters())
    for p in params:
        p.grad = torch.zeros_like(p)       # autograd accumulates here: the addresses stay
    opt = Optimizer(params, z.hparams(lr=1e-3, max_grad_norm=1.0), weight_decay=0.01)
    gen = torch.Generator(device=dev).manual_seed(3)
    losses = []
    for k in range(steps):
        if bits == 8 and k == steps // 2:
            opt.to_8_bits()
        x = torch.randn(batch, 64, device=dev, generator=gen)
        with torch.no_grad():
            y = teacher(x)
        loss = torch.nn.functional.mse_loss(model(x.bfloat16()).float(), y)
        loss.backward()
        opt.step()                         # writes the bf16 parameters in place
        for p in params:
            p.grad.zero_()
        losses.append(loss.detach())
        if log and (k + 1) % log == 0:
            s = z.zero_step_state_read(opt.st)
            print(f"step {k + 1:5d}  loss {loss.item():.5f}  gradient norm {s.norm:.4f}  states of {opt.bits} bits")
    return [float(x) for x in losses], opt


def space(bytes_: int, like: torch.Tensor) -> torch.Tensor:
    return torch.empty(bytes_, dtype=torch.uint8, device=like.device)


def gradient(table: torch.Tensor) -> torch.Tensor:
    """table.grad, zeros where there is none yet (zero_grad lets gradients go; the list then takes the
    new ones by set_grad)."""
    if table.grad is None:
        table.grad = torch.zeros_like(table)
    return table.grad


class Embed(torch.autograd.Function):
    """Rows of the table; their gradient is added to table.grad, where the head's went."""

    @staticmethod
    def forward(ctx, table, tokens, scale):
        out = torch.empty(*tokens.shape, table.shape[1], dtype=table.dtype, device=table.device)
        z.zero_embedding(tokens, table, out, scale=scale)
        ctx.save_for_backward(tokens)
        ctx.table, ctx.scale = table, scale
        return out

    @staticmethod
    def backward(ctx, dout):
        (tokens,), (vocab, dim) = ctx.saved_tensors, ctx.table.shape
        work = space(z.zero_embedding_workspace_bytes(tokens.numel(), dim, vocab), dout)
        z.zero_embedding_backward(tokens, dout.contiguous(), gradient(ctx.table), work, scale=ctx.scale, accumulate=True)
        return None, None, None


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        y, rows = torch.empty_like(x), x.numel() // x.shape[-1]
        mean, rstd = torch.empty(2, rows, device=x.device).unbind()
        z.zero_layernorm(x, weight, bias, y, mean, rstd)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        dx, dweight, dbias = torch.empty_like(x), torch.empty_like(weight), torch.empty_like(weight)
        work = space(z.zero_layernorm_workspace_bytes(mean.numel(), x.shape[-1]), x)
        z.zero_layernorm_backward(x, weight, mean, rstd, dy.contiguous(), dx, dweight, dbias, work)
        return dx, dweight, dbias


class HeadLoss(torch.autograd.Function):
    """Each token's cross entropy against the table's rows, without the logits.  The backward pass
    multiplies by the step state's loss scale and adds to table.grad (zeros before the first
    micro-batch of a step)."""

    @staticmethod
    def forward(ctx, hidden, table, targets, st):
        loss, lse = torch.empty(2, targets.numel(), device=hidden.device).unbind()
        work = space(z.zero_head_workspace_bytes(targets.numel(), *reversed(table.shape)), hidden)
        z.zero_head_loss(hidden, table, targets, loss, lse, work)
        ctx.save_for_backward(hidden, targets, lse, work)
        ctx.table, ctx.st = table, st
        return loss

    @staticmethod
    def backward(ctx, dloss):
        hidden, targets, lse, work = ctx.saved_tensors
        dhidden = torch.empty_like(hidden)
        z.zero_head_loss_backward(hidden, ctx.table, targets, lse, dhidden, gradient(ctx.table), work,
                                  row_scale=dloss.contiguous(), st=ctx.st, accumulate=True)
        return dhidden, None, None, None


class TokenModel(torch.nn.Module):
    def __init__(self, vocab: int, dim: int, seed: int):
        super().__init__()
        torch.manual_seed(seed)
        self.table = torch.nn.Parameter(torch.randn(vocab, dim) * dim ** -0.5)
        self.norms = torch.nn.ModuleList([torch.nn.LayerNorm(dim) for _ in range(2)])
        self.up, self.down = torch.nn.Linear(dim, 4 * dim), torch.nn.Linear(4 * dim, dim)

    def forward(self, tokens, targets, st):
        scale = self.table.shape[1] ** 0.5
        x = Embed.apply(self.table, tokens, scale)
        a, b = self.norms
        x = x + self.down(torch.nn.functional.gelu(self.up(Norm.apply(x, a.weight, a.bias))))
        return HeadLoss.apply(Norm.apply(x, b.weight, b.bias), self.table, targets, st)


def token_model(vocab: int, dim: int, loss_scale: float = 1.0) -> tuple[TokenModel, Optimizer]:
    model = TokenModel(vocab, dim, 5).to("cuda", torch.bfloat16)
    params = list(model.parameters())
    for p in params:
        p.grad = torch.zeros_like(p)
    return model, Optimizer(params, z.hparams(lr=2e-3, max_grad_norm=1.0), weight_decay=0.01, loss_scale=loss_scale)


def sequence(step: int, vocab: int, rows: int = 8, length: int = 128) -> tuple:
    """Tokens that each follow from the one before, and their targets; the last has none."""
    gen = torch.Generator(device="cuda").manual_seed(step)
    t = torch.randint(0, vocab, (rows, 1), device="cuda", generator=gen)
    tokens = (t + 7 * torch.arange(length, device="cuda")) % vocab
    targets = torch.full_like(tokens, -100)
    targets[:, :-1] = tokens[:, 1:]
    return tokens, targets


def train_tokens(steps: int, bits: int, vocab: int = 5003, dim: int = 256, log=None) -> tuple[list, Optimizer]:
    model, opt = token_model(vocab, dim)
    losses = []
    for k in range(steps):
        if bits == 8 and k == steps // 2:
            opt.to_8_bits()
        tokens, targets = sequence(k, vocab)
        loss = model(tokens, targets, opt.st).sum() / (targets >= 0).sum()
        loss.backward()
        opt.step()
        for p in opt.params:
            p.grad.zero_()
        losses.append(loss.detach())
        if log and (k + 1) % log == 0:
            s = z.zero_step_state_read(opt.st)
            print(f"step {k + 1:5d}  loss {loss.item():.5f}  gradient norm {s.norm:.4f}  states of {opt.bits} bits")
    return [float(x) for x in losses], opt


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--task", choices=["network", "tokens"], default="network")
    ap.add_argument("--steps", type=int, default=300)
    ap.add_argument("--states", choices=["32", "8", "both"], default="both")
    a = ap.parse_args()
    for bits in ([32, 8] if a.states == "both" else [int(a.states)]):
        losses, opt = (train_tokens if a.task == "tokens" else train)(a.steps, bits, log=max(1, a.steps // 6))
        ck = opt.checkpoint()
        held = sum(t.numel() * t.element_size() for k in ("m", "v", "exps") for t in opt.list.tensors.get(k, []))
        n = sum(t.numel() for t in ck["m"])
        print(f"{bits}-bit run: mean loss of the last tenth {sum(losses[-a.steps // 10:]) / max(1, len(losses[-a.steps // 10:])):.5f}, "
              f"m and v hold {held / n:.2f} bytes per parameter")


if __name__ == "__main__":
    main()
