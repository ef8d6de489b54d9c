"""Trains a small bf16 model with the list-of-tensors step: gradients where autograd leaves
them, fp32 master weights, per-tensor weight decay, optimizer states of 32 or of 8 bits.

  python examples/train_tensors.py [--steps 300] [--states 32|8|both]

The task is regression onto a fixed random network.  With 8-bit states the run changes over
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

    def __init__(self, params: list, hp, weight_decay: float, seed: int = 1):
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
        z.zero_tensors_state_init(1, 1.0, False, 0, self.st)

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


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=300)
    ap.add_argument("--states", choices=["32", "8", "both"], default="both")
    a = ap.parse_args()
    for bits in ([32, 8] if a.states == "both" else [int(a.states)]):
        losses, opt = train(a.steps, bits, log=max(1, a.steps // 6))
        ck = opt.checkpoint()
        held = sum(t.numel() * t.element_size() for k in ("m", "v", "exps") for t in opt.list.tensors.get(k, []))
        n = sum(t.numel() for t in ck["m"])
        print(f"{bits}-bit run: mean loss of the last tenth {sum(losses[-a.steps // 10:]) / max(1, len(losses[-a.steps // 10:])):.5f}, "
              f"m and v hold {held / n:.2f} bytes per parameter")


if __name__ == "__main__":
    main()
