"""One pre-norm MoE block trained as a whole, the library's operators from end to end.

    h = x + residual;  z = RMS norm of h          Norm
    logits = z Wr                                  fp32 product (torch)
    experts, gates = softmax top-k                 Routing
    balance loss and penalty on large logits       Balance, per packed sequence
    out = h + routed experts of z                  MoELayer(router=False)
    clipped AdamW over every weight                grad_norm, AdamW (8-bit moments)

Run on a GPU: ``python -m examples.moe_training`` trains a few steps, one of them captured in a
CUDA graph.
"""
from __future__ import annotations

import dataclasses

import torch

from grouped_gemm_built_gb300.balance import Balance
from grouped_gemm_built_gb300.layer import MoELayer
from grouped_gemm_built_gb300.norm import Norm
from grouped_gemm_built_gb300.optim import AdamW, grad_norm
from grouped_gemm_built_gb300.routing import Routing


@dataclasses.dataclass(frozen=True)
class Sizes:
    H: int = 256          # hidden
    I: int = 128          # expert intermediate size
    E: int = 16           # routed experts
    k: int = 4            # experts per token
    coef: float = 0.02    # of the balance loss
    z_coef: float = 1e-3  # of the penalty on large logits


NAMES = ("norm", "Wr", "W_up", "W_gate", "W_down")
GRADS = {"norm": "dnorm", "Wr": "dWr", "W_up": "dW_up", "W_gate": "dW_gate", "W_down": "dW_down"}


def make_weights(s: Sizes, seed: int = 0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)

    def draw(*shape, std=0.05, dtype=torch.bfloat16):
        return torch.empty(shape, device=device).normal_(0, std, generator=g).to(dtype)

    return {"norm": torch.ones(s.H, dtype=torch.bfloat16, device=device),
            "Wr": draw(s.H, s.E, dtype=torch.float32), "W_up": draw(s.E, s.H, s.I),
            "W_gate": draw(s.E, s.H, s.I), "W_down": draw(s.E, s.I, s.H)}


class MoEBlock:
    """The block for T tokens; the weights are read where they lie, so a step on them is seen."""

    def __init__(self, s: Sizes, T: int, w):
        self.s, self.w = s, w
        self.norm = Norm(w["norm"], kind="rms", eps=1e-5)
        self.rule = Routing(s.E, s.k)
        self.balance = Balance(s.E, s.k, coef=s.coef, z_coef=s.z_coef)
        self.experts = MoELayer(T, s.H, s.I, s.E, s.k, router=False, precision="bf16_plain")
        self.expert_w = self.experts.weights(w["W_up"], w["W_gate"], w["W_down"])

    def forward(self, x, residual, seqs=None):
        """(out [T,H] bf16, losses [2], counts [E]); ``seqs``: offsets of packed sequences."""
        z, h, stats = self.norm.forward(x, add=residual)
        logits = z.float() @ self.w["Wr"]
        idx, gates = self.rule.forward(logits)
        losses, counts, saved = self.balance.forward(logits, idx, seqs)
        self.experts.plan(topk_idx=idx, gates=gates)
        out = h + self.experts.forward(z, self.expert_w)
        self.kept = (z, h, stats, logits, idx, saved, seqs)
        return out, losses, counts

    def backward(self, dout):
        """Gradients for dout [T,H] bf16 of a loss to which both balance losses are added."""
        z, h, stats, logits, idx, saved, seqs = self.kept
        g = self.experts.backward(z, None, self.expert_w, dout)
        dlogits = self.rule.backward(logits, idx, g["dgates"])
        dlogits = self.balance.backward(logits, saved, seqs, add=dlogits)
        g["dWr"] = z.float().t() @ dlogits
        dz = (g["dX"].float() + dlogits @ self.w["Wr"].t()).to(torch.bfloat16)
        n = self.norm.backward(dz, h, stats, add=dout)
        g["dX"], g["dnorm"] = n["dX"], n["dW"]
        return g

    def status(self) -> int:
        return self.experts.status()


def make_optimizer(w, bits: int = 8) -> AdamW:
    """Matrices decay, the norm's weight does not."""
    return AdamW([w[n] for n in NAMES], weight_decay=[0.0 if n == "norm" else 0.1 for n in NAMES],
                 bits=bits)


def train_step(block: MoEBlock, opt: AdamW, x, residual, target, lr, step=None, seqs=None):
    """(loss, balance losses, gradient norm) of one step towards ``target``, all on the device."""
    out, losses, _ = block.forward(x, residual, seqs)
    err = out.float() - target
    grads = block.backward((2.0 / err.numel() * err).to(torch.bfloat16))
    grads = [grads[GRADS[n]] for n in NAMES]
    norm, coef = grad_norm(grads, max_norm=1.0)
    opt.step(grads, lr=lr, coef=coef, step=step)
    return (err * err).mean(), losses, norm


def main():
    s, T = Sizes(), 512
    w = make_weights(s)
    block, opt = MoEBlock(s, T, w), make_optimizer(w)
    x, residual = (torch.randn(T, s.H, device="cuda").to(torch.bfloat16) for _ in range(2))
    target = residual.float() + 0.3 * torch.tanh(x.float())
    seqs = torch.tensor([0, 100, 300, 500], dtype=torch.int32, device="cuda")   # 12 padding rows
    t = torch.zeros(1, dtype=torch.int32, device="cuda")
    lr = torch.full((1,), 2e-3, device="cuda")

    def step():
        t.add_(1)
        return train_step(block, opt, x, residual, target, lr, step=t, seqs=seqs)

    side = torch.cuda.Stream()                             # the first steps, then a graph of one
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        first = step()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            last = step()
    for _ in range(40):
        graph.replay()
    torch.cuda.synchronize()
    for name, (loss, losses, norm) in (("first", first), ("last", last)):
        print(f"{name}: loss {float(loss):.4f}, balance {float(losses[0]):.5f}, logits "
              f"{float(losses[1]):.5f}, gradient norm {float(norm):.4f}")
    print("steps", int(t), "status", block.status())


if __name__ == "__main__":
    main()
