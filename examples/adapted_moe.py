"""An MoE block for many tenants: one frozen model, low-rank adapters per request.

    logits = x Wr (+ adapter)                      AdaptedLinear, fp32 result
    experts, gates = sigmoid scores, groups, top-k Routing
    y = routed experts                             MoELayer(router=False)
      + shared expert, its three projections with  AdaptedLinear, dropout on the
        adapters                                   adapters' input while training

Run on a GPU: ``python -m examples.adapted_moe`` trains the adapters of three tenants for a few
steps and then serves a batch of single tokens.
"""
from __future__ import annotations

import dataclasses

import torch

from grouped_gemm_built_gb300.dropout import dropout
from grouped_gemm_built_gb300.layer import MoELayer
from grouped_gemm_built_gb300.lora import AdaptedLinear
from grouped_gemm_built_gb300.routing import Routing


@dataclasses.dataclass(frozen=True)
class Sizes:
    H: int = 256          # hidden
    I: int = 128          # expert intermediate size
    E: int = 16           # routed experts
    k: int = 4            # experts per token
    Is: int = 128         # shared expert
    tenants: int = 3
    rank: int = 8
    p: float = 0.1        # adapter dropout


def make_weights(s: Sizes, seed: int = 0, device="cuda"):
    """Frozen bf16 weights, and adapters whose B starts at zero."""
    g = torch.Generator(device=device).manual_seed(seed)

    def draw(*shape, std=0.05):
        t = torch.empty(shape, dtype=torch.float32, device=device).normal_(0, std, generator=g)
        return t.to(torch.bfloat16)

    shapes = {"router": (s.H, s.E), "gate": (s.H, s.Is), "up": (s.H, s.Is), "down": (s.Is, s.H)}
    w = {"W_up": draw(s.E, s.H, s.I), "W_gate": draw(s.E, s.H, s.I), "W_down": draw(s.E, s.I, s.H),
         "bias": torch.zeros(s.E, device=device), "scale": torch.full((s.tenants,), 2.0, device=device)}
    for name, (K, N) in shapes.items():
        w[name] = draw(K, N)
        w[name + ".A"] = draw(s.tenants, s.rank, K)
        w[name + ".B"] = torch.zeros(s.tenants, s.rank, N, dtype=torch.bfloat16, device=device)
    return w


class AdaptedMoEBlock:
    """The block for batches of T tokens; ``ids`` names each token's tenant (-1: none)."""

    PROJECTIONS = ("router", "gate", "up", "down")

    def __init__(self, s: Sizes, T: int, w):
        self.s, self.w = s, w
        self.proj = {n: AdaptedLinear(w[n], w[n + ".A"], w[n + ".B"], w["scale"])
                     for n in self.PROJECTIONS}
        self.rule = Routing(s.E, s.k, score="sigmoid", groups=4, top_groups=2, group_score="top2",
                            scale=1.5)
        self.experts = MoELayer(T, s.H, s.I, s.E, s.k, router=False, precision="bf16_plain")
        self.expert_w = self.experts.weights(w["W_up"], w["W_gate"], w["W_down"])

    def forward(self, x, ids, seed=None):
        """y [T,H] bf16; ``seed``: train with adapter dropout. Keeps what backward needs."""
        P, p = self.proj, self.s.p
        xa = dropout(x, p, seed) if seed is not None else None
        logits, s_r = P["router"].forward(x, ids, x_ad=xa, out=torch.float32)
        idx, gates = self.rule.forward(logits, self.w["bias"])
        self.experts.plan(topk_idx=idx, gates=gates)
        y = self.experts.forward(x, self.expert_w)
        g, s_g = P["gate"].forward(x, ids, x_ad=xa)
        u, s_u = P["up"].forward(x, ids, x_ad=xa)
        h = (torch.nn.functional.silu(g.float()) * u.float()).to(torch.bfloat16)
        ys, s_d = P["down"].forward(h, ids)
        self.kept = (x, xa, ids, seed, logits, idx, g, u, h,
                     {"router": s_r, "gate": s_g, "up": s_u, "down": s_d})
        return y + ys

    def backward(self, dY):
        """(dX, {projection: (dA, dB)}) for dY [T,H] bf16, after ``forward``."""
        x, xa, ids, seed, logits, idx, g, u, h, saved = self.kept
        P, grads = self.proj, {}
        moe = self.experts.backward(x, None, self.expert_w, dY)
        d = P["down"].backward(h, ids, saved["down"], dY)
        grads["down"] = d["dA"], d["dB"]
        sig = torch.sigmoid(g.float())
        dh = d["dX"].float()
        dlogits = self.rule.backward(logits, idx, moe["dgates"], dtype=torch.bfloat16)
        upstream = {"gate": (dh * u.float() * sig * (1 + g.float() * (1 - sig))).to(torch.bfloat16),
                    "up": (dh * g.float() * sig).to(torch.bfloat16), "router": dlogits}
        dX = moe["dX"].float()
        for name, dy in upstream.items():
            b = P[name].backward(x, ids, saved[name], dy, x_ad=xa)
            grads[name] = b["dA"], b["dB"]
            dX += (dropout(b["dXa"], self.s.p, seed, add=b["dX"]) if xa is not None else b["dX"]).float()
        return dX.to(torch.bfloat16), grads

    def status(self) -> int:
        return self.experts.status() or max((q.status() for q in self.proj.values()), key=abs)


def train(block: AdaptedMoEBlock, x, ids, target, steps: int, lr: float, seed: int = 1):
    """Plain gradient descent on the adapters (fp32 copies) towards ``target``; the losses."""
    master = {(n, m): block.w[f"{n}.{m}"].float() for n in block.PROJECTIONS for m in "AB"}
    losses = []
    for step in range(steps):
        y = block.forward(x, ids, seed=seed + step)
        err = y.float() - target
        losses.append(float((err ** 2).mean()))
        _, grads = block.backward((2.0 / err.numel() * 1e3 * err).to(torch.bfloat16))
        for n, (dA, dB) in grads.items():
            for m, d in (("A", dA), ("B", dB)):
                master[n, m] -= lr / 1e3 * d.float()
                block.w[f"{n}.{m}"].copy_(master[n, m])    # the projections read these tensors
    return losses


def main():
    s = Sizes()
    w = make_weights(s)
    T = 384
    x = torch.randn(T, s.H, device="cuda").to(torch.bfloat16)
    ids = (torch.arange(T, device="cuda") * (s.tenants + 1) // T - 1).to(torch.int32)   # packed prompts
    block = AdaptedMoEBlock(s, T, w)
    target = block.forward(x, ids).float() + 0.3 * torch.randn(T, s.H, device="cuda") @ torch.randn(
        s.H, s.H, device="cuda") / s.H ** 0.5
    losses = train(block, x, ids, target, steps=30, lr=30.0)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    serve = AdaptedMoEBlock(s, 8, w)                       # one token each of eight requests
    y = serve.forward(torch.randn(8, s.H, device="cuda").to(torch.bfloat16),
                      torch.tensor([0, 2, 1, -1, 0, 0, 2, 1], dtype=torch.int32, device="cuda"))
    print("served", tuple(y.shape), "status", block.status(), serve.status())


if __name__ == "__main__":
    main()
