#!/usr/bin/env python3
"""Training steps of a tensor-parallel feed-forward block on one GPU: layer norm
of each rank's rows, the gated first projection over the gathered rows, the last
projection with bias and the residual stream, and the way back through all.

    python examples/feed_forward_step.py [--steps 20]

The rows come as the shards of a sequence-parallel layer, one buffer per rank;
the hidden columns are cut into slices, one per rank.

  forward   norm the shards; per slice the gated product, which keeps its
            pre-activations in 8 bits, and the slice's part of the last
            projection; the parts add up (on several GPUs: a reduce-scatter), the
            first one brings the bias and the residual
  backward  per slice: the hidden activations again from the 8 bits, the last
            projection's gradients, the gated product's; the normed rows'
            gradients add up over the slices, and go back through the norm
  update    plain SGD on fp32 master weights
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import all_gather_gemm_agmm_amd as agmm  # noqa: E402


class Block:
    def __init__(self, shards=4, rows=64, width=256, hidden=512, slices=2, activation="silu", keep=8, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def noise(*shape, scale=1.0):
            return torch.randn(shape, generator=g, device="cuda") * scale

        self.shards, self.rows, self.m, self.width, self.keep = shards, rows, shards * rows, width, keep
        self.part = hidden // slices
        # fp32 masters: norm weights, per slice the gate's and the factor's rows, and the last projection
        self.gain, self.shift = 1 + noise(width, scale=0.1), noise(width, scale=0.1)
        self.first = [noise(2 * self.part, width, scale=width ** -0.5) for _ in range(slices)]
        self.last = [noise(width, self.part, scale=hidden ** -0.5) for _ in range(slices)]
        self.bias = noise(width, scale=0.1)
        self.x = [noise(rows, width).bfloat16() for _ in range(shards)]
        self.goal = noise(self.m, width).bfloat16()
        self.norm_plan = agmm.NormPlan(rows, width, agmm.AGMM_BF16, agmm.AGMM_FP32)
        self.first_plan = agmm.FeedForwardPlan(shards, rows, width, self.part, agmm.AGMM_BF16, activation=activation, gated=True)
        self.last_plan = agmm.FeedForwardPlan(1, self.m, self.part, width, agmm.AGMM_BF16)

    def step(self, rate=0.0):
        """One step on the loss mean((y - goal)^2) / 2; returns the loss and the gradients by name."""
        x = torch.cat(self.x)
        normed = [self.norm_plan.forward(s, self.gain, self.shift) for s in self.x]
        rows = [n[0] for n in normed]
        y, kept = None, []
        first = [w.bfloat16() for w in self.first]
        last = [w.bfloat16() for w in self.last]
        bias = self.bias.bfloat16()
        for i, (w, v) in enumerate(zip(first, last)):
            h, saved = self.first_plan.forward(rows, w, keep=self.keep)
            kept.append(saved)                        # h itself is not kept
            part = self.last_plan.forward([h], v, bias if i == 0 else None, x if i == 0 else None)
            y = part.float() if y is None else y + part.float()
        off = y - self.goal.float()
        loss = (off * off).mean() / 2
        dy = (off / off.numel() * 1024).bfloat16()     # the loss is scaled, the updates are not
        # back
        drows = torch.zeros_like(off)
        grads = {"first": [], "last": []}
        for i, (w, v, saved) in enumerate(zip(first, last, kept)):
            h = self.first_plan.recompute(saved)
            dh, dlast, dbias = self.last_plan.backward([h], v, None, dy, need_dbias=i == 0)
            if i == 0:
                grads["bias"] = dbias.float() / 1024
            da, dfirst, _ = self.first_plan.backward(rows, w, saved, dh)
            drows += da.float()
            grads["first"].append(dfirst.float() / 1024)
            grads["last"].append(dlast.float() / 1024)
        grads["gain"], grads["shift"], grads["x"] = torch.zeros_like(self.gain), torch.zeros_like(self.shift), []
        for r, (s, n) in enumerate(zip(self.x, normed)):
            own = slice(r * self.rows, (r + 1) * self.rows)
            dx, dgain, dshift = self.norm_plan.backward(s, drows[own].bfloat16(), self.gain, n[1], n[2])
            grads["x"].append((dx.float() + dy[own].float()) / 1024)   # and the residual's
            grads["gain"] += dgain / 1024
            grads["shift"] += dshift / 1024
        if rate:
            for i in range(len(self.first)):
                self.first[i] -= rate * grads["first"][i]
                self.last[i] -= rate * grads["last"][i]
            self.bias -= rate * grads["bias"]
            self.gain -= rate * grads["gain"]
            self.shift -= rate * grads["shift"]
        return loss, grads

    def close(self):
        for p in (self.norm_plan, self.first_plan, self.last_plan):
            p.close()


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    block = Block()
    for i in range(a.steps):
        loss, _ = block.step(rate=20.0)
        if i % 5 == 0 or i == a.steps - 1:
            print(f"step {i:3d}  loss {loss.item():.4f}", flush=True)
    block.close()


if __name__ == "__main__":
    main()
