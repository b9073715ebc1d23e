#!/usr/bin/env python3
"""Training steps of the end of a tensor-parallel model on one GPU: an 8-bit
projection of the shards' rows, the vocabulary loss without logits, and the
way back through both.

    python examples/vocab_head_step.py [--steps 20]

The rows come as the shards of a sequence-parallel layer, one buffer per rank.

  forward   quantise the shards and the projection's weight, multiply (block
            scales, bf16 out), loss over each rank's slice of the vocabulary,
            merge the slices
  backward  gradient of the slices with the merged log-sum-exp; the hidden
            rows' gradients add up over the slices (on several GPUs: a
            reduce-scatter); quantise them both ways; the rows' gradient dx
            from the transposed weight, the weight's from both transposed
            activations, with fp32 results
  update    plain SGD on fp32 master weights
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import all_gather_gemm_agmm_amd as agmm  # noqa: E402


class Head:
    def __init__(self, shards=4, rows=64, width=256, hidden=512, vocab=2000, slices=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.shards, self.rows, self.m = shards, rows, shards * rows
        self.part = vocab // slices
        self.vocab = self.part * slices
        self.project = torch.randn((hidden, width), generator=g, device="cuda") / width ** 0.5   # fp32 masters
        self.table = [torch.randn((self.part, hidden), generator=g, device="cuda") / hidden ** 0.5 for _ in range(slices)]
        self.x = [torch.randn((rows, width), generator=g, device="cuda").bfloat16() for _ in range(shards)]
        self.labels = torch.randint(0, self.vocab, (self.m,), generator=g, device="cuda")
        self.labels[::16] = -100                     # rows without a target
        self.forward_plan = agmm.ScaledPlan(shards, rows, width, hidden, "e4m3", 128, agmm.AGMM_BF16)
        self.dx_plan = agmm.ScaledPlan(1, self.m, hidden, width, "e5m2", 128, agmm.AGMM_BF16)
        self.dw_plan = agmm.ScaledPlan(1, hidden, self.m, width, "e5m2", 1, agmm.AGMM_FP32)
        self.loss_plans = [agmm.LossPlan(1, self.m, hidden, self.part, agmm.AGMM_BF16, vocab_start=i * self.part,
                                         vocab_size=self.vocab) for i in range(slices)]

    def step(self, rate=0.5):
        """One step; returns the mean loss and the rows' gradient dx."""
        # 8-bit projection of the gathered rows; every scale block is quantised once, for both directions
        rows = [agmm.quantize(s, out="both") for s in self.x]
        weight, weight_t = agmm.quantize(self.project, block_rows=128, out="both")
        h = self.forward_plan.run([r[0] for r in rows], weight)
        # loss over the slices of the vocabulary
        tables = [t.bfloat16() for t in self.table]
        out = [p.forward([h], t, self.labels) for p, t in zip(self.loss_plans, tables)]
        loss, lse = agmm.merge_vocab_slices(torch.stack([o[1] for o in out]), torch.stack([o[2] for o in out]), self.labels,
                                            self.vocab)
        kept = (self.labels != -100).sum()
        grad = (self.labels != -100).float() / kept
        # back: every slice with the merged lse, their dh added up
        dh = torch.zeros(h.shape, dtype=torch.float32, device="cuda")
        for i, (p, t) in enumerate(zip(self.loss_plans, tables)):
            dh_i, dt = p.backward([h], t, self.labels, lse, grad)
            dh += dh_i
            self.table[i] -= rate * 10 * dt.float()
        # through the projection: dx = dh W, dW = dh^T x, both block-scaled products
        d, d_t = agmm.quantize(dh, "e5m2", out="both")
        dx = self.dx_plan.run([d], weight_t)
        # the shards' transposed activations, side by side, are those of the gathered rows where a
        # shard's rows are whole scale blocks; otherwise the gathered rows are quantised
        if self.rows % 128 == 0:
            x_t = agmm.Scaled(torch.cat([r[1].values for r in rows], dim=1), torch.cat([r[1].scales for r in rows]), self.m, 1)
        else:
            x_t = agmm.quantize(torch.cat(self.x), out="cols")
        self.project -= rate * self.dw_plan.run([d_t], x_t)
        return loss.sum() / kept, dx

    def close(self):
        for p in [self.forward_plan, self.dx_plan, self.dw_plan, *self.loss_plans]:
            p.close()


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    head = Head()
    for i in range(a.steps):
        loss, _ = head.step()
        if i % 5 == 0 or i == a.steps - 1:
            print(f"step {i:3d}  loss {loss.item():.4f}", flush=True)
    head.close()


if __name__ == "__main__":
    main()
