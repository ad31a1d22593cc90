"""Distilling into a model's last ZeRO-3 unit (final norm + head), N_d ranks
simulated as buffers on one GPU, every operator of the unit's forward and
backward and of its step from this package:

    python examples/distil_head.py [--steps 30] [--tokens 512] [--width 256] [--vocab 1000]

Each step
  1. every owner quantises its part of the head to 4 bits, and the unit is
     gathered in 4.25 bits per parameter (the norm's weight in 16);
  2. every rank, on its own tokens: h = x + residual and y = RMSnorm(h) w;
     logits = y W^T with both operands in 4 bits; the loss against the teacher's
     k largest logits and, in the logits' place, its gradient, scaled by the
     loss scale that the device chain holds; dW = dlogits^T y and
     dy = dlogits W in 4 bits; the norm's backward pass; both gradients land in
     the rank's bucket;
  3. one fused partial pass reduces the buckets and updates every owner's
     shard, and a commit takes the step or, on an overflow, skips it.

The hidden states x, residual stand in for a frozen body; the teacher is the
same head with other weights.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import zero_dp_partitioned_gb300 as Z  # noqa: E402

DEV, BF16 = "cuda", torch.bfloat16
EPS = 1e-5


class HeadUnit:
    """The unit's flat parameters [norm weight | head, row by row] in N_d equal parts."""

    def __init__(self, width, vocab, ranks, seed=0):
        self.width, self.vocab, self.ranks = width, vocab, ranks
        self.numel = width + vocab * width
        self.part = self.numel // ranks
        assert self.numel % ranks == 0 and self.part % 64 == 0 and width % 64 == 0
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.params = torch.cat([torch.ones(width, device=DEV),
                                 torch.randn(vocab * width, generator=g, device=DEV) * 0.02]).to(BF16)
        self.state = [torch.empty(self.numel, device=DEV) for _ in range(6)]
        self.buckets = [torch.empty(self.numel, dtype=BF16, device=DEV) for _ in range(ranks)]
        P = self.part
        self.shards = [Z.shard(P, r * P, r * P, *(s[r * P:(r + 1) * P] for s in self.state)) for r in range(ranks)]
        Z.zero_shard_init(self.shards, self.params, Z.ZERO_BF16)
        # the 4-bit form of each owner's part, and what is gathered from them
        self.parts4 = [Z.mx4(1, P, layout=Z.ZERO_MX4_ROWS, device=DEV) for _ in range(ranks)]
        self.data = torch.empty(self.numel // 2, dtype=torch.uint8, device=DEV)
        self.scales = torch.empty(self.numel // 32, dtype=torch.uint8, device=DEV)
        self.norm_weight = torch.empty(width, dtype=BF16, device=DEV)
        head = (self.data[width // 2:], self.scales[width // 32:])
        self.gathered = Z.mx4(vocab, width, *head, layout=Z.ZERO_MX4_ROWS)
        self.head = Z.mx4(vocab, width, head[0],
                          torch.empty(Z.zero_mx4_bytes(vocab, width)[2], dtype=torch.uint8, device=DEV))
        self.head_values = torch.empty(vocab, width, dtype=BF16, device=DEV)
        self.head_t = Z.mx4(width, vocab, device=DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def gather(self):
        P = self.part
        for r, q in enumerate(self.parts4):
            Z.zero_mx4_quantize(self.params[r * P:(r + 1) * P], 1, P, q, None)
        # bytes in pairs: the gathers move 16-bit elements
        Z.zero3_gather_bulk([q.tensors[0] for q in self.parts4], [P // 4] * self.ranks, Z.ZERO_BF16, self.data, 0, self.status)
        Z.zero3_gather_segments([q.tensors[1] for q in self.parts4], [P // 64] * self.ranks, Z.ZERO_BF16, self.scales)
        Z.zero3_gather_segments([self.params], [self.width], Z.ZERO_BF16, self.norm_weight)
        Z.zero_mx4_tile_scales(self.gathered, self.head)

    def forward_backward(self, rank, x, residual, ids, teacher, temperature, chain):
        """This rank's losses; its gradients go into its bucket."""
        tokens, width, vocab = x.shape[0], self.width, self.vocab
        h, y = torch.empty_like(x), torch.empty_like(x)
        rstd, loss = torch.empty(tokens, device=DEV), torch.empty(tokens, device=DEV)
        logits = torch.empty(tokens, vocab, dtype=BF16, device=DEV)
        Z.zero_norm_forward(x, residual, self.norm_weight, tokens, width, EPS, h, y, None, 0, rstd)
        yq, yt = Z.mx4(tokens, width, device=DEV), Z.mx4(width, tokens, device=DEV)
        Z.zero_mx4_quantize(y, tokens, width, yq, yt)
        Z.zero_mx4_matmul(yq, self.head, 1.0, logits, self.status)
        Z.zero_distill_loss(logits, tokens, vocab, ids, teacher, ids.shape[1], None, temperature, None, 1.0 / tokens,
                            chain, loss, None, logits)
        dq, dt = Z.mx4(tokens, vocab, device=DEV), Z.mx4(vocab, tokens, device=DEV)
        Z.zero_mx4_quantize(logits, tokens, vocab, dq, dt)
        bucket = self.buckets[rank]
        Z.zero_mx4_matmul(dt, yt, 1.0, bucket[width:].view(vocab, width), self.status)
        # dy = dlogits W sums over the vocabulary: W along its columns
        Z.zero_mx4_dequantize(self.head, self.head_values)
        Z.zero_mx4_quantize(self.head_values, vocab, width, None, self.head_t)
        dy, dx = torch.empty_like(x), torch.empty_like(x)
        Z.zero_mx4_matmul(dq, self.head_t, 1.0, dy, self.status)
        ws = torch.empty(Z.zero_norm_workspace_bytes(width), dtype=torch.uint8, device=DEV)
        Z.zero_norm_backward(dy, h, self.norm_weight, tokens, width, rstd, None, dx, bucket[:width], 0, ws, ws.numel())
        return loss, dx


def run(steps=30, tokens=512, width=256, vocab=1000, ranks=4, k=32, temperature=2.0, lr=2e-3, loss_scale=1024.0):
    """The mean loss of every step (and the chain at the end)."""
    unit = HeadUnit(width, vocab, ranks)
    g = torch.Generator(device=DEV).manual_seed(1)
    teacher_head = torch.randn(vocab, width, generator=g, device=DEV) * 0.2
    batches = []
    for _ in range(ranks):
        x = (torch.randn(tokens, width, generator=g, device=DEV) * 0.5).to(BF16)
        residual = torch.randn(tokens, width, generator=g, device=DEV).to(BF16)
        hidden = torch.nn.functional.normalize((x + residual).float(), dim=1) * width ** 0.5
        top = (hidden @ teacher_head.t()).topk(k, dim=1)
        batches.append((x, residual, top.indices, top.values.to(BF16)))
    hyper = Z.hyper(lr=lr, weight_decay=0.0)
    table = torch.from_numpy(Z.zero_adam_scalar_table(hyper, 1, steps)).to(DEV)
    chain = torch.frombuffer(bytearray(bytes(Z.chain(loss_scale=loss_scale))), dtype=torch.uint8).to(DEV)
    ws = torch.zeros(Z.zero_workspace_bytes(), dtype=torch.uint8, device=DEV)
    stats, result = (torch.zeros(n, dtype=torch.uint8, device=DEV) for n in (16, 48))
    losses = []
    for _ in range(steps):
        unit.gather()
        losses.append(torch.stack([unit.forward_backward(r, *batches[r], temperature, chain)[0].mean()
                                   for r in range(ranks)]).mean())
        Z.zero_shard_step_partial(unit.buckets, Z.ZERO_BF16, unit.shards, unit.params, Z.ZERO_BF16, hyper, loss_scale, 0,
                                  stats, ws, ws.numel(), scalar_table=table, table_t0=1, n_table=steps, chain_dev=chain)
        Z.zero_shard_step_commit(unit.shards, unit.params, Z.ZERO_BF16, loss_scale, stats, 0.0, 0, result, table_t0=1,
                                 n_table=steps, chain_dev=chain)
    torch.cuda.synchronize()
    assert int(unit.status) == 0
    return [float(x) for x in losses], Z.read_chain(chain)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description="Distil into the last ZeRO-3 unit (final norm + head).")
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--vocab", type=int, default=1000)
    a = ap.parse_args()
    losses, chain = run(a.steps, a.tokens, a.width, a.vocab)
    for i, x in enumerate(losses):
        print(f"step {i + 1:3d}  loss {x:.4f}")
    print(f"applied {chain.applied}, skipped {chain.skipped}, loss scale {chain.loss_scale:g}")
