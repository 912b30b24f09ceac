"""A small mixture-of-experts language model, trained and then asked for tokens.

    python examples/train_and_serve.py [--steps 60] [--tokens 2048]

Every large product of a step runs in this library: the experts' forward and
data-gradient GEMMs on MXFP8 operands (fwd), the loss over the vocabulary with
its gradients (vocab_cross_entropy), the experts' weight gradients (wgrad) and
their orthogonalised updates (orthogonalize).  Afterwards the same experts,
quantised once more, answer single tokens and small batches (moe_layer).

The task is synthetic: the next word is a fixed function of the current one, so
a table look-up through the experts can learn it.  The embedding and the router
stay as they were drawn; the experts and the output vocabulary learn.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_ragged_grouped_amd as mxw  # noqa: E402

VOCAB, HIDDEN, WIDTH, EXPERTS, TOP_K = 1000, 256, 128, 8, 2


def quantize_rows(x):
    """MXFP8 of bf16 x [..., R, C] with the 32-element blocks along C."""
    rows = x.reshape(-1, x.shape[-1])
    q, s = mxw.quantize_tokens(rows.t().contiguous())
    return q.view(x.shape), s.view(*x.shape[:-1], x.shape[-1] // 32)


class Model:
    def __init__(self, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def draw(*shape, scale):
            return torch.randn(shape, generator=g, device=device) * scale

        self.embedding = draw(VOCAB, HIDDEN, scale=1.0).to(torch.bfloat16)
        self.router = draw(EXPERTS, HIDDEN, scale=1 / math.sqrt(HIDDEN)).to(torch.bfloat16)
        # float32 master weights and momenta; each expert: gate rows, then up rows
        self.gate_up = draw(EXPERTS, 2 * WIDTH, HIDDEN, scale=1 / math.sqrt(HIDDEN))
        self.down = draw(EXPERTS, HIDDEN, WIDTH, scale=1 / math.sqrt(WIDTH))
        self.words = draw(VOCAB, HIDDEN, scale=0.02)
        self.momenta = [torch.zeros_like(self.gate_up), torch.zeros_like(self.down)]

    def routing(self, x):
        p = torch.softmax(x.float() @ self.router.float().t(), 1)
        w, ids = p.topk(TOP_K, dim=1)
        return ids, w / w.sum(1, keepdim=True)

    def group(self, ids):
        """Rows by expert, each expert's run padded to a multiple of 32 (the
        weight gradient's block): source token of every row (-1: padding), the
        choice it came from, and the runs' cumulative ends."""
        flat = ids.flatten()
        order = torch.argsort(flat, stable=True)
        counts = torch.bincount(flat, minlength=EXPERTS)
        padded = (counts + 31) // 32 * 32
        ends = padded.cumsum(0)
        first = ends - padded - (counts.cumsum(0) - counts)
        rows = torch.arange(len(flat), device=flat.device) + first[flat[order]]
        choice = torch.full((int(ends[-1]),), -1, dtype=torch.int64, device=flat.device)
        choice[rows] = order
        return choice, ends.to(torch.int32)

    def step(self, words, targets, lr):
        """One training step; the loss as a tensor."""
        x = self.embedding[words]
        ids, weights = self.routing(x)
        choice, offs = self.group(ids)
        token, real = choice.clamp(min=0) // TOP_K, (choice >= 0)[:, None]
        xs = torch.where(real, x[token], torch.zeros_like(x[token]))
        share = torch.where(real[:, 0], weights.flatten()[choice.clamp(min=0)], torch.zeros_like(token, dtype=torch.float32))

        # forward
        gate_up, down = self.gate_up.to(torch.bfloat16), self.down.to(torch.bfloat16)
        gu = mxw.fwd(*quantize_rows(xs), *quantize_rows(gate_up), offs).float()
        gate, up = gu[:, :WIDTH], gu[:, WIDTH:]
        sig = torch.sigmoid(gate)
        h = (gate * sig * up).to(torch.bfloat16)
        out = mxw.fwd(*quantize_rows(h), *quantize_rows(down), offs).float()
        y = x.float().index_add(0, token, out * share[:, None] * real)

        # the loss, and back
        loss, dy, dwords = mxw.vocab_cross_entropy(y.to(torch.bfloat16), self.words.to(torch.bfloat16), targets)
        dout = (dy.float()[token] * share[:, None] * real).to(torch.bfloat16)
        dh = mxw.fwd(*quantize_rows(dout), *quantize_rows(down.transpose(1, 2).contiguous()), offs).float()
        dgate = dh * up * (sig + gate * sig * (1 - sig))
        dgu = torch.cat([dgate, dh * gate * sig], 1).to(torch.bfloat16)
        grads = [mxw.wgrad(*mxw.quantize_tokens(dgu, offs), *mxw.quantize_tokens(xs, offs), offs),
                 mxw.wgrad(*mxw.quantize_tokens(dout, offs), *mxw.quantize_tokens(h, offs), offs)]

        # the experts: orthogonalised momentum; the vocabulary: plain descent
        for weight, momentum, grad in zip((self.gate_up, self.down), self.momenta, grads):
            momentum.mul_(0.9).add_(grad.float())
            scale = math.sqrt(max(1.0, weight.shape[1] / weight.shape[2]))
            weight.sub_(mxw.orthogonalize(momentum).float(), alpha=lr * scale)
        self.words.sub_(dwords.float(), alpha=100 * lr)
        return loss

    def serve(self):
        """The layer for single tokens and small batches: words -> logits."""
        qgu, sgu = quantize_rows(self.gate_up.to(torch.bfloat16))
        qd, sd = quantize_rows(self.down.to(torch.bfloat16))
        words = self.words.to(torch.bfloat16).float().t()

        def logits(prompt):
            x = self.embedding[prompt]
            out, _, _ = mxw.moe_layer(x, self.router, qgu, sgu, qd, sd, TOP_K)
            return (x.float() + out.float()) @ words

        return logits


def next_word(words):
    return (words * 37 + 11) % VOCAB


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--lr", type=float, default=0.05)
    a = ap.parse_args(argv)
    model = Model()
    g = torch.Generator(device="cuda").manual_seed(1)
    losses = []
    for i in range(a.steps):
        words = torch.randint(0, VOCAB, (a.tokens,), generator=g, device="cuda")
        loss = model.step(words, next_word(words), a.lr)
        losses.append(loss)
        if i % 10 == 0 or i + 1 == a.steps:
            print("step %3d  loss %.3f" % (i, loss.item()), flush=True)
    logits = model.serve()
    word = torch.tensor([5], device="cuda")
    said = [5]
    for _ in range(10):  # one token at a time
        word = logits(word).argmax(1)
        said.append(int(word))
    batch = torch.randint(0, VOCAB, (64,), generator=g, device="cuda")
    right = (logits(batch).argmax(1) == next_word(batch)).float().mean().item()
    print("said", said)
    print("next word right for %d%% of a batch of 64" % round(100 * right))
    return [v.item() for v in losses], right


if __name__ == "__main__":
    main()
