"""A small Monarch student distilled from a dense teacher's top logits.

The student is a residual stream of feed-forward blocks whose dense layers are
MonarchLinear layers (up with ReLU, down), joined by SandwichNorm modules; it is
trained with distill_step, which gives the loss and the logits' gradient in one
pass, against the stored top logits of a dense model of the same widths. Tokens
and the teacher are synthetic (seeded draws).

    python -m monarch_block_diagonal_amd.distill_student --steps 60

--no-logits takes the same loss with head_loss_step instead, from the head's input, without
the logits; --dropout 0.1 drops a tenth of every block's output while it trains.
"""
from __future__ import annotations

import argparse

import torch

from . import binding as B
from . import torch_api as T


class MonarchStudent(torch.nn.Module):
    """Embedding, `blocks` Monarch feed-forward blocks, a dense head."""

    def __init__(self, vocab: int, features: int, hidden: int, blocks: int, nblocks: int = 4,
                 device="cuda", dtype=torch.bfloat16, dropout: float = 0.0):
        super().__init__()
        kw = dict(device=device, dtype=dtype)
        self.embed = torch.nn.Embedding(vocab, features, **kw)
        self.first = torch.nn.Parameter(torch.ones(features, **kw))
        self.up = torch.nn.ModuleList(T.MonarchLinear(features, hidden, nblocks, act=B.ACT_RELU, **kw)
                                      for _ in range(blocks))
        self.down = torch.nn.ModuleList(T.MonarchLinear(hidden, features, nblocks, **kw)
                                        for _ in range(blocks))
        self.join = torch.nn.ModuleList(T.SandwichNorm(features, gated=True, branch_scale=blocks ** -0.5, **kw)
                                        for _ in range(blocks))
        self.head = torch.nn.Linear(features, vocab, bias=False, **kw)
        self.drop = torch.nn.ModuleList(T.Dropout(dropout) if dropout else torch.nn.Identity() for _ in range(blocks))

    def hidden(self, tokens):
        """The head's input."""
        h = self.embed(tokens)
        n = T.SandwichFunction.apply(h, None, None, None, None, self.first, None,
                                     dict(post_norm=B.NORM_NONE, pre_norm=B.NORM_RMS, skip_scale=1.0,
                                          branch_scale=1.0, eps=1e-5))
        for up, down, drop, join in zip(self.up, self.down, self.drop, self.join):
            h, n = join(h, drop(down(up(n))))
        return n

    def forward(self, tokens):
        return self.head(self.hidden(tokens))


def dense_teacher(vocab: int, features: int, hidden: int, generator, device="cuda"):
    """A dense model's logits for tokens [rows], fp32."""
    draw = lambda *s: torch.randn(s, generator=generator, device=device) * s[-1] ** -0.5  # noqa: E731
    embed, up, down, head = draw(vocab, features), draw(hidden, features), draw(features, hidden), draw(vocab, features)

    def logits(tokens):
        h = embed[tokens] * features ** 0.5
        h = h + torch.relu(h @ up.T) @ down.T
        return 4.0 * h @ head.T

    return logits


def train(steps: int = 60, rows: int = 2048, vocab: int = 5003, features: int = 256, hidden: int = 1024,
          blocks: int = 2, top: int = 32, temperature: float = 2.0, mix: float = 0.8, seed: int = 0,
          log=lambda step, loss: None, keep_logits: bool = True, dropout: float = 0.0):
    """Trains a student; returns (student, mean losses of the steps as one tensor). Without keep_logits
    the head's logits are not kept: its gradient and its input's come with the loss."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    torch.manual_seed(seed)
    teacher = dense_teacher(vocab, features, hidden, g)
    student = MonarchStudent(vocab, features, hidden, blocks, dropout=dropout)
    opt = torch.optim.Adam(student.parameters(), lr=2e-3)
    weight = torch.full((rows,), 1.0 / rows, device="cuda")
    losses = []
    for step in range(steps):
        tokens = torch.randint(0, min(vocab, 512), (rows,), generator=g, device="cuda")
        with torch.no_grad():
            known, ids = teacher(tokens).topk(top, dim=1)   # what a stored teacher would hold
        labels = ids[:, 0].contiguous()
        opt.zero_grad(set_to_none=True)
        if keep_logits:
            logits = student(tokens)
            # loss and gradient in one pass, the gradient in the logits' own memory
            loss, dlogits = T.distill_step(logits.detach(), known, ids, labels, weight, temperature=temperature,
                                           mix=mix, out=logits.detach())
            logits.backward(dlogits)
        else:
            n = student.hidden(tokens)
            loss, dn, dw = T.head_loss_step(n.detach(), student.head.weight.detach(), labels, known, ids, weight,
                                            temperature=temperature, mix=mix)
            student.head.weight.grad = dw
            n.backward(dn)
        opt.step()
        losses.append(loss.mean())
        log(step, losses[-1])
    return student, torch.stack(losses)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--rows", type=int, default=2048)
    ap.add_argument("--vocab", type=int, default=5003)
    ap.add_argument("--no-logits", action="store_true", help="the loss from the head's input, without its logits")
    ap.add_argument("--dropout", type=float, default=0.0, help="share of a block's output that is dropped")
    a = ap.parse_args()
    train(a.steps, a.rows, a.vocab, keep_logits=not a.no_logits, dropout=a.dropout,
          log=lambda step, loss: print(f"step {step:4d}  loss {float(loss):.4f}", flush=True)
          if step % 10 == 0 or step == a.steps - 1 else None)


if __name__ == "__main__":
    main()
