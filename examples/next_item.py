"""Next-item prediction over a large catalogue: a TT embedding bag in, a vocabulary-head loss out.

A session is a bag of items.  ``TTEmbeddingBag`` pools it (cores updated inside the backward),
a linear layer turns the pooled row into a hidden state, and an output table [V, D] scores every
item of the catalogue -- through ``linear_cross_entropy``, so the [sessions, V] logits are never
stored.  A second, narrower model is then trained on the first one's top logits with
``linear_distillation``, and one session's next items are scored token by token.

    python examples/next_item.py [--items 100000] [--steps 60]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import torch

from tensor_train_compressed_ttembeddingbag_amd import loss as L
from tensor_train_compressed_ttembeddingbag_amd.module import TTEmbeddingBag


class NextItem(torch.nn.Module):
    def __init__(self, items, embed, hidden, seed):
        super().__init__()
        self.bag = TTEmbeddingBag(items, embed, tt_ranks=(16, 16), sparse=True, learning_rate=0.1,
                                  mode="mean", seed=seed)
        self.proj = torch.nn.Linear(embed, hidden, device="cuda")
        self.out = torch.nn.Parameter(
            (torch.randn(items, hidden, device="cuda") * hidden ** -0.5).bfloat16())

    def forward(self, indices, offsets):
        return self.proj(self.bag(indices, offsets)).bfloat16()


def batches(items, sessions, length, seed):
    """Sessions walk through the catalogue in a fixed direction: the next item follows from the
    bag, the third of the targets that the session does not reach is ignored."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    topics = max(1, items // 64)
    while True:
        topic = torch.randint(0, topics, (sessions, 1), device="cuda", generator=g)
        step = torch.randint(0, 32, (sessions, length), device="cuda", generator=g)
        indices = (topic * 64 + step) % items
        target = (topic[:, 0] * 64 + 48) % items
        target[torch.rand(sessions, device="cuda", generator=g) < 0.33] = -100
        yield indices.reshape(-1), torch.arange(0, sessions * length, length, device="cuda"), target


def train(model, steps, data, loss_of):
    opt = torch.optim.Adam([model.out, *model.proj.parameters()], lr=0.02)
    first = last = None
    for _ in range(steps):
        indices, offsets, target = next(data)
        opt.zero_grad()
        value = loss_of(model(indices, offsets), target, (indices, offsets))
        value.backward()
        opt.step()
        last = value.detach()
        first = last if first is None else first
    model.bag.check_status()
    return float(first), float(last)


def main(items=100_000, steps=60, sessions=2048, seed=0):
    torch.manual_seed(seed)
    teacher = NextItem(items, 64, 256, seed)
    data = batches(items, sessions, 10, seed)
    hard = train(teacher, steps, data,
                 lambda h, t, _: L.linear_cross_entropy(h, teacher.out, t, label_smoothing=0.05))
    print("teacher: cross entropy %.3f -> %.3f" % hard)

    student = NextItem(items, 64, 128, seed + 1)

    def distil(h, t, batch):
        with torch.no_grad():  # the teacher's 16 top logits, a slice of sessions at a time
            ht = teacher(*batch)
            top = [(x @ teacher.out.t()).float().topk(16, 1) for x in ht.split(256)]
        return L.linear_distillation(h, student.out, torch.cat([x.values for x in top]),
                                     torch.cat([x.indices for x in top]), temperature=2.0)

    soft = train(student, steps, data, distil)
    print("student: divergence %.3f -> %.3f" % soft)

    indices, offsets, target = next(data)
    with torch.no_grad():
        h, known = student(indices, offsets), target >= 0
        h, target = h[known], target[known]
        scores = [-L.linear_cross_entropy(h[i:i + 1], student.out, target[i:i + 1],
                                          reduction="none") for i in range(4)]
    print("log-probability of four next items:", ["%.2f" % float(s) for s in scores])
    return hard, soft


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--items", type=int, default=100_000)
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    main(a.items, a.steps)
