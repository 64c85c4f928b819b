"""A dense table at both ends of a model: looked up, trained through policy and preference losses,
served in 8 bits.

A token's row, times sqrt(D), goes through one hidden layer, and the same table scores every token
that may follow.  The model is first trained by the clipped policy loss (an action is rewarded when it
is the token after next in the vocabulary), with the actions drawn from the model and an older copy
of it as the reference; then by pairs of sequences of which one follows that rule and one does
not.  At last the table is held in int8, and a few sequences are continued from it.

    python examples/tied_policy.py [--rows 20000] [--steps 30]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import torch

from tensor_train_compressed_ttembeddingbag_amd import loss as L
from tensor_train_compressed_ttembeddingbag_amd.embedding import embedding
from tensor_train_compressed_ttembeddingbag_amd.quant import int8_linear, quantize_rows


class Tied(torch.nn.Module):
    def __init__(self, rows, width, seed):
        super().__init__()
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.table = torch.nn.Parameter(
            (torch.randn(rows, width, device="cuda", generator=g) * width ** -0.5).bfloat16())
        self.layer = torch.nn.Parameter(
            (torch.randn(width, width, device="cuda", generator=g) * width ** -0.5).bfloat16())
        self.scale = width ** 0.5

    def hidden(self, tokens, table=None):
        rows = embedding(tokens, self.table if table is None else table, scale=self.scale,
                         dtype=torch.bfloat16)
        return rows + torch.tanh(rows @ self.layer)

    def logps(self, tokens, actions):
        return -L.linear_cross_entropy(self.hidden(tokens), self.table, actions, reduction="none")


def goal(tokens, rows):
    return (tokens + 2) % rows


def policy_step(model, reference, opt, tokens, rows, g):
    with torch.no_grad():  # one action in two is the rewarded one, the others are drawn
        drawn = torch.randint(0, rows, tokens.shape, device="cuda", generator=g)
        keep = torch.rand(tokens.shape, device="cuda", generator=g) < 0.5
        actions = torch.where(keep, goal(tokens, rows), drawn)
        reward = (actions == goal(tokens, rows)).float()
        advantages = (reward - reward.mean()) / (reward.std() + 1e-4)
        old, ref = model.logps(tokens, actions), reference.logps(tokens, actions)
    for _ in range(2):  # the second step is off the policy that took the actions
        opt.zero_grad()
        loss = L.linear_policy(model.hidden(tokens), model.table, actions, advantages, old, ref,
                               kl_coef=0.01)
        loss.backward()
        opt.step()
    return float(loss.detach())


def preference_step(model, reference, opt, tokens, rows, g):
    """tokens [P, T]: the first halves of the batch's sequences follow the rule, the second ones do not."""
    pairs, length = tokens.shape
    both = torch.cat([tokens, tokens])
    targets = torch.cat([goal(tokens, rows),
                         torch.randint(0, rows, tokens.shape, device="cuda", generator=g)])
    targets[:, 0] = -100  # prompts do not count
    offsets = torch.arange(0, 2 * pairs * length + 1, length, device="cuda")
    with torch.no_grad():
        ref = reference.logps(both, targets)
    opt.zero_grad()
    loss, ratios = L.linear_preference(model.hidden(both), model.table, targets, offsets, ref,
                                       return_ratios=True)
    loss.backward()
    opt.step()
    return float(loss.detach()), float((ratios[0] > ratios[1]).float().mean())


def main(rows=20000, steps=30, width=256, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    model, reference = Tied(rows, width, seed), Tied(rows, width, seed)
    reference.load_state_dict(model.state_dict())
    opt = torch.optim.Adam(model.parameters(), lr=2e-3)
    policy, prefer = [], []
    for _ in range(steps):
        tokens = torch.randint(0, rows, (16, 64), device="cuda", generator=g)
        policy.append(policy_step(model, reference, opt, tokens, rows, g))
        prefer.append(preference_step(model, reference, opt, tokens[:, :16], rows, g))
    print("policy loss %.3f -> %.3f" % (policy[0], policy[-1]))
    print("preference loss %.3f -> %.3f, pairs in order %.2f" % (prefer[0][0], *prefer[-1]))

    table = quantize_rows(model.table.detach())
    with torch.no_grad():
        tokens = torch.randint(0, rows, (4,), device="cuda", generator=g)
        said = [tokens]
        for _ in range(5):
            tokens = int8_linear(model.hidden(tokens, table), table).argmax(-1)
            said.append(tokens)
    print("continued from int8 rows:", torch.stack(said, 1).tolist())
    return policy, prefer, torch.stack(said, 1)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--rows", type=int, default=20000)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    main(a.rows, a.steps)
