"""A TT table as the output head, with the gradient of its cores: a bag of its own for every row
gives the rows as a differentiable [V, D], which full_weight() (detached) does not."""
import pytest
import torch

from tensor_train_compressed_ttembeddingbag_amd import abi, loss as L
from tensor_train_compressed_ttembeddingbag_amd.module import TTEmbeddingBag

pytestmark = pytest.mark.gpu


def test_gradient_reaches_the_cores():
    """The table is linear in each core: along a direction r of one core the loss changes by
    <dW, table with r in the core's place>, so <gradient of the core, r> has to be that.  Bound:
    both are fp32 sums of the same products, 2^-16 of their terms' size."""
    print("case tt head", flush=True)
    v, d, n = 3000, 32, 200
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    bag = TTEmbeddingBag(v, d, tt_ranks=(8, 8), sparse=False, seed=1)
    rows = torch.arange(v, device="cuda")
    h = torch.randn(n, d, device="cuda", generator=g)
    t = torch.randint(0, v, (n,), device="cuda", generator=g)
    table = bag(rows, rows)
    assert float((table.detach() - bag.full_weight()).abs().max()) <= \
        2.0 ** -20 * float(table.detach().abs().max())
    table.retain_grad()
    h.requires_grad_(True)
    L.linear_cross_entropy(h, table, t).backward()
    assert h.grad.abs().max() > 0
    for k in range(3):
        r = torch.randn(bag.cores[k].shape, device="cuda", generator=g)
        cores = [c.data if j != k else r for j, c in enumerate(bag.cores)]
        along = abi.tt_full_weight(bag.desc, cores, 0, v)
        terms = (table.grad * along).double()
        got = (bag.cores[k].grad * r).double()
        size = float(terms.abs().sum() + got.abs().sum())
        assert abs(float(got.sum()) - float(terms.sum())) <= 2.0 ** -16 * size
        assert float(got.abs().max()) > 0
    bag.check_status()


def test_the_head_learns_through_its_cores():
    print("case tt head trains", flush=True)
    v, d, n = 2000, 32, 512
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    bag = TTEmbeddingBag(v, d, tt_ranks=(16, 16), sparse=False, seed=1)
    rows = torch.arange(v, device="cuda")
    h = torch.randn(n, d, device="cuda", generator=g)
    t = torch.randint(0, 50, (n,), device="cuda", generator=g)
    opt = torch.optim.Adam(bag.cores.parameters(), lr=0.02)
    losses = []
    for _ in range(40):
        opt.zero_grad()
        out = L.linear_cross_entropy(h, bag(rows, rows), t)
        out.backward()
        opt.step()
        losses.append(float(out.detach()))
    assert losses[-1] < 0.8 * losses[0], losses


def test_views_of_one_shape_share_a_plan():
    """What is kept per kind of call depends on shapes, strides and types, not on an address."""
    print("case plans", flush=True)
    big = torch.randn(100, 48, device="cuda").bfloat16()
    h = torch.randn(5, 32, device="cuda").bfloat16()
    t = torch.zeros(5, dtype=torch.int64, device="cuda")
    L.linear_cross_entropy(h, big[:, :32], t)
    n = len(L._plans)
    for a in range(1, 16):
        L.linear_cross_entropy(h, big[:, a:a + 32], t)
    assert len(L._plans) == n
