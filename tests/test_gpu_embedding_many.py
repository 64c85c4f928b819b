"""The table's gradient of many tokens, exactly: gradients are whole numbers up to 4 and every sum stays far below
2^24, so fp32 sums in any order have one right answer and a token that is lost or counted twice shows.

Past 32768 tokens whole pieces of 64 sorted tokens of one row are summed by a launch of their own, a run's blocks lie
beside each other along the row (every 512 columns) and the pieces' too (every 2048); past 131072 the sort's tiles are
larger and their counts have a launch."""
import pytest
import torch

from tensor_train_compressed_ttembeddingbag_amd import abi
from tensor_train_compressed_ttembeddingbag_amd.embedding import embedding, embedding_gradient

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
WIDTHS = [24, 520, 4104]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def whole(n, d, dtype, g):
    return torch.randint(-4, 5, (n, d), device="cuda", generator=g, dtype=torch.int8).to(dtype)


def exact(i, up, v, scale=1.0):
    return torch.zeros(v, up.shape[1], device="cuda").index_add_(0, i, up.float()) * scale


def tokens(n, v, g, hot=0.1):
    i = (v * torch.rand(n, device="cuda", generator=g) ** 3).long().clamp_(max=v - 1)
    i[torch.rand(n, device="cuda", generator=g) < hot] = v // 3
    return i


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("n", [32768, 32769, 131072, 131073])
def test_both_sides_of_the_borders(n, d):
    g = gen(n + d)
    v = 70001
    i, up = tokens(n, v, g), whole(n, d, torch.bfloat16, g)
    dw = embedding_gradient(up, i, v, scale=2.0, dtype=torch.float32)
    assert torch.equal(dw, exact(i, up, v, 2.0))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", WIDTHS + [5])
def test_runs_of_every_length(dtype, d):
    """Runs around a group's 16 tokens, a piece's 64 and two of them, of rows in any order, so that they start anywhere
    in a piece; and a few very long ones."""
    g = gen(d)
    lengths = [0, 1, 2, 15, 16, 17, 63, 64, 65, 126, 127, 128, 129, 130, 191, 192, 193, 255, 256, 257] * 12 + \
        [1000, 4096, 9000]
    order = torch.randperm(len(lengths), generator=torch.Generator().manual_seed(d)).tolist()
    lengths = [lengths[k] for k in order]
    i = torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(lengths)).cuda()
    n, v = i.numel(), len(lengths) + 3
    assert n > 32768
    i = i[torch.randperm(n, device="cuda", generator=g)]
    up = whole(n, d, dtype, g)
    assert torch.equal(embedding_gradient(up, i, v, dtype=torch.float32), exact(i, up, v))


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("n", [32769, 70001, 140003])
def test_one_token_all_over(n, d):
    """A run as long as the batch, with whole pieces in its middle."""
    g = gen(n)
    for v, row in ((1, 0), (5000, 4999)):
        i = torch.full((n,), row, dtype=torch.int64, device="cuda")
        up = whole(n, d, torch.float16, g)
        assert torch.equal(embedding_gradient(up, i, v, dtype=torch.float32), exact(i, up, v))


@pytest.mark.parametrize("d", WIDTHS)
def test_bad_indices_padding_and_strides(d):
    """Tokens without a row behind all others, rows of grad_out any distance apart."""
    g = gen(d)
    n, v = 40000, 9001
    i = tokens(n, v, g)
    i[::9], i[3::9] = -5, v + 77
    bad = (i < 0) | (i >= v)
    drop = bad | (i == v // 3)
    up = whole(n, 2 * d + 1, torch.bfloat16, g)[:, d:2 * d]
    up[drop] = float("nan")  # not read into anything
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dw = embedding_gradient(up, i, v, padding_idx=v // 3, dtype=torch.float32, dev_status=status)
    assert int(status) == abi.TT_DEV_BAD_INDEX
    assert torch.equal(dw, exact(i[~drop], up[~drop], v))
    status.zero_()
    embedding_gradient(up[~bad], i[~bad], v, dev_status=status)
    assert int(status) == 0


def test_rows_of_three_digits():
    g = gen(2)
    n, v, d = 40000, (1 << 20) + 5, 24
    i, up = tokens(n, v, g), whole(n, d, torch.float32, g)
    i[-1], i[-2] = v - 1, 0
    assert torch.equal(embedding_gradient(up, i, v), exact(i, up, v))


@pytest.mark.parametrize("n,d", [(40000, 520), (140000, 24)])
def test_captured(n, d):
    """Replayed with other tokens between eager work, through autograd and by itself."""
    g = gen(n)
    v = 3000
    w = torch.zeros(v, d, device="cuda", requires_grad=True)
    i, up = tokens(n, v, g), whole(n, d, torch.float32, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        embedding_gradient(up, i, v)
        torch.autograd.grad(embedding(i, w), w, up)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = embedding_gradient(up, i, v)
        b, = torch.autograd.grad(embedding(i, w), w, up)
    for k in range(4):
        i.copy_(tokens(n, v, g, 0.2 * k))
        up.copy_(whole(n, d, torch.float32, g))
        graph.replay()
        eager = embedding_gradient(up, i, v)
        torch.cuda.synchronize()
        want = exact(i, up, v)
        assert torch.equal(eager, want) and torch.equal(a, want) and torch.equal(b, want)


@pytest.mark.parametrize("n", [33000, 200000])
def test_the_same_bits_again(n):
    """Sums of any values in an order that depends on the tokens alone."""
    g = gen(n)
    i, up = tokens(n, 2000, g, 0.3), torch.randn(n, 520, device="cuda", generator=g)
    first = embedding_gradient(up, i, 2000)
    for _ in range(3):
        assert torch.equal(embedding_gradient(up, i, 2000), first)
