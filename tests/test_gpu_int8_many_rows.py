"""``quantize_rows`` of more rows than one launch has workgroups for: there are several launches then.

Every row is held against the scale and the values in float32 operations, bit for bit (divisions of tensors by
tensors, which are rounded correctly; torch divides by a number through its reciprocal)."""
import pytest
import torch

from tensor_train_compressed_ttembeddingbag_amd.quant import quantize_rows

pytestmark = pytest.mark.gpu


# rows of three columns, four a workgroup; of a whole workgroup each; and past 2^32 lanes, a wave a row
@pytest.mark.parametrize("n,d,dtype", [((1 << 22) + 7, 3, torch.float32), ((1 << 20) + 9, 2056, torch.bfloat16),
                                       ((1 << 26) + 5, 8, torch.float16)])
def test_many_rows(n, d, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    x = torch.empty(n, d, dtype=dtype, device="cuda").normal_(0, 1, generator=g)
    rows = quantize_rows(x)
    step = max(1, (1 << 27) // d)
    for a in range(0, n, step):
        part = x[a:a + step].float()
        top = part.abs().amax(1)
        s = top / torch.full_like(top, 127.0)
        assert torch.equal(rows.scales[a:a + step], s)
        q = torch.round(part / s[:, None]).clamp(-127, 127)
        q[s == 0] = 0
        assert torch.equal(rows.values[a:a + step].float(), q)
        pad = rows.values.as_strided((len(part), rows.pitch - d), (rows.pitch, 1), a * rows.pitch + d)
        assert not bool(pad.any())
