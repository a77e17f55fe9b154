"""sq_paged_attention over the range of values: queries whose largest element
ends an octave, rows of very different size side by side, logits far from one.
Lengths, layouts and masks are test_paged_attention_gpu's; the bound is
pagedlib.attention_ref's where no other is derived."""
import pytest
import torch

from pagedlib import Batch
from test_paged_attention_gpu import verify

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
FEW, MANY = [1, 3], [2, 40]  # tokens of two sequences: 4 heads to a group, so 12 or 160 rows


@pytest.fixture(scope="session")
def sq():
    from smoothquant_w8a8_int8_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load()
    return binding


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q", [FEW, MANY])
@pytest.mark.parametrize("top", [2.0 ** -33, 2.0 ** -16, 2.0 ** -8, 1.0, 2.0, 256.0, 2.0 ** 16])
def test_largest_element_at_an_octaves_end(sq, top, q, D, dtype):
    """Every row's largest element is the largest float below `top`, whose
    rounding to fewer bits is `top`; keys that make logits of order one."""
    t = Batch(q, [200, 333], 8, 2, D, 32, dtype, seed=D + sum(q))
    rows = t.Q.view(t.T * t.Hq, D)
    rows.mul_(0.3).clamp_(-0.9, 0.9)
    at = torch.arange(rows.shape[0])
    rows[at, at % D] = torch.where(at % 2 == 0, 1.0, -1.0) * (1 - 2.0 ** -24)
    rows.mul_(top)
    t.k = (t.k.float() * (3 / top)).clamp(-65504.0, 65504.0).to(dtype)
    verify(sq, t.cuda())
