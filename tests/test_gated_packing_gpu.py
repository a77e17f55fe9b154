"""sq_pack_gated_weight's row norms where they leave 32 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="session")
def sq():
    from smoothquant_w8a8_int8_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load()
    return binding


@pytest.mark.parametrize("K,norm", [(16909312, 127 * 16909312), (16909328, 2 ** 31 - 1),
                                    (33818656, 2 ** 31 - 1)])
def test_norms_saturate(sq, K, norm):
    """Rows of codes of 127 alone: the last that fits 32 bits, the first that does not, and
    one whose wrapped norm would be a small positive number."""
    assert norm == min(127 * K, 2 ** 31 - 1)
    one = torch.ones(1, K, device="cuda")
    _, w, l1 = sq.pack_gated_weight(one, -one, one[0], want_l1=True)
    want = torch.zeros(64, dtype=torch.int32)
    want[0] = want[32] = norm
    assert torch.equal(l1.cpu(), want)
    assert (w[0] == 127).all() and (w[32] == -127).all()
