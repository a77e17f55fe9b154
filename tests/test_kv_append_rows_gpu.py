"""kv_append without q_out: rows of no sequence are zeros, as paged_attention's."""
import pytest
import torch

from pagedlib import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="session")
def sq():
    from smoothquant_w8a8_int8_gb300 import binding, build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    binding.load()
    return binding


@pytest.mark.parametrize("stream", [False, True])
def test_rows_of_no_sequence_are_zeros(sq, stream):
    t = Batch([3, 0, 2], [9, 4, 40], 4, 2, 64, 16, torch.bfloat16, seed=3, front=2, behind=5).cuda()
    qkv = torch.randn(t.T, 8 * 64, device="cuda")
    side = torch.cuda.Stream() if stream else None
    torch.cuda.synchronize()
    for _ in range(4):
        with torch.cuda.stream(side):
            old = torch.full((t.T, 4 * 64), float("nan"), device="cuda")
            del old  # what the next allocation of this size holds
        q = sq.kv_append(qkv, 4, t.k_d, t.v_d, t.table_d, t.q_start_d, t.kv_len_d, stream=side)
        torch.cuda.synchronize()
        first, last = int(t.q_start[0]), int(t.q_start[-1])
        assert torch.equal(q[first:last], qkv[first:last, :4 * 64])
        assert not q[:first].any() and not q[last:].any()
