"""The compiled binding raises what torch raises: out of memory in an output's allocation
(the limit is the allocator's own, far below the GPU's memory), before anything is
launched; and a refusal for a tensor without dimensions."""
import pytest
import torch

from exact_tiled_attention_40_b200 import fa

pytestmark = pytest.mark.gpu


def test_out_of_memory_is_torchs_own_error(cuda_device):
    dev = cuda_device
    table = torch.zeros(2, 3, dtype=torch.int32, device=dev)
    lens = torch.zeros(2, dtype=torch.int32, device=dev)
    new = torch.full_like(lens, 20)
    free = torch.arange(9, dtype=torch.int32, device=dev)
    count = torch.full((1,), 9, dtype=torch.int32, device=dev)
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(0.02)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            fa.extend_pages(table, lens, new, free, count, 9, 2 ** 31 - 1)    # 26 GB of rows
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    torch.cuda.synchronize()
    assert not table.any()                       # nothing ran
    out = fa.extend_pages(table, lens, new, free, count, 9, 40)
    assert out[0].tolist() == [20, 20] and table[:, :2].tolist() == [[8, 7], [6, 5]]
    assert fa.device_status() == 0


@pytest.mark.parametrize("positions", [0, 7])
def test_positions_of_no_dimension_or_too_many_are_refused(cuda_device, positions):
    dev = cuda_device
    x = torch.zeros(1, 7, 2, 128, dtype=torch.bfloat16, device=dev)
    w = torch.ones(128, dtype=torch.bfloat16, device=dev)
    p = torch.tensor(3, device=dev) if positions == 0 else torch.zeros(1, 1, 7, device=dev)
    with pytest.raises(fa.FAError) as e:
        fa.qk_norm_rope(x, x, w, w, torch.ones(8, 128, device=dev), p.int())
    assert e.value.code == 1 and "positions" in str(e.value)
