"""fa_extend_pages with as many token rows as its sizes allow."""
import pytest
import torch

from exact_tiled_attention_40_b200 import fa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_tokens", [2 ** 31 - 1, 2 ** 31 - 512])
def test_the_most_token_rows(cuda_device, max_tokens):
    """Three requests of 40 tokens, and padding up to the bound (26 GB of rows)."""
    dev = cuda_device
    table = torch.zeros(3, 5, dtype=torch.int32, device=dev)
    lens = torch.tensor([7, 0, 16], dtype=torch.int32, device=dev)
    new = torch.tensor([40, 40, 40], dtype=torch.int32, device=dev)
    table[0, 0], table[2, 0] = 20, 21
    free = torch.arange(22, dtype=torch.int32, device=dev)
    count = torch.tensor([20], dtype=torch.int32, device=dev)
    small = table.clone()
    want = fa.extend_pages(small, lens, new, free, count, 22, 120)
    lens_out, cu, pos, slots, left = fa.extend_pages(table, lens, new, free, count, 22, max_tokens)
    assert torch.equal(table, small)
    assert torch.equal(lens_out, want[0]) and torch.equal(cu, want[1]) and torch.equal(left, want[4])
    assert torch.equal(pos[:120], want[2]) and torch.equal(slots[:120], want[3])
    # (in pieces: a comparison of the whole would double the memory)
    for at in range(120, max_tokens, 1 << 28):
        assert int(pos[at:at + (1 << 28)].abs().max()) == 0
        part = slots[at:at + (1 << 28)]
        assert int(part.min()) == -1 and int(part.max()) == -1
    assert fa.device_status() == 0
    del pos, slots, part
    torch.cuda.empty_cache()
