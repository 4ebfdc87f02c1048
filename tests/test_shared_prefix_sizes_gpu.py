"""fa_decode_shared_prefix over the longest prefixes that 31-bit lengths allow."""
import math

import pytest
import torch

from exact_tiled_attention_40_b200 import fa

pytestmark = pytest.mark.gpu
MOST = (2 ** 31 - 1) // 16               # pages of a sequence


@pytest.mark.parametrize("P,own", [(MOST, 0), (MOST - 1, 16), (MOST - 7, 16 * 7), (MOST - 8, 3)])
def test_a_prefix_of_2_to_the_31_tokens(cuda_device, P, own):
    """All keys score -60 but one in the first shared page, one in the last and, where there
    are any, the first own one, which score 0: 2^31 exp(-60) is below 2^-55, so O is the
    mean of the three values (whole numbers, so exactly) and the LSE the logarithm of their
    number, to 2^-18.  Keys past the prefix, taken for zero vectors, would score 0 too."""
    dev = cuda_device
    kc = torch.zeros(17, 16, 1, 128, dtype=torch.bfloat16, device=dev)
    kc[..., 0] = -60
    vc = torch.full_like(kc, 7)
    for page, slot, value in ((14, 9, 1), (15, 15, 3), (16, 0, 5)):
        kc[page, slot, :, 0] = 0
        vc[page, slot] = value
    table = torch.full((1, MOST), 16, dtype=torch.int32, device=dev)
    table[0, :P] = torch.arange(P, dtype=torch.int32, device=dev).remainder_(14)
    table[0, P:] = 0
    table[0, 0], table[0, P - 1] = 14, 15
    if own:
        table[0, P] = 16
    q = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device=dev)
    q[..., 0] = 1
    lens = torch.tensor([P * 16 + own], dtype=torch.int32, device=dev)
    o, lse = fa.decode_shared_prefix(q, kc, vc, table, lens, table[0],
                                     torch.tensor([P], dtype=torch.int32, device=dev), scale=1.0)
    assert torch.all(o == (3 if own else 2)), o
    assert (lse - math.log(3 if own else 2)).abs().max() <= 2.0 ** -18
    assert fa.device_status() == 0
    del table
    torch.cuda.empty_cache()
