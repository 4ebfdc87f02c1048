"""What the serving operators leave in the page pool, token by token, and decode over a
shared prefix at the bounds of its roundings: with lengths that are not allowed among the
others, and with tables much wider than their sequences, as a serving loop keeps them."""
import numpy as np
import pytest
import torch

import oracle
from exact_tiled_attention_40_b200 import fa
from test_serving_step_gpu import Book, D, EPS, Hkv, Hq, f64, rotary
from test_shared_prefix_gpu import check, i32, make, on_device, spread

pytestmark = pytest.mark.gpu


def test_the_pool_holds_every_token_in_its_place(cuda_device):
    """Steps of page extension and append: V as it is, K within its one rounding to bf16
    (2^-8 of it) and the fp32 arithmetic before (a sum of 128 squares, a reciprocal root,
    five products: below 2^-18 of the row's largest element), in the slot that the block
    table gives; then one decode step against the fp64 softmax over what the pool holds."""
    dev = cuda_device
    gen = torch.Generator().manual_seed(3)
    B, max_pages, num_pages, P = 6, 40, 200, 3
    table = rotary(700, dev)
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=gen)).bfloat16().to(dev) for _ in range(2))
    kc = torch.zeros(num_pages, 16, Hkv, D, dtype=torch.bfloat16, device=dev)
    vc = torch.zeros_like(kc)
    blocks = torch.zeros(B, max_pages, dtype=torch.int32, device=dev)
    lens = torch.zeros(B, dtype=torch.int32, device=dev)
    free = torch.randperm(num_pages, generator=gen).int().to(dev)
    count = torch.tensor([num_pages], dtype=torch.int32, device=dev)
    book = Book(B, table, wq, wk)
    for new in ([70, 49, 0, 48, 15, 100], [0, 1, 3, 16, 33, 7], [300, 1, 1, 1, 1, 1], [1] * 6):
        total = sum(new) + 5
        lens, cu, pos, slots, count = fa.extend_pages(blocks, lens, i32(new, dev), free, count,
                                                      num_pages, total)
        qkv = torch.randn(total, Hq + 2 * Hkv, D, generator=gen).bfloat16().to(dev)
        q = fa.append_paged(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], kc, vc, slots, wq,
                            wk, table, pos, eps=EPS)
        ends = cu.tolist()
        for b in range(B):
            rows = slice(ends[b], ends[b + 1])
            book.add(b, f64(qkv[rows, Hq:Hq + Hkv]), f64(qkv[rows, Hq + Hkv:]))
        assert [len(k) for k in book.k] == lens.tolist()
        for b in range(B):
            n = int(lens[b])
            k = f64(kc[blocks[b].long()].view(-1, Hkv, D)[:n])
            v = f64(vc[blocks[b].long()].view(-1, Hkv, D)[:n])
            assert np.array_equal(v, book.v[b])
            top = np.abs(book.k[b]).max(-1, keepdims=True)
            assert (np.abs(k - book.k[b]) <= 2.0 ** -8 * np.abs(book.k[b]) + 2.0 ** -18 * top).all()
    # every slot that no token has is as it was
    used = torch.zeros(num_pages * 16, dtype=torch.bool, device=dev)
    for b in range(B):
        t = torch.arange(int(lens[b]), device=dev)
        used[blocks[b, t // 16].long() * 16 + t % 16] = True
    assert int(used.sum()) == int(lens.sum())
    assert not kc.view(-1, Hkv, D)[~used].any() and not vc.view(-1, Hkv, D)[~used].any()
    # the first sequence's pages as the prefix of a batch made from it
    s = dict(q=q[:B].cpu(), kc=kc.cpu(), vc=vc.cpu(), P=P, own=np.array([5] * B), scale=D ** -0.5,
             lens=np.array([P * 16 + 5] * B), table=np.repeat(blocks[:1].cpu().numpy(), B, 0))
    o, lse = fa.decode_shared_prefix(q[:B], kc, vc, i32(s["table"], dev), i32(s["lens"], dev),
                                     blocks[0], i32([P], dev))
    check(o, lse, s)


@pytest.mark.parametrize("Hq,Hkv,P", [(8, 2, 9), (8, 2, 230), (16, 16, 120), (6, 3, 250),
                                      (32, 8, 40)])
def test_lengths_that_are_not_allowed_among_others(cuda_device, Hq, Hkv, P):
    """They count as no keys and are flagged; the live rows at the bounds of `check`."""
    dev = cuda_device
    own = np.array([0, 1, 33, 48, 7, -16 * P, 70, -7, 16] + [3] * 40)
    s = make(P, len(own), Hq, Hkv, P, own, dev)
    q, kc, vc, table, lens, prefix, pages = on_device(s, dev)
    width = table.shape[1]
    for b, bad in ((3, -3), (4, 16 * width + 1), (8, 2 ** 31 - 1), (11, -2 ** 31)):
        lens[b] = bad
        s["lens"][b] = 0
    o, lse = fa.decode_shared_prefix(q, kc, vc, table, lens, prefix, pages)
    assert fa.device_status() == 5
    check(o, lse, s)


@pytest.mark.parametrize("B,P,hi", [(7, 32, 200), (7, 65, 200), (64, 16, 100), (64, 256, 300),
                                    (1, 3, 40), (200, 5, 30)])
@pytest.mark.parametrize("width", [512, 2048])
def test_tables_wider_than_their_sequences(cuda_device, B, P, hi, width):
    """A row of a wide block table as prefix_table: the count alone says what is shared."""
    s = make(B + P, B, 8, 2, P, spread(P, B, hi), cuda_device)
    narrow = s["table"]
    s["table"] = np.full((B, width), 1 << 28)
    s["table"][:, :narrow.shape[1]] = narrow
    q, kc, vc, _, lens, _, pages = on_device(s, cuda_device)
    table = i32(s["table"], cuda_device)
    o, lse = fa.decode_shared_prefix(q, kc, vc, table, lens, table[B // 2], pages)
    s["table"] = narrow
    check(o, lse, s)
    # and the bits of a second call are the first one's
    again = fa.decode_shared_prefix(q, kc, vc, table, lens, table[B // 2], pages)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
