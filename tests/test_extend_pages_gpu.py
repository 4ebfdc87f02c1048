"""fa_extend_pages against the sequence-by-sequence oracle; whole numbers, so equal."""
import numpy as np
import pytest
import torch

import oracle
from exact_tiled_attention_40_b200 import fa

pytestmark = pytest.mark.gpu
INDEX, PAGES = 5, 8      # FA_ERR_DEVICE_INDEX, FA_ERR_DEVICE_NO_PAGES


def i32(a, dev):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)


def inputs(seed, B, hi, new_hi, max_pages, spare=0, new_lo=0):
    """Lengths, a table of scattered pages for the cached tokens, and the free list."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, hi + 1, B)
    new = rng.integers(new_lo, new_hi + 1, B)
    need = -(-(lens + new) // 16)
    num_pages = int(need.sum()) + spare + 1
    ids = rng.permutation(num_pages)
    table = np.zeros((B, max_pages), np.int64)
    at = 0
    for b in range(B):
        n = -(-int(lens[b]) // 16)
        table[b, :n] = ids[at:at + n]
        at += n
    free = np.zeros(num_pages, np.int64)
    free[:num_pages - at] = ids[at:]
    return dict(table=table, lens=lens, new=new, free=free, count=num_pages - at,
                num_pages=num_pages)


def call(s, max_tokens, dev):
    table = i32(s["table"], dev)
    lens, cu, pos, slots, left = fa.extend_pages(
        table, i32(s["lens"], dev), i32(s["new"], dev), i32(s["free"], dev), i32([s["count"]], dev),
        s["num_pages"], max_tokens)
    return dict(table=table, lens=lens, cu=cu, positions=pos, slots=slots, left=left)


def check(got, s, max_tokens):
    want, faults = oracle.extend_pages(s["table"], s["lens"], s["new"], s["free"], s["count"],
                                       max_tokens, s["num_pages"])
    for name in want:
        assert np.array_equal(got[name].cpu().numpy().ravel(),
                              np.asarray(want[name]).ravel()), name
    status = fa.device_status()
    assert status == (INDEX if "index" in faults else PAGES if "pages" in faults else 0)
    assert fa.device_status() == 0


@pytest.mark.parametrize("B,hi,new_hi,new_lo", [
    (1, 0, 1, 1), (1, 40, 17, 0), (3, 40, 0, 0), (64, 500, 1, 1), (33, 60, 100, 0),
    (1000, 70, 9, 0), (1025, 40, 3, 1), (2500, 0, 33, 0), (16384, 20, 2, 0),
    (256, 90, 7, 0), (257, 90, 7, 0), (301, 300, 60, 1)])
def test_extension_matches_the_oracle(cuda_device, B, hi, new_hi, new_lo):
    s = inputs(B + hi, B, hi, new_hi, -(-(hi + new_hi) // 16) + 1, spare=5, new_lo=new_lo)
    total = int(s["new"].sum())
    for max_tokens in (total, total + 77):       # exactly enough rows, and padding behind
        check(call(s, max_tokens, cuda_device), s, max_tokens)


def test_a_long_sequence_and_no_sequence(cuda_device):
    s = inputs(1, 1, 0, 0, 6251)
    s["new"] = np.array([100001])
    s["num_pages"], s["free"], s["count"] = 7000, np.arange(7000)[::-1].copy(), 7000
    check(call(s, 100001, cuda_device), s, 100001)
    s = inputs(2, 0, 0, 0, 4)
    check(call(s, 9, cuda_device), s, 9)


def test_lengths_and_count_in_place(cuda_device):
    """A step after step on the same buffers, as a serving loop keeps them."""
    s = inputs(7, 300, 90, 20, 30, spare=3000)
    dev = cuda_device
    B, maxp, np_ = 300, 30, s["num_pages"]
    table, lens, free = i32(s["table"], dev), i32(s["lens"], dev), i32(s["free"], dev)
    count = i32([s["count"]], dev)
    cu = torch.empty(B + 1, dtype=torch.int32, device=dev)
    pos = torch.empty(7000, dtype=torch.int32, device=dev)
    slots = torch.empty(7000, dtype=torch.int64, device=dev)
    rng = np.random.default_rng(8)
    for _ in range(4):
        s["new"] = rng.integers(0, 21, B)
        fa.fa_extend_pages(table, lens, i32(s["new"], dev), free, count, lens, count, cu, pos, slots,
                           B, maxp, np_, 16, 7000)
        want, _ = oracle.extend_pages(s["table"], s["lens"], s["new"], s["free"], s["count"], 7000,
                                      np_)
        got = dict(table=table, lens=lens, cu=cu, positions=pos, slots=slots, left=count)
        for name in want:
            assert np.array_equal(got[name].cpu().numpy().ravel(), np.ravel(want[name])), name
        s["table"], s["lens"], s["count"] = want["table"], want["lens"], want["left"]
    assert fa.device_status() == 0


def test_too_few_pages_and_too_few_rows(cuda_device):
    s = inputs(9, 200, 50, 40, 7)
    s["count"] = 130                              # runs out in the middle
    check(call(s, 8000, cuda_device), s, 8000)
    s = inputs(10, 200, 50, 40, 7)
    check(call(s, 1000, cuda_device), s, 1000)
    check(call(s, 0, cuda_device), s, 0)
    s["count"] = 0
    check(call(s, 8000, cuda_device), s, 8000)


def test_impossible_lengths_ids_and_counts(cuda_device):
    s = inputs(11, 64, 60, 30, 6, spare=9)
    s["lens"][3], s["new"][5], s["lens"][8] = -4, -1, 97      # 97 tokens of at most 96
    s["new"][20] = 2 ** 31 - 1
    check(call(s, 4000, cuda_device), s, 4000)
    s = inputs(12, 64, 60, 30, 6, spare=9)
    s["free"][s["count"] - 3] = s["num_pages"]
    s["free"][s["count"] - 9] = -1
    b = int(np.argmax((s["lens"] % 16 != 0) & (s["new"] > 0)))
    s["table"][b, s["lens"][b] // 16] = s["num_pages"] + 1
    check(call(s, 4000, cuda_device), s, 4000)
    s = inputs(13, 64, 60, 30, 6, spare=9)
    for count in (-1, s["num_pages"] + 1):
        s["count"] = count
        got = call(s, 4000, cuda_device)
        want, _ = oracle.extend_pages(s["table"], s["lens"], s["new"], s["free"], count, 4000,
                                      s["num_pages"])
        for name in want:
            assert np.array_equal(got[name].cpu().numpy().ravel(), np.ravel(want[name])), name
        assert fa.device_status() == INDEX


def test_captured_and_replayed(cuda_device):
    """The replay extends the lengths that the buffers then hold."""
    dev = cuda_device
    s = inputs(14, 100, 30, 8, 12, spare=2000, new_lo=1)
    table, lens, new, free = (i32(s[n], dev) for n in ("table", "lens", "new", "free"))
    count = i32([s["count"]], dev)
    cu = torch.empty(101, dtype=torch.int32, device=dev)
    pos = torch.empty(900, dtype=torch.int32, device=dev)
    slots = torch.empty(900, dtype=torch.int64, device=dev)

    def step():
        fa.fa_extend_pages(table, lens, new, free, count, lens, count, cu, pos, slots, 100, 12,
                           s["num_pages"], 16, 900)

    step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    table.copy_(i32(s["table"], dev))
    lens.copy_(i32(s["lens"], dev))
    count.fill_(s["count"])
    for _ in range(3):
        graph.replay()
        want, _ = oracle.extend_pages(s["table"], s["lens"], s["new"], s["free"], s["count"], 900,
                                      s["num_pages"])
        got = dict(table=table, lens=lens, cu=cu, positions=pos, slots=slots, left=count)
        for name in want:
            assert np.array_equal(got[name].cpu().numpy().ravel(), np.ravel(want[name])), name
        s["table"], s["lens"], s["count"] = want["table"], want["lens"], want["left"]
    assert fa.device_status() == 0
