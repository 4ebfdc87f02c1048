"""fa_decode_shared_prefix against the fp64 paged-decode oracle, which knows no sharing.

Tolerances.  The weights of the shared keys (and of the streamed own keys) are rounded to
bf16 for the second product, the row sum is not: at most 2^-8 of sum p |v|; the output is
rounded to bf16: 2^-8 of |o|.  A score is a sum of 128 exact products of bf16 numbers in
fp32, in 8 steps of the tensor core and a few more additions, each off by at most a few
units of 2^-24 of the sum of absolute products: below 2^-18 of L1 = scale * sum |q k|; ex2
and its argument add 2^-18 of 1 + |score - max| <= 1 + 2 L1.  So a weight and the LSE are
off by less than 2^-16 (L1 + 1), the LSE also by its own rounding 2^-23 |lse|.
"""
import numpy as np
import pytest
import torch

import oracle
from exact_tiled_attention_40_b200 import fa

pytestmark = pytest.mark.gpu
NEVER = 1 << 28          # an id far behind every pool


def make(seed, B, Hq, Hkv, P, own, dev, max_prefix=None, garbage=True):
    """own: tokens behind the shared pages, one number for each sequence; below zero: a
    sequence that many tokens short of the shared pages, with pages of its own."""
    gen = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    own = np.asarray(own)
    lens = P * 16 + own
    max_prefix = P if max_prefix is None else max_prefix
    pages_of = [-(-int(n) // 16) if o < 0 else -(-int(o) // 16) for n, o in zip(lens, own)]
    num_pages = P + sum(pages_of) + 3
    ids = rng.permutation(num_pages)
    width = P + max(max(pages_of), 1) + 1
    table = np.zeros((B, width), np.int64)
    at = P
    for b in range(B):
        n = pages_of[b]
        if own[b] < 0:
            table[b, :n] = ids[at:at + n]
        else:
            table[b, :P] = ids[:P]
            table[b, P:P + n] = ids[at:at + n]
        at += n
    kc = torch.randn(num_pages, 16, Hkv, 128, generator=gen).bfloat16()
    vc = torch.randn(num_pages, 16, Hkv, 128, generator=gen).bfloat16()
    if garbage:           # slots that hold no token: what a reused pool may hold
        used = np.zeros(num_pages * 16, bool)
        for b in range(B):
            t = np.arange(max(lens[b], 0))
            used[table[b, t // 16] * 16 + t % 16] = True
        free = torch.tensor(~used)
        kc.view(-1, Hkv, 128)[free] = float("nan")
        vc.view(-1, Hkv, 128)[free] = float("inf")
    q = torch.randn(B, Hq, 128, generator=gen).bfloat16()
    prefix = np.full(max(max_prefix, 1), NEVER)
    prefix[:P] = ids[:P]
    return dict(q=q, kc=kc, vc=vc, table=table, lens=lens, prefix=prefix[:max_prefix], P=P, own=own,
                scale=128 ** -0.5)


def i32(a, dev):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)


def on_device(s, dev):
    table = np.where((np.arange(s["table"].shape[1])[None] < s["P"]) & (s["own"][:, None] >= 0),
                     NEVER, s["table"])          # of the sharers these entries are not read
    return (s["q"].to(dev), s["kc"].to(dev), s["vc"].to(dev), i32(table, dev), i32(s["lens"], dev),
            i32(s["prefix"], dev), i32([s["P"]], dev))


def reference(s):
    q, kc, vc = s["q"].double().numpy(), s["kc"].float().numpy(), s["vc"].float().numpy()
    O, LSE = oracle.decode_paged(q, kc, vc, s["table"], s["lens"], s["scale"], 16)
    B, Hq, _ = q.shape
    G = Hq // kc.shape[2]
    A, L1 = np.zeros_like(O), np.zeros_like(LSE)
    for b in range(B):
        n = int(s["lens"][b])
        if n <= 0:
            continue
        k = oracle.gather_paged_kv(kc, s["table"], n, b, 16)
        v = oracle.gather_paged_kv(vc, s["table"], n, b, 16)
        for h in range(Hq):
            z = k[h // G] @ q[b, h] * s["scale"]
            A[b, h] = np.exp(z - LSE[b, h]) @ np.abs(v[h // G])
            L1[b, h] = (np.abs(k[h // G]) @ np.abs(q[b, h])).max() * s["scale"]
    return O, LSE, A, L1


def check(o, lse, s):
    O, LSE, A, L1 = reference(s)
    o, lse = o.cpu().double().numpy(), lse.cpu().double().numpy()
    dead = s["lens"] <= 0
    assert (o[dead] == 0).all() and (lse[dead] == -np.inf).all()
    live = ~dead
    e = 2.0 ** -16 * (L1[live] + 1)
    lim = 2.0 ** -8 * (np.abs(O[live]) + A[live]) * 1.01 + 2 * e[..., None] * A[live]
    assert (np.abs(o[live] - O[live]) <= lim).all(), np.abs(o[live] - O[live]).max()
    assert (np.abs(lse[live] - LSE[live]) <= e + 2.0 ** -23 * np.abs(LSE[live])).all()
    assert fa.device_status() == 0, fa.last_error()


def spread(seed, B, hi):
    return np.random.default_rng(seed).integers(0, hi + 1, B)


@pytest.mark.parametrize("B,Hq,Hkv,P,hi", [
    (1, 1, 1, 1, 1), (1, 8, 2, 8, 40), (2, 8, 8, 9, 0), (5, 16, 2, 7, 33), (7, 8, 2, 65, 200),
    (33, 16, 16, 12, 50), (64, 32, 8, 16, 100), (65, 4, 1, 40, 20), (129, 4, 2, 3, 17),
    (257, 8, 8, 5, 20), (40, 64, 8, 33, 30), (3, 10, 5, 130, 9), (300, 8, 1, 17, 3),
    (70, 9, 9, 16, 40), (5, 22, 11, 220, 30), (600, 8, 1, 3, 5), (9, 32, 16, 120, 90),
    (2, 8, 8, 800, 70), (4200, 4, 1, 1, 20), (2, 8, 1, 800, 30000), (3, 64, 64, 70, 40),
    (128, 8, 2, 10, 90), (129, 8, 2, 10, 90), (257, 8, 8, 7, 20)])
def test_matches_the_oracle(cuda_device, B, Hq, Hkv, P, hi):
    s = make(B + P, B, Hq, Hkv, P, spread(P, B, hi), cuda_device)
    o, lse = fa.decode_shared_prefix(*on_device(s, cuda_device))
    check(o, lse, s)


# a few copies of the shared keys are streamed with the own ones, many are attended at
# once; 16 KV heads go through the stream kernel in two groups
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (16, 16)])
@pytest.mark.parametrize("P", [25, 140])
def test_shorter_sequences_and_padding_rows(cuda_device, Hq, Hkv, P):
    own = np.array([-16 * P, -1, 0, 1, 15, 16, 17, -384, -16, 1 - 16 * P, 250, -16 * P])
    s = make(3, 12, Hq, Hkv, P, own, cuda_device)
    assert s["lens"].min() == 0
    check(*fa.decode_shared_prefix(*on_device(s, cuda_device)), s)


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (16, 16)])
@pytest.mark.parametrize("P", [4, 320])
def test_all_rows_empty(cuda_device, Hq, Hkv, P):
    s = make(4, 5, Hq, Hkv, P, [-16 * P] * 5, cuda_device)
    check(*fa.decode_shared_prefix(*on_device(s, cuda_device)), s)


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (16, 16)])
def test_count_below_its_bound_and_none_shared(cuda_device, Hq, Hkv):
    for P, bound in ((3, 50), (0, 50), (0, 0), (3, 180), (0, 180)):
        s = make(5, 9, Hq, Hkv, P, spread(1, 9, 70), cuda_device, max_prefix=bound)
        s["table"] = np.pad(s["table"], ((0, 0), (0, 180)))
        check(*fa.decode_shared_prefix(*on_device(s, cuda_device)), s)


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (16, 16)])
@pytest.mark.parametrize("P", [10, 270])
def test_a_row_of_the_block_table_as_the_prefix(cuda_device, Hq, Hkv, P):
    s = make(6, 6, Hq, Hkv, P, spread(2, 6, 40), cuda_device)
    q, kc, vc, _, lens, _, pages = on_device(s, cuda_device)
    table = i32(s["table"], cuda_device)
    check(*fa.decode_shared_prefix(q, kc, vc, table, lens, table[2], pages), s)


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (16, 16)])
@pytest.mark.parametrize("P", [10, 270])
def test_counts_and_ids_out_of_range(cuda_device, Hq, Hkv, P):
    s = make(7, 6, Hq, Hkv, P, spread(3, 6, 40), cuda_device)
    q, kc, vc, _, lens, prefix, pages = on_device(s, cuda_device)
    table = i32(s["table"], cuda_device)
    for bad in (-1, P + 1, 2 ** 31 - 1):             # counts as no shared page
        o, lse = fa.decode_shared_prefix(q, kc, vc, table, lens, prefix,
                                         torch.full_like(pages, bad))
        assert fa.device_status() == 5
        check(o, lse, s)
    for bad in (-1, kc.shape[0], -2 ** 31, 2 ** 31 - 1):     # its keys count as zero vectors
        prefix[3] = bad
        o, lse = fa.decode_shared_prefix(q, kc, vc, table, lens, prefix, pages)
        assert fa.device_status() == 5
        z = dict(s, kc=s["kc"].clone(), vc=s["vc"].clone())
        z["kc"][s["prefix"][3]] = 0
        z["vc"][s["prefix"][3]] = 0
        check(o, lse, z)


@pytest.mark.parametrize("P", [20, 400])
def test_lowest_and_infinite_scores(cuda_device, P):
    """Scores of -inf over the whole prefix: it takes no weight; large scores saturate."""
    s = make(8, 4, 8, 2, P, np.array([5, 0, 40, 1]), cuda_device, garbage=False)
    s["q"][:] = 0
    s["q"][..., 0] = 1
    at = torch.tensor(s["prefix"])
    s["kc"][at, :, :, 0] = float("-inf")
    q, kc, vc, table, lens, prefix, pages = on_device(s, cuda_device)
    o, lse = fa.decode_shared_prefix(q, kc, vc, table, lens, prefix, pages)
    t = dict(s, lens=np.array([5, 0, 40, 1]), table=s["table"][:, P:], P=0,
             own=np.array([5, 0, 40, 1]))
    check(o, lse, t)
    s["kc"][at, :, :, 0] = 3e4                    # far above the own keys', one far above all
    s["kc"][at[7], 3, :, 0] = 6e4
    q, kc, vc, table, lens, prefix, pages = on_device(s, cuda_device)
    o, lse = fa.decode_shared_prefix(q, kc, vc, table, lens, prefix, pages)
    want = s["vc"][at[7], 3].repeat_interleave(4, 0).double()
    assert torch.equal(o.cpu().double(), want[None].expand(4, 8, 128))
    assert fa.device_status() == 0


@pytest.mark.parametrize("P", [50, 80])
def test_equal_to_plain_decode_without_lse(cuda_device, P):
    """The same numbers as fa_decode_paged within both calls' roundings."""
    s = make(9, 20, 32, 8, P, spread(4, 20, 300), cuda_device)
    q, kc, vc, _, lens, prefix, pages = on_device(s, cuda_device)
    table = i32(s["table"], cuda_device)
    o, none = fa.decode_shared_prefix(q, kc, vc, table, lens, prefix, pages, return_lse=False)
    assert none is None
    p, _ = fa.decode_paged(q, kc, vc, table, lens)
    A = reference(s)[2]
    assert ((o - p).abs().cpu().double().numpy() <= 2.0 ** -6 * A * 1.1).all()


def test_long_prefix_over_every_sm(cuda_device):
    """Few rows, thousands of pages: shares that end inside items; a pool past 2^32 bytes."""
    dev = cuda_device
    B, Hq, Hkv, P = 3, 16, 8, 2500
    num_pages = 140000
    gen = torch.Generator(device=dev).manual_seed(1)
    kc = torch.empty(num_pages, 16, Hkv, 128, dtype=torch.bfloat16, device=dev)
    vc = torch.empty_like(kc)
    ids = torch.randperm(num_pages, generator=gen, device=dev)[:P + 3 * 9]
    ids[:40] = torch.arange(num_pages - 40, num_pages, device=dev)
    ids = torch.unique(ids)
    P = ids.numel() - 27
    ids = ids.flip(0)
    kc[ids] = torch.randn(ids.numel(), 16, Hkv, 128, generator=gen, device=dev).bfloat16()
    vc[ids] = torch.randn(ids.numel(), 16, Hkv, 128, generator=gen, device=dev).bfloat16()
    q = torch.randn(B, Hq, 128, generator=gen, device=dev).bfloat16()
    table = torch.cat([ids[None, :P].expand(3, P), ids[P:].view(3, 9)], 1).int()
    lens = torch.tensor([P * 16, P * 16 + 133, P * 16 + 144], dtype=torch.int32, device=dev)
    o, lse = fa.decode_shared_prefix(q, kc, vc, table, lens, ids[:P].int(),
                                     torch.tensor([P], dtype=torch.int32, device=dev))
    for b in range(B):
        n = int(lens[b])
        k = kc[table[b].long()].view(-1, Hkv, 128)[:n].double().repeat_interleave(2, 1)
        v = vc[table[b].long()].view(-1, Hkv, 128)[:n].double().repeat_interleave(2, 1)
        z = torch.einsum("hd,nhd->hn", q[b].double(), k) * 128 ** -0.5
        p = torch.softmax(z, -1)
        want = torch.einsum("hn,nhd->hd", p, v)
        A = torch.einsum("hn,nhd->hd", p, v.abs())
        L1 = torch.einsum("hd,nhd->hn", q[b].double().abs(), k.abs()).amax(-1) * 128 ** -0.5
        e = 2.0 ** -16 * (L1 + 1)
        lim = 2.0 ** -8 * (want.abs() + A) * 1.01 + 2 * e[:, None] * A
        assert ((o[b].double() - want).abs() <= lim).all()
        ref = torch.logsumexp(z, -1)
        assert ((lse[b].double() - ref).abs() <= e + 2.0 ** -23 * ref.abs()).all()
    assert fa.device_status() == 0


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (16, 16)])
def test_graphs_streams_and_calls_at_once(cuda_device, Hq, Hkv):
    """Two captured graphs replayed at once on two streams, beside eager calls."""
    dev = cuda_device
    cases = [make(11, 30, Hq, Hkv, 60, spread(5, 30, 90), dev),
             make(12, 11, Hq, Hkv, 90, spread(6, 11, 200), dev)]
    ins = [on_device(s, dev) for s in cases]
    for a in ins:
        fa.decode_shared_prefix(*a)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fa.decode_shared_prefix(*a))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        eager = [fa.decode_shared_prefix(*a) for a in ins]
    torch.cuda.synchronize()
    for s, o, e in zip(cases, outs, eager):
        check(*o, s)
        check(*e, s)
    # other lengths in the captured buffers, a shorter prefix among them
    s = cases[0]
    short = dict(s, lens=s["lens"].copy(), own=s["own"].copy())
    short["own"] = np.minimum(short["own"], 16)
    short["lens"] = 960 + short["own"]           # (60 shared pages)
    ins[0][4].copy_(i32(short["lens"], dev))
    graphs[0].replay()
    check(*outs[0], short)
