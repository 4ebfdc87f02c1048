"""The operators together, as a serving loop and a training step run them: page
extension, norm + rotation into the pool, prefill and decode over it; norm + rotation,
attention, and both backward passes."""
import numpy as np
import pytest
import torch

import oracle
from exact_tiled_attention_40_b200 import fa

pytestmark = pytest.mark.gpu
Hq, Hkv, D, ROT, EPS = 8, 2, 128, 128, 1e-6


def rotary(max_pos, dev):
    inv = 10000.0 ** (-torch.arange(0, ROT, 2, dtype=torch.float64) / ROT)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().to(dev)


def f64(t):
    return t.detach().cpu().double().numpy()


class Book:
    """Every sequence's keys and values in fp64, from the definition."""

    def __init__(self, B, table, wq, wk):
        self.k = [np.zeros((0, Hkv, D)) for _ in range(B)]
        self.v = [np.zeros((0, Hkv, D)) for _ in range(B)]
        self.table, self.wq, self.wk = f64(table), f64(wq), f64(wk)

    def add(self, b, k, v):
        n = len(self.k[b])
        R = oracle.rotation(self.table, np.arange(n, n + len(k))[None], None, D, False)
        self.k[b] = np.concatenate([self.k[b], oracle.norm_rope(k, self.wk, R, EPS)])
        self.v[b] = np.concatenate([self.v[b], v])

    def attend(self, b, q, scale):
        """q [n, Hq, D]: the last n positions of sequence b, causal."""
        n, have = len(q), len(self.k[b])
        R = oracle.rotation(self.table, np.arange(have - n, have)[None], None, D, False)
        q = oracle.norm_rope(q, self.wq, R, EPS).transpose(1, 0, 2)[None]
        o, _ = oracle.attention(q, self.k[b].transpose(1, 0, 2)[None],
                                self.v[b].transpose(1, 0, 2)[None], scale, causal=True)
        return o[0].transpose(1, 0, 2)


def test_a_serving_loop(cuda_device):
    """A shared prompt, then each request's own tokens in two chunks, then decode steps."""
    dev = cuda_device
    gen = torch.Generator().manual_seed(0)
    B, P, max_pages, num_pages = 5, 6, 20, 120
    scale = D ** -0.5
    table = rotary(400, dev)
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=gen)).bfloat16().to(dev) for _ in range(2))
    kc = torch.zeros(num_pages, 16, Hkv, D, dtype=torch.bfloat16, device=dev)
    vc = torch.zeros_like(kc)
    blocks = torch.zeros(B + 1, max_pages, dtype=torch.int32, device=dev)
    lens = torch.zeros(B + 1, dtype=torch.int32, device=dev)
    free = torch.randperm(num_pages, generator=gen).int().to(dev)
    count = torch.tensor([num_pages], dtype=torch.int32, device=dev)
    pages = torch.tensor([P], dtype=torch.int32, device=dev)
    book = Book(B + 1, table, wq, wk)

    def step(new):
        """Row B holds the shared prompt, which the others then begin with."""
        nonlocal lens, count
        total = int(sum(new)) + 3                          # three padding rows
        lens, cu, pos, slots, count = fa.extend_pages(
            blocks, lens, torch.tensor(new, dtype=torch.int32, device=dev), free, count, num_pages,
            total)
        qkv = torch.randn(total, Hq + 2 * Hkv, D, generator=gen).bfloat16().to(dev)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        out = fa.append_paged(q, k, v, kc, vc, slots, wq, wk, table, pos, eps=EPS)
        ends = cu.tolist()
        for b in range(B + 1):
            book.add(b, f64(k[ends[b]:ends[b + 1]]), f64(v[ends[b]:ends[b + 1]]))
        return out, cu, f64(q), ends

    def compare(o, b, q):
        # q, k rounded to bf16 move a score by at most 2^-7 of sum |q k| scale (about 7),
        # so a weight by 6 %; v is of order 1 and averages over the keys: 2e-1 bounds both
        assert np.abs(o - book.attend(b, q, scale)).max() <= 2e-1
        assert np.abs(o - book.attend(b, q, scale)).mean() <= 1e-2

    q, cu, raw, ends = step([0] * B + [P * 16])
    o, _ = fa.prefill_paged(q, kc, vc, blocks, cu, lens, P * 16, scale)
    compare(f64(o[:P * 16]), B, raw[:P * 16])
    blocks[:B, :P] = blocks[B, :P]
    lens[:B] = P * 16
    for b in range(B):
        book.k[b], book.v[b] = book.k[B].copy(), book.v[B].copy()
    for new in ([17, 1, 30, 16, 5, 0], [3, 40, 0, 1, 16, 0]):
        q, cu, raw, ends = step(new)
        o, _ = fa.prefill_paged(q, kc, vc, blocks, cu, lens, max(new), scale)
        for b in range(B):
            if new[b]:
                compare(f64(o[ends[b]:ends[b + 1]]), b, raw[ends[b]:ends[b + 1]])
    for _ in range(18):                                    # past a page's end
        q, cu, raw, ends = step([1] * B + [0])
        o, lse = fa.decode_shared_prefix(q[:B], kc, vc, blocks[:B], lens[:B], blocks[B, :P], pages,
                                         scale)
        plain, plain_lse = fa.decode_paged(q[:B], kc, vc, blocks[:B], lens[:B], scale)
        for b in range(B):
            compare(f64(o[b:b + 1]), b, raw[b:b + 1])
        # the same inputs: only the roundings of the weights and of the output differ,
        # each 2^-8 of values of at most 4
        assert (o.float() - plain.float()).abs().max() <= 4 * 4 * 2.0 ** -8
        assert (lse - plain_lse).abs().max() <= 1e-4
    assert fa.device_status() == 0
    left = int(count)
    assert left == num_pages - P - sum(-(-int(n) // 16) - P for n in lens[:B].tolist())


def test_a_training_step(cuda_device):
    """Gradients of q, k (before the norm) and of the weights through attention."""
    dev = cuda_device
    gen = torch.Generator().manual_seed(1)
    B, N = 2, 150
    scale = D ** -0.5
    qkv = torch.randn(B, N, Hq + 2 * Hkv, D, generator=gen).bfloat16()
    wq, wk = ((1 + 0.2 * torch.randn(D, generator=gen)).bfloat16() for _ in range(2))
    do = torch.randn(B, Hq, N, D, generator=gen).bfloat16()
    table = rotary(N, "cpu")
    pos = torch.arange(N).repeat(B).int()

    leaves = [qkv[:, :, :Hq].double(), qkv[:, :, Hq:Hq + Hkv].double(), wq.double(), wk.double()]
    for t in leaves:
        t.requires_grad_()
    v64 = qkv[:, :, Hq + Hkv:].double().transpose(1, 2)
    R = torch.tensor(oracle.rotation(f64(table), pos.numpy()[None], None, D, False))
    R = R.view(B, N, D, D)

    def normed(x, w):
        y = x * (x.square().mean(-1, keepdim=True) + EPS) ** -0.5 * w
        return torch.einsum("bnij,bnhj->bhni", R, y)

    q64, k64 = normed(leaves[0], leaves[2]), normed(leaves[1], leaves[3])
    G = Hq // Hkv
    z = q64 @ k64.repeat_interleave(G, 1).transpose(2, 3) * scale
    z = z.masked_fill(torch.ones(N, N, dtype=torch.bool).triu(1), float("-inf"))
    o64 = torch.softmax(z, -1) @ v64.repeat_interleave(G, 1)
    want = torch.autograd.grad((o64 * do.double()).sum(), leaves)

    x = qkv.to(dev)
    q_in, k_in = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]
    v = x[:, :, Hq + Hkv:].transpose(1, 2).contiguous()
    args = (wq.to(dev), wk.to(dev), table.to(dev), pos.to(dev))
    q, k = fa.qk_norm_rope(q_in, k_in, *args, eps=EPS)
    o, lse = fa.attention(q, k, v, scale, causal=True)
    dq, dk, _ = fa.attention_backward(q, k, v, o, lse, do.to(dev), scale, causal=True)
    got = fa.qk_norm_rope_backward(q_in, k_in, dq, dk, *args, eps=EPS)
    # bf16 roundings of q, k, o, P, dS, dq, dk on the way, each 2^-8: in the mean of the
    # squares below eight of them
    for g, w in zip(got, want):
        err = (g.cpu().double() - w).square().mean().sqrt()
        assert err <= 8 * 2.0 ** -8 * w.square().mean().sqrt()
    assert fa.device_status() == 0
