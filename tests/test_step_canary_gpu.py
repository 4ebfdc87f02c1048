"""The operators around attention write their outputs and nothing else, and read no
further than their inputs: tensors sit between margins of a pattern (NaN around inputs),
strided outputs between columns that must stay; calls of several streams at once; and
sizes at the ends of what is allowed."""
import numpy as np
import pytest
import torch

import oracle
from exact_tiled_attention_40_b200 import fa

pytestmark = pytest.mark.gpu
PAD = 4096               # elements on either side


class Guarded:
    def __init__(self, like=None, shape=None, dtype=None, dev="cuda"):
        shape = tuple(like.shape) if shape is None else shape
        dtype = like.dtype if dtype is None else dtype
        self.n = int(np.prod(shape))
        self.full = torch.empty(self.n + 2 * PAD, dtype=dtype, device=dev)
        if dtype.is_floating_point:
            self.full.fill_(float("nan"))
        else:
            self.full.fill_(-77 if dtype != torch.uint8 else 177)
        self.before = self.full.clone()
        self.t = self.full[PAD:PAD + self.n].view(shape)
        if like is not None:
            self.t.copy_(like)

    def intact(self):
        bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32, 8: torch.int64}
        a, b = (x.view(bits[x.element_size()]) for x in (self.full, self.before))
        return torch.equal(a[:PAD], b[:PAD]) and torch.equal(a[PAD + self.n:], b[PAD + self.n:])


def rope_inputs(dtype, T=37, Hq=5, Hkv=3, D=128, rot=96, axes=1, lead=None):
    gen = torch.Generator().manual_seed(3)
    qkv = Guarded(torch.randn(*(lead or (T,)), Hq + 2 * Hkv, D, generator=gen).to(dtype))
    w = [Guarded(torch.randn(D, generator=gen).to(dtype)) for _ in range(2)]
    ang = torch.rand(20, rot // 2, generator=gen) * 6
    table = Guarded(torch.cat([ang.cos(), ang.sin()], 1))
    pos = Guarded(torch.randint(0, 20, (axes, T), generator=gen).int())
    axis = Guarded(torch.randint(0, axes, (rot // 2,), generator=gen).to(torch.uint8))
    return qkv, w, table, pos, axis


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,rot,axes,inter,first", [(128, 128, 1, False, True),
                                                    (64, 48, 3, True, False),
                                                    (128, 96, 2, False, True)])
def test_norm_rope_and_backward_between_margins(cuda_device, dtype, D, rot, axes, inter, first):
    """The backward into views of one gradient of the projection: V's columns stay."""
    B, N, Hq, Hkv = 2, 37, 5, 3
    qkv, w, table, pos, axis = rope_inputs(dtype, B * N, Hq, Hkv, D, rot, axes, (B, N))
    x = qkv.t
    q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]
    shape = (lambda H: (B, H, N, D)) if first else (lambda H: (B, N, H, D))
    qo, ko = (Guarded(shape=shape(H), dtype=dtype) for H in (Hq, Hkv))
    args = (w[0].t, w[1].t, table.t, pos.t, axis.t)
    step = (Hq + 2 * Hkv) * D
    fa.fa_qk_norm_rope(q, k, *args, qo.t, ko.t, B, N, Hq, Hkv, D, step, step, rot, 20, axes, inter,
                       first, 1e-6)
    want = fa.qk_norm_rope(q, k, *args, interleaved=inter, heads_first=first)
    assert torch.equal(qo.t, want[0]) and torch.equal(ko.t, want[1])
    assert not torch.isnan(qo.t).any()

    dqo, dko = (Guarded(torch.randn(shape(H)).to(dtype)) for H in (Hq, Hkv))
    dqkv = Guarded(torch.full((B, N, Hq + 2 * Hkv, D), 7.0, dtype=dtype))
    dw = [Guarded(shape=(D,), dtype=torch.float32) for _ in range(2)]
    scratch = Guarded(shape=(2 * fa.QK_NORM_ROPE_SCRATCH_ROWS * D,), dtype=torch.float32)
    fa.fa_qk_norm_rope_bwd(q, k, dqo.t, dko.t, *args, dqkv.t[:, :, :Hq],
                           dqkv.t[:, :, Hq:Hq + Hkv], dw[0].t, dw[1].t, scratch.t, B, N, Hq, Hkv, D,
                           step, step, step, step, rot, 20, axes, inter, first, 1e-6)
    ref = fa.qk_norm_rope_backward(q, k, dqo.t, dko.t, *args, interleaved=inter, heads_first=first)
    assert torch.equal(dqkv.t[:, :, :Hq], ref[0])
    assert torch.equal(dqkv.t[:, :, Hq:Hq + Hkv], ref[1])
    assert torch.all(dqkv.t[:, :, Hq + Hkv:] == 7)
    assert torch.equal(dw[0].t, ref[2]) and torch.equal(dw[1].t, ref[3])
    for g in (qkv, *w, table, pos, axis, qo, ko, dqo, dko, dqkv, *dw, scratch):
        assert g.intact()
    assert fa.device_status() == 0


@pytest.mark.parametrize("T", [1, 64, 3001])
def test_append_between_margins(cuda_device, T):
    Hq, Hkv, D = 8, 2, 128
    qkv, w, table, pos, axis = rope_inputs(torch.bfloat16, T, Hq, Hkv, D, 128)
    pages = -(-T // 16) + 1
    kc, vc = (Guarded(torch.zeros(pages, 16, Hkv, D, dtype=torch.bfloat16)) for _ in range(2))
    slots = Guarded(torch.randperm(pages * 16)[:T])
    qo = Guarded(shape=(T, Hq, D), dtype=torch.bfloat16)
    x, step = qkv.t, (Hq + 2 * Hkv) * D
    fa.fa_append_paged(x[:, :Hq], x[:, Hq:], x[:, Hq + Hkv:], w[0].t, w[1].t, table.t, pos.t, None,
                       slots.t, qo.t, kc.t, vc.t, T, Hq, Hkv, D, 16, pages, step, step, step, 128,
                       20, 1, False, 1e-6)
    q, k = fa.qk_norm_rope(x[None, :, :Hq], x[None, :, Hq:Hq + Hkv], w[0].t, w[1].t, table.t, pos.t,
                           heads_first=False)
    assert torch.equal(qo.t, q[0])
    assert torch.equal(kc.t.view(-1, Hkv, D)[slots.t], k[0])
    assert torch.equal(vc.t.view(-1, Hkv, D)[slots.t], x[:, Hq + Hkv:])
    empty = torch.ones(pages * 16, dtype=torch.bool, device=cuda_device)
    empty[slots.t] = False
    assert torch.all(kc.t.view(-1, Hkv, D)[empty] == 0)
    for g in (qkv, *w, table, pos, kc, vc, slots, qo):
        assert g.intact()
    assert fa.device_status() == 0


@pytest.mark.parametrize("B,new,rows", [(0, 0, 5), (1, 1, 1), (70, 3, 300), (300, 40, 13000)])
def test_extend_between_margins(cuda_device, B, new, rows):
    rng = np.random.default_rng(B)
    maxp, num_pages = 6, 6 * B + 2
    lens, add = rng.integers(0, 50, B), rng.integers(0, new + 1, B)
    table = np.zeros((B, maxp), np.int64)
    ids = rng.permutation(num_pages)
    at = 0
    for b in range(B):
        n = -(-int(lens[b]) // 16)
        table[b, :n] = ids[at:at + n]
        at += n
    free = np.zeros(num_pages, np.int64)
    free[:num_pages - at] = ids[at:]
    g = {n: Guarded(torch.tensor(np.asarray(v), dtype=torch.int32)) for n, v in
         dict(table=table, lens=lens, new=add, free=free, count=[num_pages - at]).items()}
    out = {n: Guarded(shape=(k,), dtype=torch.int32) for n, k in
           dict(lens=B, left=1, cu=B + 1, positions=rows).items()}
    slots = Guarded(shape=(rows,), dtype=torch.int64)

    def call():
        fa.fa_extend_pages(g["table"].t, g["lens"].t, g["new"].t, g["free"].t, g["count"].t,
                           out["lens"].t, out["left"].t, out["cu"].t, out["positions"].t, slots.t, B,
                           maxp, num_pages, 16, rows)

    def compare():
        want, faults = oracle.extend_pages(table, lens, add, free, num_pages - at, rows, num_pages)
        assert not faults
        got = dict(table=g["table"].t, slots=slots.t, **{n: v.t for n, v in out.items()})
        for name in want:
            assert np.array_equal(got[name].cpu().numpy().ravel(), np.ravel(want[name])), name
        for t in (*g.values(), *out.values(), slots):
            assert t.intact()

    call()
    compare()
    graph = torch.cuda.CUDAGraph()                   # the two grids of many rows in a graph
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for v in (*out.values(), slots):
        v.t.fill_(-5)
    graph.replay()
    compare()
    assert fa.device_status() == 0


@pytest.mark.parametrize("Hq,Hkv,P", [(8, 2, 9), (8, 2, 230), (16, 16, 120), (6, 3, 250)])
def test_shared_prefix_between_margins(cuda_device, Hq, Hkv, P):
    """Lengths that are not allowed among the others, margins around everything."""
    dev, B = cuda_device, 7
    gen = torch.Generator(device=dev).manual_seed(5)
    own = [0, 1, 33, 48, 7, -16 * P, 70]
    maxp = P + 5
    num_pages = P + 5 * B
    ids = torch.randperm(num_pages, generator=gen, device=dev).int()
    table = torch.cat([ids[None, :P].expand(B, P), ids[P:].view(B, 5)], 1)
    lens = torch.tensor([16 * P + o for o in own], dtype=torch.int32, device=dev)
    lens[3], lens[4] = -3, 16 * maxp + 1             # count as no keys
    kc, vc = (Guarded(torch.randn(num_pages, 16, Hkv, 128, generator=gen, device=dev).bfloat16())
              for _ in range(2))
    q = Guarded(torch.randn(B, Hq, 128, generator=gen, device=dev).bfloat16())
    tb, ln, px = Guarded(table), Guarded(lens), Guarded(ids[:P])
    pages = Guarded(torch.tensor([P], dtype=torch.int32))
    o = Guarded(shape=(B, Hq, 128), dtype=torch.bfloat16)
    lse = Guarded(shape=(B, Hq), dtype=torch.float32)
    fa.fa_decode_shared_prefix(q.t, kc.t, vc.t, tb.t, ln.t, px.t, pages.t, o.t, B, Hq, Hkv, 128, 16,
                               0.1, maxp, P, num_pages, lse.t)
    assert fa.device_status() == 5
    lens[3] = lens[4] = 0
    po, pl = fa.decode_paged(q.t, kc.t, vc.t, tb.t, lens, 0.1)
    # the same inputs: weights and outputs rounded to bf16 on either side, of values that
    # a mean of normals keeps below 4
    assert (o.t.float() - po.float()).abs().max() <= 4 * 4 * 2.0 ** -8
    live = lens > 0
    assert (lse.t[live] - pl[live]).abs().max() <= 1e-3
    assert torch.all(lse.t[~live] == -float("inf")) and torch.all(o.t[~live] == 0)
    for g in (kc, vc, q, tb, ln, px, pages, o, lse):
        assert g.intact()
    assert fa.device_status() == 0


def test_many_calls_of_all_kinds_on_two_streams(cuda_device):
    """The same calls alone and beside those of another stream: the same bits where the
    order of sums is fixed, and the same whole numbers."""
    dev = cuda_device
    gen = torch.Generator(device=dev).manual_seed(6)
    T = 2000
    x = torch.randn(T, 24, 128, generator=gen, device=dev).bfloat16()
    w = torch.ones(128, dtype=torch.bfloat16, device=dev)
    tab = torch.rand(64, 128, generator=gen, device=dev)
    pos = torch.randint(0, 64, (T,), generator=gen, device=dev).int()
    dy = [torch.randn(1, H, T, 128, generator=gen, device=dev).bfloat16() for H in (16, 4)]
    q, k = x[None, :, :16], x[None, :, 16:20]
    lens = torch.randint(0, 90, (500,), generator=gen, device=dev).int()
    new = torch.randint(0, 20, (500,), generator=gen, device=dev).int()
    free = torch.randperm(9000, generator=gen, device=dev).int()
    count = torch.tensor([9000], dtype=torch.int32, device=dev)

    def calls():
        table = torch.zeros(500, 8, dtype=torch.int32, device=dev)
        out = [*fa.qk_norm_rope(q, k, w, w, tab, pos),
               *fa.qk_norm_rope_backward(q, k, *dy, w, w, tab, pos),
               *fa.extend_pages(table, lens, new, free, count, 9000, 6000)]
        return out + [table]

    alone = calls()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    results = [[], []]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                results[i].append(calls())
    torch.cuda.synchronize()
    for rs in results:
        for r in rs:
            for a, b in zip(alone, r):
                assert torch.equal(a, b)
    assert fa.device_status() == 0


def test_offsets_past_32_bits(cuda_device):
    """270,000 tokens of 64 heads of 128: 2.2e9 elements a tensor.  Rows at the start, in the
    middle and at the end are what a call on those tokens alone gives, in both layouts."""
    dev = cuda_device
    T, H, D = 270000, 64, 128
    gen = torch.Generator(device=dev).manual_seed(7)
    x = torch.empty(1, T, H, D, dtype=torch.bfloat16, device=dev)
    dy = torch.empty(1, H, T, D, dtype=torch.bfloat16, device=dev)
    spots = [slice(0, 40), slice(131060, 131100), slice(T - 40, T)]
    x.fill_(0.5)
    dy.fill_(0.25)
    for at in spots:
        x[:, at] = torch.randn(1, 40, H, D, generator=gen, device=dev).bfloat16()
        dy[:, :, at] = torch.randn(1, H, 40, D, generator=gen, device=dev).bfloat16()
    none = torch.empty(1, T, 0, D, dtype=torch.bfloat16, device=dev)
    few = torch.empty(1, 40, 0, D, dtype=torch.bfloat16, device=dev)
    w = torch.randn(D, generator=gen, device=dev).bfloat16()
    tab = torch.rand(64, D, generator=gen, device=dev)
    pos = torch.arange(T, device=dev).remainder(64).int()
    for first in (True, False):
        y, _ = fa.qk_norm_rope(x, none, w, None, tab, pos, heads_first=first)
        for at in spots:
            z, _ = fa.qk_norm_rope(x[:, at], few, w, None, tab, pos[at], heads_first=first)
            assert torch.equal(y[:, :, at] if first else y[:, at], z)
        del y
    dx, _, _, _ = fa.qk_norm_rope_backward(x, none, dy, none.transpose(1, 2), w, None, tab, pos)
    for at in spots:
        dz, _, _, _ = fa.qk_norm_rope_backward(x[:, at], few, dy[:, :, at], few.transpose(1, 2), w,
                                               None, tab, pos[at])
        assert torch.equal(dx[:, at], dz)
    assert fa.device_status() == 0


def test_the_binding_refuses_other_types_and_shapes(cuda_device):
    dev = cuda_device
    bf, i32 = torch.bfloat16, torch.int32

    def z(*shape, dtype=bf):
        return torch.zeros(*shape, dtype=dtype, device=dev)

    q, k, w, tab, pos = z(2, 3, 4, 64), z(2, 3, 2, 64), z(64), z(9, 64, dtype=torch.float32), z(
        6, dtype=i32)
    kc = z(5, 16, 2, 64)
    slots = z(3, dtype=torch.int64)
    d = z(2, 8, 128)
    pool = z(7, 16, 2, 128)
    table, lens, pages = z(2, 4, dtype=i32), z(2, dtype=i32), z(1, dtype=i32)
    rope = [q, k, w, w, tab, pos]
    bwd = [q, k, z(2, 4, 3, 64), z(2, 2, 3, 64), w, w, tab, pos]
    app = [q[0], k[0], k[0], kc, kc.clone(), slots, w, w, tab, pos[:3]]
    ext = [table, lens, lens, z(7, dtype=i32), pages, 7, 5]
    dec = [d, pool, pool, table, lens, table[0], pages]
    for fn, args, changes in (
            (fa.qk_norm_rope, rope, [(0, q.float()), (0, q[0]), (1, k.half()), (1, k[:1]),
                                     (1, z(2, 3, 2, 128)), (2, z(65)), (3, w.half()), (4, w),
                                     (4, tab.to(bf)), (5, pos.long()), (5, pos[:5]),
                                     (5, z(2, 6, dtype=i32)), (0, q.cpu()), (4, tab.cpu())]),
            (fa.qk_norm_rope_backward, bwd, [(2, z(2, 3, 4, 64)), (3, z(2, 2, 3, 64).half()),
                                             (2, z(2, 4, 3, 64).cpu()), (4, z(32))]),
            (fa.append_paged, app, [(0, q[0].half()), (2, z(3, 1, 64)), (3, z(5, 16, 1, 64)),
                                    (3, kc.transpose(0, 1)), (4, z(4, 16, 2, 64)), (5, slots.int()),
                                    (5, slots[:2]), (3, kc[:, ::2])]),
            (fa.extend_pages, ext, [(0, table.long()), (0, lens), (0, table.t()), (1, lens[:1]),
                                    (2, lens.long()), (3, z(6, dtype=i32)), (4, lens), (6, -1),
                                    (1, lens.cpu())]),
            (fa.decode_shared_prefix, dec, [(0, d.half()), (0, d[0]), (1, z(7, 16, 2, 64)),
                                            (2, pool[:6]), (3, table[:1]), (4, lens.long()),
                                            (5, table), (6, lens), (5, z(5, dtype=i32))])):
        for at, wrong in changes:
            bad = list(args)
            bad[at] = wrong
            with pytest.raises(fa.FAError):
                fn(*bad)
        fn(*args)                                    # and takes what is right
    with pytest.raises(fa.FAError, match="pair_axis"):
        fa.qk_norm_rope(q, k, w, w, tab, z(2, 6, dtype=i32))
    assert fa.device_status() == 0
