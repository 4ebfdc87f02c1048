"""A NaN among the live numbers of a decode shows in every output that it is part of and in
no other: the softmax of a row with a NaN score is NaN in O and in the LSE, however the
keys are split and joined.  Rows that do not see it keep their bits."""
import numpy as np
import pytest
import torch

from exact_tiled_attention_40_b200 import fa
from test_shared_prefix_gpu import make, on_device

pytestmark = pytest.mark.gpu
NAN = float("nan")

# (B, Hq, Hkv, P): attended together and joined by 8 warps a row, and by one; streamed with
# a scan kernel, one warp and 8; streamed without; two groups of heads, either way
CASES = [(7, 8, 2, 300), (64, 32, 8, 30), (200, 16, 2, 5), (140, 2, 1, 5), (7, 8, 2, 20),
         (5, 16, 16, 330), (5, 16, 16, 12)]


def inputs(B, Hq, Hkv, P, dev):
    own = np.random.default_rng(B).integers(1, 60, B)
    own[0], own[1] = -5, 33                     # the first is too short to take part
    return make(B + P, B, Hq, Hkv, P, own, dev)


def same_elsewhere(got, want, hit):
    """NaN where `hit` [B, Hq] holds, the bits of `want` elsewhere."""
    for g, w in zip(got, want):
        assert torch.isnan(g[hit]).all()
        assert torch.equal(g[~hit], w[~hit]) and not torch.isnan(w).any()
    assert fa.device_status() == 0


@pytest.mark.parametrize("B,Hq,Hkv,P", CASES)
def test_shared_prefix_with_a_nan(cuda_device, B, Hq, Hkv, P):
    s = inputs(B, Hq, Hkv, P, cuda_device)
    q, kc, vc, table, lens, prefix, pages = on_device(s, cuda_device)

    def call():
        return fa.decode_shared_prefix(q, kc, vc, table, lens, prefix, pages)

    want = call()
    heads = torch.arange(Hq, device=cuda_device)[None] // (Hq // Hkv)
    seq = torch.arange(B, device=cuda_device)[:, None]
    g = Hkv - 1
    # a key that all but the first sequence have: the first one, one inside, the last
    for page, slot in ((0, 0), (P // 2, 7), (P - 1, 15)):
        at = (int(s["prefix"][page]), slot, g, 5)
        keep = kc[at].clone()
        kc[at] = NAN
        same_elsewhere(call(), want, (heads == g) & (seq > 0))
        kc[at] = keep
    # a key of one sequence: of one behind the shared pages, of the one without them
    for b, t in ((1, P * 16 + 20), (0, 3)):
        at = (int(s["table"][b, t // 16]), t % 16, g, 100)
        keep = kc[at].clone()
        kc[at] = NAN
        same_elsewhere(call(), want, (heads == g) & (seq == b))
        kc[at] = keep
    # one query row
    keep = q[2, 1].clone()
    q[2, 1] = NAN
    same_elsewhere(call(), want, (seq == 2) & (torch.arange(Hq, device=cuda_device)[None] == 1))
    q[2, 1] = keep
    # a value: only its column, and no LSE
    at = (int(s["prefix"][P // 2]), 3, g)
    vc[at[0], at[1], at[2], 9] = NAN
    o, lse = call()
    hit = ((heads == g) & (seq > 0))[..., None] & (torch.arange(128, device=cuda_device) == 9)
    assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], want[0][~hit])
    assert torch.equal(lse, want[1])
    assert fa.device_status() == 0


@pytest.mark.parametrize("noalloc", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv", [(5, 8, 2), (70, 32, 8), (3, 16, 16), (40, 9, 9)])
def test_paged_decode_with_a_nan(cuda_device, B, Hq, Hkv, noalloc):
    """The streamed schedule and, above 8 KV heads, the one of fixed chunks."""
    s = make(B, B, Hq, Hkv, 0, np.random.default_rng(B).integers(30, 900, B), cuda_device)
    q, kc, vc, table, lens, _, _ = on_device(s, cuda_device)

    def call():
        if not noalloc:
            return fa.decode_paged(q, kc, vc, table, lens)
        o = torch.empty_like(q)
        lse = torch.empty(B, Hq, dtype=torch.float32, device=cuda_device)
        fa.decode_paged_noalloc(q, kc, vc, table, lens, o, lse)
        return o, lse

    want = call()
    heads = torch.arange(Hq, device=cuda_device)[None] // (Hq // Hkv)
    seq = torch.arange(B, device=cuda_device)[:, None]
    for b, t, g in ((0, 0, 0), (1, 17, Hkv - 1), (2, int(s["lens"][2]) - 1, 1)):
        at = (int(s["table"][b, t // 16]), t % 16, g, 77)
        keep = kc[at].clone()
        kc[at] = NAN
        same_elsewhere(call(), want, (heads == g) & (seq == b))
        kc[at] = keep
    q[1, 1] = NAN
    same_elsewhere(call(), want, (seq == 1) & (torch.arange(Hq, device=cuda_device)[None] == 1))
