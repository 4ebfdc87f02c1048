"""fa_qk_norm_rope, its backward and fa_append_paged against the fp64 oracle.

Tolerances.  The kernels compute in fp32 and round once, so an output is off by half a
step of its type (eps / 2 of the value; for fp16 also half its smallest step, 2^-25) and
by the fp32 errors below.  Units are u = 2^-24, a rounding in fp32.
Forward, y = a c - b s with a, b the normalised pair: the sum of squares is off by at
most 13 u (8 products in a lane, log2(D / 8) <= 4 shuffled sums, 1 / D and eps exact or
1 u), half of that after the root, rsqrtf by 4 u (2 ulp), two products 2 u, the
rotation 3 u: below 16 u = 2^-20 of |a| + |b|.
Backward: g is off by 3 u of |g_a| + |g_b|; w g xhat, its mean over D and the last
product by at most 55 u of their absolute values, which is below 2^-18.
dw: terms off by 15 u; they are summed in chains of at most 128 additions between the
rows and the result for the sizes here: below 2^-16 of the sum of absolute values.
"""
import numpy as np
import pytest
import torch

import oracle
from exact_tiled_attention_40_b200 import fa

pytestmark = pytest.mark.gpu
EPS = 1e-6


def table_of(rng, max_pos, rot):
    ang = rng.uniform(-3, 3, (max_pos, rot // 2))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def make(seed, lead, Hq, Hkv, D, rot, axes, dtype, dev, max_pos=50, fused=True, pad=0):
    rng = np.random.default_rng(seed)
    T = int(np.prod(lead))
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(*lead, Hq + 2 * Hkv, D, generator=gen).to(dtype)
    if pad:                                       # a wider stride from token to token
        wide = torch.zeros(*lead, Hq + 2 * Hkv + pad, D, dtype=dtype)
        wide[..., :Hq + 2 * Hkv, :] = x
        x = wide
    x = x.to(dev)
    q, k, v = x[..., :Hq, :], x[..., Hq:Hq + Hkv, :], x[..., Hq + Hkv:Hq + 2 * Hkv, :]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    wq, wk = (torch.randn(D, generator=gen).to(dtype).to(dev) for _ in range(2))
    table = table_of(rng, max_pos, rot)
    pos = rng.integers(0, max_pos, (axes, T))
    axis = rng.integers(0, axes, rot // 2) if axes > 1 else None
    return dict(q=q, k=k, v=v, wq=wq, wk=wk, table=table, pos=pos, axis=axis, T=T, lead=lead, D=D,
                args=(torch.tensor(table, device=dev).reshape(max_pos, rot),
                      torch.tensor(pos, dtype=torch.int32, device=dev),
                      None if axis is None else torch.tensor(axis, dtype=torch.uint8, device=dev)))


def f64(t):
    return t.detach().cpu().float().double().numpy()


def rows(t, s):
    return f64(t).reshape(s["T"], -1, s["D"])


def partner_abs(x, rot, inter):
    """|x| + |its partner in the rotation|."""
    a = np.abs(x)
    out = a.copy()
    h = rot // 2
    if inter:
        out[..., 0:rot:2] += a[..., 1:rot:2]
        out[..., 1:rot:2] += a[..., 0:rot:2]
    else:
        out[..., :h] += a[..., h:rot]
        out[..., h:rot] += a[..., :h]
    return out


def half_step(want, err, dtype):
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    return torch.finfo(dtype).eps / 2 * (np.abs(want) + err) + err + tiny


def check_forward(got, x, w, s, rot, inter, dtype, eps=EPS):
    """got: [T, H, D] float64."""
    R = oracle.rotation(s["table"], s["pos"], s["axis"], s["D"], inter)
    want = oracle.norm_rope(x, w, R, eps)
    xn = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    err = 2.0 ** -20 * partner_abs(xn, rot, inter)
    bad = np.abs(got - want) - half_step(want, err, dtype)
    assert (bad <= 0).all(), bad.max()


def tokens_first(t, heads_first):
    return t.transpose(1, 2) if heads_first else t


CASES = [
    # lead, Hq, Hkv, D, rot, axes, interleaved, heads_first, dtype
    ((1, 1), 8, 2, 128, 128, 1, False, True, torch.bfloat16),
    ((1, 1), 1, 1, 64, 64, 1, True, False, torch.float16),
    ((2, 37), 8, 2, 128, 128, 1, False, True, torch.bfloat16),
    ((2, 37), 8, 2, 128, 64, 2, True, True, torch.float16),
    ((3, 5), 7, 3, 64, 48, 3, False, False, torch.bfloat16),
    ((1, 101), 5, 5, 64, 16, 8, True, True, torch.bfloat16),
    ((1, 33), 6, 1, 128, 48, 3, False, True, torch.float16),
    ((4, 9), 3, 0, 128, 128, 1, False, False, torch.bfloat16),
    ((4, 9), 0, 3, 128, 96, 1, True, True, torch.bfloat16),
    ((2, 11), 4, 4, 64, 0, 1, False, True, torch.float16),
    ((1, 300), 9, 1, 128, 32, 1, True, False, torch.bfloat16),
]


@pytest.mark.parametrize("lead,Hq,Hkv,D,rot,axes,inter,first,dtype", CASES)
@pytest.mark.parametrize("weights", ["both", "none", "q"])
def test_forward(cuda_device, lead, Hq, Hkv, D, rot, axes, inter, first, dtype, weights):
    s = make(sum(lead) + Hq, lead, Hq, Hkv, D, rot, axes, dtype, cuda_device)
    wq = None if weights == "none" else s["wq"]
    wk = s["wk"] if weights == "both" else None
    q, k = fa.qk_norm_rope(s["q"], s["k"], wq, wk, *s["args"], eps=EPS, interleaved=inter,
                           heads_first=first)
    for got, x, w in ((q, s["q"], wq), (k, s["k"], wk)):
        assert got.is_contiguous()
        if x.numel():
            check_forward(rows(tokens_first(got, first), s), rows(x, s),
                          None if w is None else f64(w), s, rot, inter, dtype)
    assert fa.device_status() == 0


@pytest.mark.parametrize("fused,pad", [(True, 0), (True, 3), (False, 0)])
def test_strides(cuda_device, fused, pad):
    s = make(77, (2, 19), 6, 2, 128, 128, 1, torch.bfloat16, cuda_device, fused=fused, pad=pad)
    q, k = fa.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], *s["args"], heads_first=False)
    check_forward(rows(q, s), rows(s["q"], s), f64(s["wq"]), s, 128, False, torch.bfloat16)
    check_forward(rows(k, s), rows(s["k"], s), f64(s["wk"]), s, 128, False, torch.bfloat16)
    # an order that the kernel cannot read in place is copied first
    qt = s["q"].transpose(1, 2).contiguous().transpose(1, 2)
    q2, _ = fa.qk_norm_rope(qt, s["k"], s["wq"], s["wk"], *s["args"], heads_first=False)
    assert torch.equal(q, q2)
    one = s["q"][:, :1].expand(2, 19, 6, 128)                # a broadcast token
    q3, _ = fa.qk_norm_rope(one, s["k"], s["wq"], s["wk"], *s["args"], heads_first=False)
    q4, _ = fa.qk_norm_rope(one.contiguous(), s["k"], s["wq"], s["wk"], *s["args"],
                            heads_first=False)
    assert torch.equal(q3, q4)


def test_zero_rows_and_large_values(cuda_device):
    s = make(5, (1, 4), 4, 1, 64, 64, 1, torch.float16, cuda_device, fused=False)
    s["q"][0, 0] = 0
    s["q"][0, 1] = 60000
    s["q"][0, 2] = 2.0 ** -24
    q, _ = fa.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], *s["args"], heads_first=False)
    assert torch.all(q[0, 0] == 0)
    check_forward(rows(q, s), rows(s["q"], s), f64(s["wq"]), s, 64, False, torch.float16)


def test_not_a_number_stays_in_its_row(cuda_device):
    s = make(6, (1, 9), 5, 2, 128, 128, 1, torch.bfloat16, cuda_device, fused=False)
    clean, _ = fa.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], *s["args"], heads_first=False)
    s["q"][0, 3, 2, 7] = float("nan")
    s["q"][0, 5, 1, 9] = float("inf")
    got, _ = fa.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], *s["args"], heads_first=False)
    assert torch.isnan(got[0, 3, 2]).all() and torch.isnan(got[0, 5, 1]).any()
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[0, 3, 2] = keep[0, 5, 1] = False
    assert torch.equal(got[keep], clean[keep])


def test_positions_and_axes_out_of_range_count_as_zero(cuda_device):
    for axes in (1, 2):
        s = make(8 + axes, (1, 20), 4, 2, 128, 128, axes, torch.bfloat16, cuda_device)
        s["args"][1][0, 3] = -1
        s["args"][1][0, 7] = 50
        s["pos"][0, [3, 7]] = 0
        if axes > 1:
            s["args"][2][5] = 9
            s["axis"][5] = 0
        q, _ = fa.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], *s["args"], heads_first=False)
        check_forward(rows(q, s), rows(s["q"], s), f64(s["wq"]), s, 128, False, torch.bfloat16)
        assert fa.device_status() == 5


def check_backward(dx, x, w, dy, s, rot, inter, dtype):
    R = oracle.rotation(s["table"], s["pos"], s["axis"], s["D"], inter)
    want, want_dw = oracle.norm_rope_backward(x, w, R, dy, EPS)
    ga = partner_abs(dy, rot, inter)
    if w is None:
        err = 2.0 ** -22 * ga
    else:
        rstd = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
        xh = np.abs(x * rstd)
        wga = np.abs(w) * ga
        err = 2.0 ** -18 * rstd * (wga + xh * (wga * xh).mean(-1, keepdims=True))
    bad = np.abs(dx - want) - half_step(want, err, dtype)
    assert (bad <= 0).all(), bad.max()
    if w is None:
        return None, None
    return want_dw, 2.0 ** -16 * (ga * xh).sum((0, 1))


@pytest.mark.parametrize("lead,Hq,Hkv,D,rot,axes,inter,first,dtype", CASES + [
    ((1, 1500), 32, 8, 128, 128, 1, False, True, torch.bfloat16),
    ((2, 700), 4, 1, 64, 32, 2, True, True, torch.float16),
])
@pytest.mark.parametrize("weights", ["both", "none", "k"])
def test_backward(cuda_device, lead, Hq, Hkv, D, rot, axes, inter, first, dtype, weights):
    s = make(sum(lead) + Hq + 1, lead, Hq, Hkv, D, rot, axes, dtype, cuda_device)
    gen = torch.Generator().manual_seed(9)
    wq = s["wq"] if weights == "both" else None
    wk = None if weights == "none" else s["wk"]
    grads = [torch.randn(*lead, H, D, generator=gen).to(dtype).to(cuda_device) for H in (Hq, Hkv)]
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(
        s["q"], s["k"], *(tokens_first(g, first).contiguous() for g in grads), wq, wk, *s["args"],
        eps=EPS, interleaved=inter, heads_first=first)
    for dx, dw, x, w, dy in ((dq, dwq, s["q"], wq, grads[0]), (dk, dwk, s["k"], wk, grads[1])):
        assert (dw is None) == (w is None)
        if not x.numel():
            assert dw is None or torch.all(dw == 0)
            continue
        want, lim = check_backward(rows(dx, s), rows(x, s), None if w is None else f64(w),
                                   rows(dy, s), s, rot, inter, dtype)
        if w is not None:
            assert dw.dtype == torch.float32
            assert (np.abs(f64(dw) - want) <= lim).all()
    assert fa.device_status() == 0


def test_backward_gradients_match_differences(cuda_device):
    """Central differences of the kernels' own fp16 forward, x moved by h = 2^-3 either
    way, the loss summed in fp64.  The 64 outputs of the row, of at most 8, are each off
    by at most 2^-11 of themselves at either point; the third-order term is below h^2
    times the row's sum of |dy| (derivatives in x / |x| of order 1)."""
    s = make(21, (1, 3), 2, 1, 64, 64, 1, torch.float16, cuda_device, fused=False)
    dy = torch.randn(1, 3, 2, 64, generator=torch.Generator().manual_seed(4)).half().to(cuda_device)
    dyk = torch.zeros(1, 3, 1, 64, dtype=torch.float16, device=cuda_device)
    dq, _, _, _ = fa.qk_norm_rope_backward(s["q"], s["k"], dy, dyk, s["wq"], s["wk"], *s["args"],
                                           heads_first=False)

    def loss(q):
        y, _ = fa.qk_norm_rope(q, s["k"], s["wq"], s["wk"], *s["args"], heads_first=False)
        return float((y.double() * dy.double()).sum())

    h = 2.0 ** -3
    for at in [(0, 0, 0, 0), (0, 1, 1, 31), (0, 2, 0, 32), (0, 2, 1, 63)]:
        up, down = s["q"].clone(), s["q"].clone()
        up[at] += h
        down[at] -= h
        step = float(up[at].double() - down[at].double())
        diff = (loss(up) - loss(down)) / step
        row_dy = dy[at[0], at[1], at[2]].double().abs().sum().item()
        # roundings of the 64 outputs, each at most 2^-11 * 8, at two points; third order
        assert abs(diff - float(dq[at])) <= 2 * row_dy * 8 * 2.0 ** -11 / step + row_dy * h * h


def test_backward_is_deterministic_and_captures(cuda_device):
    s = make(31, (1, 700), 8, 2, 128, 128, 1, torch.bfloat16, cuda_device)
    dy = [torch.randn(1, H, 700, 128, device=cuda_device).bfloat16() for H in (8, 2)]
    args = (s["q"], s["k"], *dy, s["wq"], s["wk"], *s["args"])
    first = fa.qk_norm_rope_backward(*args)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = fa.qk_norm_rope_backward(*args)
    for _ in range(3):
        graph.replay()
        for a, b in zip(first, out):
            assert torch.equal(a, b)
    dy[0].mul_(2)
    graph.replay()
    again = fa.qk_norm_rope_backward(*args)
    for a, b in zip(again, out):
        assert torch.equal(a, b)


def test_backward_of_no_tokens_gives_zero_weight_gradients(cuda_device):
    s = make(32, (2, 0), 4, 2, 128, 128, 1, torch.bfloat16, cuda_device)
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(
        s["q"], s["k"], torch.empty(2, 4, 0, 128, dtype=torch.bfloat16, device=cuda_device),
        torch.empty(2, 2, 0, 128, dtype=torch.bfloat16, device=cuda_device), s["wq"], s["wk"],
        *s["args"])
    assert dq.numel() == 0 and torch.all(dwq == 0) and torch.all(dwk == 0)


# ---------------------------------------------------------------------- append
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,axes,inter", [
    (1, 8, 2, 128, 128, 1, False), (64, 32, 8, 128, 128, 1, False), (37, 7, 1, 128, 64, 3, True),
    (301, 5, 5, 64, 64, 1, True), (50, 4, 3, 64, 48, 2, False), (19, 0, 4, 128, 128, 1, False),
    (19, 4, 0, 128, 0, 1, False)])
@pytest.mark.parametrize("padded", [True, False])
def test_append(cuda_device, T, Hq, Hkv, D, rot, axes, inter, padded):
    s = make(T + Hq, (T,), Hq, Hkv, D, rot, axes, torch.bfloat16, cuda_device)
    pages = -(-T // 16) + 3
    gen = torch.Generator().manual_seed(T)
    kc, vc = (torch.randn(pages, 16, Hkv, D, generator=gen).bfloat16().to(cuda_device)
              for _ in range(2))
    kc0, vc0 = kc.clone(), vc.clone()
    slots = torch.randperm(pages * 16, generator=gen)[:T]
    if padded:                                               # padding rows among the others
        slots[T // 2::7] = -1
    live = (slots >= 0).numpy()
    q = fa.append_paged(s["q"], s["k"], s["v"], kc, vc, slots.to(cuda_device), s["wq"], s["wk"],
                        *s["args"], eps=EPS, interleaved=inter)
    sub = dict(s, T=int(live.sum()), pos=s["pos"][:, live])
    if Hq:
        check_forward(rows(q, s)[live], rows(s["q"], s)[live], f64(s["wq"]), sub, rot, inter,
                      torch.bfloat16)
    if Hkv:
        at = slots[slots >= 0].to(cuda_device)
        check_forward(f64(kc.view(-1, Hkv, D)[at]), rows(s["k"], s)[live], f64(s["wk"]), sub, rot,
                      inter, torch.bfloat16)
        assert torch.equal(vc.view(-1, Hkv, D)[at], s["v"][torch.tensor(live, device=cuda_device)])
        other = torch.ones(pages * 16, dtype=torch.bool, device=cuda_device)
        other[at] = False
        for c, c0 in ((kc, kc0), (vc, vc0)):
            assert torch.equal(c.view(-1, Hkv, D)[other], c0.view(-1, Hkv, D)[other])
    assert fa.device_status() == 0


def test_append_leaves_padding_rows_and_bad_slots_alone(cuda_device):
    s = make(41, (8,), 4, 2, 128, 128, 1, torch.bfloat16, cuda_device)
    kc = torch.zeros(2, 16, 2, 128, dtype=torch.bfloat16, device=cuda_device)
    vc = torch.zeros_like(kc)
    slots = torch.tensor([0, -1, 32, 5, -7, 2 ** 40, 31, 1], device=cuda_device)
    q = torch.full((8, 4, 128), 7.0, dtype=torch.bfloat16, device=cuda_device)
    pos = s["args"][1].clone()
    pos[0, 1] = 1 << 30                                      # a padding row's is not read
    fa.fa_append_paged(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["args"][0], pos, None, slots, q,
                       kc, vc, 8, 4, 2, 128, 16, 2, 8 * 128, 8 * 128, 8 * 128, 128, 50, 1, False,
                       EPS)
    assert fa.device_status() == 5                           # the slots behind the pool
    for t in (1, 2, 4, 5):
        assert torch.all(q[t] == 7)
    written = vc.view(32, 2, 128).ne(0).any(-1).any(-1)
    assert written.nonzero().ravel().tolist() == [0, 1, 5, 31]
    slots.fill_(-1)
    fa.fa_append_paged(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["args"][0], pos, None, slots, q,
                       kc, vc, 8, 4, 2, 128, 16, 2, 8 * 128, 8 * 128, 8 * 128, 128, 50, 1, False,
                       EPS)
    assert fa.device_status() == 0


def test_append_far_into_a_long_cache(cuda_device):
    """Slots whose byte offset passes 2^32."""
    pages, Hkv = 140000, 8
    kc = torch.empty(pages, 16, Hkv, 128, dtype=torch.bfloat16, device=cuda_device)
    vc = torch.empty_like(kc)
    s = make(43, (5,), 8, Hkv, 128, 128, 1, torch.bfloat16, cuda_device)
    slots = torch.tensor([pages * 16 - 1, 3, 1 << 20, (1 << 21) + 17, pages * 16 - 16],
                         device=cuda_device)
    fa.append_paged(s["q"], s["k"], s["v"], kc, vc, slots, s["wq"], s["wk"], *s["args"])
    check_forward(f64(kc.view(-1, Hkv, 128)[slots]), rows(s["k"], s), f64(s["wk"]), s, 128, False,
                  torch.bfloat16)
    assert torch.equal(vc.view(-1, Hkv, 128)[slots], s["v"])
    assert fa.device_status() == 0
