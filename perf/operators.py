"""Workloads of the serving and training operators around the attention kernels.

Each case is one call of one operator at a size that a program makes:

  extend   pages, positions and cache slots of a step's new tokens, from request lengths
  append   per-head RMS norm and rotation of q and k, with K and V written to the page pool
  rope     the same norm and rotation for training (no cache), outputs as attention takes them
  rope_bwd its backward pass
  prefix   one query per sequence over a paged cache whose first pages the whole batch shares

``run`` computes a case in plain torch operations, in 32 bits, rounded once at the
end; with ``own`` set it calls the library instead.  ``exact`` computes it in 64
bits, sequence by sequence or element by element from the definition.
"""
import math

import torch

own = False

PAGE = 16
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 64 requests: every length grows by one token; launch latency
        dict(name="extend_decode_b64", op="extend", B=64, lo=512, hi=8191, new_lo=1, new_hi=1,
             max_pages=512, num_pages=40000),
        # a prefill step of many ragged requests, some new, some continued; ~131 k tokens
        dict(name="extend_prefill_b301", op="extend", B=301, lo=0, hi=4096, new_lo=1, new_hi=871,
             max_pages=320, num_pages=100000),
        # the projections of one decode step of 64 requests; launch latency
        dict(name="append_decode_t64", op="append", T=64, Hq=32, Hkv=8, D=128, rot=128,
             inter=False, axes=1, max_pos=8192, num_pages=2048),
        # a step of chunked prefill (16 chunks of 512, one token short)
        dict(name="append_chunks_t8191", op="append", T=8191, Hq=32, Hkv=8, D=128, rot=128,
             inter=False, axes=1, max_pos=8192, num_pages=1024),
        # training forward at the headline sequence
        dict(name="rope_train_n8192", op="rope", dtype="bf16", B=1, N=8192, Hq=32, Hkv=8, D=128,
             rot=128, inter=False, axes=1, max_pos=8192),
        # image and video tokens: three axes, fp16, heads of 64, an odd length
        dict(name="rope_axes_fp16_d64", op="rope", dtype="fp16", B=2, N=4093, Hq=8, Hkv=8, D=64,
             rot=64, inter=False, axes=3, max_pos=4096),
        # training backward at the headline sequence
        dict(name="rope_bwd_n8192", op="rope_bwd", dtype="bf16", B=1, N=8192, Hq=32, Hkv=8, D=128,
             rot=128, inter=False, axes=1, max_pos=8192),
        # a small fp16 batch, half of each head rotated in adjacent pairs, two axes
        dict(name="rope_bwd_small_fp16", op="rope_bwd", dtype="fp16", B=3, N=333, Hq=8, Hkv=2,
             D=128, rot=64, inter=True, axes=2, max_pos=512),
        # few requests after a short system prompt; launch latency
        dict(name="prefix_b7_p1040", op="prefix", B=7, Hq=8, Hkv=2, prefix=65, suffix=200),
        # a decode batch whose requests share the first half of a long prompt
        dict(name="prefix_b64_p4096", op="prefix", B=64, Hq=32, Hkv=8, prefix=256, suffix=4096),
        # no grouped heads, more KV heads than the streamed decode takes, a ragged prefix
        dict(name="prefix_mha_b33_p4000", op="prefix", B=33, Hq=16, Hkv=16, prefix=250,
             suffix=301),
        # many samples of one long document
        dict(name="prefix_b256_p32768", op="prefix", B=256, Hq=32, Hkv=8, prefix=2048, suffix=512),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["extend", "append", "rope", "rope_bwd", "prefix"])
    if op == "extend":
        B = _log_int(rng, 1, 600)
        new_hi = _log_int(rng, 1, max(1, 250000 // B))
        hi = _log_int(rng, 1, 8191)
        max_pages = -(-(hi + new_hi) // PAGE) + rng.randint(0, 40)
        return dict(op=op, B=B, lo=rng.choice([0, hi // 16]), hi=hi, new_lo=rng.choice([0, 1]),
                    new_hi=new_hi, max_pages=max_pages, num_pages=B * max_pages + rng.randint(0, 999))
    if op == "prefix":
        Hkv, G = rng.choice([(8, 4), (8, 1), (4, 8), (2, 2), (1, 8), (16, 1), (10, 2)])
        B = _log_int(rng, 1, 256)
        rows = B * Hkv * G
        prefix = _log_int(rng, 1, max(2, min(2048, 256 * 32 * 2048 // rows)))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, prefix=prefix,
                    suffix=_log_int(rng, 1, max(2, min(4096, 64 * 4096 // B))))
    D = rng.choice([64, 128])
    Hkv, G = rng.choice([(9, 4), (6, 1), (4, 7), (2, 8), (1, 8), (5, 3)])
    rot = rng.choice([D, D, D // 2, D // 4, 48])
    T = _log_int(rng, 1, 8192 * 40 * 128 // ((G + 1) * Hkv * D))
    common = dict(op=op, Hq=Hkv * G, Hkv=Hkv, D=D, rot=rot, inter=rng.random() < 0.4,
                  axes=rng.choice([1, 1, 2, 3]))
    if op == "append":
        T = min(T, 8191)
        return dict(common, T=T, max_pos=rng.choice([2048, 32768]),
                    num_pages=-(-T // PAGE) + rng.randint(1, 500))
    B = rng.choice([1, 1, 2, 3])
    return dict(common, dtype=rng.choice(["bf16", "fp16"]), B=B, N=max(1, T // B),
                max_pos=rng.choice([2048, 32768]))


def work(case):
    op = case["op"]
    if op == "extend":
        B, new = case["B"], (case["new_lo"] + case["new_hi"]) / 2
        tokens = B * new
        # lengths in and out, offsets, one table entry and 12 bytes for each token row
        return {"bytes": B * 20 + tokens / PAGE * 8 + B * case["new_hi"] * 12, "flops": tokens * 4}
    Hq, Hkv = case["Hq"], case["Hkv"]
    if op == "prefix":
        B, D = case["B"], 128
        own_keys = B * (case["suffix"] + 1) / 2
        keys = case["prefix"] * PAGE + own_keys
        rows = B * Hq
        return {"bytes": keys * Hkv * D * 4 + rows * (D * 4 + 4),
                "flops": 4 * rows * D * case["prefix"] * PAGE + 4 * own_keys * Hq * D}
    D = case["D"]
    T = case["T"] if op == "append" else case["B"] * case["N"]
    rows = T * (Hq + Hkv)
    side = T * case["axes"] * 4 + min(case["max_pos"], T) * case["rot"] * 4
    if op == "rope_bwd":
        return {"bytes": rows * D * 6 + side, "flops": rows * D * 20}
    copied = T * Hkv * D * 4 + T * 8 if op == "append" else 0
    return {"bytes": rows * D * 4 + copied + side, "flops": rows * D * 8}


# ------------------------------------------------------------------------ inputs
def _rotary_table(max_pos, rot, dev):
    """[max_pos, rot] fp32: the cosines of the pairs, then their sines."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / max(rot, 1))
    ang = torch.arange(max_pos, dtype=torch.float64, device=dev)[:, None] * inv[None, :]
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def _pages_for(gen, dev, lens, max_pages, num_pages):
    """A block table of scattered pages for lens tokens, and the ids left over."""
    perm = torch.randperm(num_pages, generator=gen, device=dev).to(torch.int32)
    need = (lens + PAGE - 1) // PAGE
    start = need.cumsum(0) - need
    j = torch.arange(max_pages, device=dev)
    idx = (start[:, None] + j[None, :]).clamp(max=num_pages - 1)
    table = torch.where(j[None, :] < need[:, None], perm[idx], torch.zeros_like(perm[idx]))
    used = int(need.sum())
    return table.to(torch.int32).contiguous(), perm, used


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]

    def ints(lo, hi, n):
        return torch.randint(lo, hi + 1, (n,), generator=gen, device=dev)

    def normal(*shape, dtype):
        return torch.randn(shape, generator=gen, device=dev, dtype=dtype)

    if op == "extend":
        B = case["B"]
        lens = ints(case["lo"], case["hi"], B)
        new = ints(case["new_lo"], case["new_hi"], B)
        table, perm, used = _pages_for(gen, dev, lens, case["max_pages"], case["num_pages"])
        free = torch.zeros_like(perm)
        free[:case["num_pages"] - used] = perm[used:]
        return dict(case=case, table=table, lens=lens.to(torch.int32), new=new.to(torch.int32),
                    free=free, count=torch.tensor([case["num_pages"] - used], dtype=torch.int32,
                                                  device=dev),
                    max_tokens=B * case["new_hi"], num_pages=case["num_pages"])
    Hq, Hkv = case["Hq"], case["Hkv"]
    if op == "prefix":
        B, P, D = case["B"], case["prefix"], 128
        own_len = ints(1, case["suffix"], B)
        own_max = -(-case["suffix"] // PAGE)
        num_pages = P + B * own_max + 1
        own_table, perm, used = _pages_for(gen, dev, own_len, own_max, num_pages)
        shared = perm[used:used + P]
        table = torch.cat([shared[None, :].expand(B, P), own_table], 1).contiguous()
        shape = (num_pages, PAGE, Hkv, D)
        return dict(case=case, q=normal(B, Hq, D, dtype=torch.bfloat16),
                    kc=normal(*shape, dtype=torch.bfloat16), vc=normal(*shape, dtype=torch.bfloat16),
                    table=table, lens=(own_len + P * PAGE).to(torch.int32), shared=shared.contiguous(),
                    pages=torch.tensor([P], dtype=torch.int32, device=dev), scale=D ** -0.5)
    D, rot, axes = case["D"], case["rot"], case["axes"]
    dt = DTYPES[case.get("dtype", "bf16")]
    lead = (case["T"],) if op == "append" else (case["B"], case["N"])
    T = math.prod(lead)
    heads = Hq + 2 * Hkv
    qkv = normal(*lead, heads, D, dtype=dt)          # the projection, q | k | v by heads
    s = dict(case=case, q=qkv[..., :Hq, :], k=qkv[..., Hq:Hq + Hkv, :], v=qkv[..., Hq + Hkv:, :],
             wq=(1 + 0.1 * normal(D, dtype=torch.float32)).to(dt),
             wk=(1 + 0.1 * normal(D, dtype=torch.float32)).to(dt),
             rows=_rotary_table(case["max_pos"], rot, dev), eps=1e-6)
    s["pos"] = ints(0, case["max_pos"] - 1, axes * T).to(torch.int32).view(axes, T)
    if op != "append" and axes == 1:                 # training: positions run along the sequence
        s["pos"] = (torch.arange(T, device=dev) % case["N"] % case["max_pos"]).to(torch.int32)[None]
    s["axis"] = None
    if axes > 1:                                     # contiguous sections of the pairs
        s["axis"] = (torch.arange(rot // 2, device=dev) * axes // (rot // 2)).to(torch.uint8)
    if op == "append":
        slots = torch.randperm(case["num_pages"] * PAGE, generator=gen, device=dev)[:T]
        shape = (case["num_pages"], PAGE, Hkv, D)
        s.update(slots=slots.to(torch.int64), kc=normal(*shape, dtype=dt), vc=normal(*shape, dtype=dt))
    if op == "rope_bwd":
        B, N = lead
        s.update(dq=normal(B, Hq, N, D, dtype=dt), dk=normal(B, Hkv, N, D, dtype=dt))
    return s


# ------------------------------------------------------------------------ plain forms
def _extend_plain(s):
    table, lens, new = s["table"], s["lens"].long(), s["new"].long()
    dev, max_pages, max_tokens = table.device, table.shape[1], s["max_tokens"]
    count = s["count"].long()
    first, last = (lens + PAGE - 1) // PAGE, (lens + new + PAGE - 1) // PAGE
    need = last - first
    fits = (lens + new <= max_pages * PAGE)
    need, new = need * fits, new * fits
    ends, tokens = need.cumsum(0), new.cumsum(0)
    admit = (ends <= count) & (tokens <= max_tokens)
    need, new = need * admit, new * admit
    before = ends - need
    j = torch.arange(max_pages, device=dev)
    rank = count - 1 - (before[:, None] + j[None, :] - first[:, None])
    mine = (j[None, :] >= first[:, None]) & (j[None, :] < (first + need)[:, None])
    got = s["free"][rank.clamp(0, s["free"].numel() - 1)]
    table.copy_(torch.where(mine, got, table))
    cu = torch.zeros(lens.numel() + 1, dtype=torch.int64, device=dev)
    cu[1:] = new.cumsum(0)
    t = torch.arange(max_tokens, device=dev)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=lens.numel() - 1)
    live = t < cu[-1]
    pos = torch.where(live, lens[b] + t - cu[b], torch.zeros_like(t))
    slot = table[b, pos // PAGE].long() * PAGE + pos % PAGE
    slot = torch.where(live, slot, torch.full_like(slot, -1))
    return dict(table=table, lens=(lens + new).to(torch.int32), cu=cu.to(torch.int32),
                pos=pos.to(torch.int32), slots=slot, count=(count - need.sum()).to(torch.int32))


def _angles(s, lead):
    """cos and sin [*lead, 1, rot/2] of every token's pairs."""
    half = s["rows"].shape[1] // 2
    pos = s["pos"].long()
    if s["axis"] is None:
        rows = s["rows"][pos[0]]
        cos, sin = rows[:, :half], rows[:, half:]
    else:
        at = pos[s["axis"].long()].T                 # [T, rot/2]: the row of each pair
        cos, sin = s["rows"][:, :half].gather(0, at), s["rows"][:, half:].gather(0, at)
    return cos.view(*lead, 1, half), sin.view(*lead, 1, half)


def _split(x, rot, inter):
    if inter:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def _join(a, b, rest, inter):
    turned = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([turned, rest], -1)


def _norm_rotate(x, w, cos, sin, rot, inter, eps):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()
    a, b = _split(y, rot, inter)
    return _join(a * cos - b * sin, b * cos + a * sin, y[..., rot:], inter)


def _norm_rotate_bwd(x, w, dy, cos, sin, rot, inter, eps):
    x, w = x.float(), w.float()
    dy = dy.float().transpose(1, 2)                  # [B, N, H, D]
    a, b = _split(dy, rot, inter)
    g = _join(a * cos + b * sin, b * cos - a * sin, dy[..., rot:], inter)
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    xhat = x * rstd
    dw = (g * xhat).double().flatten(0, -2).sum(0).float()
    g = g * w
    return rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True)), dw


def _rope_plain(s):
    c = s["case"]
    lead = s["q"].shape[:-2]
    cos, sin = _angles(s, lead)
    dt = s["q"].dtype
    q = _norm_rotate(s["q"], s["wq"], cos, sin, c["rot"], c["inter"], s["eps"]).to(dt)
    k = _norm_rotate(s["k"], s["wk"], cos, sin, c["rot"], c["inter"], s["eps"]).to(dt)
    if c["op"] == "rope":
        return dict(q=q.transpose(1, 2).contiguous(), k=k.transpose(1, 2).contiguous())
    Hkv, D = c["Hkv"], c["D"]
    s["kc"].view(-1, Hkv, D)[s["slots"]] = k
    s["vc"].view(-1, Hkv, D)[s["slots"]] = s["v"]
    return dict(q=q, kc=s["kc"], vc=s["vc"])


def _rope_bwd_plain(s):
    c = s["case"]
    cos, sin = _angles(s, s["q"].shape[:-2])
    dt = s["q"].dtype
    dq, dwq = _norm_rotate_bwd(s["q"], s["wq"], s["dq"], cos, sin, c["rot"], c["inter"], s["eps"])
    dk, dwk = _norm_rotate_bwd(s["k"], s["wk"], s["dk"], cos, sin, c["rot"], c["inter"], s["eps"])
    return dict(dq=dq.to(dt), dk=dk.to(dt), dwq=dwq, dwk=dwk)


def _prefix_plain(s):
    c = s["case"]
    q, lens, table = s["q"], s["lens"].long(), s["table"].long()
    B, Hq, D = q.shape
    Hkv, P = c["Hkv"], c["prefix"]
    G = Hq // Hkv
    qg = q.float().view(B, Hkv, G, D) * s["scale"]
    # all rows of a KV head against the shared keys at once
    kp = s["kc"][s["shared"].long()].view(-1, Hkv, D).float().permute(1, 2, 0)       # [Hkv, D, n]
    vp = s["vc"][s["shared"].long()].view(-1, Hkv, D).float().transpose(0, 1)        # [Hkv, n, D]
    s1 = torch.matmul(qg.transpose(0, 1).reshape(Hkv, B * G, D), kp).view(Hkv, B, G, -1)
    s1 = s1.transpose(0, 1)                                                          # [B, Hkv, G, n]
    # each row against its own keys, padded to the longest
    ks = s["kc"][table[:, P:]].view(B, -1, Hkv, D).float().permute(0, 2, 3, 1)       # [B, Hkv, D, S]
    vs = s["vc"][table[:, P:]].view(B, -1, Hkv, D).float().transpose(1, 2)           # [B, Hkv, S, D]
    s2 = torch.matmul(qg, ks)
    behind = torch.arange(s2.shape[-1], device=q.device)[None, :] >= (lens - P * PAGE)[:, None]
    s2 = s2.masked_fill(behind[:, None, None, :], float("-inf"))
    m = torch.maximum(s1.amax(-1, keepdim=True), s2.amax(-1, keepdim=True))
    p1, p2 = (s1 - m).exp(), (s2 - m).exp()
    total = p1.sum(-1, keepdim=True) + p2.sum(-1, keepdim=True)
    o1 = torch.matmul(p1.transpose(0, 1).reshape(Hkv, B * G, -1), vp).view(Hkv, B, G, D)
    o = (o1.transpose(0, 1) + torch.matmul(p2, vs)) / total
    lse = (m + total.log()).squeeze(-1)
    return dict(o=o.reshape(B, Hq, D).to(q.dtype), lse=lse.reshape(B, Hq))


# ------------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        plain = dict(extend=_extend_plain, append=_rope_plain, rope=_rope_plain,
                     rope_bwd=_rope_bwd_plain, prefix=_prefix_plain)
        return plain[op](s)
    from exact_tiled_attention_40_b200 import fa
    if op == "extend":
        lens, cu, pos, slots, count = fa.extend_pages(s["table"], s["lens"], s["new"], s["free"],
                                                      s["count"], s["num_pages"], s["max_tokens"])
        return dict(table=s["table"], lens=lens, cu=cu, pos=pos, slots=slots, count=count)
    if op == "prefix":
        o, lse = fa.decode_shared_prefix(s["q"], s["kc"], s["vc"], s["table"], s["lens"],
                                         s["shared"], s["pages"], scale=s["scale"])
        return dict(o=o, lse=lse)
    if op == "append":
        q = fa.append_paged(s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"], s["wq"], s["wk"],
                            s["rows"], s["pos"], s["axis"], eps=s["eps"], interleaved=c["inter"])
        return dict(q=q, kc=s["kc"], vc=s["vc"])
    if op == "rope":
        q, k = fa.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["rows"], s["pos"], s["axis"],
                               eps=s["eps"], interleaved=c["inter"], heads_first=True)
        return dict(q=q, k=k)
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(
        s["q"], s["k"], s["dq"], s["dk"], s["wq"], s["wk"], s["rows"], s["pos"], s["axis"],
        eps=s["eps"], interleaved=c["inter"], heads_first=True)
    return dict(dq=dq, dk=dk, dwq=dwq, dwk=dwk)


# ------------------------------------------------------------------------ 64 bits
def _extend_exact(s):
    table, lens, new = s["table"].tolist(), s["lens"].tolist(), s["new"].tolist()
    free, count = s["free"].tolist(), int(s["count"])
    out_lens, cu, pos, slots = [], [0], [], []
    for b, (have, more) in enumerate(zip(lens, new)):
        for t in range(have, have + more):
            if t % PAGE == 0:
                count -= 1
                table[b][t // PAGE] = free[count]
            pos.append(t)
            slots.append(table[b][t // PAGE] * PAGE + t % PAGE)
        out_lens.append(have + more)
        cu.append(len(pos))
    pad = s["max_tokens"] - len(pos)
    return dict(table=torch.tensor(table, dtype=torch.int32), lens=torch.tensor(out_lens, dtype=torch.int32),
                cu=torch.tensor(cu, dtype=torch.int32), pos=torch.tensor(pos + [0] * pad, dtype=torch.int32),
                slots=torch.tensor(slots + [-1] * pad, dtype=torch.int64),
                count=torch.tensor([count], dtype=torch.int32))


def _rotation(s, T, D):
    """Per token the partner element of each element, and the 64-bit factors of both."""
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    d = torch.arange(D, device=s["q"].device)
    if c["inter"]:
        pair, upper, partner = d // 2, d % 2 == 1, d ^ 1
    else:
        pair, upper = d % max(half, 1), d >= half
        partner = torch.where(upper, d - half, d + half)
    inside = d < rot
    pair, partner = torch.where(inside, pair, 0), torch.where(inside, partner, d)
    axis = s["axis"].long()[pair] if s["axis"] is not None else torch.zeros_like(pair)
    row = s["pos"].long()[axis].T                                        # [T, D]
    cos = torch.where(inside, s["rows"].double()[row, pair], 1.0)
    sin = torch.where(inside, s["rows"].double()[row, half + pair], 0.0)
    return partner, cos, torch.where(upper, sin, -sin)


def _rope_exact(s):
    c = s["case"]
    D, lead = c["D"], s["q"].shape[:-2]
    T = math.prod(lead)
    partner, cos, sin = _rotation(s, T, D)

    def one(x, w):
        x = x.reshape(T, -1, D).double()
        y = x / (x.pow(2).sum(-1, keepdim=True) / D + s["eps"]).sqrt() * w.double()
        return y * cos[:, None] + y[..., partner] * sin[:, None]

    q, k = one(s["q"], s["wq"]), one(s["k"], s["wk"])
    if c["op"] == "rope":
        return dict(q=q.view(*lead, -1, D).transpose(1, 2).contiguous(),
                    k=k.view(*lead, -1, D).transpose(1, 2).contiguous())
    kc, vc = s["kc"].double(), s["vc"].double()
    kc.view(-1, *k.shape[1:]).index_copy_(0, s["slots"], k)
    vc.view(-1, *k.shape[1:]).index_copy_(0, s["slots"], s["v"].double())
    return dict(q=q, kc=kc, vc=vc)


def _rope_bwd_exact(s):
    """Through autograd of the definition in 64 bits."""
    D, lead = s["case"]["D"], s["q"].shape[:-2]
    T = math.prod(lead)
    partner, cos, sin = _rotation(s, T, D)
    out = {}
    for n, x, w, dy in (("q", s["q"], s["wq"], s["dq"]), ("k", s["k"], s["wk"], s["dk"])):
        x = x.double().requires_grad_()
        w = w.double().requires_grad_()
        y = x * (x.square().mean(-1, keepdim=True) + s["eps"]) ** -0.5 * w
        y = y * cos.view(*lead, 1, D) + y[..., partner] * sin.view(*lead, 1, D)
        out["d" + n], out["dw" + n] = torch.autograd.grad(y, (x, w), dy.double().transpose(1, 2))
    return out


def _prefix_exact(s):
    """Sequence by sequence over its whole block table row."""
    c = s["case"]
    B, Hq, D = s["q"].shape
    Hkv = c["Hkv"]
    o, lse = [], []
    for b, n in enumerate(s["lens"].tolist()):
        pages = s["table"][b, :-(-n // PAGE)].long()
        k = s["kc"][pages].reshape(-1, Hkv, D)[:n].double().transpose(0, 1)
        v = s["vc"][pages].reshape(-1, Hkv, D)[:n].double().transpose(0, 1)
        q = s["q"][b].double().view(Hkv, Hq // Hkv, D)
        z = torch.bmm(q, k.transpose(1, 2)) * s["scale"]
        lse.append(torch.logsumexp(z, -1).reshape(Hq))
        o.append(torch.bmm(torch.softmax(z, -1), v).reshape(Hq, D))
    return dict(o=torch.stack(o), lse=torch.stack(lse))


def exact(case, seed):
    s = prepare(case, seed)
    return dict(extend=_extend_exact, append=_rope_exact, rope=_rope_exact,
                rope_bwd=_rope_bwd_exact, prefix=_prefix_exact)[case["op"]](s)
