"""Host validation of the operators around attention (no kernel is launched) and the
binding's own checks."""
import pytest
import torch

from exact_tiled_attention_40_b200 import fa

E = {v: k for k, v in fa.STATUS.items()}
FAKE = 0x1000000         # 16-byte aligned fake addresses, far apart; never dereferenced


def at(i):
    return FAKE + (i << 32)


@pytest.fixture(scope="module")
def lib():
    return fa.lib()


# The calls without a fault pass validation: on a machine with a GPU they would launch
# kernels on the fake addresses, so they are made only where no device exists.
NO_DEVICE_ONLY = pytest.mark.skipif(torch.cuda.is_available(),
                                    reason="fake pointers must never reach a device")
INVALID, UNSUPPORTED = E["FA_ERR_INVALID_ARG"], E["FA_ERR_UNSUPPORTED"]


def rope(lib, fp16=False, q=at(1), k=at(2), wq=at(3), wk=at(4), table=at(5), pos=at(6), axis=None,
         qo=at(7), ko=at(8), B=2, N=5, Hq=4, Hkv=2, D=128, qs=512, ks=256, rot=128, maxp=10, axes=1,
         inter=0, first=1, eps=1e-6):
    fn = lib.fa_qk_norm_rope_fp16 if fp16 else lib.fa_qk_norm_rope
    return fn(q, k, wq, wk, table, pos, axis, qo, ko, B, N, Hq, Hkv, D, qs, ks, rot, maxp, axes,
              inter, first, eps, None)


ROPE_BAD = [
    (dict(B=-1), INVALID), (dict(N=-1), INVALID), (dict(Hq=-1), INVALID), (dict(Hkv=-4), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(rot=8), UNSUPPORTED), (dict(rot=144), UNSUPPORTED),
    (dict(rot=-16), UNSUPPORTED), (dict(axes=0), UNSUPPORTED), (dict(axes=9), UNSUPPORTED),
    (dict(axes=2), INVALID), (dict(maxp=0), INVALID), (dict(table=None), INVALID),
    (dict(pos=None), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(q=at(1) + 8), INVALID),
    (dict(wq=at(3) + 2), INVALID), (dict(table=at(5) + 4), INVALID), (dict(pos=at(6) + 2), INVALID),
    (dict(qs=504), INVALID), (dict(ks=260), INVALID), (dict(qs=1 << 33), INVALID),
    (dict(B=1 << 15, N=1 << 15), UNSUPPORTED),
]
ROPE_OUT_BAD = [(dict(qo=None), INVALID), (dict(ko=None), INVALID), (dict(qo=at(1)), INVALID),
                (dict(ko=at(1) + 64), INVALID), (dict(ko=at(7) + 16), INVALID)]


@pytest.mark.parametrize("kw,code", ROPE_BAD + ROPE_OUT_BAD)
@pytest.mark.parametrize("fp16", [False, True])
def test_norm_rope_rejects(lib, kw, code, fp16):
    assert rope(lib, fp16, **kw) == code
    assert lib.fa_last_error_string()


def test_norm_rope_of_nothing(lib):
    assert rope(lib, B=0) == 0 and rope(lib, N=0, q=None, table=None, pos=None) == 0
    assert rope(lib, Hq=0, Hkv=0) == 0


@NO_DEVICE_ONLY
def test_norm_rope_accepts(lib):
    none = E["FA_ERR_NO_DEVICE"]
    assert rope(lib) == none
    assert rope(lib, wq=None, wk=None, eps=0.0) == none
    assert rope(lib, rot=0, table=None, pos=None, maxp=0) == none
    assert rope(lib, k=at(1) + 1024, qs=1024, ks=1024) == none       # one projection
    assert rope(lib, axes=3, axis=at(9)) == none
    assert rope(lib, Hkv=0, k=None, ko=None, wk=None) == none


def rope_bwd(lib, fp16=False, q=at(1), k=at(2), dqo=at(11), dko=at(12), wq=at(3), wk=at(4),
             table=at(5), pos=at(6), axis=None, dq=at(7), dk=at(8), dwq=at(9), dwk=at(10),
             scratch=at(13), B=2, N=5, Hq=4, Hkv=2, D=128, qs=512, ks=256, dqs=512, dks=256,
             rot=128, maxp=10, axes=1, inter=0, first=1, eps=1e-6):
    fn = lib.fa_qk_norm_rope_bwd_fp16 if fp16 else lib.fa_qk_norm_rope_bwd
    return fn(q, k, dqo, dko, wq, wk, table, pos, axis, dq, dk, dwq, dwk, scratch, B, N, Hq, Hkv, D,
              qs, ks, dqs, dks, rot, maxp, axes, inter, first, eps, None)


@pytest.mark.parametrize("kw,code", ROPE_BAD + [
    (dict(dqo=None), INVALID), (dict(dko=at(12) + 4), INVALID), (dict(dq=None), INVALID),
    (dict(dk=None), INVALID), (dict(dqs=500), INVALID), (dict(dks=128), INVALID),
    (dict(dwq=None), INVALID), (dict(dwk=None), INVALID), (dict(scratch=None), INVALID),
    (dict(scratch=at(13) + 4), INVALID), (dict(dq=at(1)), INVALID), (dict(dk=at(11)), INVALID)])
@pytest.mark.parametrize("fp16", [False, True])
def test_norm_rope_backward_rejects(lib, kw, code, fp16):
    assert rope_bwd(lib, fp16, **kw) == code


@NO_DEVICE_ONLY
def test_norm_rope_backward_accepts(lib):
    none = E["FA_ERR_NO_DEVICE"]
    assert rope_bwd(lib) == none
    assert rope_bwd(lib, wq=None, wk=None, dwq=None, dwk=None, scratch=None) == none
    assert rope_bwd(lib, dk=at(7) + 1024, dqs=768, dks=768) == none  # one gradient
    assert rope_bwd(lib, N=0) == none                                # zero weight gradients
    assert rope_bwd(lib, N=0, wq=None, wk=None) == 0


def append(lib, q=at(1), k=at(2), v=at(3), wq=at(4), wk=at(5), table=at(6), pos=at(7), axis=None,
           slots=at(8), qo=at(9), kc=at(10), vc=at(11), T=5, Hq=4, Hkv=2, D=128, page=16, pages=9,
           qs=512, ks=256, vs=256, rot=128, maxp=10, axes=1, inter=0, eps=1e-6):
    return lib.fa_append_paged(q, k, v, wq, wk, table, pos, axis, slots, qo, kc, vc, T, Hq, Hkv, D,
                               page, pages, qs, ks, vs, rot, maxp, axes, inter, eps, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(pages=-1), INVALID), (dict(pages=0), INVALID),
    (dict(page=32), UNSUPPORTED), (dict(D=80), UNSUPPORTED), (dict(slots=None), INVALID),
    (dict(slots=at(8) + 4), INVALID), (dict(v=None), INVALID), (dict(vs=192), INVALID),
    (dict(kc=None), INVALID), (dict(vc=at(11) + 2), INVALID), (dict(vc=at(10) + 4096), INVALID),
    (dict(qo=at(10)), INVALID), (dict(kc=at(2)), INVALID), (dict(rot=24), UNSUPPORTED),
    (dict(axes=4), INVALID), (dict(eps=-1.0), INVALID)])
def test_append_rejects(lib, kw, code):
    assert append(lib, **kw) == code


@NO_DEVICE_ONLY
def test_append_accepts(lib):
    assert append(lib) == E["FA_ERR_NO_DEVICE"]
    assert append(lib, T=0, q=None) == 0


def extend(lib, table=at(1), lens=at(2), new=at(3), free=at(4), count=at(5), lens_out=at(6),
           left=at(7), cu=at(8), pos=at(9), slots=at(10), B=4, maxp=8, pages=20, page=16, tokens=9):
    return lib.fa_extend_pages(table, lens, new, free, count, lens_out, left, cu, pos, slots, B,
                               maxp, pages, page, tokens, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(tokens=-1), INVALID), (dict(pages=-1), INVALID),
    (dict(maxp=0), INVALID), (dict(pages=0), INVALID), (dict(page=8), UNSUPPORTED),
    (dict(B=16385), UNSUPPORTED), (dict(maxp=1 << 28), INVALID), (dict(pages=1 << 28), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(new=None), INVALID),
    (dict(free=None), INVALID), (dict(count=None), INVALID), (dict(lens_out=None), INVALID),
    (dict(left=None), INVALID), (dict(cu=None), INVALID), (dict(pos=None), INVALID),
    (dict(slots=None), INVALID), (dict(lens=at(2) + 2), INVALID), (dict(slots=at(10) + 4), INVALID)])
def test_extend_rejects(lib, kw, code):
    assert extend(lib, **kw) == code


def shared(lib, q=at(1), kc=at(2), vc=at(3), table=at(4), lens=at(5), prefix=at(6), pages=at(7),
           o=at(8), B=2, Hq=8, Hkv=2, D=128, page=16, scale=0.1, maxp=9, max_prefix=4, npages=20):
    return lib.fa_decode_shared_prefix(q, kc, vc, table, lens, prefix, pages, o, B, Hq, Hkv, D,
                                       page, scale, None, maxp, max_prefix, npages, None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=64), UNSUPPORTED), (dict(page=32), UNSUPPORTED), (dict(Hq=6), UNSUPPORTED),
    (dict(Hq=5), INVALID), (dict(B=-1), INVALID), (dict(maxp=0), INVALID), (dict(npages=0), INVALID),
    (dict(q=None), INVALID), (dict(table=None), INVALID), (dict(kc=at(2) + 8), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(max_prefix=-1), INVALID), (dict(max_prefix=10), INVALID), (dict(prefix=None), INVALID),
    (dict(pages=None), INVALID), (dict(prefix=at(6) + 2), INVALID)])
def test_shared_prefix_rejects(lib, kw, code):
    assert shared(lib, **kw) == code


@NO_DEVICE_ONLY
def test_shared_prefix_accepts(lib):
    assert shared(lib) == E["FA_ERR_NO_DEVICE"]
    assert shared(lib, max_prefix=0, prefix=None, pages=None) == E["FA_ERR_NO_DEVICE"]
    assert shared(lib, B=0) == 0


def test_the_binding_refuses_host_tensors():
    i = torch.zeros(2, 3, dtype=torch.int32)
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    w, tab = torch.zeros(64, dtype=torch.bfloat16), torch.zeros(4, 64)
    calls = [
        lambda: fa.extend_pages(i, i[0, :2], i[0, :2], i[0], i[0, :1], 3, 4),
        lambda: fa.qk_norm_rope(x, x, w, w, tab, i[:1, :2]),
        lambda: fa.qk_norm_rope_backward(x, x, x, x, w, w, tab, i[:1, :2]),
        lambda: fa.append_paged(x[0], x[0], x[0], x, x, i[0].long(), w, w, tab, i[:1, :2]),
        lambda: fa.decode_shared_prefix(x[0], x, x, i, i[0], i[0], i[0, :1]),
    ]
    for call in calls:
        with pytest.raises(fa.FAError, match="CUDA device"):
            call()


def test_head_rows_reads_views_in_place_and_copies_the_rest():
    x = torch.randn(2, 5, 8, 64).bfloat16()
    q = x[:, :, :4]
    head_rows = fa._native().head_rows
    t, stride = head_rows(q)
    assert t.data_ptr() == q.data_ptr() and t.stride() == q.stride() and stride == 512
    t, stride = head_rows(x[:, ::2, :4])                 # a step of two tokens
    assert stride == 256 and t.is_contiguous()
    t, stride = head_rows(x[:1, ::2, :4])
    assert t.data_ptr() == x.data_ptr() and stride == 1024
    t, stride = head_rows(x[:, :1, :4])                  # one token a batch row
    assert t.data_ptr() == x.data_ptr() and stride == 5 * 512
    for odd in (x.transpose(1, 2)[:, :4], x[..., :32], x[:, :1].expand(2, 5, 8, 64)):
        t, stride = head_rows(odd)
        assert t.is_contiguous() and torch.equal(t, odd)
        assert stride == odd.shape[-1] * odd.shape[-2]
    t, stride = head_rows(x.view(-1)[1:1 + 512 * 3].view(3, 8, 64))
    assert t.data_ptr() % 16 == 0 and stride == 512
    assert head_rows(x[:1, :1].expand(1, 1, 8, 64))[1] == 512
    assert head_rows(x[:, :0])[1] == 512
