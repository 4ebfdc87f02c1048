"""A call that could not launch reports so once: the calls after it do not inherit its
error.  The failure is the host's: a stream whose capture has been invalidated takes no
work, so nothing of the failing call reaches the GPU."""
import contextlib
import ctypes

import pytest
import torch

from exact_tiled_attention_40_b200 import fa

pytestmark = pytest.mark.gpu
CUDA = 3                 # FA_ERR_CUDA
RELAXED, NON_BLOCKING = 2, 1


@contextlib.contextmanager
def stream_that_takes_no_work():
    rt = ctypes.CDLL("libcudart.so.12")          # the one that torch has loaded
    s, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreateWithFlags(ctypes.byref(s), NON_BLOCKING) == 0
    assert rt.cudaStreamBeginCapture(s, RELAXED) == 0
    assert rt.cudaStreamSynchronize(s) != 0      # not allowed in a capture: invalidates it
    rt.cudaGetLastError()                        # (torch asks for it after its launches)
    try:
        yield s.value
    finally:
        assert rt.cudaStreamEndCapture(s, ctypes.byref(graph)) != 0
        assert rt.cudaStreamDestroy(s) == 0
        rt.cudaGetLastError()


def ints(n, dev, value=0):
    return torch.full((n,), value, dtype=torch.int32, device=dev)


def extend(rows):
    def call(dev, stream=None):
        B = 4
        fa.fa_extend_pages(ints(B * 8, dev).view(B, 8), ints(B, dev), ints(B, dev, 3),
                           torch.arange(64, dtype=torch.int32, device=dev), ints(1, dev, 64),
                           ints(B, dev), ints(1, dev), ints(B + 1, dev), ints(rows, dev),
                           torch.empty(rows, dtype=torch.int64, device=dev), B, 8, 64, 16, rows,
                           stream=stream)
    return call


def cache(dev):
    q = torch.randn(4, 8, 128, device=dev).bfloat16()
    kv = [torch.randn(64, 16, 2, 128, device=dev).bfloat16() for _ in range(2)]
    table = (torch.arange(4 * 600, device=dev) % 64).int().view(4, 600)
    return q, *kv, table, ints(4, dev, 9600), torch.empty_like(q)


def shared(pages):
    def call(dev, stream=None):
        q, kc, vc, table, lens, o = cache(dev)
        fa.fa_decode_shared_prefix(q, kc, vc, table, lens, table[0], ints(1, dev, pages), o, 4, 8, 2,
                                   128, 16, 0.1, 600, pages, 64, stream=stream)
    return call


def paged(dev, stream=None):
    q, kc, vc, table, lens, o = cache(dev)
    fa.fa_decode_paged(q, kc, vc, table, lens, o, 4, 8, 2, 128, 16, 0.1, 600, 64, stream=stream)


def norm_rope_bwd(dev, stream=None):
    x = torch.randn(1, 9, 2, 128, device=dev).bfloat16()
    dy = torch.randn(1, 2, 9, 128, device=dev).bfloat16()
    w = torch.ones(128, dtype=torch.bfloat16, device=dev)
    scratch = torch.empty(2 * fa.QK_NORM_ROPE_SCRATCH_ROWS * 128, device=dev)
    dw = [torch.empty(128, device=dev) for _ in range(2)]
    fa.fa_qk_norm_rope_bwd(x, x, dy, dy, w, w, torch.ones(16, 128, device=dev),
                           torch.arange(9, dtype=torch.int32, device=dev), None,
                           torch.empty_like(x), torch.empty_like(x), *dw, scratch, 1, 9, 2, 2, 128,
                           256, 256, 256, 256, 128, 16, 1, False, True, 1e-6, stream=stream)


@pytest.mark.parametrize("call", [extend(12), extend(5000), shared(600), shared(3), paged,
                                  norm_rope_bwd],
                         ids=["extend", "extend_rows", "shared", "shared_streamed", "paged", "bwd"])
def test_a_failed_launch_is_reported_once(cuda_device, call):
    dev = cuda_device
    call(dev)                                    # kernels loaded, limits raised
    torch.cuda.synchronize()
    x = torch.randn(1, 5, 2, 128, device=dev).bfloat16()
    w = torch.ones(128, dtype=torch.bfloat16, device=dev)
    args = (x, x, w, w, torch.ones(8, 128, device=dev), ints(5, dev))
    want = fa.qk_norm_rope(*args)
    with stream_that_takes_no_work() as stream:
        with pytest.raises(fa.FAError) as e:
            call(dev, stream)
    assert e.value.code == CUDA
    got = fa.qk_norm_rope(*args)
    assert all(torch.equal(g, t) for g, t in zip(got, want))
    call(dev)
    assert fa.device_status() == 0
