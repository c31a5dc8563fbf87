"""A failed call's error is its own: it is reported once, and the next call starts from a clean state."""
import ctypes
import time

import pytest
import torch

from test_gpu_parity import DEV, q  # noqa: F401  (q: fixture)

pytestmark = pytest.mark.gpu


def failed_wait(q):  # noqa: F811
    """quarot_check_error on a stream under capture: refused by the runtime on the host."""
    cu = ctypes.CDLL("libcuda.so.1")
    side = torch.cuda.Stream()
    graph = ctypes.c_void_p()
    assert cu.cuStreamBeginCapture_v2(ctypes.c_void_p(side.cuda_stream), 2) == 0
    with pytest.raises(q.QuarotError):
        q.quarot_check_error(stream=side)
    assert cu.cuStreamEndCapture(ctypes.c_void_p(side.cuda_stream), ctypes.byref(graph)) != 0 and not graph


@pytest.mark.parametrize("op", ["rotate_quant", "gemm", "kv_write", "quant_fp8", "norm_fp8"])
def test_the_call_after_a_failed_one(q, op):  # noqa: F811
    g = torch.Generator().manual_seed(7)
    x = torch.randn((64, 4096), generator=g).half().to(DEV)
    a, s, _ = q.quarot_rotate_quant(x)
    kv = torch.randn((2, 3, 4, 128), generator=g).half().to(DEV)

    def call():
        if op == "rotate_quant":
            return q.quarot_rotate_quant(x)[:2]
        if op == "gemm":
            return q.quarot_w4a4_gemm(a, s, a, s)[:1]
        if op == "kv_write":
            cache = q.QuarotKVCache(2, 4, 3, device=DEV)
            cache.append(kv, kv)
            return [t.contiguous() for t in cache.tensors]
        if op == "quant_fp8":
            return q.quarot_quant_fp8(x)
        h = x.clone()
        return q.quarot_add_rmsnorm_quant_fp8(x, h, residual_out=h)

    want = call()
    failed_wait(q)
    for w, v in zip(want, call()):
        assert torch.equal(w.view(torch.uint8), v.view(torch.uint8))
    q.quarot_check_error()


def test_both_bounded_waits_end_after_about_a_second(q):  # noqa: F811
    """The self-test runs the library's wait and the 8-bit products' own, one after the other: a second each."""
    q.quarot_check_error()
    t0 = time.perf_counter()
    q.quarot_selftest_wait()
    with pytest.raises(q.QuarotError) as e:
        q.quarot_check_error()
    dt = time.perf_counter() - t0
    assert e.value.status == q.QUAROT_ERR_TIMEOUT
    assert 1.7 <= dt <= 3.5, dt
    q.quarot_check_error()
