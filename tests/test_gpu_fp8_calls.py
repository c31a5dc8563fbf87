"""An 8-bit call is made once, whatever went wrong before it or in it."""
import ctypes

import pytest
import torch

from test_gpu_errors import failed_wait
from test_gpu_fp8 import E4M3, FP16, _Sub, _operand, _rand
from test_gpu_parity import DEV, q  # noqa: F401  (q: fixture)

pytestmark = pytest.mark.gpu

NAMES = ("quarot_quant_fp8", "quarot_quant_fp8_block", "quarot_add_rmsnorm_quant_fp8", "quarot_fp8_gemm",
         "quarot_fp8_gated_gemm")


@pytest.fixture
def stubs(q, monkeypatch):  # noqa: F811
    """Entry points that launch nothing: they count their calls and return `status`."""
    class Stubs:
        status, count, lib = 4, 0, None

    def called(*_):
        Stubs.count += 1
        return Stubs.status

    fns = {n: ctypes.CFUNCTYPE(*q._SIGS[n][:1], *q._SIGS[n][1])(called) for n in NAMES}
    real = q.load()
    stub_lib = type("Lib", (), {n: staticmethod(f) for n, f in fns.items()})
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    monkeypatch.setattr(q, "_lib", stub_lib)
    q._calls.bind(*(address(fns[n]) for n in NAMES))
    yield Stubs
    q._calls.bind(*(address(getattr(real, n)) for n in NAMES))


def _all_calls(q, like=lambda t: t):  # noqa: F811
    x, r = like(_rand((4, 256), FP16, 1)), _rand((4, 256), FP16, 2)
    a, sa = _operand(4, 256, 3, False)
    w, sw = _operand(144, 256, 4, True)
    a = like(a)
    return {"quarot_quant_fp8": lambda: q.quarot_quant_fp8(x), "quarot_quant_fp8_block": lambda: q.quarot_quant_fp8_block(x),
            "quarot_add_rmsnorm_quant_fp8": lambda: q.quarot_add_rmsnorm_quant_fp8(x, r, residual_out=r),
            "quarot_fp8_gemm": lambda: q.quarot_fp8_gemm(a, sa, w, sw),
            "quarot_fp8_gated_gemm": lambda: q.quarot_fp8_gated_gemm(a, sa, w, sw, w, sw)}


@pytest.mark.parametrize("status", [4, 5, 6])
@pytest.mark.parametrize("general", [False, True])
def test_a_call_that_fails_is_not_made_again(q, stubs, status, general):  # noqa: F811
    stubs.status = status
    for name, call in _all_calls(q, (lambda t: t.as_subclass(_Sub)) if general else lambda t: t).items():
        stubs.count = 0
        with pytest.raises(q.QuarotError, match=name) as e:
            call()
        assert stubs.count == 1 and e.value.status == status


@pytest.mark.parametrize("status", [1, 2, 3])
def test_a_refused_call_names_its_reason(q, stubs, status):  # noqa: F811
    """Refusals come before any launch: the general path makes the call again and raises."""
    stubs.status = status
    for name, call in _all_calls(q).items():
        with pytest.raises(q.QuarotError, match=name) as e:
            call()
        assert e.value.status == status


@pytest.mark.parametrize("target", ["residual", "x"])
def test_in_place_after_an_earlier_error_adds_once(q, target):  # noqa: F811
    x0, r0 = _rand((37, 528), FP16, 5), _rand((37, 528), FP16, 6)
    want = q.quarot_add_rmsnorm_quant_fp8(x0, r0)
    x, r = x0.clone(), r0.clone()
    failed_wait(q)
    codes, scale, h = q.quarot_add_rmsnorm_quant_fp8(x, r, residual_out=r if target == "residual" else x)
    assert torch.equal(h, want[2]) and torch.equal(scale, want[1])
    assert torch.equal(codes.view(torch.uint8), want[0].view(torch.uint8)) and codes.dtype == E4M3
    q.quarot_check_error()


def test_the_general_path_alone_gives_the_same_bits(q, monkeypatch):  # noqa: F811
    raw = lambda v: [t.view(torch.uint8).clone() for t in (v if isinstance(v, tuple) else (v,))]  # noqa: E731
    calls = _all_calls(q)
    calls["quarot_add_rmsnorm_quant_fp8"] = lambda: q.quarot_add_rmsnorm_quant_fp8(_rand((4, 256), FP16, 1), _rand((4, 256), FP16, 2))
    want = {n: raw(c()) for n, c in calls.items()}
    monkeypatch.setattr(q, "_calls", q._GeneralOnly())
    for n, c in calls.items():
        got = raw(c())
        assert len(got) == len(want[n]) and all(torch.equal(g, w) for g, w in zip(got, want[n]))
