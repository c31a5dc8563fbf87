"""What the 8-bit sources and their build have to keep to, checked without a GPU."""
import glob
import os
import re
import warnings

import pytest
import torch

import __graft_entry__
import w4a4_rotated_quantized_gb300 as q
import w4a4_rotated_quantized_gb300.build as B

CSRC = os.path.join(os.path.dirname(q.__file__), "csrc")


def test_no_bulk_load_writes_another_cta():
    """The library runs as replicas on several GPUs too: every CTA loads its own tiles into its own shared memory."""
    found = []
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        with open(path) as f:
            text = re.sub(r'"\s*"', "", f.read())  # asm strings that the source breaks over lines, joined
        for ins in re.findall(r"cp\.async\.bulk[\w.:]*", text):
            if "multi" + "cast" in ins:
                found.append((os.path.basename(path), ins))
    assert found == []


def test_accumulators_are_handed_over_behind_a_fence():
    """A read of tensor memory comes before another thread's next MMA into it only across a fence on both sides of the
    barrier: every arrival on acc_empty has one before it, and the MMA loops one after their wait."""
    with open(os.path.join(CSRC, "fp8_gemm.cu")) as f:
        lines = [ln.strip() for ln in f]
    arrivals = [i for i, ln in enumerate(lines) if ln.startswith("mbar_arrive_if(acc_empty")]
    waits = [i for i, ln in enumerate(lines) if "wait_one(acc_empty" in ln]
    assert len(arrivals) == len(waits) == 2
    assert all(lines[i - 1] == "fence_before_sync();" for i in arrivals)
    assert all("fence_after_sync();" in lines[i + 1:i + 3] for i in waits)


def test_the_version_tells_of_the_8_bit_layer():
    __graft_entry__.build()
    assert q.quarot_version() >> 16 == 1 and q.quarot_version() & 0xFFFF >= 2
    with open(os.path.join(os.path.dirname(CSRC), os.pardir, "include", "quarot.h")) as f:
        told = " ".join(f.read().split("1.2 adds")[1].split("*/")[0].replace("*", " ").split())
    for name in ("quant_fp8", "quant_fp8_block", "add_rmsnorm_quant_fp8", "fp8_gemm", "fp8_gated_gemm"):
        assert f"quarot_{name}" in told


# ---------------------------------------------------------------- without the compiled form
def _load_again(monkeypatch, path):
    monkeypatch.setattr(B, "calls_path", lambda: str(path))
    monkeypatch.setattr(q, "_lib", None)
    monkeypatch.setattr(q, "_calls", None)
    return q.load()


def _serves(lib):
    x = torch.zeros((4, 128), dtype=torch.float16)
    assert lib.quarot_version() >> 16 == 1 and lib.quarot_decode_workspace_bytes(16, 32, 128, 4096) > 0
    assert q._calls.quant(x, None, None, False) is None and q._calls.norm(x, None, None, 1e-6, None, None, None) is None
    assert q._calls.gemm(x, x, x, x, None, 0) is None and q._calls.gated(x, x, x, x, x, x, None, None) is None
    with pytest.raises(q.QuarotError, match="CUDA tensor"):  # the general path's answer
        q.quarot_quant_fp8(x)


def test_the_library_loads_without_the_compiled_form(monkeypatch, tmp_path):
    __graft_entry__.build()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        _serves(_load_again(monkeypatch, tmp_path / "absent.so"))


def test_the_library_loads_beside_a_compiled_form_that_does_not(monkeypatch, tmp_path):
    __graft_entry__.build()
    broken = tmp_path / "broken.so"
    broken.write_bytes(b"built for something else")
    with pytest.warns(RuntimeWarning, match="general path"):
        lib = _load_again(monkeypatch, broken)
    _serves(lib)


def test_the_library_builds_without_the_compiled_form(monkeypatch, tmp_path):
    __graft_entry__.build()

    def no_compiler(nvcc):
        raise FileNotFoundError("g++")

    monkeypatch.setattr(B, "calls_path", lambda: str(tmp_path / "absent.so"))
    monkeypatch.setattr(B, "_build_calls", no_compiler)
    assert not B.up_to_date()
    with pytest.warns(RuntimeWarning, match="general path"):
        assert B.build() == B.LIB


@pytest.mark.parametrize("what", ["torch", "python"])
def test_another_torch_or_python_gets_a_compiled_form_of_its_own(monkeypatch, what):
    __graft_entry__.build()
    here = B.calls_path()
    assert os.path.exists(here) and B.up_to_date()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "99.0")
    else:
        monkeypatch.setattr(B.sys.implementation, "cache_tag", "cpython-399")
    assert B.calls_path() != here and not B.up_to_date()
