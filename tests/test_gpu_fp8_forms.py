"""Every form of the 8-bit products (few tokens at each tile width, the depth split, whole tiles, one or several to a
CTA), at every number of CTAs that can share a tile's depth, against the float64 forms."""
import os
import re

import pytest
import torch

import w4a4_rotated_quantized_gb300 as package
from test_gpu_fp8 import BF16, E4M3, FP16, GATED, GEMM, _check_gated, _check_product, _operand
from test_gpu_parity import DEV, q  # noqa: F401  (q: fixture)

SMS = 152

GEMM_MORE = [(9, 300, 1040), (16, 777, 2064), (17, 1031, 1040), (24, 4096, 2064), (32, 1000, 4096), (31, 1002, 4112),
             (50, 640, 2064), (64, 1000, 4096), (63, 129, 4112),
             # an output head's columns
             (1, 131073, 1040), (37, 131080, 272), (129, 131080, 144)]
GATED_MORE = [(9, 304, 1040), (16, 784, 2064), (20, 144, 272), (17, 1040, 1040), (24, 400, 2064), (32, 1040, 4096),
              (31, 144, 4112), (130, 784, 2064), (33, 1920, 2064), (257, 640, 4112)]


def _form(M, N, K, gated):
    """The rule of fp8_gemm.cu, its numbers read from there, on a GPU of SMS SMs."""
    with open(os.path.join(os.path.dirname(package.__file__), "csrc", "fp8_gemm.cu")) as f:
        src = f.read()
    narrow = re.search(r"constexpr int kNarrow = GATED \? (\d+) : (\d+);", src).groups()
    splits = re.findall(r"if \(tiles(?: \* (\d+)) <= sms(?: \* (\d+) / (\d+))? && nkb >= (\d+)\) return (\d+);", src)
    assert len(splits) == 3 and "while (cl < 8 && wbs * cl * 2 <= 2 * sms && nkb / (2 * cl) >= 4) cl *= 2;" in src
    nkb, wbs = -(-K // 128), -(-N // 128)
    if M <= int(narrow[0 if gated else 1]):
        cl = 1
        while cl < 8 and wbs * cl * 2 <= 2 * SMS and nkb // (2 * cl) >= 4:
            cl *= 2
        return "few", 16 if M <= 16 else 32 if M <= 32 else 64, cl
    tiles = -(-M // 128) * -(-N // (128 if gated else 256))
    for by, num, den, least, ranks in splits:
        if tiles * int(by) <= SMS * int(num or 1) // int(den or 1) and nkb >= int(least):
            return "split", int(ranks)
    return ("one",) if tiles <= SMS else ("several",)


def test_the_sizes_reach_every_form():
    few = lambda widths: {("few", w, r) for w in widths for r in (1, 2, 4, 8)}  # noqa: E731
    rest = {("split", 2), ("split", 4), ("split", 8), ("one",), ("several",)}
    assert {_form(*s, False) for s in GEMM + GEMM_MORE} == few((16, 32, 64)) | rest
    assert {_form(*s, True) for s in GATED + GATED_MORE} == few((16, 32)) | rest


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", GEMM_MORE)
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_gemm_forms(q, M, N, K, dtype):  # noqa: F811
    a, sa = _operand(M, K, M + N + K, False)
    w, sw = _operand(N, K, M + N + K + 1, True)
    guard = torch.full((M * N + 64,), 5.0, dtype=dtype, device=DEV)
    y = guard[:M * N].view(M, N)
    assert q.quarot_fp8_gemm(a, sa, w, sw, y=y) is y
    q.quarot_check_error()
    _check_product(y, a, sa, w, sw)
    assert (guard[M * N:] == 5.0).all()
    assert torch.equal(q.quarot_fp8_gemm(a, sa, w, sw, out_dtype=dtype), y)


@pytest.mark.gpu
@pytest.mark.parametrize("M,I,K", GATED_MORE)
def test_gated_forms(q, M, I, K):  # noqa: F811
    a, sa = _operand(M, K, M + I + K, False)
    g, sg = _operand(I, K, M + I + K + 1, True)
    u, su = _operand(I, K, M + I + K + 2, True)
    sg.mul_(2.0 ** -8 * (12.0 / K ** 0.5))  # gate values of a few units
    guard = torch.full((M * I + 64,), 0x55, dtype=torch.uint8, device=DEV)
    qo = guard[:M * I].view(E4M3).view(M, I)
    codes, scale = q.quarot_fp8_gated_gemm(a, sa, g, sg, u, su, q_out=qo)
    q.quarot_check_error()
    assert codes is qo and (guard[M * I:] == 0x55).all()
    _check_gated(codes, scale, a, sa, g, sg, u, su)
    again = q.quarot_fp8_gated_gemm(a, sa, g, sg, u, su)
    assert torch.equal(again[0].view(torch.uint8), codes.view(torch.uint8)) and torch.equal(again[1], scale)
