"""The 4-bit calls and the block norms refuse what they do not take, before any device work; their
symbols are exported, and the packing order of the codes is the header's."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import int8_mixed_precision_absmax_b200 as i8
from int8_mixed_precision_absmax_b200 import build as lib_build

import block_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(0x10000)  # aligned, never dereferenced: the checks come first
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def L():
    lib_build.build()
    return i8.load_library()


def test_declared_and_exported(L):
    text = open(os.path.join(ROOT, "include", "int8mm.h"), encoding="utf-8").read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(int4_\w+|int8_block_\w+)\s*\(", text))
    assert names == {"int4_quant_weight", "int4_dequant_weight", "int4_linear_forward",
                     "int8_block_norm", "int8_block_residual"}
    for name in names:
        assert hasattr(L, name)
    for code in (-12, -13):
        assert i8.int8_status_string(code) not in ("", "unknown status")


def linear(L, X=FAKE, M=4, K=64, codes=FAKE, scales=FAKE, zeros=None, bias=None, N=8, group=64,
           flags=0, Y=FAKE, status=None):
    return L.int4_linear_forward(X, M, K, codes, scales, zeros, bias, N, group, flags, Y, status,
                                 None)


@pytest.mark.parametrize("change,status", [
    (dict(X=None), -1), (dict(codes=None), -1), (dict(scales=None), -1), (dict(Y=None), -1),
    (dict(M=0), -2), (dict(M=-1), -2), (dict(N=0), -2), (dict(K=0), -2),
    (dict(K=65536 + 32), -2), (dict(K=48), -3), (dict(X=ODD), -3), (dict(codes=ODD), -3),
    (dict(scales=ODD), -3), (dict(zeros=ODD), -3), (dict(bias=ODD), -3), (dict(Y=ODD), -3),
    (dict(status=ctypes.c_void_p(0x10002)), -3), (dict(flags=2), -11), (dict(flags=16), -11),
    (dict(group=0), -12), (dict(group=-128), -12), (dict(group=16), -12), (dict(group=96), -12),
    (dict(group=192), -12)])
def test_linear_refusals(L, change, status):
    assert linear(L, **change) == status


def test_weight_refusals(L):
    q, d = L.int4_quant_weight, L.int4_dequant_weight
    assert q(None, 8, 64, 64, 0, FAKE, FAKE, None, None) == -1
    assert q(FAKE, 8, 64, 64, 0, None, FAKE, None, None) == -1
    assert q(FAKE, 8, 64, 64, 0, FAKE, None, None, None) == -1
    assert q(FAKE, 8, 80, 64, 0, FAKE, FAKE, None, None) == -3
    assert q(FAKE, 0, 64, 64, 0, FAKE, FAKE, None, None) == -2
    assert q(FAKE, 8, 64, 48, 0, FAKE, FAKE, None, None) == -12
    assert q(FAKE, 8, 64, 64, 4, FAKE, FAKE, None, None) == -11
    assert q(FAKE, 8, 64, 64, 0, FAKE, FAKE, ODD, None) == -3
    assert d(None, FAKE, None, 8, 64, 64, 0, FAKE, None) == -1
    assert d(FAKE, FAKE, None, 8, 64, 64, 0, None, None) == -1
    assert d(FAKE, FAKE, None, 8, 64, 96, 0, FAKE, None) == -12
    assert d(FAKE, FAKE, None, 8, 64, 64, 0, ODD, None) == -3


def test_norm_refusals(L):
    n, r = L.int8_block_norm, L.int8_block_residual
    assert n(None, 4, 32, None, None, 1e-6, 0, FAKE, None) == -1
    assert n(FAKE, 4, 32, None, None, 1e-6, 0, None, None) == -1
    assert n(FAKE, 0, 32, None, None, 1e-6, 0, FAKE, None) == -2
    assert n(FAKE, 4, 65536 + 16, None, None, 1e-6, 0, FAKE, None) == -2
    assert n(FAKE, 4, 40, None, None, 1e-6, 0, FAKE, None) == -3
    assert n(FAKE, 4, 32, ODD, None, 1e-6, 0, FAKE, None) == -3
    assert n(FAKE, 4, 32, None, None, 1e-6, 8, FAKE, None) == -11  # POST_NORM is not its flag
    for eps in (-1e-6, math.nan, math.inf):
        assert n(FAKE, 4, 32, None, None, eps, 0, FAKE, None) == -13
    ok = dict(f=FAKE, x=FAKE, M=6, D=32, pw=None, pb=None, gate=None, rows=0, xs=1.0, fs=1.0,
              nw=None, nb=None, eps=1e-6, flags=0, y=FAKE, h=FAKE)

    def call(**change):
        return r(*{**ok, **change}.values(), None)

    assert call(f=None) == -1 and call(x=None) == -1 and call(y=None, h=None) == -1
    assert call(pw=FAKE) == -11 and call(pb=FAKE) == -11  # weights of a norm that is not taken
    assert call(h=None, nw=FAKE) == -1 and call(h=None, nb=FAKE) == -1
    assert call(gate=FAKE, rows=4) == -2 and call(gate=FAKE, rows=0) == -2  # 4 does not divide 6
    assert call(gate=FAKE, rows=12) == -2 and call(rows=1) == -2
    assert call(xs=math.inf) == -13 and call(fs=math.nan) == -13 and call(eps=math.nan) == -13
    assert call(gate=ODD, rows=2) == -3 and call(y=ODD) == -3 and call(h=ODD) == -3
    assert call(flags=16) == -11


def test_cpu_tensors_are_refused():
    x = torch.zeros(2, 64, dtype=torch.float16)
    codes = torch.zeros(8, 32, dtype=torch.uint8)
    scales = torch.zeros(8, 1, dtype=torch.float16)
    for call in (lambda: i8.int4_quant_weight(x), lambda: i8.int4_dequant_weight(codes, scales),
                 lambda: i8.int4_linear_forward(x, codes, scales), lambda: i8.int8_block_norm(x),
                 lambda: i8.int8_block_residual(x, x), lambda: i8.Int4Linear(x)):
        with pytest.raises(TypeError, match="CUDA"):
            call()


def test_reference_packing_round_trip():
    u = np.random.default_rng(0).integers(0, 16, (3, 64)).astype(np.uint8)
    codes = ref.pack(u)
    assert np.array_equal(ref.unpack(codes), u)
    # the header's words: neighbours 0 and 1 in the lowest nibbles of the two halves
    word = int(codes[0, :4].view("<u4")[0])
    assert [word >> 4 * i & 15 for i in range(8)] == [int(u[0, k]) for k in
                                                      (0, 2, 4, 6, 1, 3, 5, 7)]


def test_sizes_past_an_int_are_not_cut_off():
    assert i8._int4_shapes(8, 100, 64) == (8, 2)
    for N, group in ((8, 2 ** 32 + 128), (2 ** 32 + 8, 128)):
        with pytest.raises(ValueError, match="2\\^31"):
            i8._int4_shapes(N, 256, group)
