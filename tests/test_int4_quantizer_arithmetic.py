"""The 4-bit quantizer's rounding of w / s by a reciprocal, on the CPU.

The kernel takes t = RN(w r + 768) with r within one step of 1 / s, then RN(t + (1.5 2^23 - 768)):
two float32 roundings in place of the float32 quotient and its rounding to a whole number.  For w and
s of a 16-bit type the two agree wherever |w / s| < 16; here for sampled scales and every w in reach,
with r one step too small, right, and one step too large.  float64 holds w r + 768 exactly (11 by 24
bits, above 2^-43), so one conversion is the fused operation's rounding.
"""
import numpy as np
import pytest

F32 = np.float32


def all_positive(T):
    bits = np.arange(0x7C00 if T == "fp16" else 0x7F80, dtype=np.uint16)
    if T == "fp16":
        return bits.view(np.float16).astype(np.float64)
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


@pytest.mark.parametrize("T,lo,hi", [("fp16", 6.2e-5, 9400.0), ("bf16", 1e-30, 1e30)])
def test_two_roundings_are_the_quotients(T, lo, hi):
    values = all_positive(T)
    scales = values[(values >= lo) & (values <= hi)]
    rng = np.random.default_rng(1)
    for s in np.concatenate((rng.choice(scales, 300, replace=False), scales[:3], scales[-3:])):
        w = values[(values < 15.99 * s) & (values > s / 64)]
        want = np.rint((w.astype(F32) / F32(s)))
        exact = F32(1) / F32(s)
        for r in (np.nextafter(exact, F32(0)), exact, np.nextafter(exact, F32(np.inf))):
            t = (w * np.float64(r) + 768.0).astype(F32)
            whole = (t + F32(12582912.0 - 768.0)) - F32(12582912.0)
            assert np.array_equal(whole, want), (s, w[whole != want][:4])


@pytest.mark.parametrize("T,D", [("fp16", 7), ("bf16", 7), ("fp16", 15), ("bf16", 15)])
def test_division_by_a_constant_is_correctly_rounded(T, D):
    """q = RN(a c), RN(q + RN(a - q D) c) with c = RN(1 / D), for every a of the type from 1e-30 on."""
    a = all_positive(T)
    a = a[a >= 1e-30]
    c = F32(1) / F32(D)
    q = (a.astype(F32) * c).astype(np.float64)
    rest = (a - q * D).astype(F32).astype(np.float64)  # exact in float64: 24 by 4 bits
    got = (q + rest * np.float64(c)).astype(F32)
    # (the last sum is in float64: where its rounding and float32's could differ twice, the exact
    # quotient decides)
    want = (a.astype(F32) / F32(D))
    assert np.array_equal(got, want)


def test_codes_of_a_half_word_are_one_number():
    """Four codes by Horner's rule in float32, and 2^23 added: the low 16 bits are the nibbles."""
    rng = np.random.default_rng(2)
    u = rng.integers(0, 16, (1000, 4)).astype(F32)
    acc = ((u[:, 3] * F32(16) + u[:, 2]) * F32(16) + u[:, 1]) * F32(16) + u[:, 0]
    bits = (acc + F32(8388608.0)).view(np.uint32) & 0xFFFF
    n = u.astype(np.uint32)
    assert np.array_equal(bits, n[:, 0] | n[:, 1] << 4 | n[:, 2] << 8 | n[:, 3] << 12)
