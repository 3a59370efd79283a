"""The product on 4-bit weights where a few activations are far larger than the others, by the terms
that the formula has.

A large activation whose code equals its zero point adds exactly 0 to its output: what the others add
has to come out as if the large one were not there.  So a product Y[m,n] = T(sum_k x s (u - z) + b) is
held to the magnitudes of its own terms, A = sum |x| s |u - z| + |b|:
  v |Y| + t        its one rounding to T (v = half a step: 2^-11 or 2^-8; t = half a step of the
                   least numbers of T)
  2^-23 n 3 A      float32 sums of n = K / min(group, 128) + 64 roundings on the way of a term (2^-23:
                   a matrix instruction may cut off); a term may be taken in digits of both signs,
                   whose magnitudes are together at most 3 times its own
  6 v sqrt(sum (x W)^2)   for more than 8 tokens only, whose weights are rounded to T: by Hoeffding's
                   bound over the independent signs of X exceeded with probability 2 exp(-18)
"""
import numpy as np
import pytest
import torch

import int8_mixed_precision_absmax_b200 as i8

import block_reference as ref

pytestmark = pytest.mark.gpu

FP16, BF16 = torch.float16, torch.bfloat16
HALF_STEP = {FP16: 2.0 ** -11, BF16: 2.0 ** -8}
LEAST = {FP16: 2.0 ** -25, BF16: 2.0 ** -134}


def f64(t):
    return t.detach().double().cpu().numpy()


def case(M, N, K, group, T, affine, cols, big, std, seed=0, scale=1.0):
    """Inputs whose activations are `big` in `cols` and of spread `std` elsewhere; in the even output
    channels the codes of `cols` equal their zero points."""
    g = np.random.default_rng(seed)
    G = -(-K // group)
    u = g.integers(0, 16, (N, K)).astype(np.uint8)
    z = g.integers(0, 16, (N, G)).astype(np.uint8) if affine else None
    zk = ref.spread(z, group, K) if affine else np.full((N, K), 8, np.uint8)
    u[::2, cols] = zk[::2, cols]
    scales = torch.from_numpy((g.random((N, G)) * 0.02 + 0.005) * scale).to(T)
    X = torch.from_numpy(g.standard_normal((M, K)) * std).to(T)
    X[:, cols] = torch.tensor(big, dtype=torch.float64).to(T)
    return (X.cuda(), torch.from_numpy(ref.pack(u)).cuda(), scales.cuda(),
            torch.from_numpy(z).cuda() if affine else None)


def check(Y, X, codes, scales, zeros, bias, group):
    T = X.dtype
    x, W = f64(X), ref.values(codes.cpu().numpy(), f64(scales),
                              None if zeros is None else zeros.cpu().numpy(), group)
    b = 0.0 if bias is None else f64(bias)
    want, A = x @ W.T + b, np.abs(x) @ np.abs(W).T + np.abs(b)
    M, K = x.shape
    tol = (HALF_STEP[T] * np.abs(want) + LEAST[T]
           + 2.0 ** -23 * (K / min(group, 128) + 64) * 3 * A)
    if M > 8:
        tol += 6 * HALF_STEP[T] * np.sqrt((x * x) @ (W * W).T)
    got = f64(Y)
    assert np.isfinite(got).all()
    over = np.abs(got - want) - tol
    assert (over <= 0).all(), (float((over / tol).max()), np.unravel_index(over.argmax(), over.shape))


# the large activations over the spread of the others: an ordinary outlier, a massive one, and the
# ends of the type's range
RATIOS = [(FP16, 60.0, 1.0), (FP16, 1000.0, 0.2), (FP16, 1000.0, 0.01), (FP16, 30000.0, 0.01),
          (FP16, 65504.0, 1e-4), (FP16, -65504.0, 2e-7), (BF16, 60.0, 1.0), (BF16, 2.0 ** 20, 0.1),
          (BF16, -1e8, 1e-3), (BF16, 1e12, 1e-12), (BF16, 1e30, 1.0), (BF16, 1e30, 1e-30)]


@pytest.mark.parametrize("M", [1, 2, 8, 16, 200])
@pytest.mark.parametrize("T,big,std", RATIOS)
def test_large_activations_of_no_weight(T, big, std, M):
    """One large activation in each 256, or in one of them only."""
    for K, group, affine in ((1024, 128, False), (1312, 64, True), (544, 32, True), (2048, 512, True)):
        for cols in (list(range(100, K, 256)), [300]):
            X, codes, scales, zeros = case(M, 75, K, group, T, affine, cols, big, std, seed=K)
            check(i8.int4_linear_forward(X, codes, scales, zeros, None, group), X, codes, scales, zeros,
                  None, group)


@pytest.mark.parametrize("T", [FP16, BF16])
@pytest.mark.parametrize("K", [8192, 12288, 16384, 18432, 24576, 32768, 49152, 65536])
def test_one_token_of_long_rows(T, K):
    cols = [5, 300, K - 20]
    X, codes, scales, zeros = case(1, 100, K, 128, T, True, cols, 2000.0, 0.01, seed=K)
    bias = torch.linspace(-1, 1, 100).to(T).cuda()
    check(i8.int4_linear_forward(X, codes, scales, zeros, bias, 128), X, codes, scales, zeros, bias, 128)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_one_token_of_many_channels(group):
    """Every block takes several pairs of units; the last unit is alone in some."""
    for N in (5000, 19000):
        X, codes, scales, zeros = case(1, N, 768, group, FP16, True, [1, 257, 700], 500.0, 0.01, seed=N)
        check(i8.int4_linear_forward(X, codes, scales, zeros, None, group), X, codes, scales, zeros, None,
              group)


def test_one_token_near_the_least_numbers():
    """bf16 activations down to the subnormal ones, whose products with large scales are normal."""
    for std in (2.0 ** -120, 2.0 ** -126, 2.0 ** -131):
        for group in (32, 64, 128):
            X, codes, scales, zeros = case(1, 40, 512, group, BF16, True, [3], 0.0, std, scale=2.0 ** 60)
            check(i8.int4_linear_forward(X, codes, scales, zeros, None, group), X, codes, scales, zeros,
                  None, group)


@pytest.mark.parametrize("T", [FP16, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_one_token_of_nan_or_infinity(T, group):
    for value in (float("nan"), float("inf"), -float("inf")):
        for col in (0, 300, 1000):
            X, codes, scales, zeros = case(1, 33, 1024, group, T, True, [col], value, 1.0)
            assert not torch.isfinite(i8.int4_linear_forward(X, codes, scales, zeros, None, group)).any()
    X = torch.zeros(1, 1024, dtype=T, device="cuda")
    X[0, 512:] = -0.0
    assert (i8.int4_linear_forward(X, codes, scales, zeros, None, group) == 0).all()


def test_a_token_alone_and_in_a_pair():
    """The same row in a batch of two: both within one rounding of the same sum, large column or not."""
    X, codes, scales, zeros = case(2, 64, 1024, 128, FP16, True, [7, 600], 30000.0, 0.01)
    two = i8.int4_linear_forward(X, codes, scales, zeros, None, 128)
    for m in (0, 1):
        one = i8.int4_linear_forward(X[m:m + 1], codes, scales, zeros, None, 128)
        check(one, X[m:m + 1], codes, scales, zeros, None, 128)
        assert torch.allclose(one[0, ::2].float(), two[m, ::2].float(), rtol=2.0 ** -10, atol=2.0 ** -20)
