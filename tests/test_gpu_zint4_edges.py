"""The product on 4-bit weights at the ends of its ranges: rows that end inside a step, offsets past
32 bits on the streaming kernel, weights that are not rounded for few tokens."""
import numpy as np
import pytest
import torch

import int8_mixed_precision_absmax_b200 as i8

import block_reference as ref

pytestmark = pytest.mark.gpu

FP16, BF16 = torch.float16, torch.bfloat16


@pytest.mark.parametrize("M", [1, 5, 9, 40, 130, 300])
@pytest.mark.parametrize("K,group", [(32, 32), (96, 64), (160, 32), (160, 128), (480, 256), (1056, 64)])
def test_nothing_behind_a_row_is_multiplied(M, K, group):
    """Scales with which a weight is finite only for codes near the zero point: the steps of 128 k that
    are filled up behind the row's end must not bring in others.  Codes are the zero point, or 1 beside
    it in the last 32 columns, so each result is a sum of at most 32 exact products."""
    N = 70
    g = np.random.default_rng(K)
    G = -(-K // group)
    for scale, zero in ((9000.0, 8), (5000.0, 15), (60000.0, 1)):
        z = np.full((N, G), zero, np.uint8)
        u = np.full((N, K), zero, np.uint8)
        u[:, K - 32:] -= g.integers(0, 2, (N, 32)).astype(np.uint8)
        s = np.full((N, G), scale)
        x = g.integers(-2, 3, (M, K)) / 64.0
        want = x @ ref.values(ref.pack(u), s, z, group).T
        Y = i8.int4_linear_forward(torch.from_numpy(x).half().cuda(), torch.from_numpy(ref.pack(u)).cuda(),
                                   torch.from_numpy(s).half().cuda(), torch.from_numpy(z).cuda(),
                                   group_size=group)
        # x is a multiple of 2^-6 and at most 2^-5, and a result a multiple of scale 2^-6: float32 sums
        # of 32 of them are exact, and the result is rounded once
        assert torch.equal(Y.cpu(), torch.from_numpy(want).half()), (scale, zero)


@pytest.mark.parametrize("M,N,K", [(1, 560000, 16384), (1, 270000, 32768), (2, 270000, 32768)])
def test_streaming_offsets_past_32_bits(M, N, K):
    """More than 4 GiB of codes through the streaming kernel: one token in digits, one in 16 bits, two."""
    group = 128
    gen = torch.Generator(device="cuda").manual_seed(N + M)
    codes = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda").random_(0, 256, generator=gen)
    scales = (torch.rand(N, K // group, device="cuda", generator=gen) * 0.02 + 0.005).half()
    X = (torch.randn(M, K, device="cuda", generator=gen) * 0.1).half()
    assert codes.numel() > 2 ** 32
    Y = i8.int4_linear_forward(X, codes, scales, None, None, group)
    edge = 2 ** 32 // (K // 2)  # the channel whose codes begin past 4 GiB
    for rows in (slice(0, 3), slice(edge - 2, edge + 3), slice(N - 3, N)):
        x = X.double().cpu().numpy()
        W = ref.values(codes[rows].cpu().numpy(), scales[rows].double().cpu().numpy(), None, group)
        want, A = x @ W.T, np.abs(x) @ np.abs(W).T
        # one rounding to fp16, and float32 sums of terms in digits of both signs
        tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 2.0 ** -23 * (K / 128 + 64) * 3 * A
        assert (np.abs(Y[:, rows].double().cpu().numpy() - want) <= tol).all(), rows


@pytest.mark.parametrize("T", [FP16, BF16])
@pytest.mark.parametrize("M", [1, 2, 8])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_few_tokens_multiply_weights_that_are_not_rounded(T, M, group):
    """Nearly every result is the formula's, rounded once.  The sums' float32 error, of the order of
    sqrt(100) 2^-24 A with A = sum |x W|, is 1 / 60 of the steps of T at |Y| ~ A / sqrt(K): some 3 % of
    the results are rounded to the other side.  Weights rounded to T would move each sum by about as
    much as its own rounding, and 4 of 10 results."""
    N, K = 500, 1024
    g = np.random.default_rng(M)
    u = g.integers(0, 16, (N, K)).astype(np.uint8)
    s = torch.from_numpy(g.random((N, K // group)) * 0.02 + 0.005).to(T)
    X = torch.from_numpy(g.standard_normal((M, K))).to(T)
    want = X.double().numpy() @ ref.values(ref.pack(u), s.double().numpy(), None, group).T
    Y = i8.int4_linear_forward(X.cuda(), torch.from_numpy(ref.pack(u)).cuda(), s.cuda(), group_size=group)
    same = (Y.cpu() == torch.from_numpy(want).to(T)).double().mean()
    assert same >= 0.9, float(same)
