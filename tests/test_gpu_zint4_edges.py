"""The product on 4-bit weights at the ends of its ranges: rows that end inside a step, offsets past
32 bits on the streaming kernel."""
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
