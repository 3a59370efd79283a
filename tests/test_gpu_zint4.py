"""4-bit weights on the GPU against their formulas in 64 bits.

Tolerances.  The codes, scales and zero points are compared bit for bit: every step of the
quantizer is an IEEE float32 operation.  A product Y[m,n] is off by at most
  u |Y|                              its one rounding to T (u = half a step: 2^-11 or 2^-8)
  2^-23 n A                          n = G/4 + K/G + 32 float32 roundings on the way of a term (a
                                     matrix instruction adds 16 products; a group, then the groups,
                                     then lanes and warps are summed), A = sum s |x| (u + z) the
                                     magnitudes, zero point and code apart
  6 u sqrt(sum (x W)^2)              where a kernel multiplies by weights rounded to T (more than
                                     the few tokens of the streaming kernel): by Hoeffding's bound
                                     over the independent signs of X exceeded with probability
                                     2 exp(-18)
"""
import numpy as np
import pytest
import torch

import int8_mixed_precision_absmax_b200 as i8

import block_reference as ref

pytestmark = pytest.mark.gpu

FP16, BF16 = torch.float16, torch.bfloat16
U = {FP16: 2.0 ** -11, BF16: 2.0 ** -8}


def f64(t):
    return t.detach().double().cpu().numpy()


def weight(N, K, group, T, affine, seed=0):
    """Random codes, scales and zero points on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    G = -(-K // group)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = (torch.rand(N, G, device="cuda", generator=g) * 0.02 + 0.001).to(T)
    zeros = torch.randint(0, 16, (N, G), dtype=torch.uint8, device="cuda", generator=g)
    return codes, scales, zeros if affine else None


def acts(M, K, T, seed=1, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(M, K, device="cuda", generator=g) * std).to(T)


def reference(X, codes, scales, zeros, bias, group):
    x, s = f64(X), f64(scales)
    c = codes.cpu().numpy()
    z = None if zeros is None else zeros.cpu().numpy()
    W = ref.values(c, s, z, group)
    Y = x @ W.T + (0.0 if bias is None else f64(bias))
    K = x.shape[1]
    zz = 8.0 if z is None else ref.spread(z.astype(np.float64), group, K)
    A = np.abs(x) @ ((ref.unpack(c) + zz) * ref.spread(np.abs(s), group, K)).T
    if bias is not None:
        A += np.abs(f64(bias))
    return Y, A, np.sqrt((x * x) @ (W * W).T)


def check(Y, X, codes, scales, zeros, bias, group, rows=None):
    T = X.dtype
    if rows is not None:
        X, Y = X[rows], Y[rows]
    Yr, A, L2 = reference(X, codes, scales, zeros, bias, group)
    K = X.shape[1]
    n = min(group, K) / 4 + K / min(group, K) + 32
    tol = U[T] * np.abs(Yr) + 2.0 ** -23 * n * A + 6 * U[T] * L2
    got = f64(Y)
    assert np.isfinite(got).all()
    over = np.abs(got - Yr) - tol
    assert (over <= 0).all(), (float(over.max()), np.unravel_index(over.argmax(), over.shape))
    # most errors are far below their bounds: the norm of all of them
    rel = np.linalg.norm(got - Yr) / np.linalg.norm(Yr)
    assert rel <= 2 * U[T] + 2.0 ** -20, rel


@pytest.mark.parametrize("T", [FP16, BF16])
@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("N,K,group", [
    (1, 32, 32), (5, 64, 128), (3, 96, 64), (17, 288, 128), (33, 256, 32), (7, 4096, 64),
    (9, 544, 256), (4, 1056, 384), (3, 2080, 512), (2, 65536, 65536), (130, 1024, 128)])
def test_quantizer_is_its_definition(T, symmetric, N, K, group):
    g = torch.Generator(device="cuda").manual_seed(N + K)
    W = torch.randn(N, K, device="cuda", generator=g) * 0.05
    W[:, ::7] *= 3
    W[0, : K // 2] = 0.0
    W[N // 2, :32] = W[N // 2, :32].abs()
    W = W.to(T)
    codes, scales, zeros = i8.int4_quant_weight(W, group, symmetric)
    u, s, z = ref.quantize(f64(W), group, symmetric,
                           lambda a: f64(torch.from_numpy(np.asarray(a, np.float32)).to(T)))
    assert np.array_equal(f64(scales), s)
    assert np.array_equal(ref.unpack(codes.cpu().numpy()), u)
    assert (zeros is None) == symmetric
    if not symmetric:
        assert np.array_equal(zeros.cpu().numpy(), z)
    What = i8.int4_dequant_weight(codes, scales, zeros, group)
    want = torch.from_numpy(ref.values(codes.cpu().numpy(), s, None if symmetric else z, group))
    assert torch.equal(What.cpu(), want.float().to(T))  # a 5-bit by 11-bit product is exact in f32


@pytest.mark.parametrize("T", [FP16, BF16])
def test_quantizer_extremes(T):
    big = torch.finfo(T).max
    tiny = torch.finfo(T).smallest_normal * torch.finfo(T).eps  # the least subnormal
    W = torch.zeros(8, 128, dtype=T, device="cuda")
    W[1, 0], W[2, 0], W[2, 1] = big, big, -big
    W[3] = tiny
    W[4, 3], W[5, 5], W[6, 40] = float("nan"), float("inf"), -float("inf")
    W[7] = -2.0
    for symmetric in (True, False):
        codes, scales, zeros = i8.int4_quant_weight(W, 32, symmetric)
        u, s, z = ref.quantize(f64(W), 32, symmetric,
                               lambda a: f64(torch.from_numpy(np.asarray(a, np.float32)).to(T)))
        assert np.array_equal(f64(scales), s, equal_nan=True)
        assert np.array_equal(ref.unpack(codes.cpu().numpy()), u)
        if not symmetric:
            assert np.array_equal(zeros.cpu().numpy(), z)
        # a group that held a NaN or an infinity makes its products NaN, the others do not
        Y = i8.int4_linear_forward(torch.ones(1, 128, dtype=T, device="cuda"), codes, scales, zeros,
                                   group_size=32)
        assert torch.isnan(Y[0, 4:7]).all() and torch.isfinite(Y[0, 7])


SHAPES = [  # M, N, K, group
    (1, 1, 32, 32), (1, 16, 64, 64), (2, 17, 96, 64), (3, 31, 128, 128), (4, 33, 288, 32),
    (5, 100, 544, 128), (7, 129, 1056, 256), (8, 257, 4096, 128), (8, 48, 2080, 32),
    (9, 65, 320, 64), (12, 200, 1024, 128), (16, 128, 4096, 64), (17, 130, 256, 32),
    (31, 333, 800, 128), (33, 64, 2048, 512), (64, 129, 1024, 32), (65, 257, 160, 128),
    (100, 50, 4128, 128), (127, 128, 96, 32), (128, 384, 512, 64), (129, 65, 640, 128),
    (255, 140, 288, 64), (257, 300, 1024, 128), (300, 1, 64, 32), (700, 260, 192, 65536)]


@pytest.mark.parametrize("T", [FP16, BF16])
@pytest.mark.parametrize("M,N,K,group", SHAPES)
def test_linear_against_64_bits(T, M, N, K, group):
    for affine in (False, True):
        codes, scales, zeros = weight(N, K, group, T, affine, seed=M)
        X = acts(M, K, T, seed=N)
        bias = acts(1, N, T, seed=5)[0] if affine else None
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        Y = i8.int4_linear_forward(X, codes, scales, zeros, bias, group, dev_status=status)
        check(Y, X, codes, scales, zeros, bias, group)
        assert int(status) == 0


@pytest.mark.parametrize("T", [FP16, BF16])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 6, 8, 10, 16, 24, 40, 96])
def test_linear_every_few_tokens(T, M):
    N, K, group = 200, 1312, 128  # the last group is short
    codes, scales, zeros = weight(N, K, group, T, True)
    X = acts(M, K, T)
    check(i8.int4_linear_forward(X, codes, scales, zeros, None, group), X, codes, scales, zeros, None,
          group)


@pytest.mark.parametrize("T", [FP16, BF16])
@pytest.mark.parametrize("M,N,K,group", [
    (1, 4096, 4096, 128), (8, 4096, 4096, 64), (3, 5120, 13824, 128), (6, 1000, 65536, 32),
    (1, 300, 65536, 128), (16, 640, 13824, 128), (40, 3000, 11008, 32)])
def test_linear_layer_sizes(T, M, N, K, group):
    codes, scales, zeros = weight(N, K, group, T, True)
    X = acts(M, K, T)
    check(i8.int4_linear_forward(X, codes, scales, zeros, None, group), X, codes, scales, zeros, None,
          group)


def test_linear_long_prompt_sampled_rows():
    M, N, K, group = 2048, 1376, 4096, 128
    codes, scales, zeros = weight(N, K, group, FP16, False)
    X = acts(M, K, FP16)
    Y = i8.int4_linear_forward(X, codes, scales, zeros, None, group)
    check(Y, X, codes, scales, zeros, None, group, rows=[0, 1, 127, 128, 255, 256, 1000, 2047])


@pytest.mark.parametrize("M", [1, 5, 16, 50, 300])
def test_linear_wide_range_of_activations(M):
    """bf16 activations far outside fp16's range, large and small in one row: each output keeps
    the accuracy of a 32-bit sum."""
    N, K, group = 70, 512, 64
    codes, scales, zeros = weight(N, K, group, BF16, True)
    X = acts(M, K, torch.float32)
    for factor in (1e30, 1e-30):
        Xf = (X * factor).to(BF16)
        check(i8.int4_linear_forward(Xf, codes, scales, zeros, None, group), Xf, codes, scales, zeros,
              None, group)
    X[:, ::3] *= 1e12
    X[:, 1::3] *= 1e-12
    X = X.to(BF16)
    check(i8.int4_linear_forward(X, codes, scales, zeros, None, group), X, codes, scales, zeros, None,
          group)
    X = torch.zeros(M, K, dtype=BF16, device="cuda")
    Y = i8.int4_linear_forward(X, codes, scales, zeros, None, group)
    assert (Y == 0).all()


@pytest.mark.parametrize("M", [1, 8, 16, 50, 300])
def test_linear_small_fp16_activations(M):
    """fp16 subnormal activations and scales count exactly."""
    N, K, group = 40, 256, 32
    codes, scales, zeros = weight(N, K, group, FP16, True)
    X = (acts(M, K, torch.float32) * 2.0 ** -20).to(FP16)
    scales = scales * 1000.0  # so that the results are normal numbers
    Y = i8.int4_linear_forward(X, codes, scales, zeros, None, group)
    Yr, A, L2 = reference(X, codes, scales, zeros, None, group)
    tol = U[FP16] * np.abs(Yr) + 2.0 ** -25 + 2.0 ** -23 * 48 * A + 6 * U[FP16] * L2
    assert (np.abs(f64(Y) - Yr) <= tol).all()


@pytest.mark.parametrize("M", [1, 7, 12, 40, 200])
def test_non_finite_activations_stay_in_their_row(M):
    N, K, group = 50, 320, 64
    for T in (FP16, BF16):
        codes, scales, zeros = weight(N, K, group, T, True)
        X = acts(M + 2, K, T)
        bad = X.clone()
        bad[M // 2, 7] = float("nan")
        bad[M + 1, 70] = float("inf")
        Y = i8.int4_linear_forward(X, codes, scales, zeros, None, group)
        Z = i8.int4_linear_forward(bad, codes, scales, zeros, None, group)
        keep = [m for m in range(M + 2) if m not in (M // 2, M + 1)]
        assert torch.equal(Z[keep], Y[keep])
        assert torch.isnan(Z[M // 2]).all()
        assert not torch.isfinite(Z[M + 1]).any()


@pytest.mark.parametrize("M", [1, 8, 16, 60, 260])
def test_linear_leaves_what_is_not_its_own(M):
    """Nothing behind Y is written, no input changes, the same call gives the same bits."""
    N, K, group = 77, 352, 32
    codes, scales, zeros = weight(N, K, group, FP16, True)
    X = acts(M, K, FP16)
    whole = torch.full((M * N + 512,), 7.0, dtype=FP16, device="cuda")
    Y = whole[: M * N].view(M, N)
    before = [t.clone() for t in (X, codes, scales, zeros)]
    i8.int4_linear_forward(X, codes, scales, zeros, None, group, Y=Y)
    first = Y.clone()
    assert (whole[M * N:] == 7.0).all()
    for a, b in zip(before, (X, codes, scales, zeros)):
        assert torch.equal(a, b)
    for _ in range(3):
        i8.int4_linear_forward(X, codes, scales, zeros, None, group, Y=Y)
        assert torch.equal(Y, first)


def test_a_row_does_not_depend_on_its_batch():
    """The rows of one call with few tokens equal the calls of one token."""
    codes, scales, zeros = weight(300, 1024, 128, FP16, False)
    X = acts(4, 1024, FP16)
    Y = i8.int4_linear_forward(X, codes, scales, zeros, None, 128)
    for m in range(4):
        one = i8.int4_linear_forward(X[m:m + 1], codes, scales, zeros, None, 128)
        check(one, X[m:m + 1], codes, scales, zeros, None, 128)
        assert torch.allclose(one[0].float(), Y[m].float(), rtol=2 * U[FP16], atol=1e-4)


@pytest.mark.parametrize("M", [1, 8, 24, 200])
def test_streams_and_graphs(M):
    """On a stream of its own, and captured and replayed with other inputs while calls on another
    stream run."""
    N, K, group = 256, 1024, 64
    codes, scales, zeros = weight(N, K, group, BF16, True)
    X1, X2 = acts(M, K, BF16, 1), acts(M, K, BF16, 2)
    want = [i8.int4_linear_forward(x, codes, scales, zeros, None, group) for x in (X1, X2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = i8.int4_linear_forward(X1, codes, scales, zeros, None, group, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want[0])
    X, Y = X1.clone(), torch.empty_like(want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        i8.int4_linear_forward(X, codes, scales, zeros, None, group, Y=Y)
    for x, w in ((X2, want[1]), (X1, want[0])):
        X.copy_(x)
        Y.fill_(float("nan"))
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        other = i8.int4_linear_forward(X2, codes, scales, zeros, None, group, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(Y, w) and torch.equal(other, want[1])


def test_weights_and_activations_made_just_before():
    """Quantizer, dequantizer and products back to back on one stream read what the call before
    wrote."""
    W = (torch.randn(512, 1024, device="cuda") * 0.05).half()
    X = acts(8, 1024, FP16)
    for _ in range(20):
        codes, scales, zeros = i8.int4_quant_weight(W, 64, False)
        Y = i8.int4_linear_forward(X, codes, scales, zeros, None, 64)
        Z = i8.int4_linear_forward(Y, *i8.int4_quant_weight(W[:, :512].contiguous(), 64, False),
                                   group_size=64)
        check(Y, X, codes, scales, zeros, None, 64)
        c2, s2, z2 = i8.int4_quant_weight(W[:, :512].contiguous(), 64, False)
        check(Z, Y, c2, s2, z2, None, 64)
        W = W.roll(1, 0).contiguous()


def test_two_threads_on_two_streams():
    """Two threads at once, each on a stream of its own, through every kernel of the product: each
    result is that of the same calls one after the other."""
    import threading

    Ws = [(torch.randn(512, 1024, device="cuda") * 0.05).half() for _ in range(2)]
    Xs = [acts(M, 1024, FP16, M) for M in (1, 4, 30, 160)]

    def calls(W):
        out = []
        for X in Xs:
            weight = i8.int4_quant_weight(W, 64, False)
            Y = i8.int4_linear_forward(X, *weight, group_size=64)
            out.append((Y, i8.int8_block_norm(Y)))
        return out

    want = [calls(W) for W in Ws]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                for _ in range(30):
                    got[i] = calls(Ws[i])
            side.synchronize()
        except Exception as e:  # pragma: no cover
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_offsets_past_32_bits():
    """More than 4 GiB of codes, and more than 4 GiB of outputs."""
    N, K, group = 140000, 65536, 128
    codes = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda").random_(0, 256)
    scales = torch.full((N, K // group), 2.0 ** -7, dtype=FP16, device="cuda")
    X = acts(2, K, FP16, std=0.1)
    Y = i8.int4_linear_forward(X, codes, scales, None, None, group)
    for rows in (slice(0, 3), slice(131070, 131075), slice(N - 3, N)):
        check(Y[:, rows].contiguous(), X, codes[rows], scales[rows], None, None, group)
    X = acts(20, K, FP16, std=0.1)
    Y = i8.int4_linear_forward(X, codes, scales, None, None, group)
    check(Y[:, N - 3:].contiguous(), X, codes[N - 3:], scales[N - 3:], None, None, group)
    del codes, scales
    M, N, K = 70000, 32768, 64
    codes, scales, zeros = weight(N, K, 32, FP16, False)
    X = acts(M, K, FP16)
    Y = i8.int4_linear_forward(X, codes, scales, None, None, 32)
    rows = [0, 65535, 65536, M - 1]
    check(Y, X, codes, scales, None, None, 32, rows=rows)


def test_python_refusals():
    codes, scales, zeros = weight(16, 64, 32, FP16, True)
    X = acts(2, 64, FP16)
    call = i8.int4_linear_forward
    with pytest.raises(TypeError):
        call(X.float(), codes, scales, zeros, None, 32)
    with pytest.raises(TypeError):
        call(X.bfloat16(), codes, scales, zeros, None, 32)
    with pytest.raises(ValueError):
        call(X[:, :32].contiguous(), codes, scales, zeros, None, 32)
    with pytest.raises(ValueError):
        call(X, codes, scales, zeros, None, 64)  # scales of another group size
    with pytest.raises(ValueError):
        call(X.t().contiguous().t(), codes, scales, zeros, None, 32)
    with pytest.raises(ValueError):
        call(X, codes, scales, zeros[:8], None, 32)
    with pytest.raises(ValueError):
        call(X, codes, scales, zeros, None, 32, Y=torch.empty(2, 15, dtype=FP16, device="cuda"))
    with pytest.raises(ValueError):
        call(X, codes, scales, zeros, torch.zeros(17, dtype=FP16, device="cuda"), 32)
    with pytest.raises(ValueError):
        call(X, codes, scales, zeros, torch.zeros(16, dtype=FP16), 32)  # on the CPU
    with pytest.raises(i8.Int8mmError):
        call(X[:0], codes, scales, zeros, None, 32)  # no token
    with pytest.raises(i8.Int8mmError):
        i8.int4_quant_weight(acts(4, 48, FP16), 32)
    with pytest.raises(i8.Int8mmError):
        i8.int4_quant_weight(acts(4, 64, FP16), 48)
    with pytest.raises(i8.Int8mmError):
        i8.int4_quant_weight(acts(4, 64, FP16), 0)
    with pytest.raises(ValueError):
        i8.int4_quant_weight(acts(4, 64, FP16), 32, True, zeros=zeros)
    with pytest.raises(i8.Int8mmError):  # rows that do not start on 16 bytes
        flat = torch.empty(2 * 64 + 8, dtype=FP16, device="cuda")
        call(flat[4:4 + 128].view(2, 64), codes, scales, zeros, None, 32)
    torch.cuda.synchronize()


def test_layer():
    W = (torch.randn(96, 256, device="cuda") * 0.1).to(BF16)
    b = torch.randn(96, device="cuda").to(BF16)
    layer = i8.Int4Linear(W, b, group_size=64, symmetric=False)
    X = acts(10, 256, BF16).view(2, 5, 256)
    Y = layer(X)
    assert Y.shape == (2, 5, 96)
    check(Y.view(10, 96), X.view(10, 256), layer.codes, layer.scales, layer.zeros, layer.bias, 64)
    assert torch.equal(layer(X[:, ::2]), layer(X[:, ::2].contiguous()))  # a strided batch
    # off by at most half a step, and 15 roundings of the scale to T (15 * 2^-8 of a step)
    step = layer.scales.float().repeat_interleave(64, 1)
    assert ((layer.dequantize().float() - W.float()).abs() <= 0.56 * step).all()
    assert int(layer.dev_status) == 0
