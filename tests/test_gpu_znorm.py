"""The norms before and after a block on the GPU against their formulas in 64 bits.

Tolerances, with u half a step of the stored type.  The residual sum: u |y| for its rounding and
2^-21 of the magnitudes of its terms for the float32 operations in between (the output norm's sum
of D squares by 64 or more accumulators: below 2^-17 for D = 65536 by worst case, 2^-21 by its
square root; at most ten further roundings).  The norm h of y, y as stored: u |h| and 2^-18 of
(|y| + |mean|) / deviation * |w| + |b|.
"""
import numpy as np
import pytest
import torch

import int8_mixed_precision_absmax_b200 as i8

import block_reference as ref

pytestmark = pytest.mark.gpu

FP16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = {FP16: 2.0 ** -11, BF16: 2.0 ** -8, F32: 2.0 ** -24}
TINY = {FP16: 2.0 ** -25, BF16: 2.0 ** -134, F32: 0.0}  # half a step of the least numbers


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def rand(*shape, T=FP16, seed=0, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * std + mean).to(T)


def spread(v, layer_norm, eps):
    """What 1 stands for in the norm's errors, per element."""
    m = v.mean(axis=1, keepdims=True) if layer_norm else 0.0
    return (np.abs(v) + np.abs(m)) / np.sqrt(((v - m) ** 2).mean(axis=1, keepdims=True) + eps)


def check_norm(h, v, w, b, eps, layer_norm):
    """h against norm(v; w, b) of what is stored."""
    v64, w64, b64 = f64(v), f64(w), f64(b)
    want = ref.norm(v64, w64, b64, eps, layer_norm)
    size = spread(v64, layer_norm, eps) * (1.0 if w64 is None else np.abs(w64)) + (
        0.0 if b64 is None else np.abs(b64))
    tol = U[h.dtype] * np.abs(want) + TINY[h.dtype] + 2.0 ** -18 * size
    over = np.abs(f64(h) - want) - tol
    assert (over <= 0).all(), (float(over.max()), np.unravel_index(over.argmax(), over.shape))


def check_sum(y, f, x, post, pw, pb, gate, xs, fs, eps, layer_norm):
    p, x64 = f64(f), f64(x)
    size = np.abs(p)
    if post:
        size = spread(p, layer_norm, eps) * (1.0 if pw is None else np.abs(f64(pw))) + (
            0.0 if pb is None else np.abs(f64(pb)))
        p = ref.norm(p, f64(pw), f64(pb), eps, layer_norm)
    if gate is not None:
        g = f64(gate).reshape(-1, p.shape[1])
        g = np.repeat(g, p.shape[0] // g.shape[0], axis=0)
        p, size = p * g, size * np.abs(g)
    want = xs * x64 + fs * p
    size = abs(xs) * np.abs(x64) + abs(fs) * size
    tol = U[y.dtype] * np.abs(want) + TINY[y.dtype] + 2.0 ** -18 * size
    over = np.abs(f64(y) - want) - tol
    assert (over <= 0).all(), (float(over.max()), np.unravel_index(over.argmax(), over.shape))


TYPES = [(FP16, FP16), (BF16, BF16), (FP16, F32), (BF16, F32)]
SIZES = [(1, 16), (3, 48), (2, 256), (5, 1040), (1, 4096), (9, 4112), (4, 8192), (3, 12288),
         (2, 16400), (2, 32768), (1, 65536), (3, 65520), (1000, 64), (600, 2064)]


@pytest.mark.parametrize("T,R", TYPES)
@pytest.mark.parametrize("M,D", SIZES)
def test_norm_before(T, R, M, D):
    for layer_norm in (False, True):
        x = rand(M, D, T=R, seed=D, std=2.0, mean=0.5)
        w, b = rand(D, T=T, seed=1, mean=1.0), rand(D, T=T, seed=2)
        check_norm(i8.int8_block_norm(x, w, b, 1e-5, layer_norm), x, w, b, 1e-5, layer_norm)
        h = torch.empty(M, D, dtype=T, device="cuda")
        assert i8.int8_block_norm(x, None, None, 1e-6, layer_norm, h=h) is h
        check_norm(h, x, None, None, 1e-6, layer_norm)


@pytest.mark.parametrize("T,R", TYPES)
@pytest.mark.parametrize("M,D", SIZES)
def test_norms_after(T, R, M, D):
    f = rand(M, D, T=T, seed=D, std=3.0, mean=-0.25)
    x = rand(M, D, T=R, seed=D + 1, std=2.0)
    pw, pb = rand(D, T=T, seed=3, mean=1.0), rand(D, T=T, seed=4)
    nw, nb = rand(D, T=T, seed=5, mean=1.0), rand(D, T=T, seed=6)
    gates = [None, rand(D, T=T, seed=7), rand(M, D, T=T, seed=8)]
    for i, (post, nxt, layer_norm) in enumerate([(True, True, False), (True, True, True),
                                                 (False, True, False), (True, False, True),
                                                 (False, False, False)]):
        gate = gates[i % 3]
        xs, fs = ((1.0, 0.25), (0.5, -2.0))[i % 2]
        y, h = i8.int8_block_residual(f, x, post, pw if post else None, pb if post else None, gate,
                                      xs, fs, nxt, nw if nxt else None, nb if nxt else None, 1e-6,
                                      layer_norm)
        assert y.dtype == R and (h is None) == (not nxt)
        check_sum(y, f, x, post, pw if post else None, pb if post else None, gate, xs, fs, 1e-6,
                  layer_norm)
        if nxt:
            assert h.dtype == T
            check_norm(h, y, nw, nb, 1e-6, layer_norm)


@pytest.mark.parametrize("T,R", TYPES)
def test_fused_is_the_two_calls(T, R):
    """y and h of one call: the sum alone, then the norm before the next block, bit for bit."""
    for M, D in ((5, 4096), (130, 1024), (2, 32768)):
        f, x = rand(M, D, T=T, seed=1), rand(M, D, T=R, seed=2)
        pw, nw, gate = (rand(D, T=T, seed=s, mean=1.0) for s in (3, 4, 5))
        y, h = i8.int8_block_residual(f, x, True, pw, None, gate, 1.0, 0.5, True, nw)
        y2, none = i8.int8_block_residual(f, x, True, pw, None, gate, 1.0, 0.5)
        assert none is None and torch.equal(y, y2)
        assert torch.equal(h, i8.int8_block_norm(y2, nw, h=torch.empty_like(f)))


@pytest.mark.parametrize("T,R", TYPES)
@pytest.mark.parametrize("M,D", [(700, 64), (616, 1040), (600, 4096)])
def test_usual_calls_of_many_rows(T, R, M, D):
    """Root-mean-square norms with weights, layer norms with weights and biases, every result wanted:
    with and without the output norm and the gate."""
    f = rand(M, D, T=T, seed=D, std=3.0, mean=-0.25)
    x = rand(M, D, T=R, seed=D + 1, std=2.0)
    w, pw, nw = (rand(D, T=T, seed=s, mean=1.0) for s in (3, 4, 5))
    for layer_norm in (False, True):
        pb, nb = (rand(D, T=T, seed=s) if layer_norm else None for s in (6, 7))
        check_norm(i8.int8_block_norm(x, w, pb, 1e-5, layer_norm, h=torch.empty_like(f)), x, w, pb,
                   1e-5, layer_norm)
        for post in (False, True):
            for gate in (None, rand(4, D, T=T, seed=8)):
                y, h = i8.int8_block_residual(f, x, post, pw if post else None, pb if post else None,
                                              gate, 1.0, 0.25, True, nw, nb, 1e-6, layer_norm)
                check_sum(y, f, x, post, pw if post else None, pb if post else None, gate, 1.0, 0.25,
                          1e-6, layer_norm)
                check_norm(h, y, nw, nb, 1e-6, layer_norm)


def test_gate_rows():
    """One gate row for each sequence of a batch: the rows of its tokens."""
    B, S, D = 3, 7, 320
    f, x, gate = rand(B * S, D, seed=1), rand(B * S, D, seed=2), rand(B, D, seed=3)
    y, _ = i8.int8_block_residual(f, x, gate=gate)
    check_sum(y, f, x, False, None, None, gate, 1.0, 1.0, 1e-6, False)
    whole, _ = i8.int8_block_residual(f, x, gate=gate.repeat_interleave(S, 0).contiguous())
    assert torch.equal(y, whole)
    with pytest.raises(ValueError):
        i8.int8_block_residual(f, x, gate=rand(2, D, seed=3))


@pytest.mark.parametrize("D", [64, 4096, 16384, 65536])
def test_in_place(D):
    """y on x, h on f, and the norm on its own input."""
    M = 5
    for T in (FP16, BF16):
        f, x = rand(M, D, T=T, seed=1), rand(M, D, T=T, seed=2)
        pw, nw = rand(D, T=T, seed=3, mean=1.0), rand(D, T=T, seed=4, mean=1.0)
        want = i8.int8_block_residual(f, x, True, pw, next_norm=True, next_weight=nw)
        f2, x2 = f.clone(), x.clone()
        i8.int8_block_residual(f2, x2, True, pw, next_norm=True, next_weight=nw, y=x2, h=f2)
        assert torch.equal(x2, want[0]) and torch.equal(f2, want[1])
        h = i8.int8_block_norm(x, nw)
        x3 = x.clone()
        i8.int8_block_norm(x3, nw, h=x3)
        assert torch.equal(x3, h)


def test_only_h():
    """Without y (the C call alone offers it): the same h."""
    L = i8.load_library()
    M, D = 6, 512
    f, x = rand(M, D, seed=1), rand(M, D, seed=2)
    want = i8.int8_block_residual(f, x, next_norm=True)[1]
    h = torch.empty_like(f)
    s = torch.cuda.current_stream().cuda_stream
    assert L.int8_block_residual(f.data_ptr(), x.data_ptr(), M, D, None, None, None, 0, 1.0, 1.0,
                                 None, None, 1e-6, 0, None, h.data_ptr(), s) == 0
    assert torch.equal(h, want)


def test_rows_of_zeros_and_of_one_value():
    x = torch.zeros(3, 256, dtype=FP16, device="cuda")
    x[1] = 5.0
    for layer_norm in (False, True):
        h = i8.int8_block_norm(x, eps=1e-6, layer_norm=layer_norm)
        assert (h[0] == 0).all() and (h[2] == 0).all()
        assert (h[1] == (0.0 if layer_norm else 1.0)).all()
    assert torch.isnan(i8.int8_block_norm(x, eps=0.0)[0]).all()  # 0 / 0


def test_layer_norm_far_from_zero():
    """A mean a thousand deviations away: the deviations are taken about the mean, not from the
    difference of two squares."""
    x = rand(4, 4096, T=F32, seed=1, std=1.0, mean=1000.0)
    h = i8.int8_block_norm(x, layer_norm=True)
    check_norm(h, x, None, None, 1e-6, True)
    assert abs(float(h.float().std()) - 1.0) < 1e-2


def test_large_and_non_finite_rows():
    """Squares past fp16's range do not matter; a NaN stays in its row."""
    x = rand(4, 1024, seed=1, std=20000.0).clamp(-60000, 60000)
    check_norm(i8.int8_block_norm(x), x, None, None, 1e-6, False)
    y = x.clone()
    y[2, 3] = float("nan")
    a, b = i8.int8_block_norm(x), i8.int8_block_norm(y)
    assert torch.equal(a[[0, 1, 3]], b[[0, 1, 3]]) and torch.isnan(b[2]).all()


def test_leaves_what_is_not_its_own_and_repeats():
    M, D = 37, 1040
    whole = torch.full((M * D + 1024,), 3.0, dtype=FP16, device="cuda")
    f, x = rand(M, D, seed=1), rand(M, D, seed=2)
    keep = f.clone(), x.clone()
    h = whole[: M * D].view(M, D)
    y, _ = i8.int8_block_residual(f, x, True, next_norm=True, h=h)
    first = h.clone()
    assert (whole[M * D:] == 3.0).all()
    assert torch.equal(f, keep[0]) and torch.equal(x, keep[1])
    for _ in range(3):
        i8.int8_block_residual(f, x, True, next_norm=True, y=y, h=h)
        assert torch.equal(h, first)


@pytest.mark.parametrize("M", [2, 700])
def test_streams_and_graphs(M):
    D = 2048
    f1, x1, f2 = rand(M, D, seed=1), rand(M, D, seed=2), rand(M, D, seed=3)
    want = [i8.int8_block_residual(f, x1, True, next_norm=True) for f in (f1, f2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, h = i8.int8_block_residual(f1, x1, True, next_norm=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want[0][0]) and torch.equal(h, want[0][1])
    f, y, h = f1.clone(), torch.empty_like(x1), torch.empty_like(x1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        i8.int8_block_residual(f, x1, True, next_norm=True, y=y, h=h)
    for src, w in ((f2, want[1]), (f1, want[0])):
        f.copy_(src)
        graph.replay()
        assert torch.equal(y, w[0]) and torch.equal(h, w[1])


def test_offsets_past_32_bits():
    M, D = 33000, 65536
    x = torch.empty(M, D, dtype=FP16, device="cuda").normal_()
    h = i8.int8_block_norm(x)
    for rows in (slice(0, 2), slice(32766, 32770), slice(M - 2, M)):
        check_norm(h[rows], x[rows], None, None, 1e-6, False)
    y, h = i8.int8_block_residual(h, x, True, next_norm=True, y=x, h=h)
    check_norm(h[M - 2:], y[M - 2:], None, None, 1e-6, False)


def test_python_refusals():
    x, w = rand(2, 64), rand(64)
    with pytest.raises(TypeError):
        i8.int8_block_norm(x.double())
    with pytest.raises(TypeError):
        i8.int8_block_norm(x, w.float())
    with pytest.raises(TypeError):
        i8.int8_block_norm(x, w.bfloat16())
    with pytest.raises(ValueError):
        i8.int8_block_norm(x, w[:32])
    with pytest.raises(ValueError):
        i8.int8_block_norm(x.t())
    with pytest.raises(ValueError):
        i8.int8_block_norm(x.float(), h=x[:1])
    with pytest.raises(i8.Int8mmError):
        i8.int8_block_norm(rand(2, 40))
    with pytest.raises(i8.Int8mmError):
        i8.int8_block_norm(x[:0])
    with pytest.raises(i8.Int8mmError):
        i8.int8_block_norm(x, eps=-1.0)
    with pytest.raises(ValueError):
        i8.int8_block_residual(x, x, post_weight=w)
    with pytest.raises(ValueError):
        i8.int8_block_residual(x, x, next_weight=w)
    with pytest.raises(TypeError):
        i8.int8_block_residual(x, x.bfloat16())
    with pytest.raises(ValueError):
        i8.int8_block_residual(x, x[:1])
    with pytest.raises(i8.Int8mmError):
        i8.int8_block_residual(x, x, f_scale=float("inf"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["int8", "int4"])
@pytest.mark.parametrize("M", [1, 6, 40])
def test_blocks_of_layers(kind, M):
    """Two blocks as a decoder runs them: norm, up, down, output norm, gate, residual, through the
    layers; each step from the one before is the direct call's result."""
    D, F = 256, 512
    g = torch.Generator(device="cuda").manual_seed(3)

    def mat(n, k):
        return (torch.randn(n, k, device="cuda", generator=g) * k ** -0.5).half()

    def layer(W, **norms):
        if kind == "int8":
            return i8.Int8Linear(W, threshold=6.0, **norms)
        return i8.Int4Linear(W, group_size=64, symmetric=False, **norms)

    pre = i8.BlockNorm(rand(D, seed=1, mean=1.0), eps=1e-5)
    post = i8.BlockNorm(rand(D, seed=2, mean=1.0), rand(D, seed=3), layer_norm=True)
    gate = rand(D, seed=4, mean=0.5)
    blocks = [(layer(mat(F, D), pre_norm=pre), layer(mat(D, F), post_norm=post)) for _ in range(2)]
    x = rand(M, D, seed=5)
    for up, down in blocks:
        u = up(x)
        h = i8.int8_block_norm(x, pre.weight, None, 1e-5)
        assert torch.equal(pre(x), h)
        assert torch.equal(u, up._product(h, None))
        a = torch.nn.functional.gelu(u)
        y = down(a, residual=x, gate=gate, f_scale=0.5)
        f = down._product(a, None)
        assert torch.equal(y, i8.int8_block_residual(f, x, True, post.weight, post.bias, gate, 1.0,
                                                     0.5, layer_norm=True)[0])
        check_sum(y, f, x, True, post.weight, post.bias, gate, 1.0, 0.5, 1e-6, True)
        x = y
    with pytest.raises(ValueError):
        blocks[0][1](a)  # an output norm without the residual it belongs to
    with pytest.raises(ValueError):
        blocks[0][0](x, gate=gate)


def test_layers_without_ends_are_as_before():
    W = rand(64, 128, seed=1, std=0.1)
    X = rand(3, 2, 128, seed=2)
    layer = i8.Int8Linear(W)
    Y = layer(X)
    assert Y.shape == (3, 2, 64)
    assert torch.equal(Y.view(6, 64), i8.int8_linear_forward(X.view(6, 128), layer.Wq, layer.w_scale,
                                                             None))


@pytest.mark.parametrize("T", [torch.float16, torch.bfloat16])
def test_layer_of_a_float32_stream_without_norm_weights(T):
    """The norm's output takes the layer's type where no weight says it."""
    layer = i8.Int4Linear(rand(64, 128, seed=1, std=0.1).to(T), pre_norm=i8.BlockNorm())
    x = rand(5, 128, seed=2).float()
    h = i8.int8_block_norm(x, h=torch.empty(5, 128, dtype=T, device="cuda"))
    assert torch.equal(layer(x), layer._product(h, None))


def test_sizes_past_an_int_are_refused():
    with pytest.raises(ValueError, match="2\\^31"):
        i8.int8_block_norm(torch.empty(2 ** 32 + 1, 0, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError, match="2\\^31"):
        i8.int8_block_norm(torch.empty(0, 2 ** 32 + 16, dtype=torch.float16, device="cuda"))


@pytest.mark.parametrize("T,R", TYPES)
@pytest.mark.parametrize("D", [11008, 12288])
def test_usual_calls_of_rows_of_384_threads(T, R, D):
    """Rows whose blocks keep to fewer registers, three to an SM."""
    test_usual_calls_of_many_rows(T, R, 604, D)
