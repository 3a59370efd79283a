"""The 4-bit layer and the block norms from their formulas, in 64 bits (numpy, no library code)."""
import numpy as np

NIBBLE_K = (0, 2, 4, 6, 1, 3, 5, 7)  # of the 8 neighbours of a word, the one in nibble i


def unpack(codes: np.ndarray) -> np.ndarray:
    """uint8 [N, K/2] -> codes 0..15 [N, K]."""
    words = np.ascontiguousarray(codes).view("<u4")
    u = np.empty(words.shape + (8,), np.uint8)
    for i, k in enumerate(NIBBLE_K):
        u[..., k] = (words >> np.uint32(4 * i)) & np.uint32(15)
    return u.reshape(codes.shape[0], -1)


def pack(u: np.ndarray) -> np.ndarray:
    """codes 0..15 [N, K] -> uint8 [N, K/2]."""
    N, K = u.shape
    g = u.reshape(N, K // 8, 8).astype(np.uint32)
    words = np.zeros((N, K // 8), np.uint32)
    for i, k in enumerate(NIBBLE_K):
        words |= g[..., k] << np.uint32(4 * i)
    return words.astype("<u4").view(np.uint8).reshape(N, K // 2)


def spread(v: np.ndarray, group: int, K: int) -> np.ndarray:
    return np.repeat(v, group, axis=1)[:, :K] if v.shape[1] > 1 else np.repeat(v, K, axis=1)


def values(codes, scales, zeros, group):
    """scales * (code - zero) in float64 [N, K]."""
    u = unpack(codes).astype(np.float64)
    K = u.shape[1]
    z = 8.0 if zeros is None else spread(zeros.astype(np.float64), group, K)
    return (u - z) * spread(scales.astype(np.float64), group, K)


def quantize(W, group, symmetric, to_type):
    """(codes 0..15 [N, K], scales float64, zeros or None) of float64 weights; to_type rounds to
    the stored scale's type.  Quotients and the scale's sums are rounded to float32 first, as
    the definition says."""
    N, K = W.shape
    G = -(-K // group)
    u = np.empty((N, K), np.float64)
    scales, zeros = np.empty((N, G)), np.empty((N, G))
    f32 = np.float32
    for c in range(G):
        w = W[:, c * group:(c + 1) * group]
        bad = ~np.isfinite(w).all(axis=1)
        v = np.where(np.isfinite(w), w, 0.0).astype(f32)
        if symmetric:
            s = to_type(np.abs(v).max(axis=1) / f32(7))
            z = np.full(N, 8.0)
        else:
            hi, lo = np.maximum(v.max(axis=1), 0), np.minimum(v.min(axis=1), 0)
            s = to_type((hi / f32(15) - lo / f32(15)).astype(f32))
        d = np.where(s == 0, 1.0, s).astype(f32)
        if not symmetric:
            z = np.where(s == 0, 0.0, np.clip(np.rint(-lo / d), 0, 15)).astype(np.float64)
        q = np.rint((v / d[:, None]).astype(f32)).astype(np.float64)
        q = np.where((s == 0)[:, None], 0.0, q)
        code = 8 + np.clip(q, -7, 7) if symmetric else np.clip(q + z[:, None], 0, 15)
        u[:, c * group:(c + 1) * group] = np.where(bad[:, None], 8.0, code)
        scales[:, c], zeros[:, c] = np.where(bad, np.nan, s), np.where(bad, 8.0, z)
    return u.astype(np.uint8), scales, None if symmetric else zeros.astype(np.uint8)


def norm(v, w, b, eps, layer_norm):
    """norm(v; w, b) of the rows of a float64 array."""
    d = v - v.mean(axis=1, keepdims=True) if layer_norm else v
    n = d / np.sqrt((d * d).mean(axis=1, keepdims=True) + eps)
    return n * (1.0 if w is None else w) + (0.0 if b is None else b)
