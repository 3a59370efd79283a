"""The 4-bit linear layer and the block norms as workloads: what is run, on which inputs.

Each operator is here twice: as the library's calls, and in its plain form in elementary torch
operations (32 bits, rounded once at the end).  The cases are the shapes of the layers that the
library's benchmark and tests run (the 4096-wide query projection, the 11008-wide up projection,
the 13B down projection, the 175B feed-forward layer) from one token to a long prompt.
"""
import math

import torch

own = False

DTYPES = {"float16": torch.float16, "bfloat16": torch.bfloat16, "float32": torch.float32}
EPS = 1e-6
SEQ_GATES = 4  # sequences in a batch whose gates differ (one gate row for each)


def listed():
    return [
        # one new token through the query projection: launch latency counts
        dict(name="linear_1tok_q_proj", op="linear", dtype="float16", M=1, N=4096, K=4096, group=128,
             affine=False, bias=False),
        # eight sequences decoding together, small groups with zero points and a bias
        dict(name="linear_8tok_q_proj", op="linear", dtype="bfloat16", M=8, N=4096, K=4096, group=64,
             affine=True, bias=True),
        # three drafted tokens through the 13B down projection (long rows)
        dict(name="linear_3tok_down_13b", op="linear", dtype="float16", M=3, N=5120, K=13824, group=128,
             affine=True, bias=False),
        # one token through the 175B feed-forward layer: the weights' bytes are all of it
        dict(name="linear_1tok_ffn_175b", op="linear", dtype="float16", M=1, N=49152, K=12288, group=128,
             affine=False, bias=False),
        # a ragged batch of 77 tokens through the up projection, the smallest groups
        dict(name="linear_77tok_up_proj", op="linear", dtype="bfloat16", M=77, N=11008, K=4096, group=32,
             affine=False, bias=False),
        # a prompt of 2048 tokens through the up projection
        dict(name="linear_2048tok_up_proj", op="linear", dtype="float16", M=2048, N=11008, K=4096, group=128,
             affine=False, bias=True),
        # loading a layer: quantize it, and look at what its codes stand for
        dict(name="quantize_q_proj", op="quantize", dtype="bfloat16", N=4096, K=4096, group=64, affine=True),
        dict(name="quantize_ffn_175b", op="quantize", dtype="float16", N=49152, K=12288, group=128,
             affine=False),
        # the norm before a block: one decoding step of eight sequences, and a long prompt with its
        # residual stream in 32 bits
        dict(name="norm_8tok_4096", op="norm", dtype="float16", residual="float16", M=8, D=4096,
             layer_norm=False),
        dict(name="norm_4096tok_5120", op="norm", dtype="bfloat16", residual="float32", M=4096, D=5120,
             layer_norm=True),
        # after a block: norm of its output, gate, residual, and the next block's norm
        dict(name="residual_8tok_4096", op="residual", dtype="float16", residual="float16", M=8, D=4096,
             layer_norm=False, post=True, gate="channel", next=True),
        dict(name="residual_2048tok_12288", op="residual", dtype="bfloat16", residual="bfloat16", M=2048,
             D=12288, layer_norm=False, post=True, gate="sequence", next=True),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    dtype = rng.choice(["float16", "bfloat16"])
    op = rng.choice(["linear", "linear", "linear", "quantize", "norm", "residual"])
    if op in ("linear", "quantize"):
        K = _log(rng, 256, 13824, 32)
        N = _log(rng, 48, 49152)
        group = rng.choice([32, 64, 128, 256])
        affine = rng.random() < 0.5
        if op == "quantize":
            return dict(op=op, dtype=dtype, N=N, K=K, group=group, affine=affine)
        M = _log(rng, 1, 16) if rng.random() < 0.6 else _log(rng, 17, 2048)
        while M * N * K > 2048 * 11008 * 4096 or N * K > 49152 * 12288:
            N = max(48, N // 2)
        return dict(op=op, dtype=dtype, M=M, N=N, K=K, group=group, affine=affine, bias=rng.random() < 0.3)
    residual = rng.choice([dtype, dtype, "float32"])
    D = _log(rng, 256, 16384, 16)
    M = _log(rng, 1, 4096)
    while M * D > 2048 * 12288:
        M //= 2
    layer_norm = rng.random() < 0.4
    if op == "norm":
        return dict(op=op, dtype=dtype, residual=residual, M=M, D=D, layer_norm=layer_norm)
    return dict(op=op, dtype=dtype, residual=residual, M=M, D=D, layer_norm=layer_norm,
                post=rng.random() < 0.7, gate=rng.choice(["none", "channel", "row"]), next=rng.random() < 0.8)


def _groups(case):
    return -(-case["K"] // case["group"])


def work(case):
    if case["op"] in ("linear", "quantize"):
        N, K = case["N"], case["K"]
        weights = N * K // 2 + N * _groups(case) * (3 if case["affine"] else 2)
        if case["op"] == "quantize":  # weights in, codes out; codes in, values out
            return {"bytes": 4 * N * K + 2 * weights, "flops": 4 * N * K}
        M = case["M"]
        return {"bytes": weights + 2 * M * K + 2 * M * N + (2 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    M, D = case["M"], case["D"]
    r = 4 if case["residual"] == "float32" else 2
    if case["op"] == "norm":
        return {"bytes": M * D * (r + 2), "flops": 6 * M * D}
    rows = {"none": 0, "channel": 1, "sequence": SEQ_GATES, "row": M}[case["gate"]]
    return {"bytes": M * D * (2 + 2 * r + (2 if case["next"] else 0)) + 2 * rows * D, "flops": 14 * M * D}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=T):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(mean, std, generator=g)

    if case["op"] == "quantize":
        # weights of a trained layer: zero mean, each channel with a spread of its own
        W = normal(case["N"], case["K"], std=0.02)
        W *= torch.empty(case["N"], 1, dtype=T, device="cuda").uniform_(0.5, 2.0, generator=g)
        return dict(case=case, W=W)
    if case["op"] == "linear":
        M, N, K, G = case["M"], case["N"], case["K"], _groups(case)
        # codes of bell-shaped weights (the quantizer's own, about 2.5 steps of spread)
        codes = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
        for a in range(0, N, 8192):  # in slices: the normal deviates are 16 times the codes' size
            n = min(N, a + 8192) - a
            u = torch.empty(n, K // 2, 2, dtype=torch.float32, device="cuda").normal_(8.0, 2.5, generator=g)
            u = u.round_().clamp_(1, 15).to(torch.uint8)
            codes[a:a + n] = u[..., 0] | (u[..., 1] << 4)
        scales = torch.empty(N, G, dtype=torch.float32, device="cuda").uniform_(0.004, 0.016, generator=g).to(T)
        zeros = torch.randint(5, 11, (N, G), dtype=torch.uint8, device="cuda", generator=g) if case["affine"] else None
        bias = normal(N, std=0.1) if case["bias"] else None
        X = normal(M, K)
        X[:, :: max(1, K // 6)] *= 8.0  # the few feature columns of large magnitude
        # what a serving loop keeps: the output's buffer and the device status word
        return dict(case=case, X=X, codes=codes, scales=scales, zeros=zeros, bias=bias,
                    Y=torch.empty(M, N, dtype=T, device="cuda"),
                    status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    M, D, R = case["M"], case["D"], DTYPES[case["residual"]]
    s = dict(case=case, x=normal(M, D, std=2.0, mean=0.1, dtype=R), h=torch.empty(M, D, dtype=T, device="cuda"))
    s["weight"] = normal(D, std=0.2, mean=1.0)
    s["bias"] = normal(D, std=0.1) if case["layer_norm"] else None
    if case["op"] == "residual":
        s["f"] = normal(M, D, std=0.7, mean=0.05)
        s["post_weight"] = normal(D, std=0.2, mean=1.0) if case["post"] else None
        s["post_bias"] = normal(D, std=0.1) if case["post"] and case["layer_norm"] else None
        rows = {"none": 0, "channel": 1, "sequence": SEQ_GATES, "row": M}[case["gate"]]
        s["gate"] = normal(rows, D, std=0.5, mean=0.5) if rows else None
        s["x_scale"], s["f_scale"] = 1.0, 0.25
        s["y"] = torch.empty(M, D, dtype=R, device="cuda")
    return s


# ---------------------------------------------------------------------- the plain forms

_NIBBLE_OF_K = (0, 4, 1, 5, 2, 6, 3, 7)  # of 8 neighbours, k is held in this nibble of their word


def _unpack(codes, K):
    """The codes as float32 [N, K]: nibbles of a 32-bit word hold k = 0, 2, 4, 6, 1, 3, 5, 7."""
    N = codes.shape[0]
    nibbles = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(N, K // 8, 8)
    order = torch.tensor(_NIBBLE_OF_K, device=codes.device)
    return nibbles[:, :, order].reshape(N, K).float()


def _spread(v, group, K):
    """[N, groups] -> [N, K]."""
    return v.float().repeat_interleave(group, dim=1)[:, :K]


def _plain_linear(s):
    c = s["case"]
    K, G = c["K"], c["group"]
    u = _unpack(s["codes"], K)
    u -= 8.0 if s["zeros"] is None else _spread(s["zeros"], G, K)
    u *= _spread(s["scales"], G, K)
    y = s["X"].float() @ u.t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["X"].dtype)


def _by_group(w, group):
    """[N, K] -> [N, groups, group], the last group filled up with zeros."""
    N, K = w.shape
    G = -(-K // group)
    if G * group != K:
        w = torch.cat((w, w.new_zeros(N, G * group - K)), dim=1)
    return w.reshape(N, G, group)


def _plain_quantize(s):
    c = s["case"]
    W, T = s["W"], s["W"].dtype
    w = _by_group(W.float(), c["group"])
    if c["affine"]:
        fifteen = torch.full((), 15.0, device=w.device)
        lo, hi = w.amin(dim=2).clamp(max=0.0), w.amax(dim=2).clamp(min=0.0)
        scales = (hi / fifteen - lo / fifteen).to(T)
        d = torch.where(scales == 0, 1.0, scales.float())
        zeros = (-lo / d).round().clamp(0, 15)
        q = (w / d[:, :, None]).round().add_(zeros[:, :, None]).clamp_(0, 15).sub_(zeros[:, :, None])
    else:
        seven = torch.full((), 7.0, device=w.device)
        scales = (w.abs().amax(dim=2) / seven).to(T)
        d = torch.where(scales == 0, 1.0, scales.float())
        zeros = None
        q = (w / d[:, :, None]).round_().clamp_(-7, 7)
    q *= scales.float()[:, :, None]
    values = q.reshape(W.shape[0], -1)[:, : c["K"]].to(T).contiguous()
    return dict(values=values, scales=scales, zeros=None if zeros is None else zeros.to(torch.uint8))


def _normed(v, weight, bias, layer_norm):
    if layer_norm:
        v = v - v.mean(dim=1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    if weight is not None:
        v = v * weight.float()
    if bias is not None:
        v = v + bias.float()
    return v


def _plain_norm(s):
    return _normed(s["x"].float(), s["weight"], s["bias"], s["case"]["layer_norm"]).to(s["h"].dtype)


def _plain_residual(s):
    c = s["case"]
    p = s["f"].float()
    if c["post"]:
        p = _normed(p, s["post_weight"], s["post_bias"], c["layer_norm"])
    if s["gate"] is not None:
        p = p.reshape(s["gate"].shape[0], -1, c["D"]) * s["gate"].float()[:, None, :]
        p = p.reshape(c["M"], c["D"])
    y = (s["x_scale"] * s["x"].float() + s["f_scale"] * p).to(s["x"].dtype)
    if not c["next"]:
        return dict(y=y)
    return dict(y=y, h=_normed(y.float(), s["weight"], s["bias"], c["layer_norm"]).to(s["f"].dtype))


# ---------------------------------------------------------------------- one pass

def run(state):
    c = state["case"]
    if not own:
        plain = dict(linear=_plain_linear, quantize=_plain_quantize, norm=_plain_norm, residual=_plain_residual)
        return plain[c["op"]](state)
    import int8_mixed_precision_absmax_b200 as i8
    s = state
    if c["op"] == "linear":
        return i8.int4_linear_forward(s["X"], s["codes"], s["scales"], s["zeros"], s["bias"], c["group"], Y=s["Y"],
                                      dev_status=s["status"])
    if c["op"] == "quantize":
        codes, scales, zeros = i8.int4_quant_weight(s["W"], c["group"], symmetric=not c["affine"])
        values = i8.int4_dequant_weight(codes, scales, zeros, c["group"])
        return dict(values=values, scales=scales, zeros=zeros)
    if c["op"] == "norm":
        return i8.int8_block_norm(s["x"], s["weight"], s["bias"], EPS, c["layer_norm"], h=s["h"])
    y, h = i8.int8_block_residual(s["f"], s["x"], post_norm=c["post"], post_weight=s["post_weight"],
                                  post_bias=s["post_bias"], gate=s["gate"], x_scale=s["x_scale"],
                                  f_scale=s["f_scale"], next_norm=c["next"],
                                  next_weight=s["weight"] if c["next"] else None,
                                  next_bias=s["bias"] if c["next"] else None, eps=EPS, layer_norm=c["layer_norm"], y=s["y"],
                                  h=s["h"] if c["next"] else None)
    return dict(y=y, h=h) if c["next"] else dict(y=y)


# ---------------------------------------------------------------------- the definition in 64 bits

def _exact_linear(s, c):
    K, G, N = c["K"], c["group"], c["N"]
    X = s["X"].double()
    out = torch.empty(c["M"], N, dtype=torch.float64, device="cuda")
    for a in range(0, N, 8192):
        b = min(N, a + 8192)
        words = s["codes"][a:b].reshape(b - a, K // 8, 4).long()
        words = words[..., 0] + words[..., 1] * 256 + words[..., 2] * 65536 + words[..., 3] * 16777216
        W = torch.empty(b - a, K // 8, 8, dtype=torch.float64, device="cuda")
        for i, k in enumerate((0, 2, 4, 6, 1, 3, 5, 7)):
            W[:, :, k] = (words // 16 ** i % 16).double()
        W = W.reshape(b - a, K)
        for k in range(0, K, G):
            e = min(K, k + G)
            z = s["zeros"][a:b, k // G].double()[:, None] if s["zeros"] is not None else 8.0
            W[:, k:e] = s["scales"][a:b, k // G].double()[:, None] * (W[:, k:e] - z)
        out[:, a:b] = X @ W.t()
        if s["bias"] is not None:
            out[:, a:b] += s["bias"][a:b].double()
    return out


def _exact_quantize(s, c):
    W, G = s["W"], c["group"]
    values, scales = torch.empty(W.shape, dtype=torch.float64, device="cuda"), []
    for k in range(0, c["K"], G):
        w = W[:, k:k + G].double()
        if c["affine"]:
            lo, hi = torch.clamp(w.min(1).values, max=0), torch.clamp(w.max(1).values, min=0)
            sc = ((hi - lo) / 15).to(W.dtype).double()
            z = torch.clamp(torch.round(-lo / sc), 0, 15).nan_to_num(0.0)[:, None]
            q = torch.clamp(torch.round(w / sc[:, None]).nan_to_num(0.0) + z, 0, 15) - z
        else:
            sc = (w.abs().max(1).values / 7).to(W.dtype).double()
            q = torch.clamp(torch.round(w / sc[:, None]).nan_to_num(0.0), -7, 7)
        values[:, k:k + G] = q * sc[:, None]
        scales.append(sc)
    return dict(values=values, scales=torch.stack(scales, dim=1), zeros=None)


def _exact_normed(v, weight, bias, layer_norm):
    mean = torch.sum(v, 1, keepdim=True) / v.shape[1] if layer_norm else 0.0
    d = v - mean
    n = d / torch.sqrt(torch.sum(d ** 2, 1, keepdim=True) / v.shape[1] + EPS)
    n = n if weight is None else n * weight.double()
    return n if bias is None else n + bias.double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        return _exact_linear(s, case)
    if case["op"] == "quantize":
        return _exact_quantize(s, case)
    x = s["x"].double()
    if case["op"] == "norm":
        return _exact_normed(x, s["weight"], s["bias"], case["layer_norm"])
    f = s["f"].double()
    if case["post"]:
        f = _exact_normed(f, s["post_weight"], s["post_bias"], case["layer_norm"])
    if s["gate"] is not None:
        f = f * s["gate"].double().repeat_interleave(case["M"] // s["gate"].shape[0], dim=0)
    y = s["x_scale"] * x + s["f_scale"] * f
    if not case["next"]:
        return dict(y=y)
    # the next norm reads the residual stream as it is stored
    stored = y.to(DTYPES[case["residual"]]).double()
    return dict(y=y, h=_exact_normed(stored, s["weight"], s["bias"], case["layer_norm"]))
