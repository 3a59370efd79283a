"""What a layer's call does on the host beside its product: nothing to rows that are as the product
takes them (a small call's time is the host's)."""
import pytest
import torch

import int8_mixed_precision_absmax_b200 as i8


@pytest.fixture(params=["int8", "int4"])
def layer(request, monkeypatch):
    """A layer of 64 -> 8 without weights on a GPU, whose product notes its rows and returns `Y`."""
    kind = i8.Int8Linear if request.param == "int8" else i8.Int4Linear
    layer = kind.__new__(kind)
    layer.in_features, layer.out_features = 64, 8
    layer.pre_norm = layer.post_norm = layer.bias = None
    layer.seen = []

    def product(X, *args, Y=None, **kw):
        layer.seen.append(X)
        layer.Y = torch.arange(X.shape[0] * 8, dtype=torch.float16).view(-1, 8) if Y is None else Y
        return layer.Y

    if kind is i8.Int8Linear:
        monkeypatch.setattr(i8, "int8_linear_forward", product)
        layer.Wq = layer.w_scale = layer.W16 = None
        layer.threshold, layer.per_tensor_activation = 6.0, False
        layer._workspace, layer._ws_rows = torch.zeros(1), 1000
    else:
        monkeypatch.setattr(i8, "int4_linear_forward", product)
        layer.codes = layer.scales = layer.zeros = layer.dev_status = None
        layer.group_size, layer._dtype = 64, torch.float16
    return layer


def test_rows_are_passed_as_they_are(layer):
    X = torch.zeros(3, 64, dtype=torch.float16)
    Y = layer(X)
    assert layer.seen[0] is X and Y is layer.Y
    out = torch.empty(3, 8, dtype=torch.float16)
    assert layer(X, out) is out


def test_other_shapes_and_strides(layer):
    for X in (torch.zeros(64), torch.zeros(2, 3, 64), torch.zeros(5, 128)[:, ::2], torch.zeros(64, 4).t()):
        X = X.half() if X.is_contiguous() else torch.empty_like(X, dtype=torch.float16).copy_(X)
        Y = layer(X)
        assert Y.shape == (*X.shape[:-1], 8)
        seen = layer.seen[-1]
        assert seen.shape == (X.numel() // 64, 64) and seen.is_contiguous()


def test_ends_without_a_residual_are_refused(layer):
    X = torch.zeros(3, 64, dtype=torch.float16)
    for change in (dict(gate=X), dict(x_scale=0.5), dict(f_scale=2.0)):
        with pytest.raises(ValueError, match="residual"):
            layer(X, **change)
    layer.post_norm = i8.BlockNorm()
    with pytest.raises(ValueError, match="residual"):
        layer(X)
    assert not layer.seen
