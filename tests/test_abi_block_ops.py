"""Refusals of the training-block operators, on the host before any launch
(no GPU: the pointers below are never dereferenced)."""
import ctypes

import pytest
import torch

import windowed_attention_b200 as rib
from windowed_attention_b200 import _lib

INVALID, UNSUPPORTED, ALIGNMENT = 1, 2, 3
P = 256


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_dropout_refusals(lib):
    ok = [P, P, 0, 16, 0.5, 1, 2, None, None]
    for i, v, st in ((2, 3, INVALID), (4, -0.1, INVALID), (4, 1.1, INVALID), (4, float("nan"), INVALID), (0, None, INVALID),
                     (1, None, INVALID), (0, 257, ALIGNMENT), (1, 257, ALIGNMENT), (7, 260, ALIGNMENT), (3, (1 << 42) + 1, UNSUPPORTED)):
        a = list(ok)
        a[i] = v
        assert lib.rib_dropout(*a) == st, (i, v)
    a = list(ok)
    a[0], a[2] = 258, 1     # fp32 on a 2-byte boundary
    assert lib.rib_dropout(*a) == ALIGNMENT
    assert lib.rib_dropout(None, None, 0, 0, 0.5, 1, 2, None, None) == 0


def _desc(**kw):
    d = rib.residual_norm_desc(64, 48, torch.float32, torch.bfloat16, pre="layer", post="layer")
    for k, v in kw.items():
        setattr(d, k, v)
    return ctypes.byref(d)


FWD = [P] * 10 + [None, None]     # x, y, gate, scale, post_w, post_b, pre_w, pre_b, x_out, h, step, stream
BWD = [P] * 17 + [P, 1 << 30, None, None]


@pytest.mark.parametrize("kw,st", [
    ({"T": -1}, INVALID), ({"C": 0}, INVALID), ({"rows_per_group": 0}, INVALID), ({"pre": 3}, INVALID), ({"post": -1}, INVALID),
    ({"eps": 0.0}, INVALID), ({"eps": float("inf")}, INVALID), ({"p": 1.5}, INVALID), ({"p": float("nan")}, INVALID),
    ({"x_dtype": 5}, INVALID), ({"dtype": -1}, INVALID), ({"x_dtype": 2, "dtype": 0}, UNSUPPORTED), ({"x_dtype": 0, "dtype": 1}, UNSUPPORTED),
    ({"C": 4097}, UNSUPPORTED), ({"T": 2000, "rows_per_group": 1}, UNSUPPORTED), ({"T": (1 << 40) + 1}, UNSUPPORTED),
], ids=str)
def test_residual_norm_descriptor_refusals(lib, kw, st):
    assert lib.rib_residual_norm(_desc(**kw), *FWD) == st
    assert lib.rib_residual_norm_bwd(_desc(**kw), *BWD) == st


def _with(base, **at):
    a = list(base)
    for k, v in at.items():
        a[int(k[1:])] = v
    return a


def test_residual_norm_forward_refusals(lib):
    assert lib.rib_residual_norm(None, *FWD) == INVALID
    assert lib.rib_residual_norm(_desc(), *_with(FWD, _0=None)) == INVALID                     # x
    assert lib.rib_residual_norm(_desc(), *_with(FWD, _9=None)) == INVALID                     # pre norm without h
    assert lib.rib_residual_norm(_desc(pre=0), *FWD) == INVALID                                # h without a pre norm
    assert lib.rib_residual_norm(_desc(pre=0), *_with(FWD, _9=None)) == INVALID                # pre_w without a pre norm
    assert lib.rib_residual_norm(_desc(post=0), *FWD) == INVALID                               # post_w without a post norm
    assert lib.rib_residual_norm(_desc(), *_with(FWD, _1=None)) == INVALID                     # gate and scale without y
    assert lib.rib_residual_norm(_desc(pre=0, post=0), P, *[None] * 11) == INVALID             # nothing to compute
    assert lib.rib_residual_norm(_desc(pre=0, post=0), P, P, *[None] * 10) == INVALID          # nothing to write
    for i in range(10):
        assert lib.rib_residual_norm(_desc(), *_with(FWD, **{f"_{i}": 257})) == ALIGNMENT, i
    assert lib.rib_residual_norm(_desc(), *_with(FWD, _0=258)) == ALIGNMENT                    # fp32 x on 2 bytes
    assert lib.rib_residual_norm(_desc(), *_with(FWD, _10=260)) == ALIGNMENT                   # step
    assert lib.rib_residual_norm(_desc(T=0), *_with(FWD)) == 0


def test_residual_norm_backward_refusals(lib):
    # x_out, y, gate, scale, post_w, post_b, pre_w, dx_out, dh, dx, dy, dgate, dscale, dpost_w, dpost_b, dpre_w, dpre_b, ws, bytes
    b = BWD
    f = lambda d, a: lib.rib_residual_norm_bwd(d, *a)  # noqa: E731
    assert f(None, b) == INVALID
    assert f(_desc(), _with(b, _0=None)) == INVALID          # x_out
    assert f(_desc(), _with(b, _8=None)) == INVALID          # dh
    assert f(_desc(), _with(b, _1=None)) == INVALID          # y
    assert f(_desc(), _with(b, _2=None)) == INVALID          # dgate without gate
    assert f(_desc(), _with(b, _3=None)) == INVALID          # dscale without scale
    assert f(_desc(), _with(b, _17=None)) == INVALID         # workspace
    assert f(_desc(), _with(b, _18=16)) == INVALID           # workspace too small
    assert f(_desc(pre=0), b) == INVALID
    assert f(_desc(post=0), b) == INVALID
    for i in range(17):
        assert f(_desc(), _with(b, **{f"_{i}": 257})) == ALIGNMENT, i
    assert f(_desc(), _with(b, _17=258)) == ALIGNMENT
    # no gradient to start from
    assert f(_desc(pre=0, post=0), [P, P] + [None] * 7 + [P] + [None] * 8 + [0, None, None]) == INVALID


def test_workspace_sizes(lib):
    d = rib.residual_norm_desc(147456, 180, torch.float32, torch.bfloat16)
    assert rib.rib_residual_norm_bwd_workspace_size(d) == 296 * 5 * 180 * 4
    d = rib.residual_norm_desc(1, 180, torch.float32, torch.bfloat16)
    assert rib.rib_residual_norm_bwd_workspace_size(d) == 5 * 180 * 4
    assert lib.rib_residual_norm_bwd_workspace_size(None) == 0


def test_binding_refusals():
    x = torch.zeros(4, 48)
    with pytest.raises(ValueError):
        rib.rib_dropout(x, x, 0.5, 1)                       # host tensors
    with pytest.raises(ValueError):
        rib.residual_norm_desc(4, 48, torch.float64, torch.bfloat16)
    with pytest.raises(ValueError):
        rib.residual_norm_desc(4, 48, torch.float32, torch.bfloat16, pre="batch")
